// fa_split.cuh -- cutting the keys of a ragged batch over CTAs, on the device.
//
// A unit is a tile of query rows of one key/value head; all units of a sequence have
// its number of key tiles.  The host knows the number of units and of CTAs that fit, not the
// lengths.  Every CTA finds the smallest chunk c with
//   sum over units of max(1, ceil(tiles / c)) <= CTAs,
// so that one wave of CTAs, cut as evenly as whole tiles allow, does it all, and takes the
// item of its number: a unit's n-th piece.  Units of one piece are finished by their CTA; the others
// leave (O, log-sum-exp) pieces that a second kernel joins (fa_split_join.cu).  (A cluster
// per unit, joined through distributed shared memory, keeps to 8 CTAs a unit whatever the lengths:
// 8 trees over 1 to 12345 tokens took 134 us at best, with one sequence of them 8 of 152 SMs a head.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {

struct SplitPlan {
    int B, per_seq;    // sequences, units of each
    int items;         // CTAs, at least B * per_seq
    int least;         // tiles that are not worth cutting
    int whole;         // 1: sequences of about one length (none 3/2 of the mean) are not cut
};
struct SplitItem {
    int b, unit;       // sequence; unit within it; -1: no item of this number
    int j0, n;         // its tiles
    int tiles;         // of the whole unit
    int first, pieces; // the unit's items
};
// What the second kernel reads: [unit] (first piece, pieces), pieces of `rows` rows.
struct SplitParts {
    float* o;          // [item][rows][D], normalised
    float* lse;        // [item][rows], log2 units, -inf where a row saw nothing
    int2* units;
    int rows;
};

// Where a row of a unit goes: row r of a key/value head is query r % T of its group's head r / T.
struct SplitOut {
    CrossTensor o;
    __nv_bfloat16* rest;  // of the rounding, or null
    float* lse;
    int Hkv, group, T, R; // R = group * T
    int row_units, unit_rows;
};
int launch_split_join(const SplitParts& parts, const SplitOut& out, int B, int D, int items, cudaStream_t stream);

// Bytes of the pieces' workspace, and its parts.
inline size_t split_workspace(int items, long long units, int rows, int D) {
    return (static_cast<size_t>(items) * rows * D + (static_cast<size_t>(items) * rows + 1) / 2 * 2) * 4 +
           static_cast<size_t>(units) * 8;
}
inline SplitParts split_parts(void* ws, int items, int rows, int D) {
    float* o = static_cast<float*>(ws);
    float* lse = o + static_cast<size_t>(items) * rows * D;
    return {o, lse, reinterpret_cast<int2*>(lse + (static_cast<size_t>(items) * rows + 1) / 2 * 2), rows};
}

__device__ __forceinline__ int split_sum(int x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ int split_pieces(int tiles, int chunk) { return max(1, (tiles + chunk - 1) / chunk); }

// By one warp; tiles_of(b): key tiles of a sequence.
template <typename F>
__device__ __forceinline__ SplitItem split_item(const SplitPlan& p, int number, int lane, F tiles_of) {
    constexpr int kHeld = 4;  // up to 128 sequences the chunk is searched for, beyond it is an upper bound
    int held[kHeld], most = 0;
    long long total = 0;
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
        held[x] = lane + 32 * x < p.B ? tiles_of(lane + 32 * x) : -1;
        most = max(most, held[x]);
        total += max(held[x], 0);
    }
    int chunk;
    if (p.B <= 32 * kHeld) {
        int lo = max(1, p.least), hi = max(lo, __reduce_max_sync(0xffffffffu, most));
        while (lo < hi) {
            const int c = (lo + hi) >> 1;
            int count = 0;
#pragma unroll
            for (int x = 0; x < kHeld; ++x)
                if (32 * x < p.B && held[x] >= 0) count += split_pieces(held[x], c);
            if (static_cast<long long>(split_sum(count)) * p.per_seq <= p.items) hi = c;
            else lo = c + 1;
        }
        chunk = lo;
    } else {
        for (int b = 32 * kHeld + lane; b < p.B; b += 32) {
            const int tiles = tiles_of(b);
            total += tiles;
            most = max(most, tiles);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        // ceil(t / c) <= t / c + 1; the host gives more items than units here
        const long long room = p.items - static_cast<long long>(p.B) * p.per_seq;
        chunk = static_cast<int>(max(static_cast<long long>(max(1, p.least)), (total * p.per_seq + room - 1) / room));
    }
    if (p.whole) {
        if (p.B <= 32 * kHeld) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (2LL * most * p.B <= 3 * total) chunk = max(chunk, most);
    }
    SplitItem it{0, -1, 0, 0, 0, 0, 0};
    int base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane, tiles = b < p.B ? tiles_of(b) : 0;
        const int n = b < p.B ? split_pieces(tiles, chunk) : 0;
        int sum = n * p.per_seq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, base + sum > number);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            it.b = b0 + src;
            it.pieces = __shfl_sync(0xffffffffu, n, src);
            it.tiles = __shfl_sync(0xffffffffu, tiles, src);
            const int rem = number - (base + __shfl_sync(0xffffffffu, sum, src) - it.pieces * p.per_seq);
            it.unit = rem / it.pieces;
            const int k = rem - it.unit * it.pieces;
            it.first = number - k;
            it.j0 = static_cast<int>(static_cast<long long>(it.tiles) * k / it.pieces);
            it.n = static_cast<int>(static_cast<long long>(it.tiles) * (k + 1) / it.pieces) - it.j0;
            break;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    return it;
}

// Host: how many items for `units` units where `slots` CTAs run at a time.  With few units one
// wave; with more, waves of about half a unit each, which even out over the SMs; from four waves
// of whole units on nothing is cut.
inline int split_items(long long units, int slots) {
    if (units >= 4LL * slots) return static_cast<int>(units);
    return static_cast<int>(2 * units <= slots ? slots : (2 * units + slots - 1) / slots * slots);
}

}  // namespace fa
