// fa_split.cuh -- cutting the keys of a ragged batch over CTAs, on the device.
//
// A unit is a tile of query rows of one key/value head; all units of a sequence have
// its number of key tiles.  The host knows the number of units and of CTAs that fit, not the
// lengths.  Every CTA finds the smallest chunk c with
//   sum over units of max(1, ceil(tiles / c)) <= CTAs,
// so that one wave of CTAs, cut as evenly as whole tiles allow, does it all, and takes the
// item of its number: a unit's n-th piece.  Units of one piece are finished by their CTA; the others
// leave (O, log-sum-exp) pieces that a second kernel joins (fa_split_join.cu: 5 to 8 us from cold caches).  (A cluster
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
    int slots;         // CTAs that run at a time
    int share;         // pieces are no shorter than share / 4 of a slot's part of all tiles (0: as short as the items allow)
};
struct SplitItem {
    int b, unit;       // sequence; unit within it; -1: no item of this number
    int j0, n;         // its tiles
    int tiles;         // of the whole unit
    int pieces;        // of the unit
    int part, k;       // where they are left: part + k is this item's; k = 0: its first
};
// What the second kernel reads: [unit] (first piece, pieces), pieces of `rows` rows.  A unit of
// one piece leaves none, and its first piece may be `count`.
struct SplitParts {
    float* o;          // [part][rows][D], normalised
    float* lse;        // [part][rows], log2 units, -inf where a row saw nothing
    int2* units;
    int rows;
    int count;         // pieces that there is room for
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
inline size_t split_workspace(const SplitPlan& p, int rows, int D) {
    const size_t units = static_cast<size_t>(p.B) * p.per_seq, n = 2 * (p.items - units) * rows;
    return n == 0 ? 0 : n * (D + 1) * 4 + units * 8;
}
inline SplitParts split_parts(void* ws, const SplitPlan& p, int rows, int D) {
    const size_t n = 2 * (p.items - static_cast<size_t>(p.B) * p.per_seq) * rows;
    if (n == 0) return {};
    float* o = static_cast<float*>(ws);
    return {o, o + n * D, reinterpret_cast<int2*>(o + n * (D + 1)), rows, static_cast<int>(n / rows)};
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
    if (p.items == p.B * p.per_seq) {  // nothing is cut
        const int b = number / p.per_seq, tiles = tiles_of(b);
        return {b, number - b * p.per_seq, 0, tiles, tiles, 1, 0, 0};
    }
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
        for (int b = 32 * kHeld + lane; b < p.B; b += 32) total += tiles_of(b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        // ceil(t / c) <= t / c + 1; the host gives more items than units here
        const long long room = p.items - static_cast<long long>(p.B) * p.per_seq;
        chunk = static_cast<int>(max(static_cast<long long>(max(1, p.least)), (total * p.per_seq + room - 1) / room));
    }
    if (p.share > 0) {
        if (p.B <= 32 * kHeld) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        chunk = static_cast<int>(max(static_cast<long long>(chunk), total * p.per_seq * p.share / (4LL * p.slots)));
    }
    // up to 32 sequences: those with longer pieces first, as CTAs start in the order of their numbers
    int mine = lane;
    if (p.B <= 32) {
        const int size = held[0] >= 0 ? held[0] / split_pieces(held[0], chunk) : -1;
        int rank = 0;
        for (int i = 0; i < p.B; ++i) {
            const int other = __shfl_sync(0xffffffffu, size, i);
            rank += other > size || (other == size && i < lane);
        }
        for (int i = 0; i < p.B; ++i)
            if (__shfl_sync(0xffffffffu, rank, i) == lane) mine = i;
    }
    SplitItem it{0, -1, 0, 0, 0, 0, 0, 0};
    int base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + mine, tiles = b < p.B ? tiles_of(b) : 0;
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
            it.b = b0 + __shfl_sync(0xffffffffu, mine, src);
            it.pieces = __shfl_sync(0xffffffffu, n, src);
            it.tiles = __shfl_sync(0xffffffffu, tiles, src);
            const int rem = number - (base + __shfl_sync(0xffffffffu, sum, src) - it.pieces * p.per_seq);
            it.unit = rem / it.pieces;
            it.k = rem - it.unit * it.pieces;
            // items before that are a further piece of their unit; a cut unit's pieces are at most twice its further ones
            it.part = 2 * (number - it.k - ((b0 + src) * p.per_seq + it.unit));
            it.j0 = static_cast<int>(static_cast<long long>(it.tiles) * it.k / it.pieces);
            it.n = static_cast<int>(static_cast<long long>(it.tiles) * (it.k + 1) / it.pieces) - it.j0;
            break;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    return it;
}

// Host: the plan for `units` units, per_seq of each sequence, where `slots` CTAs run at a time.  Few units
// are cut as far as the CTAs go, in one wave.  Many go out whole, longest first, but for what is longer
// than share / 4 of a CTA's part, at most 4 slots / share further pieces.  Of more than 512 sequences
// none is cut, as every CTA looks through all of them: one row of 2 heads of 64 channels over 64 keys
// each, all 64 but one of 8192, and 1 to 1000, us cut / whole: 512 sequences 46 / 23, 55 / 86, 62 / 41;
// 1024: 111 / 37, 117 / 100, 138 / 72; 2048 (the long one 4096): 305 / 69, 330 / 100, 365 / 131.
inline SplitPlan split_plan(int B, long long units, int slots, int least, int share) {
    const bool few = 2 * units <= slots;
    const long long items = B > 512 ? units : few ? slots : units + (4LL * slots + share - 1) / share;
    return {B, static_cast<int>(units / B), static_cast<int>(items), least, slots, few ? 0 : share};
}

}  // namespace fa
