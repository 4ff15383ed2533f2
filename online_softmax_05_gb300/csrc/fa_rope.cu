// fa_rope.cu -- rotary positions of queries and keys, and the gradient.
//
// Pair i of a row at position p turns by the angle p f_i:
//   y1 = a (x1 cos - x2 sin),  y2 = a (x2 cos + x1 sin),
// with x1, x2 the channels (i, i + R/2) (half layout) or (2i, 2i + 1)
// (interleaved), R the rotated channels; the others are copied.  The gradient
// is the same map with -sin.
//
// Angles are exact modulo a turn at every position (fa_rope.cuh); a product in
// fp32 would be off by 0.06 rad at position 10^6.
//
// One thread takes the same pairs of one token in several heads, so that an
// angle is computed once for all of them.  Bound: HBM, each element read and
// written once.  B=2 H=16+16 T=8192 D=128 bf16 (268 MB) takes 49.4 us with the
// launch, 80 % of the measured copy rate (47.3 us with fp32's own sine and cosine);
// holding four heads' loads before the first store took 72 us (118 registers, a
// quarter of the warps), 16 heads a thread 50.4 us, against those 47.3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_internal.h"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 128;  // 256: 51.6 us instead of 47.3 in the case above, the last wave being coarser

struct RopeParams {
    RopeTensor t[2];
    int n_tensors;
    const void* positions;  // [B or 1][T], or null: 0 .. T-1
    long long pos_b;        // batch stride of positions (0: shared)
    int pos64;
    const unsigned long long* freq;
    int T, D, R;
    int units;         // units of one row: of V pairs, of 2 V channels to copy, of 16 bytes to copy
    int turns, copies; // how many of the first two
    int wide;          // channel where the third begin
    int heads_thread;  // heads per thread
    long long items;   // B * T * units
    float amp;
    int inverse;
};

template <typename E>
__device__ __forceinline__ float to_f(E x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename E>
__device__ __forceinline__ E from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

template <typename E, int V>
struct alignas(sizeof(E) * V) Vec {
    E e[V];
};

// A unit of a row: V pairs (interleaved: 2 V channels, of which those behind the
// rotated ones are copied), 2 V channels to copy, or 16 bytes of them.
// PART: the last interleaved unit's pairs are not all rotated (registers that the
// whole ones go without).
template <typename E, int V, bool INTER, bool PART>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(RopeParams p) {
    wait_for_stream();
    constexpr int W = 16 / sizeof(E);
    const long long item = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
    if (item >= p.items) return;
    const int u = static_cast<int>(item % p.units);
    const long long row = item / p.units;
    const int t = static_cast<int>(row % p.T);
    const long long b = row / p.T;
    const int half = p.R >> 1;
    const int pair0 = u * V;
    const bool turned = u < p.turns, wide = u >= p.turns + p.copies;
    // the unit's two vectors of V channels, or its one of W
    int c0, c1;
    if (turned) {
        c0 = INTER ? 2 * pair0 : pair0;
        c1 = INTER ? c0 + V : c0 + half;
    } else {
        c0 = wide ? p.wide + W * (u - p.turns - p.copies) : (INTER ? 2 * V * p.turns : p.R) + 2 * V * (u - p.turns);
        c1 = c0 + V;
    }
    float cs[V], sn[V];
    if (turned) {
        long long pos = t;
        if (p.positions != nullptr) {
            const long long at = b * p.pos_b + t;
            pos = p.pos64 ? static_cast<const long long*>(p.positions)[at]
                          : static_cast<long long>(static_cast<const int*>(p.positions)[at]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rope_angle(pos, p.freq[PART ? min(pair0 + i, half - 1) : pair0 + i], p.amp, cs[i], sn[i]);
            if (p.inverse) sn[i] = -sn[i];
        }
    }
    const int pairs = half - pair0;  // of an interleaved unit: V, or fewer in the last
    const bool tail = V > 1 || c1 < p.D;  // an odd head has a lone last channel
    int h = blockIdx.y * p.heads_thread;
    const int h_end = h + p.heads_thread;
    for (int k = 0, h_base = 0; k < p.n_tensors; h_base += static_cast<int>(p.t[k].heads), ++k) {
        const RopeTensor& x = p.t[k];
        const int heads = static_cast<int>(x.heads);
        const E* in = static_cast<const E*>(x.in) + b * x.in_b + static_cast<long long>(t) * x.in_t;
        E* out = static_cast<E*>(x.out) + b * x.out_b + static_cast<long long>(t) * x.out_t;
        const int last = min(h_end, h_base + heads);
        if (V < W && wide) {
            for (; h < last; ++h)
                *reinterpret_cast<uint4*>(out + static_cast<long long>(h - h_base) * x.out_h + c0) =
                    *reinterpret_cast<const uint4*>(in + static_cast<long long>(h - h_base) * x.in_h + c0);
            continue;
        }
#pragma unroll 4
        for (; h < last; ++h) {
            const E* src = in + static_cast<long long>(h - h_base) * x.in_h;
            E* dst = out + static_cast<long long>(h - h_base) * x.out_h;
            Vec<E, V> a = *reinterpret_cast<const Vec<E, V>*>(src + c0), c;
            if (tail) c = *reinterpret_cast<const Vec<E, V>*>(src + c1);
            if (turned) {
                E in2[2 * V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    in2[i] = a.e[i];
                    in2[V + i] = c.e[i];
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int j1 = INTER ? 2 * i : i, j2 = INTER ? 2 * i + 1 : V + i;
                    const float x1 = to_f(in2[j1]), x2 = to_f(in2[j2]);
                    const E y1 = from_f<E>(rope_turn(x1, x2, cs[i], sn[i])), y2 = from_f<E>(rope_turn(x2, x1, cs[i], -sn[i]));
                    if (!PART || i < pairs) {  // the others are copied
                        in2[j1] = y1;
                        in2[j2] = y2;
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    a.e[i] = in2[i];
                    c.e[i] = in2[V + i];
                }
            }
            *reinterpret_cast<Vec<E, V>*>(dst + c0) = a;
            if (tail) *reinterpret_cast<Vec<E, V>*>(dst + c1) = c;
        }
    }
}

template <typename E, int V>
int launch(const RopeParams& p, int inter, dim3 grid, cudaStream_t st) {
    return launch_chained(!inter ? fa_rope_kernel<E, V, false, false>
                          : p.R / 2 % V ? fa_rope_kernel<E, V, true, (V > 1)>
                                        : fa_rope_kernel<E, V, true, false>,
                          grid, kRopeThreads, 0, st, p);
}

template <typename E>
int launch16(const RopeParams& p, int V, int inter, dim3 grid, cudaStream_t st) {
    return V == 8 ? launch<E, 8>(p, inter, grid, st) : V == 2 ? launch<E, 2>(p, inter, grid, st) : launch<E, 1>(p, inter, grid, st);
}

}  // namespace

int launch_rope(const RopeTensor* tensors, int n_tensors, const void* positions, int pos64, long long pos_b,
                const void* freq, int B, int T, int D, int R, int interleaved, float amplitude, int inverse,
                int dtype, cudaStream_t stream, int num_sms) {
    // How far rows are aligned, in channels: to 16 bytes, to 4, or to one channel.
    const int size = dtype == 2 ? 4 : 2, W = 16 / size;
    RopeParams p{};
    long long heads = 0;
    uintptr_t grain = 16;
    for (int k = 0; k < n_tensors; ++k) {
        const RopeTensor& x = tensors[k];
        p.t[k] = x;
        heads += x.heads;
        grain |= reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out);
        for (long long s : {x.in_b, x.in_t, x.in_h, x.out_b, x.out_t, x.out_h}) grain |= static_cast<uintptr_t>(s) * size;
    }
    const bool by16 = (grain & 15u) == 0, by4 = (grain & 3u) == 0;
    const int half = R / 2;
    // Pairs to a unit: as many as make 16-byte vectors, else (16-bit types) 4-byte ones.
    int V = 1;
    if (interleaved) {
        if (by16 && D % (2 * W) == 0) V = W;
        else if (size == 2 && by4 && D % 4 == 0) V = 2;
    } else {
        if (by16 && half % W == 0 && (D - R) % (2 * W) == 0) V = W;
        else if (size == 2 && by4 && half % 2 == 0 && (D - R) % 4 == 0) V = 2;
    }
    p.turns = interleaved ? (half + V - 1) / V : half / V;
    const int behind = interleaved ? 2 * V * p.turns : R;  // the first channel that no turn covers
    // narrow turns, wide copies: rows of 16-byte pieces from the next border on
    p.wide = V < W && by16 && D % W == 0 ? (behind + W - 1) / W * W : D;
    p.copies = (p.wide - behind + 2 * V - 1) / (2 * V);
    p.n_tensors = n_tensors;
    p.positions = positions;
    p.pos64 = pos64;
    p.pos_b = pos_b;
    p.freq = static_cast<const unsigned long long*>(freq);
    p.T = T;
    p.D = D;
    p.R = R;
    p.units = p.turns + p.copies + (D - p.wide + W - 1) / W;
    p.items = static_cast<long long>(B) * T * p.units;
    p.amp = amplitude;
    p.inverse = inverse;
    // a thread takes up to 8 heads, fewer while the grid would leave SMs without work
    int per = 8;
    while (per > 1 && p.items * ((heads + per - 1) / per) < static_cast<long long>(num_sms) * 1024) per >>= 1;
    while ((heads + per - 1) / per > 65535) per *= 2;  // a grid's second extent
    p.heads_thread = per;
    const long long blocks = (p.items + kRopeThreads - 1) / kRopeThreads, ny = (heads + per - 1) / per;
    if (blocks > 0x7fffffffLL) return -2;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(ny));
    if (dtype == 2) return V == 4 ? launch<float, 4>(p, interleaved, grid, stream) : launch<float, 1>(p, interleaved, grid, stream);
    return dtype == 0 ? launch16<__nv_bfloat16>(p, V, interleaved, grid, stream) : launch16<__half>(p, V, interleaved, grid, stream);
}

}  // namespace fa
