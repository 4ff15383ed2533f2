// fa_kv4_cache.cu -- writing to the 4-bit paged key/value cache, reading it
// back, and evicting from it (layout: fa_kv4.cuh).
#include <cuda_runtime.h>

#include <climits>

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

__device__ int g_status_kv4 = 0;

__device__ __forceinline__ void report(int code) { atomicCAS(&g_status_kv4, 0, code); }

// ------------------------------------------------------------------ append
struct AppendParams {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    long long k_t, k_h, v_t, v_h;  // strides in elements
    Kv4Pages pages;
    const int* lengths;
    const int* cu_new;
    const void* positions;
    int pos64;
    const unsigned long long* freq;  // null: keys are stored as they come
    int R, interleaved;
    float amp;
    float* weights;       // [B][Hkv][slots] or null: zeroed at the new slots
    int* slot_positions;  // [B][Hkv][slots] or null: the tokens' positions
    long long slots;
    int B, total;
};

// Sequence of packed row t: the last b with cu[b] <= t, or -1.  `t` may differ
// between lanes; a few lookups in parallel for small batches, bisection above.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int t) {
    if (t < cu[0] || t >= cu[B]) return -1;
    if (B <= 16) {
        int b = 0;
#pragma unroll
        for (int i = 1; i < 16; ++i) b += i < B && cu[min(i, B)] <= t;
        return b;
    }
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Where a channel's partner in the rotation lies.
enum Rotation {
    kNone,         // keys are stored as they come
    kHalf,         // channels (i, i + R/2), R/2 a multiple of 8: the partners are another lane's
    kInterleaved,  // channels (2i, 2i + 1), R a multiple of 8: the thread's own
    kAny,          // any R: looked up one by one
};

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// Smallest and largest of a group's channels, 8 of them in `x`; NaN if one is.
template <int G>
__device__ __forceinline__ float2 range_of_group(const uint32_t (&x)[4]) {
    const __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(as_bf2(x[0]), as_bf2(x[1])), __hmin2_nan(as_bf2(x[2]), as_bf2(x[3])));
    const __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(as_bf2(x[0]), as_bf2(x[1])), __hmax2_nan(as_bf2(x[2]), as_bf2(x[3])));
    // (min, -max) in one word: one exchange a step serves both
    __nv_bfloat162 r = __halves2bfloat162(__hmin_nan(__low2bfloat16(lo2), __high2bfloat16(lo2)),
                                          __hneg(__hmax_nan(__low2bfloat16(hi2), __high2bfloat16(hi2))));
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) r = __hmin2_nan(r, as_bf2(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    return make_float2(__low2float(r), -__high2float(r));
}

// Two fp32 numbers in one register pair: one instruction works on both.
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two(uint64_t x) : v(x) {}
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ float2 both() const {
        float2 r;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
        return r;
    }
};
__device__ __forceinline__ Two operator*(Two a, Two b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ Two unpack(uint32_t x) {
    return Two(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(Two x) {
    const float2 f = x.both();
    return as_u32(__floats2bfloat162_rn(f.x, f.y));
}

// Quotient d / y, y of at most 8 significant bits and r within an ulp of 1 / y,
// rounded as the division rounds it: q = d r is off by an ulp or three,
// e = d - q y is exact, and q + e r differs from d / y by 2^-45 of it before its
// one rounding (Markstein's correction).  d / y is no midpoint of two fp32 numbers
// (a midpoint times y has more than d's 24 bits) and no nearer to one than 2^-33,
// so that rounding is the division's.  Ties of the codes rely on it: differences
// of bf16 numbers meet half steps often.
__device__ __forceinline__ Two quotient(Two d, Two minus_y, Two r) {
    const Two q = d * r;
    return fma2(fma2(q, minus_y, d), r, q);
}

// Codes of 8 channels, and the group's (s, m) pair.
__device__ __forceinline__ uint32_t quantise8(const uint32_t (&x)[4], float2 range, uint32_t& pair) {
    const float lo = range.x, span = __fsub_rn(range.y, lo);
    float s = __bfloat162float(__float2bfloat16_rn(
        quotient(Two(span, 0.f), Two(-15.f, -15.f), Two(1.f / 15.f, 1.f / 15.f)).both().x));
    if (s < 7.888609052210118e-31f) s = 0.f;  // 2^-100
    pair = as_u32(__floats2bfloat162_rn(s, lo));
    uint32_t word = 0;
    if (s > 0.f) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        const Two minus_lo(-lo, -lo), minus_s(-s, -s), rr(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // 1.5 2^23 more: the low bits are the nearest whole number, ties to even.
            // It is at most 15: s is span / 15 to 2^-9, so the quotient is below 15.1.
            const float2 c = (quotient(unpack(x[i]) + minus_lo, minus_s, rr) + Two(12582912.f, 12582912.f)).both();
            word += (__float_as_uint(c.x) << (8 * i)) + (__float_as_uint(c.y) << (8 * i + 4));
        }
        word -= 0x3f400000u;  // the eight shifted 0x4b400000, modulo 2^32
    }
    if (!(span <= 3.402823466e38f)) {
        pair = 0x7fff7fffu;  // NaN, NaN
        word = 0;
    }
    return word;
}

// A thread takes 8 channels of one token's keys and values in up to `heads_thread`
// heads: the angles are computed once for them, the G/8 threads of a group find
// its range with shuffles.  Bound: HBM, k and v once and the records.
template <int D, int G, int ROT>
__global__ void __launch_bounds__(256) fa_kv4_append_kernel(AppendParams p, int heads_thread) {
    using L = Kv4<D, G>;
    constexpr int kOct = D / 8;
    const int lane = threadIdx.x & 31;
    const int oct = threadIdx.x % kOct;
    const long long t_long = static_cast<long long>(blockIdx.x) * (256 / kOct) + threadIdx.x / kOct;
    const int t = static_cast<int>(t_long < p.total ? t_long : p.total - 1);
    const int b = sequence_of(p.cu_new, p.B, t);
    bool live = t_long < p.total && b >= 0;
    long long slot = 0, pos = 0;
    unsigned char* block = nullptr;
    if (live) {
        const int begin = p.cu_new[b], n = p.cu_new[b + 1] - begin;
        slot = static_cast<long long>(p.lengths[b]) - n + (t - begin);
        if (p.positions != nullptr)
            pos = p.pos64 ? static_cast<const long long*>(p.positions)[t]
                          : static_cast<long long>(static_cast<const int*>(p.positions)[t]);
        else
            pos = slot;
        if (slot < 0 || slot >= p.pages.capacity() || (p.slots != 0 && slot >= p.slots)) {
            report(kStatusBadSeqlen);
            live = false;
        } else {
            const long long at = p.pages.block_of(b, static_cast<int>(slot >> 4));
            if (at < 0) {
                report(kStatusBadPage);
                live = false;
            }
            block = p.pages.pool + at;
        }
    }
    // angles of this thread's channels: cos, and sin with the sign of the partner's term
    float cs[ROT == kInterleaved ? 4 : 8], sn[ROT == kInterleaved ? 4 : 8];
    const int half = p.R >> 1;
    const bool turned = ROT != kNone && oct * 8 < p.R;
    if constexpr (ROT != kNone) {
        if (turned) {
            constexpr int N = ROT == kInterleaved ? 4 : 8;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = oct * 8 + i;  // channel (the pair, where interleaved)
                int pair = c < half ? c : c - half;
                bool first = c < half;
                if constexpr (ROT == kInterleaved) {
                    pair = oct * 4 + i;
                    first = true;
                } else if (ROT == kAny && p.interleaved) {
                    pair = c >> 1;
                    first = (c & 1) == 0;
                }
                if (ROT == kAny && c >= p.R) continue;
                rope_angle(pos, p.freq[pair], p.amp, cs[i], sn[i]);
                if (!first) sn[i] = -sn[i];
            }
        }
    }
    const int r = static_cast<int>(slot & 15), g = oct >> 2, j = oct & 3;
    const int h1 = min(p.pages.heads, (static_cast<int>(blockIdx.y) + 1) * heads_thread);
    const int h0 = blockIdx.y * heads_thread;
    const __nv_bfloat16* krow = p.k + t * p.k_t + h0 * p.k_h;
    const __nv_bfloat16* vrow = p.v + t * p.v_t + h0 * p.v_h + oct * 8;
    block += h0 * p.pages.head_bytes() + r * L::kRow;
    uint4 kraw = *reinterpret_cast<const uint4*>(krow + oct * 8), vraw = *reinterpret_cast<const uint4*>(vrow);
    for (int h = h0; h < h1; ++h) {
        // the next head's rows are on their way while this one's are quantised
        uint4 knext = kraw, vnext = vraw;
        if (h + 1 < h1) {
            knext = *reinterpret_cast<const uint4*>(krow + p.k_h + oct * 8);
            vnext = *reinterpret_cast<const uint4*>(vrow + p.v_h);
        }
        uint32_t kx[4] = {kraw.x, kraw.y, kraw.z, kraw.w};
        const uint32_t vx[4] = {vraw.x, vraw.y, vraw.z, vraw.w};
        if constexpr (ROT == kHalf) {
            const int other = turned ? (oct * 8 < half ? oct + half / 8 : oct - half / 8) : oct;
            uint32_t y[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) y[w] = __shfl_sync(0xffffffffu, kx[w], lane - lane % kOct + other);
            if (turned) {
#pragma unroll
                for (int w = 0; w < 4; ++w)  // rope_turn of two channels
                    kx[w] = pack(fma2(unpack(kx[w]), Two(cs[2 * w], cs[2 * w + 1]),
                                      unpack(y[w]) * Two(-sn[2 * w], -sn[2 * w + 1])));
            }
        } else if constexpr (ROT == kInterleaved) {
            if (turned) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float a0 = __uint_as_float(kx[w] << 16), a1 = __uint_as_float(kx[w] & 0xffff0000u);
                    kx[w] = as_u32(__floats2bfloat162_rn(rope_turn(a0, a1, cs[w], sn[w]), rope_turn(a1, a0, cs[w], -sn[w])));
                }
            }
        } else if constexpr (ROT == kAny) {
            if (turned) {
                float z[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = oct * 8 + i;
                    z[i] = __bfloat162float(krow[c]);
                    if (c < p.R) {
                        const int other = p.interleaved ? c ^ 1 : (c < half ? c + half : c - half);
                        z[i] = rope_turn(z[i], __bfloat162float(krow[other]), cs[i], sn[i]);
                    }
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) kx[w] = as_u32(__floats2bfloat162_rn(z[2 * w], z[2 * w + 1]));
            }
        }
        uint32_t kpair, vpair;
        const uint32_t kw = quantise8(kx, range_of_group<G>(kx), kpair);
        uint32_t vw = quantise8(vx, range_of_group<G>(vx), vpair);
        // a value's 4 channels go to half-word r D/32 + g: even and odd slices meet in a word
        const uint32_t give = g & 1 ? vw & 0xffffu : vw >> 16;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
        vw = g & 1 ? got | (vw & 0xffff0000u) : (vw & 0xffffu) | got << 16;
        if (live) {
            reinterpret_cast<uint32_t*>(block + L::kKeyCodes)[j * (D / 32) + g] = kw;
            reinterpret_cast<uint32_t*>(block + L::kValueCodes)[((2 * j + (g & 1)) * (D / 32) + g) >> 1] = vw;
            if (oct % (G / 8) == 0) {
                unsigned char* to = block + r * (L::kScaleRow - L::kRow) + oct / (G / 8) * 4;
                *reinterpret_cast<uint32_t*>(to + L::kKeyScales) = kpair;
                *reinterpret_cast<uint32_t*>(to + L::kValueScales) = vpair;
            }
            if (oct == 0) {
                const long long at = (static_cast<long long>(b) * p.pages.heads + h) * p.slots + slot;
                if (p.weights != nullptr) p.weights[at] = 0.f;
                if (p.slot_positions != nullptr) p.slot_positions[at] = static_cast<int>(pos);
            }
        }
        krow += p.k_h;
        vrow += p.v_h;
        block += p.pages.head_bytes();
        kraw = knext;
        vraw = vnext;
    }
}

// ------------------------------------------------------------------ read
struct ReadParams {
    Kv4Pages pages;
    const int* lengths;
    const int* start;  // null: 0
    __nv_bfloat16* k;
    __nv_bfloat16* v;
    int B, count;
};

// One thread restores 8 channels of the keys and values of kTokensThread tokens.
// Bound: HBM, mostly the writes.
constexpr int kTokensThread = 4;
template <int D, int G>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(ReadParams p) {
    using L = Kv4<D, G>;
    constexpr int kOct = D / 8, kRows = 256 / kOct;
    const int oct = threadIdx.x % kOct, g = oct >> 2, j = oct & 3;
    const int bh = blockIdx.y, b = bh / p.pages.heads, h = bh - b * p.pages.heads;
    const int len = p.lengths[b], start = p.start != nullptr ? p.start[b] : 0;
    const int i0 = blockIdx.x * (kRows * kTokensThread) + threadIdx.x / kOct;
    const unsigned char* block[kTokensThread];
    uint32_t kw[kTokensThread], vw[kTokensThread], ks[kTokensThread], vs[kTokensThread];
#pragma unroll
    for (int x = 0; x < kTokensThread; ++x) {
        const long long slot = static_cast<long long>(start) + i0 + x * kRows;
        block[x] = nullptr;
        if (i0 + x * kRows < p.count && slot < len) {
            if (slot < 0 || slot >= p.pages.capacity()) {
                report(kStatusBadSeqlen);
            } else {
                const long long at = p.pages.block_of(b, static_cast<int>(slot >> 4));
                if (at < 0) report(kStatusBadPage);
                else block[x] = p.pages.pool + at + h * p.pages.head_bytes();
            }
        }
    }
#pragma unroll
    for (int x = 0; x < kTokensThread; ++x) {
        const int r = (start + i0 + x * kRows) & 15, so = r * L::kScaleRow + oct / (G / 8) * 4;
        kw[x] = vw[x] = ks[x] = vs[x] = 0;
        if (block[x] != nullptr) {
            kw[x] = reinterpret_cast<const uint32_t*>(block[x] + L::kKeyCodes + r * L::kRow)[j * (D / 32) + g];
            vw[x] = reinterpret_cast<const uint32_t*>(block[x] + L::kValueCodes + r * L::kRow)[((2 * j + (g & 1)) * (D / 32) + g) >> 1];
            ks[x] = *reinterpret_cast<const uint32_t*>(block[x] + L::kKeyScales + so);
            vs[x] = *reinterpret_cast<const uint32_t*>(block[x] + L::kValueScales + so);
        }
    }
#pragma unroll
    for (int x = 0; x < kTokensThread; ++x) {
        // the word holds half-words of two slices: the other one's goes to the neighbour
        const uint32_t give = g & 1 ? vw[x] & 0xffffu : vw[x] >> 16;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 4);
        const uint32_t v = g & 1 ? got | (vw[x] & 0xffff0000u) : (vw[x] & 0xffffu) | got << 16;
        if (i0 + x * kRows >= p.count) continue;
        const long long out = (static_cast<long long>(bh) * p.count + i0 + x * kRows) * kOct + oct;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint32_t word = w ? v : kw[x];
            const float2 sm = kv4_scale(w ? vs[x] : ks[x]);
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                pk[e] = as_u32(__floats2bfloat162_rn(fmaf(static_cast<float>(word >> (8 * e) & 15u), sm.x, sm.y),
                                                     fmaf(static_cast<float>(word >> (8 * e + 4) & 15u), sm.x, sm.y)));
            __stcs(reinterpret_cast<uint4*>(w ? p.v : p.k) + out, make_uint4(pk[0], pk[1], pk[2], pk[3]));
        }
    }
}

// ------------------------------------------------------------------ evict
struct EvictParams {
    Kv4Pages pages;
    const int* lengths;
    const float* weights;       // [B][Hkv][slots]
    const int* slot_positions;  // [B][Hkv][slots]
    float* weights_out;
    int* positions_out;
    int* lengths_out;
    int* source;   // [B][Hkv][budget]
    int* holes;    // workspace: [B][Hkv][budget]
    int* n_holes;  // workspace: [B][Hkv]
    long long slots;
    int budget, recent;
};

constexpr int kEvictThreads = 1024;

// Rank of a slot: larger is kept first.  Recent tokens before all others, then
// by weight; a NaN weight counts as the least.
__device__ __forceinline__ uint32_t rank_of(float w, int pos, long long newest, int recent) {
    if (static_cast<long long>(pos) > newest - recent) return 0xffffffffu;
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int warp_inclusive(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Inclusive prefix sum over the block; `total` gets the whole sum.
__device__ __forceinline__ int block_inclusive(int x, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in_warp = warp_inclusive(x, lane);
    __syncthreads();
    if (lane == 31) warp_sums[warp] = in_warp;
    __syncthreads();
    if (warp == 0) warp_sums[lane] = warp_inclusive(warp_sums[lane], lane);
    __syncthreads();
    total = warp_sums[kEvictThreads / 32 - 1];
    return in_warp + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// One CTA per (sequence, head): the rank of the budget-th token by a radix
// select of 8 bits a pass, then the kept map.  Ties go to the lowest slot.
__global__ void __launch_bounds__(kEvictThreads) fa_kv4_select_kernel(EvictParams p) {
    __shared__ int hist[256];
    __shared__ int warp_sums[32];
    __shared__ long long s_newest;
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const long long bh = static_cast<long long>(b) * p.pages.heads + h;
    const float* w = p.weights + bh * p.slots;
    const int* pos = p.slot_positions + bh * p.slots;
    float* w_out = p.weights_out + bh * p.slots;
    int* pos_out = p.positions_out + bh * p.slots;
    int* source = p.source + bh * p.budget;
    int len = p.lengths[b];
    if (len < 0 || len > p.slots || len > p.pages.capacity()) {
        report(kStatusBadSeqlen);
        len = 0;
    }
    const int left = min(len, p.budget);
    if (h == 0 && tid == 0) p.lengths_out[b] = left;
    for (long long i = left + tid; i < p.slots; i += kEvictThreads) {
        w_out[i] = 0.f;
        pos_out[i] = -1;
    }
    for (int i = left + tid; i < p.budget; i += kEvictThreads) source[i] = -1;
    if (len <= p.budget) {
        for (int i = tid; i < left; i += kEvictThreads) {
            w_out[i] = w[i];
            pos_out[i] = pos[i];
            source[i] = i;
        }
        if (tid == 0) p.n_holes[bh] = 0;
        return;
    }
    // the newest position
    long long newest = LLONG_MIN;
    for (int i = tid; i < len; i += kEvictThreads) newest = max(newest, static_cast<long long>(pos[i]));
    if (tid == 0) s_newest = LLONG_MIN;
    __syncthreads();
    atomicMax(&s_newest, newest);
    if (tid == 0) {
        s_prefix = 0;
        s_need = p.budget;
    }
    __syncthreads();
    newest = s_newest;
    // threshold: the largest rank with at least `need` slots at or above it
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix;
        for (int i = tid; i < len; i += kEvictThreads) {
            const uint32_t r = rank_of(w[i], pos[i], newest, p.recent);
            if (shift == 24 || (r >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[r >> shift & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int need = s_need, d = 255;
            while (d > 0 && hist[d] < need) need -= hist[d--];
            s_need = need;
            s_prefix = prefix | static_cast<uint32_t>(d) << shift;
        }
        __syncthreads();
    }
    const uint32_t threshold = s_prefix;
    const int ties = s_need;  // slots of exactly the threshold that are kept, the first ones
    // one walk over the slots: every hole lies before the new length and every
    // kept token to be moved behind it, so the list of holes is complete when
    // the first mover takes its place from it
    int* holes = p.holes + bh * p.budget;
    int done_ties = 0, done_holes = 0, done_movers = 0;
    for (int base = 0; base < len; base += kEvictThreads) {
        const int i = base + tid;
        const bool in = i < len;
        const uint32_t r = in ? rank_of(w[i], pos[i], newest, p.recent) : 0u;
        const bool tie = in && r == threshold;
        int n_ties, n_holes, n_movers;
        const int tie_rank = block_inclusive(tie, warp_sums, n_ties) + done_ties;
        const bool kept = in && (r > threshold || (tie && tie_rank <= ties));
        const bool hole = in && i < left && !kept, mover = kept && i >= left;
        const int hole_at = block_inclusive(hole, warp_sums, n_holes) - 1 + done_holes;
        const int mover_at = block_inclusive(mover, warp_sums, n_movers) - 1 + done_movers;
        if (hole) holes[hole_at] = i;
        __syncthreads();
        if (kept) {
            const int to = mover ? holes[mover_at] : i;
            w_out[to] = w[i];
            pos_out[to] = pos[i];
            source[to] = i;
        }
        done_ties += n_ties;
        done_holes += n_holes;
        done_movers += n_movers;
    }
    if (tid == 0) p.n_holes[bh] = done_holes;
}

// Moves the records (codes and scales of key and value) of the movers into the
// holes.  All sources lie behind the new length and all holes before it, so no
// copy touches what another one reads.  One warp per record, 4 bytes a lane.
__global__ void __launch_bounds__(256) fa_kv4_move_kernel(EvictParams p, int D, int groups) {
    const int bh = blockIdx.y, lane = threadIdx.x & 31;
    const int b = bh / p.pages.heads, h = bh % p.pages.heads;
    const int n = p.n_holes[bh];
    const int row = D / 2, scale = groups * 4;
    const int half = 16 * (row + scale);
    for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += gridDim.x * 8) {
        const int to = p.holes[static_cast<long long>(bh) * p.budget + i];
        const int from = p.source[static_cast<long long>(bh) * p.budget + to];
        const long long at = p.pages.block_of(b, from >> 4), dt = p.pages.block_of(b, to >> 4);
        if (at < 0 || dt < 0) {
            if (lane == 0) report(kStatusBadPage);
            continue;
        }
        const unsigned char* src = p.pages.pool + at + h * p.pages.head_bytes();
        unsigned char* dst = p.pages.pool + dt + h * p.pages.head_bytes();
        const int words = (row + scale) / 4;  // of the key; as many of the value
        for (int x = lane; x < 2 * words; x += 32) {
            const int is_v = x >= words, y = is_v ? x - words : x;
            const int base = is_v * half;
            const int so = y < row / 4 ? base + (from & 15) * row + y * 4
                                       : base + 16 * row + (from & 15) * scale + (y - row / 4) * 4;
            const int to_off = y < row / 4 ? base + (to & 15) * row + y * 4
                                           : base + 16 * row + (to & 15) * scale + (y - row / 4) * 4;
            *reinterpret_cast<uint32_t*>(dst + to_off) = *reinterpret_cast<const uint32_t*>(src + so);
        }
    }
}

Kv4Pages pages_of(const Kv4Shape& c, void* pool, const int* table) {
    return kv4_pages(static_cast<unsigned char*>(pool), table, c.width, c.num_pages, c.Hkv, c.page_size, c.D, c.group);
}

int last_error() { return cudaGetLastError() == cudaSuccess ? 0 : -5; }

template <int D, int G>
int append(const AppendParams& p, int rot, dim3 grid, int per, cudaStream_t stream) {
    if (rot == kNone) fa_kv4_append_kernel<D, G, kNone><<<grid, 256, 0, stream>>>(p, per);
    else if (rot == kHalf) fa_kv4_append_kernel<D, G, kHalf><<<grid, 256, 0, stream>>>(p, per);
    else if (rot == kInterleaved) fa_kv4_append_kernel<D, G, kInterleaved><<<grid, 256, 0, stream>>>(p, per);
    else fa_kv4_append_kernel<D, G, kAny><<<grid, 256, 0, stream>>>(p, per);
    return last_error();
}

}  // namespace

int launch_kv4_append(const Kv4Shape& c, void* pool, const int* table, const void* k, const void* v, long long k_t,
                      long long k_h, long long v_t, long long v_h, const int* lengths, const int* cu_new, int total,
                      const void* positions, int pos64, const void* freq, int R, int interleaved, float amplitude,
                      float* weights, int* slot_positions, long long slots, cudaStream_t stream, int num_sms) {
    AppendParams p{};
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.k_t = k_t;
    p.k_h = k_h;
    p.v_t = v_t;
    p.v_h = v_h;
    p.pages = pages_of(c, pool, table);
    p.lengths = lengths;
    p.cu_new = cu_new;
    p.positions = positions;
    p.pos64 = pos64;
    p.freq = static_cast<const unsigned long long*>(freq);
    p.R = R;
    p.interleaved = interleaved;
    p.amp = amplitude;
    p.weights = weights;
    p.slot_positions = slot_positions;
    p.slots = slots;
    p.B = c.B;
    p.total = total;
    const int rot = freq == nullptr                            ? kNone
                    : interleaved ? (R % 8 == 0 ? kInterleaved : kAny)
                                  : (R % 16 == 0 ? kHalf : kAny);
    // up to 8 heads a thread, fewer while that leaves SMs without work
    const long long rows = (total + 256 / (c.D / 8) - 1) / (256 / (c.D / 8));
    int per = 8;
    while (per > 1 && rows * ((c.Hkv + per - 1) / per) < 4LL * num_sms) per >>= 1;
    const dim3 grid(static_cast<unsigned>(rows), (c.Hkv + per - 1) / per);
    if (c.D == 64) return c.group == 32 ? append<64, 32>(p, rot, grid, per, stream) : append<64, 64>(p, rot, grid, per, stream);
    return c.group == 32 ? append<128, 32>(p, rot, grid, per, stream) : append<128, 64>(p, rot, grid, per, stream);
}

int launch_kv4_read(const Kv4Shape& c, const void* pool, const int* table, const int* lengths, const int* start,
                    int count, void* k, void* v, cudaStream_t stream) {
    ReadParams p{};
    p.pages = pages_of(c, const_cast<void*>(pool), table);
    p.lengths = lengths;
    p.start = start;
    p.k = static_cast<__nv_bfloat16*>(k);
    p.v = static_cast<__nv_bfloat16*>(v);
    p.B = c.B;
    p.count = count;
    const int rows = 256 / (c.D / 8) * kTokensThread;
    const dim3 blocks((count + rows - 1) / rows, c.B * c.Hkv);
    if (c.D == 64) {
        if (c.group == 32) fa_kv4_read_kernel<64, 32><<<blocks, 256, 0, stream>>>(p);
        else fa_kv4_read_kernel<64, 64><<<blocks, 256, 0, stream>>>(p);
    } else {
        if (c.group == 32) fa_kv4_read_kernel<128, 32><<<blocks, 256, 0, stream>>>(p);
        else fa_kv4_read_kernel<128, 64><<<blocks, 256, 0, stream>>>(p);
    }
    return last_error();
}

size_t kv4_evict_workspace(int B, int Hkv, int budget) {
    return static_cast<size_t>(B) * Hkv * (static_cast<size_t>(budget) + 1) * 4;
}

int launch_kv4_evict(const Kv4Shape& c, void* pool, const int* table, const int* lengths, const float* weights,
                     const int* slot_positions, long long slots, int budget, int recent, float* weights_out,
                     int* positions_out, int* lengths_out, int* source, void* workspace, cudaStream_t stream,
                     int num_sms) {
    EvictParams p{};
    p.pages = pages_of(c, pool, table);
    p.lengths = lengths;
    p.weights = weights;
    p.slot_positions = slot_positions;
    p.weights_out = weights_out;
    p.positions_out = positions_out;
    p.lengths_out = lengths_out;
    p.source = source;
    p.slots = slots;
    p.budget = budget;
    p.recent = recent;
    const long long bh = static_cast<long long>(c.B) * c.Hkv;
    p.holes = static_cast<int*>(workspace);
    p.n_holes = p.holes + bh * budget;
    fa_kv4_select_kernel<<<dim3(c.Hkv, c.B), kEvictThreads, 0, stream>>>(p);
    if (last_error() != 0) return -5;
    // about 8 CTAs per SM over all heads
    long long per = (8LL * num_sms + bh - 1) / bh;
    const long long most = (budget + 7) / 8;
    if (per > most) per = most;
    fa_kv4_move_kernel<<<dim3(static_cast<unsigned>(per), static_cast<unsigned>(bh)), 256, 0, stream>>>(p, c.D,
                                                                                                        c.D / c.group);
    return last_error();
}

int kv4_cache_take_status() {
    int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_kv4, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_kv4, &z, sizeof(int)) != cudaSuccess) return -5;
    return h;
}

}  // namespace fa
