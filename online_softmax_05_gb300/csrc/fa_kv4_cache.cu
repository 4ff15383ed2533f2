// fa_kv4_cache.cu -- writing to the 4-bit paged key/value cache, reading it
// back, and evicting from it (layout: fa_kv4.cuh).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <climits>

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_rope.cuh"

namespace cg = cooperative_groups;

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
    float one;  // 1, from the host (see turn2)
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

// x c + y s, both products and the sum rounded.  The compiler makes one fused
// instruction of a packed product and a packed sum, though each is written to round to
// nearest: one in 70000 of the turned channels then became another bf16 number than the
// formula's.  A product times a 1 that it cannot know leaves it nothing to fuse, and
// takes as many instructions.
__device__ __forceinline__ Two turn2(Two x, Two y, Two c, Two s, Two one) { return fma2(x * c, one, y * s); }

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
    const float q15 = __fmul_rn(span, 1.f / 15.f);  // span / 15, as quotient() has it
    float s = __bfloat162float(__float2bfloat16_rn(__fmaf_rn(__fmaf_rn(-q15, 15.f, span), 1.f / 15.f, q15)));
    if (s < 7.888609052210118e-31f) s = 0.f;  // 2^-100
    pair = as_u32(__floats2bfloat162_rn(s, lo));
    uint32_t word = 0;
    if (s > 0.f) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        const Two minus_lo(-lo, -lo), minus_s(-s, -s), rr(r, r);
        uint32_t even[4], odd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // 1.5 2^23 more: the low byte is the nearest whole number, ties to even.
            // It is at most 15: s is span / 15 to 2^-9, so the quotient is below 15.1.
            const float2 c = (quotient(unpack(x[i]) + minus_lo, minus_s, rr) + Two(12582912.f, 12582912.f)).both();
            even[i] = __float_as_uint(c.x);
            odd[i] = __float_as_uint(c.y);
        }
        auto bytes = [](const uint32_t (&n)[4]) {
            return __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
        };
        word = bytes(even) + (bytes(odd) << 4);
    }
    if (!(span <= 3.402823466e38f)) {
        pair = 0x7fff7fffu;  // NaN, NaN
        word = 0;
    }
    return word;
}

// A thread takes 8 channels of one token's keys and values in up to `heads_thread`
// heads: the angles are computed once for them, the G/8 threads of a group find
// its range with shuffles.  Bound: its instructions (about 15 a channel) ahead of
// HBM: 31 k tokens of 8 heads, D = 128 (164 MB) take 51 us, 3.2 TB/s, with the ALUs
// 61 % busy and three of four issue slots used.  Angles for every head apart and
// IEEE divisions took 298 us; one fp32 at a time instead of two 67 us.
template <int D, int G, int ROT>
__global__ void __launch_bounds__(256) fa_kv4_append_kernel(AppendParams p, int heads_thread) {
    wait_for_stream();
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
        const long long len = p.lengths[b];
        slot = len - n + (t - begin);
        if (p.positions != nullptr)
            pos = p.pos64 ? static_cast<const long long*>(p.positions)[t]
                          : static_cast<long long>(static_cast<const int*>(p.positions)[t]);
        else
            pos = slot;
        // a sequence without room for all of its tokens stores none
        if (len < n || len > p.pages.capacity() || (p.slots != 0 && len > p.slots) || slot < 0 || slot >= len) {
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
    // in rope_turn (half layout: negated, as the product is added there)
    float cs[ROT == kInterleaved ? 4 : 8], sn[ROT == kInterleaved ? 4 : 8];
    const int half = p.R >> 1;
    const bool turned = ROT != kNone && oct * 8 < p.R;
    // the lane that holds this one's partner channels (half layout)
    const int partner = lane - lane % kOct + (!turned ? oct : oct * 8 < half ? oct + half / 8 : oct - half / 8);
    if constexpr (ROT == kHalf) {
        // the two lanes of eight pairs take the angles of four each
        const bool first = oct * 8 < half;
        const int pair = (first ? oct : oct - half / 8) * 8 + (first ? 0 : 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float c = 0.f, s = 0.f;
            if (turned) rope_angle(pos, p.freq[pair + i], p.amp, c, s);
            const float oc = __shfl_sync(0xffffffffu, c, partner), os = __shfl_sync(0xffffffffu, s, partner);
            cs[i] = first ? c : oc;
            cs[4 + i] = first ? oc : c;
            sn[i] = first ? -s : os;
            sn[4 + i] = first ? -os : s;
        }
    } else if constexpr (ROT != kNone) {
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
                } else if (p.interleaved) {
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
            uint32_t y[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) y[w] = __shfl_sync(0xffffffffu, kx[w], partner);
            if (turned) {
#pragma unroll
                for (int w = 0; w < 4; ++w)  // rope_turn of two channels
                    kx[w] = pack(turn2(unpack(kx[w]), unpack(y[w]), Two(cs[2 * w], cs[2 * w + 1]),
                                       Two(sn[2 * w], sn[2 * w + 1]), Two(p.one, p.one)));
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
                if (p.slot_positions != nullptr) {
                    const long long near = max(min(pos, static_cast<long long>(INT_MAX)), static_cast<long long>(INT_MIN));
                    if (near != pos) report(kStatusBadSeqlen);
                    p.slot_positions[at] = static_cast<int>(near);
                }
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

// s * code + m of 8 codes, two at a time in bf16: 128 + code is a bf16 number whose
// low bits are the code's, 128 comes off exactly, and the product and sum are
// rounded once.  (In fp32, a code at a time, the kernel was bound by its
// instructions: 42 us instead of 38 on 201 MB of output.)
__device__ __forceinline__ uint4 restore8(uint32_t word, uint32_t pair) {
    const __nv_bfloat162 s = as_bf2(__byte_perm(pair, 0, 0x1010)), m = as_bf2(__byte_perm(pair, 0, 0x3232));
    uint32_t r[4];  // channels (i, i + 4)
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = as_u32(__hfma2(__hsub2(as_bf2((word >> (4 * i) & 0x000f000fu) | 0x43004300u), as_bf2(0x43004300u)), s, m));
    return make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                      __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
}

// One thread restores 8 channels of the keys and values of kTokensThread tokens.
// Bound: HBM, mostly the writes: 201 MB out and 36 in take 38 us, 6.3 TB/s.
constexpr int kTokensThread = 4;
template <int D, int G>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(ReadParams p) {
    wait_for_stream();
    using L = Kv4<D, G>;
    constexpr int kOct = D / 8, kRows = 256 / kOct;
    const int oct = threadIdx.x % kOct, g = oct >> 2, j = oct & 3;
    const int bh = blockIdx.y, b = bh / p.pages.heads, h = bh - b * p.pages.heads;
    const int start = p.start != nullptr ? p.start[b] : 0;
    int len = p.lengths[b];
    if (len < 0 || len > p.pages.capacity() || start < 0) {  // the sequence counts as empty
        report(kStatusBadSeqlen);
        len = 0;
    }
    const int i0 = blockIdx.x * (kRows * kTokensThread) + threadIdx.x / kOct;
    const unsigned char* block[kTokensThread];
    uint32_t kw[kTokensThread], vw[kTokensThread], ks[kTokensThread], vs[kTokensThread];
#pragma unroll
    for (int x = 0; x < kTokensThread; ++x) {
        const long long slot = static_cast<long long>(start) + i0 + x * kRows;
        block[x] = nullptr;
        if (i0 + x * kRows < p.count && slot < len) {
            const long long at = p.pages.block_of(b, static_cast<int>(slot >> 4));
            if (at < 0) report(kStatusBadPage);
            else block[x] = p.pages.pool + at + h * p.pages.head_bytes();
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
        __stcs(reinterpret_cast<uint4*>(p.k) + out, restore8(kw[x], ks[x]));
        __stcs(reinterpret_cast<uint4*>(p.v) + out, restore8(v, vs[x]));
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
    int* movers;   // workspace: [B][Hkv][budget]
    long long slots;
    int budget, recent;
    int row, scale;   // bytes of a token's codes and scales
    int slots_shared; // slots whose weights and positions fit into a CTA's shared memory
};

constexpr int kEvictThreads = 1024, kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2 * kEvictThreads;
static_assert(kEvictWarps == 32 && kBins == 1 << 11, "the block's sums are scanned by one warp");
constexpr int kEvictCluster = 8;
constexpr uint32_t kProtected = 0xffffffffu;

// Order of the weights as whole numbers; a NaN weight counts as the least.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int2 warp_inclusive(int2 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) {
            v.x += x;
            v.y += y;
        }
    }
    return v;
}
// Sums over the warps before this one of a pair that each warp holds, and over the block.
__device__ __forceinline__ int2 warps_before(int2 v, int2* warp_sums, int2& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // the sums of the scan before are read
    if (lane == 0) warp_sums[warp] = v;
    __syncthreads();
    const int2 in = warp_inclusive(warp_sums[lane], lane);
    total = make_int2(__shfl_sync(0xffffffffu, in.x, 31), __shfl_sync(0xffffffffu, in.y, 31));
    return make_int2(__shfl_sync(0xffffffffu, in.x, warp) - v.x, __shfl_sync(0xffffffffu, in.y, warp) - v.y);
}

// One cluster per (sequence, head), each CTA a slice of the slots, whose weights
// and positions stay in shared memory.  A slot's rank is its weight's order, and
// above all others where it is protected; the rank of the budget-th token is found by a radix select over the
// range that the keys span, 11 bits of it a pass, with the CTAs' histograms summed
// through distributed shared memory; ties go to the lowest slots.  Every hole lies
// below the new length and every mover at or above it, so the n-th mover takes the
// n-th hole, no copy touches what another reads, and the moves run in any order.
// Bound: the latency of about ten dependent steps (passes, scans, cluster
// barriers, 2 to 4 us each), then the moves.  128 heads of up to 8191 slots to 2048
// take 36 us, 8 heads of 60007 to 8192 38 us; select and move as two kernels with
// one CTA a head took 92 and 242 us.
__global__ void __launch_bounds__(kEvictThreads) fa_kv4_evict_kernel(EvictParams p) {
    wait_for_stream();
    extern __shared__ int2 kept_here[];  // (weight's bits, position) of the slice
    __shared__ int hist[2][kBins];
    __shared__ int2 warp_sums[kEvictWarps];
    __shared__ int s_share[8];  // what the other CTAs of the cluster read
    __shared__ uint32_t s_lo, s_hi;
    __shared__ int s_need, s_all;
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    const int b = blockIdx.y, h = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31;
    const long long bh = static_cast<long long>(b) * p.pages.heads + h;
    const float* w = p.weights + bh * p.slots;
    const int* pos = p.slot_positions + bh * p.slots;
    float* w_out = p.weights_out + bh * p.slots;
    int* pos_out = p.positions_out + bh * p.slots;
    int* source = p.source + bh * p.budget;
    int* holes = p.holes + bh * p.budget;
    int len = p.lengths[b];
    if (len < 0 || len > p.slots || len > p.pages.capacity()) {
        report(kStatusBadSeqlen);
        len = 0;
    }
    const int left = min(len, p.budget), step = C * kEvictThreads, me = rank * kEvictThreads + tid;
    if (h == 0 && me == 0) p.lengths_out[b] = left;
    for (long long i = left + me; i < p.slots; i += step) {
        w_out[i] = 0.f;
        pos_out[i] = -1;
    }
    for (int i = left + me; i < p.budget; i += step) source[i] = -1;
    if (len <= p.budget) {
        for (int i = me; i < left; i += step) {
            w_out[i] = w[i];
            pos_out[i] = pos[i];
            source[i] = i;
        }
        return;  // whole cluster
    }
    const int slice = (len + C - 1) / C, s0 = min(rank * slice, len), n = min(len, s0 + slice) - s0;
    const bool shared = slice <= p.slots_shared;
    // sum or largest over the cluster's first CTAs of what each left in s_share[at]
    auto over_cluster = [&](int at, bool largest, int upto) -> int {
        const int mine = lane < upto ? cluster.map_shared_rank(s_share, lane)[at] : largest ? INT_MIN : 0;
        return largest ? __reduce_max_sync(0xffffffffu, mine) : __reduce_add_sync(0xffffffffu, mine);
    };
    int* movers = p.movers + bh * p.budget;
    if (tid < 8) s_share[tid] = tid == 0 || tid >= 6 ? INT_MIN : 0;
    __syncthreads();
    // ---- the slice, and the newest position
    int newest = INT_MIN;
#pragma unroll 8
    for (int i = tid; i < n; i += kEvictThreads) {
        const int2 x = make_int2(shared ? __float_as_int(w[s0 + i]) : 0, pos[s0 + i]);
        newest = max(newest, x.y);
        if (shared) kept_here[i] = x;
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) atomicMax(&s_share[0], newest);
    cluster.sync();
    // positions above it are protected
    const long long border = p.recent > 0 ? static_cast<long long>(over_cluster(0, true, C)) - p.recent : LLONG_MAX;
    auto slot_at = [&](int i) -> int2 {
        return shared ? kept_here[i] : make_int2(__float_as_int(w[s0 + i]), pos[s0 + i]);
    };
    auto key_at = [&](int i) -> uint32_t {
        const int2 x = slot_at(i);
        return static_cast<long long>(x.y) > border ? kProtected : key_of(__int_as_float(x.x));
    };
    // ---- how many are protected, and the range of the others' keys
    {
        int count = 0;
        uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll 4
        for (int i = tid; i < n; i += kEvictThreads) {
            const uint32_t k = key_at(i);
            if (k == kProtected) {
                ++count;
            } else {
                lo = min(lo, k);
                hi = max(hi, k);
            }
        }
        count = __reduce_add_sync(0xffffffffu, count);
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            atomicAdd(&s_share[1], count);
            // unsigned order as signed: the top bit flipped; the least as the largest of the complement
            atomicMax(&s_share[6], static_cast<int>(~lo ^ 0x80000000u));
            atomicMax(&s_share[7], static_cast<int>(hi ^ 0x80000000u));
        }
        cluster.sync();
    }
    uint32_t lo = ~(static_cast<uint32_t>(over_cluster(6, true, C)) ^ 0x80000000u);
    uint32_t hi = static_cast<uint32_t>(over_cluster(7, true, C)) ^ 0x80000000u;
    int need = p.budget - over_cluster(1, false, C);
    // ---- the rank of the last token kept: `need` more are taken from [lo, hi]
    uint32_t threshold = kProtected;
    int ties = p.budget;  // kept among those of exactly that rank
    bool take_all = false;  // every rank from it on is kept
    for (int pass = 0; need > 0; ++pass) {
        const int bits = 32 - __clz(hi - lo), shift = max(0, bits - 11);
        int* bin = hist[pass & 1];
        for (int i = tid; i < kBins; i += kEvictThreads) bin[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int i0 = 0; i0 < n; i0 += kEvictThreads) {
            const int i = i0 + tid;
            const uint32_t k = i < n ? key_at(i) : kProtected;
            const bool in = k != kProtected && k >= lo && k <= hi;
            const int at = in ? static_cast<int>((k - lo) >> shift) : -1;
            // equal weights come in stretches: one addition for a warp that agrees
            if (__all_sync(0xffffffffu, at == __shfl_sync(0xffffffffu, at, 0))) {
                if (lane == 0 && at >= 0) atomicAdd(&bin[at], 32);
            } else if (in) {
                atomicAdd(&bin[at], 1);
            }
        }
        cluster.sync();
        // bins from the top down, two a thread
        const int top = kBins - 2 - 2 * tid;
        int2 sum = make_int2(0, 0);
#pragma unroll
        for (int c = 0; c < kEvictCluster; ++c) {  // all on their way together; past C, this CTA's again
            const int2 x = *reinterpret_cast<const int2*>(cluster.map_shared_rank(bin, c < C ? c : rank) + top);
            sum.x += c < C ? x.x : 0;
            sum.y += c < C ? x.y : 0;
        }
        const int2 in = warp_inclusive(make_int2(sum.x + sum.y, 0), lane);
        int2 all;
        const int warp_sum = __shfl_sync(0xffffffffu, in.x, 31);
        int above = warps_before(make_int2(warp_sum, 0), warp_sums, all).x + in.x - sum.x - sum.y;
        const int part[2] = {sum.y, sum.x};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (above < need && need <= above + part[x]) {
                const uint32_t at = lo + (static_cast<uint32_t>(top + 1 - x) << shift);
                s_lo = at;
                s_hi = min(hi, at + ((1u << shift) - 1u));
                s_need = need - above;
                s_all = need == above + part[x];
            }
            above += part[x];
        }
        __syncthreads();
        lo = s_lo;
        hi = s_hi;
        need = s_need;
        // done with a bin of one rank, and with one that is kept whole
        if (shift == 0 || s_all) {
            threshold = lo;
            ties = shift == 0 ? need : INT_MAX;
            take_all = s_all;
            break;
        }
    }
    // ---- what is kept: each warp walks a stretch of the slice, 32 slots a step, with
    // running counts of ties, holes and movers before it
    const int warp = tid >> 5;
    const int stretch = ((n + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
    const int r0 = min(warp * stretch, n), r1 = min(r0 + stretch, n);
    const unsigned before = (1u << lane) - 1u;
    int2 sum;
    int tie0 = 0;
    if (!take_all) {
        int mine = 0;
        for (int i = r0; i < r1; i += 32)
            mine += __popc(__ballot_sync(0xffffffffu, i + lane < r1 && key_at(i + lane) == threshold));
        tie0 = warps_before(make_int2(mine, 0), warp_sums, sum).x;
        if (tid == 0) s_share[2] = sum.x;
        cluster.sync();
        tie0 += over_cluster(2, false, rank);
    }
    // f(slot, whether there is one, whether it is kept) for the stretch, the warp together
    auto walk = [&](auto f) {
        int tie = tie0;
        for (int i = r0; i < r1; i += 32) {
            const bool in = i + lane < r1;
            const uint32_t k = in ? key_at(i + lane) : 0u;
            bool keep = in && k >= threshold;
            if (!take_all) {
                const bool eq = in && k == threshold;
                const unsigned same = __ballot_sync(0xffffffffu, eq);
                if (eq) keep = tie + __popc(same & before) < ties;
                tie += __popc(same);
            }
            f(s0 + i + lane, in, keep);
        }
    };
    int2 mine = make_int2(0, 0);  // holes, movers
    walk([&](int slot, bool in, bool keep) {
        mine.x += __popc(__ballot_sync(0xffffffffu, in && !keep && slot < left));
        mine.y += __popc(__ballot_sync(0xffffffffu, keep && slot >= left));
    });
    int2 at = warps_before(mine, warp_sums, sum);
    if (tid == 0) {
        s_share[3] = sum.x;
        s_share[4] = sum.y;
    }
    cluster.sync();
    at.x += over_cluster(3, false, rank);
    at.y += over_cluster(4, false, rank);
    const int moves = over_cluster(4, false, C);
    walk([&](int slot, bool in, bool keep) {
        const bool hole = in && !keep && slot < left, mover = keep && slot >= left;
        const unsigned all_holes = __ballot_sync(0xffffffffu, hole), all_movers = __ballot_sync(0xffffffffu, mover);
        if (hole) holes[at.x + __popc(all_holes & before)] = slot;
        if (mover) movers[at.y + __popc(all_movers & before)] = slot;
        at.x += __popc(all_holes);
        at.y += __popc(all_movers);
        if (keep && slot < left) {
            const int2 x = slot_at(slot - s0);
            w_out[slot] = __int_as_float(x.x);
            pos_out[slot] = x.y;
            source[slot] = slot;
        }
    });
    cluster.sync();  // holes and movers are listed
    // ---- move the records: a lane finds the places of one, then 10 lanes (6 at
    // D = 64) copy one, 16 bytes each and a scale row, several records at a time
    const int codes = p.row / 16, parts = 2 * (codes + 1), at_once = 32 / parts;
    const int which = lane / parts, part = lane % parts;
    const int is_v = part > codes, y = is_v ? part - codes - 1 : part;
    const bool code = y < codes;
    const int size = code ? 16 : p.scale, pitch = code ? p.row : p.scale;
    unsigned char* pool = p.pages.pool + h * p.pages.head_bytes() + is_v * 16 * (p.row + p.scale) + (code ? y * 16 : 16 * p.row);
    const int warps = C * kEvictWarps, share = min(32, (moves + warps - 1) / warps);
    for (int m0 = (rank * kEvictWarps + warp) * share; m0 < moves; m0 += warps * share) {
        long long src = -1, dst = -1;  // of the record's block, its row in the low bits
        if (lane < share && m0 + lane < moves) {
            const int from = movers[m0 + lane], to = holes[m0 + lane];
            w_out[to] = w[from];
            pos_out[to] = pos[from];
            source[to] = from;
            src = p.pages.block_of(b, from >> 4);
            dst = p.pages.block_of(b, to >> 4);
            if (src < 0 || dst < 0) {
                report(kStatusBadPage);
                src = -1;
            } else {  // blocks are multiples of 128 bytes
                src |= from & 15;
                dst |= to & 15;
            }
        }
        constexpr int kFlight = 4;
        for (int x0 = 0; x0 < share; x0 += kFlight * at_once) {
            uint4 data[kFlight];
            unsigned char* to[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const int x = x0 + f * at_once + which;
                const long long sx = __shfl_sync(0xffffffffu, src, x & 31), dx = __shfl_sync(0xffffffffu, dst, x & 31);
                to[f] = nullptr;
                if (which < at_once && x < share && sx >= 0) {
                    const unsigned char* from = pool + (sx & ~15LL) + (sx & 15) * pitch;
                    to[f] = pool + (dx & ~15LL) + (dx & 15) * pitch;
                    if (size == 16) data[f] = *reinterpret_cast<const uint4*>(from);
                    else if (size == 8) data[f].x = reinterpret_cast<const uint2*>(from)->x, data[f].y = reinterpret_cast<const uint2*>(from)->y;
                    else data[f].x = *reinterpret_cast<const uint32_t*>(from);
                }
            }
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                if (to[f] == nullptr) continue;
                if (size == 16) *reinterpret_cast<uint4*>(to[f]) = data[f];
                else if (size == 8) *reinterpret_cast<uint2*>(to[f]) = make_uint2(data[f].x, data[f].y);
                else *reinterpret_cast<uint32_t*>(to[f]) = data[f].x;
            }
        }
    }
}

Kv4Pages pages_of(const Kv4Shape& c, void* pool, const int* table) {
    return kv4_pages(static_cast<unsigned char*>(pool), table, c.width, c.num_pages, c.Hkv, c.page_size, c.D, c.group);
}

template <int D, int G>
int append(const AppendParams& p, int rot, dim3 grid, int per, cudaStream_t stream) {
    void (*const kernels[4])(AppendParams, int) = {fa_kv4_append_kernel<D, G, kNone>, fa_kv4_append_kernel<D, G, kHalf>,
                                                   fa_kv4_append_kernel<D, G, kInterleaved>,
                                                   fa_kv4_append_kernel<D, G, kAny>};
    return launch_chained(kernels[rot], grid, 256, 0, stream, p, per);
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
    p.one = 1.f;
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
    const auto kernel = c.D == 64 ? (c.group == 32 ? fa_kv4_read_kernel<64, 32> : fa_kv4_read_kernel<64, 64>)
                                  : (c.group == 32 ? fa_kv4_read_kernel<128, 32> : fa_kv4_read_kernel<128, 64>);
    return launch_chained(kernel, blocks, 256, 0, stream, p);
}

size_t kv4_evict_workspace(int B, int Hkv, int budget) {
    return static_cast<size_t>(B) * Hkv * static_cast<size_t>(budget) * 8;
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
    p.holes = static_cast<int*>(workspace);
    p.movers = p.holes + static_cast<size_t>(c.B) * c.Hkv * budget;
    p.row = c.D / 2;
    p.scale = c.D / c.group * 4;
    // CTAs of a head: as many as run at once, with two thousand slots or more each,
    // and no fewer than hold the slots in shared memory.  (Clusters of 16 do not all
    // find room at once: 8 heads of 60007 slots took 95 us against 44 us with 8.)
    constexpr int kSlotsMost = 24 * 1024;  // 192 KB
    const long long heads = static_cast<long long>(c.B) * c.Hkv;
    int cluster = 1;
    while (cluster < kEvictCluster && (2 * cluster * heads <= num_sms && slots > 2048LL * cluster)) cluster *= 2;
    while (cluster < kEvictCluster && slots > static_cast<long long>(kSlotsMost) * cluster) cluster *= 2;
    const long long slice = (slots + cluster - 1) / cluster;
    p.slots_shared = static_cast<int>(slice <= kSlotsMost ? slice : 0);
    const int smem = p.slots_shared * 8;
    static std::atomic<unsigned long long> allowed;
    if (!allow_shared_memory(fa_kv4_evict_kernel, kSlotsMost * 8, allowed)) return -5;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(c.Hkv * cluster, c.B);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fa_kv4_evict_kernel, p) == cudaSuccess ? 0 : -5;
}

int kv4_cache_take_status() {
    int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_kv4, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_kv4, &z, sizeof(int)) != cudaSuccess) return -5;
    return h;
}

}  // namespace fa
