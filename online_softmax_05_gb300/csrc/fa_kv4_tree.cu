// fa_kv4_tree.cu -- attention of a tree of drafted tokens over the 4-bit paged cache.
//
// The last N slots of a sequence are the tree's places; place i sees the context
// before them, its ancestors and itself.  The rows of a key/value head (group x N) are
// many enough for the tensor cores' 128-row tiles, which want whole operands in shared memory, so
// the codes are unpacked there.  With k = s n + m and v = s n + m per group of channels
// (fa_kv4.cuh):
//   K   s (n - 8) has eleven bits, as many as fp16: with q in fp16 too (a row scaled by a power of
//       two to [2^8, 2^9): exact down to 2^-25 of its largest), S is what fp32 sums give,
//         S = q.(s (n - 8)) + sum_g (m_g + 8 s_g) sum(q_g),
//       the last as 16 more channels: m_g and 8 s_g against two fp16 pieces (22 bits) of
//       sum(q_g).  (One bf16 number for k would put 2^-9 into each product, 2e-3 into a score and so
//       into the log-sum-exp.)  One multiply-add makes a pair of products: 16 + n is the fp16
//       number 0x4c00 | n << 6, and s (16 + n) - 24 s is exact.
//       A tile that has a scale or minimum outside [2^-17, 2^11] goes as bf16 instead, in
//       two parts, s = sa + sb its upper and lower four bits: sa n and sb n have eight bits,
//       and the minima meet three bf16 pieces of sum(q_g).
//   V   s n + m rounded once to bf16, as P is: both average out over a row's tokens and
//       are at most the output's own rounding where one token has all the weight.
// Channels stay in the order of the codes' words; Q is stored in that order, and V's is
// undone when the outputs leave.
//
// Ranges.  In bf16 K is scaled by 2^-20, V always by 2^-24, undone in the scores' factor and at the
// end: no product or sum overflows for any bf16 numbers in the cache (128 products of 2^9 and 2^109).  A
// row of queries above 2^101 goes into bf16 less its power beyond, which the factor has no room for.  A token that a row does
// not see adds nothing whatever it holds: S is replaced, and a tree's value group that is NaN
// goes into the products as 0 and into the rows that see it at the end.
//
// Per CTA, 128 rows and tiles of 128 tokens: warps 0-3 softmax of a tile's first 64 tokens, 4-7 of
// its last, the rows' maxima exchanged through shared memory (in clocks a tile of 64 that way took
// 1950, three quarters of it waits and latencies: so 128); four warps fetch and unpack keys, four
// values (a thread a token, copying the bytes that it will use two tiles ahead); the last warp
// issues tcgen05.mma, S of the next tile beside the softmax of this.  Q is in tensor memory: from
// shared memory it would take half of that memory's cycles.
// A ragged batch is cut over the CTAs by fa_split.cuh.
//
// Measured: 8 trees of 32 places, 32 heads on 8, over 1 to 12345 tokens 52 to 54 us; 4 of 64 places, 32 heads on 4,
// over up to 8111 40 us; 8 places over 117 tokens 7.5.  Neither memory (14 % of the copy's rate)
// nor the tensor cores (20 % busy) bound it but the chain of a tile: wait for S, maximum, exchange, exponentials,
// P's store, O's rescaling.  Keys as two bf16 products of tiles of 64 tokens took 60 and 45 us.
// The 8 trees with 64 channels 40.5 us; with all tiles in two bf16 parts 65 us, 46 with 64 channels.  17 warps leave
// 96 registers a thread: 108 to 136 bytes of spill stores and 216 to 264 of loads by the form.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "fa_check.cuh"
#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_ptx.cuh"
#include "fa_split.cuh"
#include "fa_tree.cuh"
#include "fa_wait.cuh"

namespace fa {

static __device__ int g_status_kv4_tree;

namespace {

constexpr int kUnpackWarps = 8;  // half of them keys, half values
constexpr int kThreads = (8 + kUnpackWarps + 1) * 32;
constexpr int kMmaWarp = 8 + kUnpackWarps;
constexpr int kTok = 128;      // of a tile
constexpr int kRaw = 2;        // tiles of codes on their way
constexpr int kInfo = 8;       // tiles whose masks are held: more than can be between their unpacking and their softmax
constexpr int kUnitRows = 128;  // of a CTA
constexpr int kLeast = 3;      // tiles that are not worth cutting
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kKeyUnit = 0x1p-20f, kValueUnit = 0x1p-24f;

template <int D_, int G_>
struct TreeCfg : Kv4<D_, G_> {
    using L = Kv4<D_, G_>;
    static constexpr int kTile = kTok * D_ * 2;            // an operand tile of keys or values
    static constexpr int kKStage = kTile + kTok * 32;      // and 16 more channels a token of keys
    static constexpr int kKStages = D_ == 128 ? 3 : 4, kVStages = D_ == 128 ? 2 : 3;
    static constexpr int kVOff = kKStages * kKStage;
    static constexpr int kQOff = kVOff + kVStages * kTile;
    static constexpr int kQAug = 128 * 32;                 // of fp16, then of bf16
    static constexpr int kRawOff = kQOff + 2 * kQAug;
    static constexpr int kRawTile = kUnpackWarps * 32 * (L::kRow + L::kScaleRow);  // of all threads: a row's codes, scales
    static constexpr int kBarOff = kRawOff + kRaw * kRawTile;
    // k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2], pv_done, o_full, q_full, mma_done
    static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 4 + 4;
    static constexpr int kMlOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // [2][2][128] row maxima of a tile's halves, by its parity
    static constexpr int kTreeOff = kMlOff + 4 * 128 * 4;    // [64] ancestors
    static constexpr int kPoisonOff = kTreeOff + 64 * 8;     // [groups] places whose value group is NaN
    static constexpr int kMaskOff = kPoisonOff + 4 * 8;      // [tiles] tokens that are there
    static constexpr int kWideOff = kMaskOff + kInfo * 16;   // [tiles] whether it is in bf16
    static constexpr int kMiscOff = kWideOff + kInfo * 4;
    static constexpr int kSmemBytes = kMiscOff + 16 + sizeof(SplitItem) + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    static_assert(kSmemBytes > 114 * 1024, "one CTA an SM: it takes all of tensor memory");
    static_assert(kQOff >= 128 * D_ * 4, "the scaled rows go where the stages were");
    // TMEM: O, two tiles of S (P over their first half), Q in fp16 and in bf16
    static constexpr uint32_t kO = 0, kQ = 384, kQWide = 448;
    __device__ static constexpr uint32_t kS(int buf) { return 128u + 128u * buf; }
    static constexpr uint32_t kIdescWide = idesc_bf16_f32(128, kTok, false, false);
    static constexpr uint32_t kIdescS = kIdescWide & ~((7u << 7) | (7u << 10));  // operand formats 0: fp16
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D_, false, true);
};

struct TreeParams {
    const __nv_bfloat16* q;
    Kv4Pages pages;
    const int* lengths;
    const int* parents;
    __nv_bfloat16* o;
    float* lse;
    SplitPlan plan;
    SplitParts parts;
    int N, R, row_units;
    float sl2;
    unsigned long long timeout_ns;
    int inject;
};

__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
// a x + b of bf16 pairs, rounded once.
__device__ __forceinline__ uint32_t fma_pair(uint32_t a, uint32_t x, uint32_t b) {
    return as_u32(__hfma2(as_bf2(a), as_bf2(x), as_bf2(b)));
}
__device__ __forceinline__ uint32_t twice(float x) { return pack_bf16x2(x, x); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t fma_f16(uint32_t a, uint32_t x, uint32_t b) {
    const __half2 h = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ bool in_range(float x) { return x == 0.f || (fabsf(x) >= 0x1p-17f && fabsf(x) <= 0x1p11f); }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t addr, uint32_t (&x)[WORDS]) {
    if constexpr (WORDS == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[0]) : "r"(addr));
    if constexpr (WORDS == 2) asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(addr));
    if constexpr (WORDS == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(addr));
}
// 16-byte chunk of a row of 16 channels: rows of 32 bytes, 32-byte swizzle.
__device__ __forceinline__ uint32_t sw32_off(uint32_t row, uint32_t chunk) {
    return row * 32u + ((chunk ^ ((row >> 2) & 1u)) << 4);
}
// Descriptor of such a K-major tile: 8 rows are 256 bytes.
__device__ __forceinline__ SDesc sdesc_sw32(uint32_t saddr) {
    SDesc d = sdesc_make(saddr, 16, 256);
    d.hi = (d.hi & 0x1fffffffu) | (6u << 29);
    return d;
}

// Barrier of `threads` threads; whether a predicate holds in any of them.
__device__ __forceinline__ bool any_of(int barrier, int threads, bool x) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(x ? 1u : 0u), "r"(barrier), "r"(threads)
        : "memory");
    return any != 0;
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) fa_kv4_tree_kernel(TreeParams p) {
    using C = TreeCfg<D, G>;
    constexpr int KST = C::kKStages, VST = C::kVStages, NG = C::kGroups, S32 = D / 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_u32(smem), bars = base + C::kBarOff;
    auto k_full = [&](int s) { return bars + 8u * s; };
    auto k_empty = [&](int s) { return bars + 8u * (KST + s); };
    auto v_full = [&](int s) { return bars + 8u * (2 * KST + s); };
    auto v_empty = [&](int s) { return bars + 8u * (2 * KST + VST + s); };
    constexpr int kFirst = 2 * KST + 2 * VST;
    auto s_full = [&](int buf) { return bars + 8u * (kFirst + buf); };
    auto p_full = [&](int buf) { return bars + 8u * (kFirst + 2 + buf); };
    const uint32_t pv_done = bars + 8u * (kFirst + 4), o_full = pv_done + 8, q_full = pv_done + 16, mma_done = pv_done + 24;
    const uint32_t sQAug = base + C::kQOff, sQWide = sQAug + C::kQAug;
    auto sK = [&](int s) { return base + s * C::kKStage; };
    auto sV = [&](int s) { return base + C::kVOff + s * C::kTile; };
    float* ml = reinterpret_cast<float*>(smem + C::kMlOff);
    unsigned long long* tree = reinterpret_cast<unsigned long long*>(smem + C::kTreeOff);
    unsigned long long* poison = reinterpret_cast<unsigned long long*>(smem + C::kPoisonOff);
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + C::kMaskOff);
    volatile uint32_t* wides = reinterpret_cast<volatile uint32_t*>(smem + C::kWideOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    const WaitCtl ctl{abort_flag, &g_status_kv4_tree, p.timeout_ns};
    SplitItem* s_item = reinterpret_cast<SplitItem*>(smem + C::kMiscOff + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    wait_for_stream();
    auto length_of = [&](int b) {
        const int len = __ldg(p.lengths + b);
        if (len >= 0 && len <= p.pages.capacity() && (len == 0 || len >= p.N)) return len;
        atomicCAS(&g_status_kv4_tree, 0, kStatusBadSeqlen);
        return 0;
    };
    if (warp == 0) {
        const SplitItem it =
            split_item(p.plan, blockIdx.x, lane, [&](int b) { return (length_of(b) + kTok - 1) / kTok; });
        if (lane == 0) *s_item = it;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    const SplitItem item = *s_item;
    if (item.unit < 0) {  // more CTAs than pieces
        if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
        return;
    }
    const int b = item.b, ru = item.unit % p.row_units, hk = item.unit / p.row_units;
    const int bh = b * p.pages.heads + hk;
    const int row0 = ru * kUnitRows, rows = min(kUnitRows, p.R - row0);
    const int len = length_of(b), ctx = len - p.N;  // tokens, and those before the tree
    const int j0 = item.j0, n = item.n;             // this CTA's tiles

    const int active = (rows + 31) / 32;  // quarters of the tile that have rows
    if (tid == 0) {
        for (int s = 0; s < KST; ++s) {
            mbar_init(k_full(s), kUnpackWarps / 2);
            mbar_init(k_empty(s), 1);
        }
        for (int s = 0; s < VST; ++s) {
            mbar_init(v_full(s), kUnpackWarps / 2);
            mbar_init(v_empty(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 2);  // the products, and the word of the warp that has seen the masks
            mbar_init(p_full(t), 2 * active);
        }
        mbar_init(pv_done, 1);
        mbar_init(o_full, 1);
        mbar_init(q_full, 4);
        mbar_init(mma_done, 1);
        for (int g = 0; g < NG; ++g) poison[g] = 0;
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();

    // a softmax thread's row, state and what it sees of the tree
    const int half = warp >> 2 & 1, r = tid & 127;
    const int row = row0 + r;
    float m = -INFINITY, l = 0.f;
    unsigned long long sees = 0;
    const uint32_t lane_base = tmem + ((32u * (warp & 3)) << 16);

    if (warp >= 8 && warp < kMmaWarp) {
        // ------------------------------------------------------------ fetch and unpack
        constexpr int CH = C::kRow / 16;  // 16-byte chunks of a row of codes
        const int th = tid - 256, tok = th & (kTok - 1);
        auto unpack = [&](auto of_values) {
        constexpr bool is_v = decltype(of_values)::value;
        const uint32_t raw = base + C::kRawOff + th * C::kRow,
                       raw_scales = base + C::kRawOff + kUnpackWarps * 32 * C::kRow + th * C::kScaleRow;
        const int turn = (tok / (8 / CH)) % CH;  // the chunks' order in shared memory, against bank conflicts
        constexpr int section = is_v ? C::kValueCodes : C::kKeyCodes, scales = is_v ? C::kValueScales : C::kKeyScales;
        const int rowb = tok & 15;
        uint32_t here = 0;  // bit i: this thread's token is there in raw tile i
        // the table's entry for this thread's token of tile i, read a tile ahead of its use; and the block in that page
        const int* entries = p.pages.table + static_cast<long long>(b) * p.pages.width;
        int page = -1, inside = 0;
        auto look_up = [&](int i) {
            const int at = (j0 + i) * kTok + tok, block = at >> 4;
            if (i < n && at < len) {
                const int e = p.pages.shift >= 0 ? block >> p.pages.shift : block / p.pages.blocks_page;
                inside = block - e * p.pages.blocks_page;
                // (len is within the table)
                page = FA_CHECK(e >= 0 && e < p.pages.width, &g_status_kv4_tree, abort_flag) ? __ldg(entries + e) : -1;
            }
        };
        look_up(0);
        auto fetch = [&](int i) {
            if (i < n) {
                const int at = (j0 + i) * kTok + tok;
                const int slot = i % kRaw;
                here &= ~(1u << slot);
                if (at < len) {
                    if (page >= 0 && page < p.pages.num_pages) {
                        here |= 1u << slot;
                        const unsigned char* from =
                            p.pages.pool + (page * static_cast<long long>(p.pages.heads) + hk) * p.pages.head_bytes() +
                            inside * C::kBlock;
#pragma unroll
                        for (int c = 0; c < CH; ++c)
                            copy_async<16>(raw + slot * C::kRawTile + ((c ^ turn) << 4), from + section + rowb * C::kRow + c * 16);
                        copy_async<C::kScaleRow>(raw_scales + slot * C::kRawTile, from + scales + rowb * C::kScaleRow);
                    } else if (rowb == 0) {
                        atomicCAS(&g_status_kv4_tree, 0, kStatusBadPage);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            look_up(i + 1);
        };
        for (int i = 0; i < kRaw; ++i) fetch(i);
        int entry = 0;   // of the keys' ring: a tile in bf16 takes two
        bool ok = true;  // a wait that ran out: the keys' warps still meet at their barrier
        for (int j = 0; j < n; ++j) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 1) : "memory");
            const int slot = j % kRaw;
            const bool there = here >> slot & 1;
            uint32_t sc[NG];  // of a token that is not there 0: its codes, whatever they are, count for nothing
            load_words(raw_scales + slot * C::kRawTile, sc);
#pragma unroll
            for (int g = 0; g < NG; ++g) sc[g] = there ? sc[g] : 0u;
            // four words of codes at a time
            auto codes = [&](int chunk, uint32_t (&w)[4]) { load_words(raw + slot * C::kRawTile + ((chunk ^ turn) << 4), w); };
            if constexpr (!is_v) {
                bool fits = true;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float2 x = kv4_scale(sc[g]);
                    fits = fits && in_range(x.x) && in_range(x.y);
                }
                const bool wide = any_of(8, kTok, !fits);
                const uint32_t mask = __ballot_sync(0xffffffffu, there);
                if (lane == 0) masks[4 * (j % kInfo) + (tok >> 5)] = mask;
                if (tok == 0) wides[j % kInfo] = wide;
                auto leave = [&]() {  // the entry is written
                    fence_proxy_async_smem();
                    __syncwarp();
                    const bool kept_back = p.inject == 5 && blockIdx.x == 0 && entry == 0;  // a test's: waits run out
                    if (lane == 0 && !kept_back) mbar_arrive(k_full(entry % KST));
                    ++entry;
                };
                ok = ok && wait_warp(k_empty(entry % KST), ((entry / KST) & 1) ^ 1, ctl);
                if (!ok) continue;  // nothing more is fetched
                uint32_t stage = sK(entry % KST);
                uint32_t extra[8];  // the 16 more channels
                if (!wide) {
                    uint32_t s2[NG], c2[NG];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const float2 x = kv4_scale(sc[g]);
                        s2[g] = pack_f16(x.x, x.x);
                        c2[g] = pack_f16(-24.f * x.x, -24.f * x.x);
                    }
#pragma unroll
                    for (int chunk = 0; chunk < CH; ++chunk) {
                        uint32_t w[4];
                        codes(chunk, w);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = 4 * chunk + k, g = c % S32 * 32 / G;
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t x = e < 2 ? w[k] << (6 - 4 * e) : w[k] >> (4 * e - 6);
                                y[e] = fma_f16(s2[g], (x & 0x03c003c0u) | 0x4c004c00u, c2[g]);
                            }
                            st_shared_v4(stage + (c >> 3) * (kTok * 128) + sw128_off(tok, c & 7), y[0], y[1], y[2], y[3]);
                        }
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float2 x = g < NG ? kv4_scale(sc[g < NG ? g : 0]) : make_float2(0.f, 0.f);
                        extra[2 * g] = pack_f16(x.y, x.y);
                        extra[2 * g + 1] = pack_f16(8.f * x.x, 8.f * x.x);
                    }
                } else {
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) {
                        uint32_t s2[NG], c2[NG];
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const float s = kv4_scale(sc[g]).x, hi = __uint_as_float(__float_as_uint(s) & 0xfff00000u);
                            const float x = (part == 0 ? hi : s - hi) * kKeyUnit;
                            s2[g] = twice(x);
                            c2[g] = twice(x * -128.f);
                        }
#pragma unroll 1
                        for (int chunk = 0; chunk < CH; ++chunk) {
                            uint32_t w[4];
                            codes(chunk, w);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int c = 4 * chunk + k, g = (S32 == 4 ? k : k % 2) * 32 / G;
                                uint32_t y[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    y[e] = fma_pair(s2[g], ((w[k] >> (4 * e)) & 0x000f000fu) | 0x43004300u, c2[g]);
                                st_shared_v4(stage + (c >> 3) * (kTok * 128) + sw128_off(tok, c & 7), y[0], y[1], y[2], y[3]);
                            }
                        }
                        if (part == 0) {
                            leave();
                            ok = wait_warp(k_empty(entry % KST), ((entry / KST) & 1) ^ 1, ctl);
                            if (!ok) break;
                            stage = sK(entry % KST);
                        }
                    }
                    if (!ok) continue;
                    float c[16];  // the minima, three times each: they go with the second part
#pragma unroll
                    for (int e = 0; e < 16; ++e) c[e] = e < 3 * NG ? kv4_scale(sc[e < 3 * NG ? e / 3 : 0]).y * kKeyUnit : 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) extra[e] = pack_bf16x2(c[2 * e], c[2 * e + 1]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    st_shared_v4(stage + C::kTile + sw32_off(tok, h), extra[4 * h], extra[4 * h + 1], extra[4 * h + 2],
                                 extra[4 * h + 3]);
                leave();
            } else {
                if (!wait_warp(v_empty(j % VST), ((j / VST) & 1) ^ 1, ctl)) break;
                const uint32_t stage = sV(j % VST);
                float vs[NG], vm[NG];
                const int place = (j0 + j) * kTok + tok - ctx;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float2 x = kv4_scale(sc[g]);
                    vs[g] = x.x * kValueUnit;
                    vm[g] = x.y * kValueUnit;
                    if (place >= 0 && !(fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY)) {
                        // rows that do not see this token must not meet it as 0 x NaN
                        if (there) atomicOr(poison + g, 1ull << place);
                        vs[g] = vm[g] = 0.f;
                    }
                }
#pragma unroll
                for (int chunk = 0; chunk < CH; ++chunk) {
                    uint32_t w[4];
                    codes(chunk, w);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 4 * chunk + k, g0 = 2 * c % S32 * 32 / G, g1 = (2 * c + 1) % S32 * 32 / G;
                        const uint32_t s2 = pack_bf16x2(vs[g0], vs[g1]), m2 = pack_bf16x2(vm[g0], vm[g1]);
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t x = ((w[k] >> (4 * e)) & 0x000f000fu) | 0x43004300u;
                            y[e] = fma_pair(as_u32(__hsub2(as_bf2(x), as_bf2(0x43004300u))), s2, m2);
                        }
                        st_shared_v4(stage + (c >> 3) * (kTok * 128) + sw128_off(tok, c & 7), y[0], y[1], y[2], y[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_full(j % VST));
            }
            fetch(j + kRaw);  // over the codes just used
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        };
        if (th < kTok) unpack(std::false_type{});
        else unpack(std::true_type{});
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ matrix instructions
        const bool leader = elect_one_sync();
        const SDesc dK = sdesc_make(sK(0), 16, 1024), dV = sdesc_make(sV(0), kTok * 128, 1024),
                    dQA = sdesc_sw32(sQAug), dKA = sdesc_sw32(sK(0) + C::kTile);
        int entry = 0;  // of the keys' ring
        // S (+)= Q K^T of the next entry
        auto products = [&](uint32_t to, uint32_t q, uint32_t idesc, bool add, bool extra, uint32_t aug) {
            const uint32_t ko = entry % KST * (C::kKStage >> 4);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                if (leader)
                    mma_ts_d(to, tmem + q + 8 * s, dK, ko + (((s >> 2) * (kTok * 128) + (s & 3) * 32) >> 4), idesc,
                             add || s > 0);
            if (leader) {
                if (extra) mma_ss_d(to, dQA, aug, dKA, ko, idesc, 1);
                mma_commit(k_empty(entry % KST));
            }
            ++entry;
        };
        auto ready = [&]() -> bool {
            if (!wait_warp(k_full(entry % KST), (entry / KST) & 1, ctl)) return false;
            tc_fence_after();
            return true;
        };
        auto issue_s = [&](int j) -> bool {
            if (!ready()) return false;
            const uint32_t to = tmem + C::kS(j & 1);
            if (wides[j % kInfo]) {
                products(to, C::kQWide, C::kIdescWide, false, false, 0);
                if (!ready()) return false;
                products(to, C::kQWide, C::kIdescWide, true, true, C::kQAug >> 4);
            } else {
                products(to, C::kQ, C::kIdescS, false, true, 0);
            }
            if (leader) {
                mma_commit(s_full(j & 1));
                mbar_arrive(s_full(j & 1));
            }
            return true;
        };
        // S(j + 1) is computed beside the softmax of tile j; its buffer's P, of tile j - 1, has been multiplied
        if (n > 0 && wait_warp(q_full, 0, ctl) && issue_s(0)) {
            for (int j = 0; j < n; ++j) {
                const int st = j % VST, buf = j & 1;
                if (j + 1 < n && !issue_s(j + 1)) break;
                if (!wait_warp(v_full(st), (j / VST) & 1, ctl)) break;
                if (!wait_warp(p_full(buf), (j >> 1) & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < kTok / 16; ++s)
                    if (leader)
                        mma_ts_d(tmem + C::kO, tmem + C::kS(buf) + s * 8, dV, st * (C::kTile >> 4) + s * (2048 >> 4),
                                 C::kIdescPV, (j > 0 || s > 0) ? 1u : 0u);
                if (leader) {
                    mma_commit(pv_done);
                    mma_commit(v_empty(st));
                }
            }
        }
        if (leader) {
            mma_commit(o_full);
            mma_commit(mma_done);
            drain(mma_done, 0, ctl);  // before tensor memory is given back
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        float factor, wide_factor;  // of the scores' sums, in fp16 and in bf16
        {
            const bool there = row < row0 + rows;
            const uint4* from = reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(bh) * p.R + row) * D);
            auto chunk = [&](int c, float (&f)[8], float up) {
                const uint4 x = there ? __ldg(from + c) : make_uint4(0, 0, 0, 0);
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = __uint_as_float(y[e] << 16) * up;
                    f[2 * e + 1] = __uint_as_float(y[e] & 0xffff0000u) * up;
                }
            };
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                float f[8];
                chunk(c, f, 1.f);
#pragma unroll
                for (int e = 0; e < 8; e += 2) top = fmax3(top, fabsf(f[e]), fabsf(f[e + 1]));
            }
            const int ex = max(-100, min(127, static_cast<int>(__float_as_uint(top) >> 23) - 127));
            const float up = p.sl2 == 0.f ? 0.f : copysignf(__int_as_float((127 + 8 - ex) << 23), p.sl2);
            factor = p.sl2 == 0.f ? 1.f : fabsf(p.sl2) * __int_as_float((127 - 8 + ex) << 23);
            const float more = __int_as_float((127 + max(0, ex - 100)) << 23);  // of q in bf16
            wide_factor = factor * (1.f / kKeyUnit / more);
            if (half == 0) {
                float sum[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) sum[g] = 0.f;
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf) {
#pragma unroll
                    for (int wide = 0; wide < 2; ++wide) {
                        uint32_t x[32];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {  // the channels of the codes' word 8 hf + k, in its pairs
                            const int word = 8 * hf + k, c = word % S32 * 4 + word / S32;
                            float f[8];
                            chunk(c, f, wide ? up * more : up);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (wide == 0) sum[c * 8 / G] += f[e];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[4 * k + e] = wide ? pack_bf16x2(f[e], f[e + 4]) : pack_f16(f[e], f[e + 4]);
                        }
                        tmem_st32(lane_base + (wide ? C::kQWide : C::kQ) + 32 * hf, x);
                    }
                }
                float c[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) c[e] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float x = sum[g] * more;
                    c[3 * g] = __bfloat162float(__float2bfloat16_rn(x));
                    c[3 * g + 1] = __bfloat162float(__float2bfloat16_rn(x - c[3 * g]));
                    c[3 * g + 2] = x - c[3 * g] - c[3 * g + 1];
                }
                uint32_t a[8];  // fp16: two pieces against the minima, two against the steps
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float x = g < NG ? sum[g < NG ? g : 0] : 0.f, hi = __half2float(__float2half_rn(x));
                    a[2 * g] = a[2 * g + 1] = pack_f16(hi, x - hi);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    st_shared_v4(sQAug + sw32_off(r, h), a[4 * h], a[4 * h + 1], a[4 * h + 2], a[4 * h + 3]);
                    st_shared_v4(sQWide + sw32_off(r, h), pack_bf16x2(c[8 * h], c[8 * h + 1]),
                                 pack_bf16x2(c[8 * h + 2], c[8 * h + 3]), pack_bf16x2(c[8 * h + 4], c[8 * h + 5]),
                                 pack_bf16x2(c[8 * h + 6], c[8 * h + 7]));
                }
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            if (warp == 0) {
                unsigned long long up[2];
                tree_ancestors(p.parents + static_cast<size_t>(b) * p.N, p.N, lane, up);
                tree[lane] = up[0];
                tree[lane + 32] = up[1];
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (row < row0 + rows && len > 0) sees = tree[row % p.N];
        }
        const uint32_t tO = lane_base + C::kO + half * (D / 2);
        bool ok = true;  // a wait that ran out ends the loop of both halves at their next barrier
        for (int j = 0; j < n && (warp & 3) < active; ++j) {
            const int buf = j & 1;
            ok = ok && wait_warp(s_full(buf), (j >> 1) & 1, ctl);
            tc_fence_after();
            const uint32_t tS = lane_base + C::kS(buf);
            uint32_t sr[64];
            tmem_ld32(tS + 64 * half, sr);
            tmem_ld32(tS + 64 * half + 32, sr + 32);
            const int t0 = (j0 + j) * kTok + 64 * half;
            const uint32_t have0 = masks[4 * (j % kInfo) + 2 * half], have1 = masks[4 * (j % kInfo) + 2 * half + 1];
            const float scale = wides[j % kInfo] ? wide_factor : factor;
            tmem_ld_wait();
            reg_fence32(sr);
            reg_fence32(sr + 32);
            float* s = reinterpret_cast<float*>(sr);
            if (t0 + 64 > ctx || (have0 & have1) != 0xffffffffu) {
                // bit c: the row sees token t0 + c
                unsigned long long vis = t0 - ctx > 63 ? 0ull
                                         : t0 >= ctx   ? sees >> (t0 - ctx)
                                         : ctx - t0 >= 64 ? ~0ull
                                                          : (sees << (ctx - t0)) | ((1ull << (ctx - t0)) - 1);
                vis &= have0 | static_cast<unsigned long long>(have1) << 32;
                const uint32_t v0 = static_cast<uint32_t>(vis), v1 = static_cast<uint32_t>(vis >> 32);
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (!((c < 32 ? v0 : v1) >> (c & 31) & 1)) s[c] = -INFINITY;
            }
            float mx4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mx4[c] = fmaxf(s[c], s[c + 4]);
#pragma unroll
            for (int c = 8; c < 64; c += 8)
#pragma unroll
                for (int a = 0; a < 4; ++a) mx4[a] = fmax3(mx4[a], s[c + a], s[c + 4 + a]);
            float mx = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]) * scale;
            // with the other half's maximum; behind the barrier both have read S, and P may go over it
            ml[256 * buf + 128 * half + r] = mx;
            if (any_of(2 + (warp & 3), 64, !ok)) break;
            mx = fmaxf(mx, ml[256 * buf + 128 * (half ^ 1) + r]);
            const bool grows = j > 0 && mx > m;
            const float m_new = fmaxf(m, mx), alpha = grows ? ex2_approx(m - m_new) : 1.f;
            l *= alpha;
            m = m_new;
            const float ref = m == -INFINITY ? 0.f : -m;  // nothing seen yet
            const uint64_t f2x = f2(scale, scale), neg2 = f2(ref, ref);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                float x0, x1;
                f2_split(fma2(f2(s[2 * c], s[2 * c + 1]), f2x, neg2), x0, x1);
                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                sum[c & 1] = add2(sum[c & 1], f2(p0, p1));
                sr[c] = pack_bf16x2(p0, p1);
            }
            float s0, s1;
            f2_split(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            tmem_st32(tS + 32 * half, sr);
            if (__any_sync(0xffffffffu, grows)) {
                ok = wait_warp(pv_done, (j - 1) & 1, ctl);  // O holds the tiles before
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    tmem_ld32(tO + 32 * c, sr);
                    tmem_ld_wait();
                    reg_fence32(sr);
#pragma unroll
                    for (int e = 0; e < 32; ++e) sr[e] = __float_as_uint(__uint_as_float(sr[e]) * alpha);
                    tmem_st32(tO + 32 * c, sr);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(buf));
        }
        wait_warp(o_full, 0, ctl);
        tc_fence_after();
    }

    // ------------------------------------------------------------ join
    __syncthreads();
    const bool whole = item.pieces == 1;
    // this item's piece, and its unit's entry, lie inside the workspace
    const bool room = (whole || FA_CHECK(item.part >= 0 && item.part + item.k < p.parts.count, &g_status_kv4_tree,
                                         abort_flag)) &&
                      FA_CHECK(bh * p.row_units + ru < p.plan.B * p.plan.per_seq, &g_status_kv4_tree, abort_flag);
    if (warp < 8) ml[128 * half + r] = l;
    __syncthreads();
    if (warp < 8) {
        const float sum = ml[r] + ml[128 + r];
        const bool used = sees != 0 && sum != 0.f;  // a place without a token gives 0
        const float factor = used ? 1.f / sum * (1.f / kValueUnit) : 0.f;
        // rows times their factors, fp32, channels in their order; 16-byte chunks turned by the row
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const int at = half * (D / 64) + c;  // 32 columns
            uint32_t o[32];
            if (n > 0) {
                tmem_ld32(lane_base + C::kO + 32 * at, o);
                tmem_ld_wait();
                reg_fence32(o);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // half-word 2 (4 at + k) + h of the codes holds channels 32 g + 4 r' .. + 3
                    const int hw = 2 * (4 * at + k) + h, g = hw % S32, chunk = 8 * g + hw / S32;
                    const bool bad = (sees & poison[g * 32 / G]) != 0;
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = __uint_as_float(o[8 * k + 2 * e + h]) * factor;
                        y[e] = used && n > 0 ? __float_as_uint(bad ? __int_as_float(0x7fffffff) : x) : 0u;
                    }
                    st_shared_v4(base + r * (D * 4) + ((chunk ^ (r & (D / 4 - 1))) << 4), y[0], y[1], y[2], y[3]);
                }
        }
        if (row < row0 + rows && half == 0) {
            const float lse2 = used ? m + __log2f(sum) : -INFINITY;
            if (whole) p.lse[static_cast<size_t>(bh) * p.R + row] = lse2 * kLn2;
            else if (room) p.parts.lse[static_cast<size_t>(item.part + item.k) * p.parts.rows + row - row0] = lse2;
        }
    }
    if (p.parts.units != nullptr && tid == 0 && item.k == 0 && room)
        p.parts.units[bh * p.row_units + ru] = make_int2(item.part, item.pieces);
    __syncthreads();
    for (int i = tid; i < rows * (D / 8); i += kThreads) {
        const int rr = i / (D / 8), c = i % (D / 8);
        float x[8];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const float4 z =
                *reinterpret_cast<const float4*>(smem + rr * (D * 4) + (((2 * c + y) ^ (rr & (D / 4 - 1))) << 4));
            x[4 * y] = z.x;
            x[4 * y + 1] = z.y;
            x[4 * y + 2] = z.z;
            x[4 * y + 3] = z.w;
        }
        if (whole) {
            *reinterpret_cast<uint4*>(p.o + (static_cast<size_t>(bh) * p.R + row0 + rr) * D + c * 8) = make_uint4(
                pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        } else if (room) {
            float4* to = reinterpret_cast<float4*>(p.parts.o +
                                                   (static_cast<size_t>(item.part + item.k) * p.parts.rows + rr) * D + c * 8);
            to[0] = make_float4(x[0], x[1], x[2], x[3]);
            to[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int G>
int launch_t(const TreeParams& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed{0};
    auto kern = fa_kv4_tree_kernel<D, G>;
    if (!allow_shared_memory(kern, TreeCfg<D, G>::kSmemBytes, allowed)) return -5;
    return launch_chained(kern, dim3(p.plan.items), kThreads, TreeCfg<D, G>::kSmemBytes, stream, p);
}

struct TreeUnits {
    int row_units, rows;  // of a head; most rows of a unit
    long long units;
    SplitPlan plan;       // items == units: nothing is cut
};
TreeUnits units_of(const Kv4Shape& c, int Hq, int N, int num_sms) {
    TreeUnits u;
    const int R = Hq / c.Hkv * N;
    u.row_units = (R + kUnitRows - 1) / kUnitRows;
    u.rows = R < kUnitRows ? R : kUnitRows;
    u.units = static_cast<long long>(c.B) * c.Hkv * u.row_units;
    u.plan = split_plan(c.B, u.units, num_sms, kLeast, 4);
    // no sequence of the table has tiles enough to be cut: an item a unit
    if (static_cast<long long>(c.width) * c.page_size <= kLeast * kTok) u.plan.items = static_cast<int>(u.units);
    return u;
}

}  // namespace

size_t kv4_tree_workspace(const Kv4Shape& c, int Hq, int N, int num_sms) {
    const TreeUnits u = units_of(c, Hq, N, num_sms);
    return split_workspace(u.plan, u.rows, c.D);
}

int launch_kv4_tree(const Kv4Shape& c, const void* pool, const int* table, const int* lengths, const int* parents,
                    const void* q, void* o, float* lse, int Hq, int N, float scale, void* workspace, cudaStream_t stream,
                    const DebugKnobs& dbg, int num_sms) {
    const TreeUnits u = units_of(c, Hq, N, num_sms);
    TreeParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.pages = kv4_pages(static_cast<unsigned char*>(const_cast<void*>(pool)), table, c.width, c.num_pages, c.Hkv,
                        c.page_size, c.D, c.group);
    p.lengths = lengths;
    p.parents = parents;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.N = N;
    p.R = Hq / c.Hkv * N;
    p.row_units = u.row_units;
    p.plan = u.plan;
    p.parts = split_parts(workspace, u.plan, u.rows, c.D);
    p.sl2 = scale * kLog2e;
    p.timeout_ns = dbg.timeout_ns;
    p.inject = dbg.inject;
    const int rc = c.D == 64 ? (c.group == 32 ? launch_t<64, 32>(p, stream) : launch_t<64, 64>(p, stream))
                             : (c.group == 32 ? launch_t<128, 32>(p, stream) : launch_t<128, 64>(p, stream));
    if (rc != 0 || u.plan.items == u.units) return rc;
    SplitOut out{};
    out.o = {o, static_cast<long long>(Hq) * N * c.D, static_cast<long long>(N) * c.D, c.D};
    out.lse = lse;
    out.Hkv = c.Hkv;
    out.group = Hq / c.Hkv;
    out.T = N;
    out.R = p.R;
    out.row_units = u.row_units;
    out.unit_rows = kUnitRows;
    return launch_split_join(p.parts, out, c.B, c.D, u.plan.items, stream);
}

int kv4_tree_take_status() {
    int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_kv4_tree, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_kv4_tree, &z, sizeof(int)) != cudaSuccess) return -5;
    return h;
}

}  // namespace fa
