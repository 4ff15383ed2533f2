// fa_kv4_tree.cu -- attention of a tree of drafted tokens over the 4-bit paged cache.
//
// The last N slots of a sequence are the tree's places; place i sees the context
// before them, its ancestors and itself.  The rows of a key/value head (group x N) are
// many enough for the tensor cores' 128-row tiles, which want whole operands in shared memory, so
// the codes are unpacked there.  With k = s n + m and v = s n + m per group of channels
// (fa_kv4.cuh):
//   K   s = sa + sb, its upper and lower four bits of significand: sa n and sb n have
//       eight bits and are exact in bf16.  S = q.(sa n) + q.(sb n) + sum_g m_g sum(q_g), the
//       last as 16 more channels: m_g against three bf16 pieces (24 bits) of sum(q_g).
//       Every operand is exact; S is what fp32 sums give.  (One bf16 number for k would put
//       2^-9 into each product, 2e-3 into a score and so into the log-sum-exp.)
//   V   s n + m rounded once to bf16, as P is: both average out over a row's tokens and
//       are at most the output's own rounding where one token has all the weight.
// One packed multiply-add makes two products: 128 + n is the bf16 number 0x4300 | n, and
// sa (128 + n) - 128 sa is exact.  Channels stay in the order of the codes' words; Q is stored
// in that order, and V's is undone when the outputs leave.
//
// Ranges.  Rows of q are scaled by a power of two to [1, 2), K by 2^-16 and V by 2^-24, undone in the
// row's score factor and at the end: no product or sum overflows for any bf16 numbers in the cache.
// A token that a row does not see adds nothing whatever it holds: S is replaced, and a tree's value
// group that is NaN goes into the products as 0 and into the rows that see it at the end.
//
// Per CTA, 128 rows: warps 0-3 softmax of a tile's first 32 tokens, 4-7 of its last, the rows' maxima
// exchanged through shared memory; two teams of four warps fetch and unpack tiles of 64 tokens
// in turn (a thread a token's keys or values, copying the bytes that it will use four tiles ahead);
// the last warp issues tcgen05.mma.  sa n and sb n lie side by side as 128 columns of one
// product, added by the softmax warps: an instruction of 64 columns takes as long as one of 128.  Q
// is in tensor memory: from shared memory it would take half of that memory's cycles.
// A ragged batch is cut over the CTAs by fa_split.cuh.
#include <cuda_runtime.h>

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

constexpr int kTeams = 2;       // of four unpacking warps, a tile each in turn
constexpr int kUnpackWarps = 4 * kTeams;
constexpr int kThreads = (8 + kUnpackWarps + 1) * 32;
constexpr int kMmaWarp = 8 + kUnpackWarps;
constexpr int kTok = 64;       // of a tile
constexpr int kRaw = 2;        // tiles of codes on their way to a team
constexpr int kUnitRows = 128;  // of a CTA
constexpr int kLeast = 6;      // tiles that are not worth cutting
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kKeyUnit = 0x1p-16f, kValueUnit = 0x1p-24f;

template <int D_, int G_>
struct TreeCfg : Kv4<D_, G_> {
    using L = Kv4<D_, G_>;
    static constexpr int kTile = kTok * D_ * 2;            // an operand tile of keys or values
    static constexpr int kAugTile = kTok * 32;             // 16 more channels a token
    static constexpr int kStage = 3 * kTile + kAugTile;    // sa n, sb n, V, minima
    static constexpr int kStages = D_ == 128 ? 3 : 4;
    static constexpr int kQAug = 128 * 32;
    static constexpr int kQOff = kStages * kStage;
    static constexpr int kRawOff = kQOff + kQAug;
    static constexpr int kRawTile = kUnpackWarps * 32 * (L::kRow + L::kScaleRow);  // of all threads: a row's codes, scales
    static constexpr int kBarOff = kRawOff + kRaw * kRawTile;
    // full[], empty[], s_full[2], p_full[2], pv_done, o_full, q_full, mma_done
    static constexpr int kNumBars = 2 * kStages + 4 + 4;
    static constexpr int kMlOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // [2][2][128] row maxima of a tile's halves, by its parity
    static constexpr int kTreeOff = kMlOff + 4 * 128 * 4;    // [64] ancestors
    static constexpr int kPoisonOff = kTreeOff + 64 * 8;     // [groups] places whose value group is NaN
    static constexpr int kMaskOff = kPoisonOff + 4 * 8;      // [stages] tokens that are there
    static constexpr int kMiscOff = kMaskOff + kStages * 8;
    static constexpr int kSmemBytes = kMiscOff + 16 + sizeof(SplitItem) + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    static_assert(kSmemBytes > 114 * 1024, "one CTA an SM: it takes all of tensor memory");
    static_assert(kQOff >= 128 * D_ * 4, "the scaled rows go where the stages were");
    // TMEM: O, two tiles of S (sa n, sb n; P over the first 32 columns), Q
    static constexpr uint32_t kO = 0, kQ = 384;
    __device__ static constexpr uint32_t kS(int buf) { return 128u + 128u * buf; }
    static constexpr uint32_t kIdescS = idesc_bf16_f32(128, 2 * kTok, false, false);
    static constexpr uint32_t kIdescAug = idesc_bf16_f32(128, kTok, false, false);
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
};

__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
// a x + b of bf16 pairs, rounded once.
__device__ __forceinline__ uint32_t fma_pair(uint32_t a, uint32_t x, uint32_t b) {
    return as_u32(__hfma2(as_bf2(a), as_bf2(x), as_bf2(b)));
}
__device__ __forceinline__ uint32_t twice(float x) { return pack_bf16x2(x, x); }

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

// Barrier of two warps; whether a predicate holds in any of their threads.
__device__ __forceinline__ bool any_of_pair(int barrier, bool x) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(x ? 1u : 0u), "r"(barrier)
        : "memory");
    return any != 0;
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) fa_kv4_tree_kernel(TreeParams p) {
    using C = TreeCfg<D, G>;
    constexpr int ST = C::kStages, NG = C::kGroups, S32 = D / 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_u32(smem), bars = base + C::kBarOff;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (ST + s); };
    auto s_full = [&](int buf) { return bars + 8u * (2 * ST + buf); };
    auto p_full = [&](int buf) { return bars + 8u * (2 * ST + 2 + buf); };
    const uint32_t pv_done = bars + 8u * (2 * ST + 4), o_full = pv_done + 8, q_full = pv_done + 16, mma_done = pv_done + 24;
    const uint32_t sQAug = base + C::kQOff;
    auto sStage = [&](int s) { return base + s * C::kStage; };
    float* ml = reinterpret_cast<float*>(smem + C::kMlOff);
    unsigned long long* tree = reinterpret_cast<unsigned long long*>(smem + C::kTreeOff);
    unsigned long long* poison = reinterpret_cast<unsigned long long*>(smem + C::kPoisonOff);
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + C::kMaskOff);
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
        for (int s = 0; s < ST; ++s) {
            mbar_init(full(s), 4);
            mbar_init(empty(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
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
        constexpr int CH = C::kRow / 16, kWords = C::kRow / 4;  // 16-byte chunks and words of a row of codes
        const int th = tid - 256, team = th >> 7, tok = th & 63;
        const bool is_v = th >> 6 & 1;
        const uint32_t raw = base + C::kRawOff + th * C::kRow,
                       raw_scales = base + C::kRawOff + kUnpackWarps * 32 * C::kRow + th * C::kScaleRow;
        const int turn = (tok / (8 / CH)) % CH;  // the chunks' order in shared memory, against bank conflicts
        const int section = is_v ? C::kValueCodes : C::kKeyCodes, scales = is_v ? C::kValueScales : C::kKeyScales;
        const int rowb = tok & 15;
        const int mine = (n + kTeams - 1 - team) / kTeams;  // this team's tiles: team, team + kTeams, ..
        uint32_t here = 0;  // bit i: this thread's token is there in raw tile i
        // the table's entry for this thread's token of tile i, read a tile ahead of its use; and the block in that page
        const int* entries = p.pages.table + static_cast<long long>(b) * p.pages.width;
        int page = -1, inside = 0;
        auto look_up = [&](int i) {
            const int at = (j0 + team + kTeams * i) * kTok + tok, block = at >> 4;
            if (i < mine && at < len) {
                const int e = p.pages.shift >= 0 ? block >> p.pages.shift : block / p.pages.blocks_page;
                inside = block - e * p.pages.blocks_page;
                page = __ldg(entries + e);  // len is within the table
            }
        };
        look_up(0);
        auto fetch = [&](int i) {
            if (i < mine) {
                const int at = (j0 + team + kTeams * i) * kTok + tok;
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
        for (int i = 0; i < mine; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 1) : "memory");
            const int j = team + kTeams * i, slot = i % kRaw, st = j % ST;
            const bool there = here >> slot & 1;
            uint32_t w[kWords], sc[NG];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint32_t x[4];
                load_words(raw + slot * C::kRawTile + ((c ^ turn) << 4), x);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * c + e] = there ? x[e] : 0u;
            }
            load_words(raw_scales + slot * C::kRawTile, sc);
#pragma unroll
            for (int g = 0; g < NG; ++g) sc[g] = there ? sc[g] : 0u;
            fetch(i + kRaw);
            if (!wait_warp(empty(st), ((j / ST) & 1) ^ 1, ctl)) break;
            const uint32_t stage = sStage(st);
            if (!is_v) {
                uint32_t sa[NG], sb[NG], ca[NG], cb[NG];  // pairs: the parts of s, and -128 of them
                float mn[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float2 x = kv4_scale(sc[g]);
                    const float hi = __uint_as_float(__float_as_uint(x.x) & 0xfff00000u), lo = x.x - hi;
                    sa[g] = twice(hi * kKeyUnit);
                    sb[g] = twice(lo * kKeyUnit);
                    ca[g] = twice(hi * kKeyUnit * -128.f);
                    cb[g] = twice(lo * kKeyUnit * -128.f);
                    mn[g] = x.y * kKeyUnit;
                }
#pragma unroll
                for (int c = 0; c < kWords; ++c) {
                    const int g = c % S32 * 32 / G;
                    uint32_t ya[4], yb[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = ((w[c] >> (4 * e)) & 0x000f000fu) | 0x43004300u;
                        ya[e] = fma_pair(sa[g], x, ca[g]);
                        yb[e] = fma_pair(sb[g], x, cb[g]);
                    }
                    const uint32_t at = stage + (c >> 3) * (2 * kTok * 128) + sw128_off(tok, c & 7);
                    st_shared_v4(at, ya[0], ya[1], ya[2], ya[3]);
                    st_shared_v4(at + kTok * 128, yb[0], yb[1], yb[2], yb[3]);
                }
                // the minima, three times each: against the three pieces of sum(q_g)
                float c[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) c[e] = e < 3 * NG ? mn[e < 3 * NG ? e / 3 : 0] : 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    st_shared_v4(stage + 3 * C::kTile + sw32_off(tok, h), pack_bf16x2(c[8 * h], c[8 * h + 1]),
                                 pack_bf16x2(c[8 * h + 2], c[8 * h + 3]), pack_bf16x2(c[8 * h + 4], c[8 * h + 5]),
                                 pack_bf16x2(c[8 * h + 6], c[8 * h + 7]));
                const uint32_t mask = __ballot_sync(0xffffffffu, there);
                if (lane == 0) masks[2 * st + (tok >> 5)] = mask;
            } else {
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
                for (int c = 0; c < kWords; ++c) {
                    const int g0 = 2 * c % S32 * 32 / G, g1 = (2 * c + 1) % S32 * 32 / G;
                    const uint32_t s2 = pack_bf16x2(vs[g0], vs[g1]), m2 = pack_bf16x2(vm[g0], vm[g1]);
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x = ((w[c] >> (4 * e)) & 0x000f000fu) | 0x43004300u;
                        y[e] = fma_pair(as_u32(__hsub2(as_bf2(x), as_bf2(0x43004300u))), s2, m2);
                    }
                    st_shared_v4(stage + 2 * C::kTile + (c >> 3) * (kTok * 128) + sw128_off(tok, c & 7), y[0], y[1],
                                 y[2], y[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(st));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ matrix instructions
        const bool leader = elect_one_sync();
        const SDesc dK = sdesc_make(sStage(0), 16, 1024), dV = sdesc_make(sStage(0) + 2 * C::kTile, kTok * 128, 1024),
                    dQA = sdesc_sw32(sQAug), dKA = sdesc_sw32(sStage(0) + 3 * C::kTile);
        constexpr uint32_t kStage16 = C::kStage >> 4;
        auto issue_s = [&](int j) -> bool {
            const int st = j % ST, buf = j & 1;
            if (!wait_warp(full(st), (j / ST) & 1, ctl)) return false;
            tc_fence_after();
            const uint32_t to = tmem + C::kS(buf), ko = st * kStage16;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                if (leader)
                    mma_ts_d(to, tmem + C::kQ + 8 * s, dK, ko + (((s >> 2) * (2 * kTok * 128) + (s & 3) * 32) >> 4),
                             C::kIdescS, s > 0);
            if (leader) {
                mma_ss_d(to, dQA, 0, dKA, ko, C::kIdescAug, 1);
                mma_commit(s_full(buf));
            }
            return true;
        };
        // S(j + 1) is computed beside the softmax of tile j; its buffer's P, of tile j - 1, has been multiplied
        if (n > 0 && wait_warp(q_full, 0, ctl) && issue_s(0)) {
            for (int j = 0; j < n; ++j) {
                const int st = j % ST, buf = j & 1;
                if (j + 1 < n && !issue_s(j + 1)) break;
                if (!wait_warp(p_full(buf), (j >> 1) & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < kTok / 16; ++s)
                    if (leader)
                        mma_ts_d(tmem + C::kO, tmem + C::kS(buf) + s * 8, dV, st * kStage16 + s * (2048 >> 4), C::kIdescPV,
                                 (j > 0 || s > 0) ? 1u : 0u);
                if (leader) {
                    mma_commit(pv_done);
                    mma_commit(empty(st));
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
        float factor;
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
            const int ex = max(-100, min(100, static_cast<int>(__float_as_uint(top) >> 23) - 127));
            const float up = p.sl2 == 0.f ? 0.f : copysignf(__int_as_float((127 - ex) << 23), p.sl2);
            factor = p.sl2 == 0.f ? 1.f : fabsf(p.sl2) * __int_as_float((127 + ex) << 23) * (1.f / kKeyUnit);
            if (half == 0) {
                float sum[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) sum[g] = 0.f;
#pragma unroll
                for (int hf = 0; hf < D / 64; ++hf) {
                    uint32_t x[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // the channels of the codes' word 8 hf + k, in its pairs
                        const int word = 8 * hf + k, c = word % S32 * 4 + word / S32;
                        float f[8];
                        chunk(c, f, up);
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[c * 8 / G] += f[e];
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[4 * k + e] = pack_bf16x2(f[e], f[e + 4]);
                    }
                    tmem_st32(lane_base + C::kQ + 32 * hf, x);
                }
                float c[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) c[e] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    c[3 * g] = __bfloat162float(__float2bfloat16_rn(sum[g]));
                    c[3 * g + 1] = __bfloat162float(__float2bfloat16_rn(sum[g] - c[3 * g]));
                    c[3 * g + 2] = sum[g] - c[3 * g] - c[3 * g + 1];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    st_shared_v4(sQAug + sw32_off(r, h), pack_bf16x2(c[8 * h], c[8 * h + 1]),
                                 pack_bf16x2(c[8 * h + 2], c[8 * h + 3]), pack_bf16x2(c[8 * h + 4], c[8 * h + 5]),
                                 pack_bf16x2(c[8 * h + 6], c[8 * h + 7]));
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
            const int st = j % ST, buf = j & 1;
            // (full has completed: what the unpacking warps wrote is seen)
            ok = ok && wait_warp(s_full(buf), (j >> 1) & 1, ctl) && wait_warp(full(st), (j / ST) & 1, ctl);
            tc_fence_after();
            const uint32_t tS = lane_base + C::kS(buf);
            uint32_t sr[32], sb[32];
            tmem_ld32(tS + 32 * half, sr);
            tmem_ld32(tS + kTok + 32 * half, sb);
            const int t0 = (j0 + j) * kTok + 32 * half;
            const uint32_t have = masks[2 * st + half];
            tmem_ld_wait();
            reg_fence32(sr);
            reg_fence32(sb);
            float* s = reinterpret_cast<float*>(sr);
#pragma unroll
            for (int c = 0; c < 32; c += 2)
                f2_split(add2(f2(s[c], s[c + 1]), f2(__uint_as_float(sb[c]), __uint_as_float(sb[c + 1]))), s[c], s[c + 1]);
            if (t0 + 32 > ctx || have != 0xffffffffu) {
                // bit c: the row sees token t0 + c
                const unsigned long long vis = t0 >= ctx ? sees >> min(t0 - ctx, 63)
                                               : ctx - t0 >= 32 ? ~0ull
                                                                : (sees << (ctx - t0)) | ((1ull << (ctx - t0)) - 1);
                const uint32_t v = t0 - ctx > 63 ? 0u : static_cast<uint32_t>(vis) & have;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (!(v >> c & 1)) s[c] = -INFINITY;
            }
            float mx4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mx4[c] = fmaxf(s[c], s[c + 4]);
#pragma unroll
            for (int c = 8; c < 32; c += 8)
#pragma unroll
                for (int a = 0; a < 4; ++a) mx4[a] = fmax3(mx4[a], s[c + a], s[c + 4 + a]);
            float mx = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]) * factor;
            // with the other half's maximum; behind the barrier both have read S, and P may go over it
            ml[256 * buf + 128 * half + r] = mx;
            if (any_of_pair(2 + (warp & 3), !ok)) break;
            mx = fmaxf(mx, ml[256 * buf + 128 * (half ^ 1) + r]);
            const bool grows = j > 0 && mx > m;
            const float m_new = fmaxf(m, mx), alpha = grows ? ex2_approx(m - m_new) : 1.f;
            l *= alpha;
            m = m_new;
            const float ref = m == -INFINITY ? 0.f : -m;  // nothing seen yet
            const uint64_t f2x = f2(factor, factor), neg2 = f2(ref, ref);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                float x0, x1;
                f2_split(fma2(f2(s[2 * c], s[2 * c + 1]), f2x, neg2), x0, x1);
                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                sum[c & 1] = add2(sum[c & 1], f2(p0, p1));
                sr[c] = pack_bf16x2(p0, p1);
            }
            float s0, s1;
            f2_split(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            tmem_st16(tS + 16 * half, sr);
            if (__any_sync(0xffffffffu, grows)) {
                ok = wait_warp(pv_done, (j - 1) & 1, ctl);  // O holds the tiles before
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    tmem_ld32(tO + 32 * c, sb);
                    tmem_ld_wait();
                    reg_fence32(sb);
#pragma unroll
                    for (int e = 0; e < 32; ++e) sb[e] = __float_as_uint(__uint_as_float(sb[e]) * alpha);
                    tmem_st32(tO + 32 * c, sb);
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
            else p.parts.lse[static_cast<size_t>(item.part + item.k) * p.parts.rows + row - row0] = lse2;
        }
    }
    if (p.parts.units != nullptr && tid == 0 && item.k == 0)
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
        } else {
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
