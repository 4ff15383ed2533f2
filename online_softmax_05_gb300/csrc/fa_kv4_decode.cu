// fa_kv4_decode.cu -- attention of a few query rows over the 4-bit paged cache.
//
// With k = s n + m and v = s n + m per group g of channels (fa_kv4.cuh),
//   S_t = scale sum_g ( s_tg (q_g . n_tg) + m_tg sum(q_g) ),  P = softmax(S),
//   O_c = sum_t P_t s_tg n_tc + sum_t P_t m_tg.
// The scales never meet the matrix operands' elements: the codes go to the
// tensor cores as they are, K's scale multiplies the 16 x 8 tile of q . n, V's
// scale multiplies P before the second product.  K's minima, bf16 numbers, are a
// small product of their own with sum(q_g) in three bf16 pieces (24 bits); V's are
// fp32 sums.  P times V's scale is rounded to fp16 (2^-11, where bf16 would lose
// 2^-8 as much as the output's own rounding), in several bands of scales where they
// lie more than 2^14 apart (kLeast); everything else is fp32.
//
// Codes as fp16.  A nibble masked into the low bits of a 16-bit half is the
// fp16 subnormal n 2^-24 (bits 0-3) or n 2^-20 (bits 4-7), which the matrix
// instructions take exactly: one AND makes two operand elements, a shift by 8
// the other four of a word.  (Converting through exponent tricks costs a
// subtraction more per pair.)  q is scaled per row by a power of two into
// fp16's range (bf16 values stay exact down to 2^-28 of the row's largest), and
// the power goes into the row's score factor.
//
// Both products put the tokens or channels on the 16-row side and the query
// rows on the 8-column side (m16n8k16), which suits 1 to 8 rows per key/value
// head: S^T = K q^T, O^T = V^T P^T.  The channel order inside a row of codes is
// the fragments' own, so there is no shuffle on K; a pair of tokens of V meets
// with one byte permute, and P^T turns from accumulator to operand by movmatrix.
// tcgen05 would need the operands dequantised into shared memory (a write and
// a read of 4 times the cache's bytes) and uses 8 of its 128 rows.
//
// Bound: HBM, the cache's bytes once.  Each warp streams units of 32 or 64
// tokens through its own ring of shared memory with asynchronous copies (16 tokens
// of a head are contiguous), 8 warps per CTA and 2 CTAs per SM.  The units of all
// sequences and heads form one line that is cut evenly over the warps, so ragged
// lengths balance without the host knowing them.  A warp works alone: it writes
// the heads that lie wholly in its stretch, and at the end the CTA joins the
// pieces that its warps share, and a second kernel those that CTAs share.  (One
// head at a time per CTA, its warps joined after each, took 85 us instead of 52
// on 24 sequences of 1 to 8111 tokens, as a short head costs all warps a barrier
// and the latency of its queries.)
//
// Measured, with the launches: B=8 H=32 T=32768 D=128 (1.21 GB) 221 us, 5.5 TB/s,
// 81 % of the copy rate; the 24 sequences above with 8 heads of 4 query rows
// (115 MB) 41.5 us, 2.8 TB/s, of which 14 are a start (three dependent loads: lengths,
// table, tokens), the joins and the second kernel.  In D = 128, 8 rows and groups of 32
// registers spill (236 bytes; 464 with weights).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <type_traits>

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

__device__ int g_status_kv4_decode = 0;

__device__ __forceinline__ void report(int code) { atomicCAS(&g_status_kv4_decode, 0, code); }

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
// The exponent's reference is set this far above the largest score so far (log2
// units), so that it seldom moves again.
constexpr float kAhead = 4.f;
// P times a value scale goes to fp16 in units that put the largest scale at 2^12 or above and
// the largest P at 2^-4 or above.  While every scale so far is kLeast or more there, 2^-14
// of the largest or so, what fp16 cannot hold of a product is 2^-25, against the 2^-6 or more
// that the heaviest token adds to a row: 2^-11.5 for 32768 tokens, at random, as much as
// their rounding.  From a smaller scale on, the values go through the products in bands: each
// P times a scale in the first of them that brings it to kLeast, a further kBand (2^16) up
// each time, the accumulators in units as much smaller meanwhile; the bands reach down to
// scales 2^-110 of the largest.  (64 heads of 32768 tokens: 67.0 us without looking for such scales, 67.7
// with it; 126, 156 and 188 where two groups lie 2^18, 2^30 and 2^60 apart, 75 where the
// steps of one are all 0.)
constexpr float kLeast = 0.25f, kBand = 65536.f, kLastBand = 0x1p96f;
// Outputs of a piece are sums of P v, P up to 1: held 2^-24 times, so that 2^24 tokens
// of the largest bf16 values do not overflow.
constexpr float kPieceUnit = 0x1p-24f;
// Places on the line for a head's start, its queries' and first copies' latency
// and its outputs, in units of 32 or 64 tokens.  (1, 2, 3, 4: 45.0, 42.9, 42.1,
// 42.2 us on 24 ragged sequences, 47.4, 41.4, 41.1, 41.2 on 8 with 16 rows a head,
// 217.6, 217.1, 219.0, 219.5 on 8 long ones.)
constexpr int kStart = 2;
// Up to this many units a warp, a CTA takes a head by itself: it need not find its
// place on the line, and nothing is left to a second kernel (2 heads of 117 tokens:
// 8.4 us instead of 12.4; above, the line's finer cut is worth its joining).
constexpr int kByHead = 2;

struct DecParams {
    const __nv_bfloat16* q;
    Kv4Pages pages;
    const int* lengths;
    float2* part_o;   // [slot][NT][D/8][32] unnormalised output pairs, in the lanes' order
    float* part_ml;   // [slot][NT][2][8] running maximum (log2 units) and sum
    float* scores;    // [B Hkv][cap][RB NT 8] in log2 units, or null
    __nv_bfloat16* o;
    float* lse;
    const float* weights;
    float* weights_out;
    long long slots, cap;
    int B, R, RB, Tq, causal, n_cta;
    int by_head;  // a CTA takes one (sequence, head, row block) alone: nothing to join between CTAs
    float sl2;  // scale log2(e)
};

template <int D_, int G_, int NT_>
struct Cfg : Kv4<D_, G_> {
    using L = Kv4<D_, G_>;
    static constexpr int UB = D_ == 128 ? 2 : 4;    // blocks of 16 tokens in a unit
    static constexpr int kTokens = UB * 16;
    static constexpr int kUnitBytes = UB * L::kBlock;
    static constexpr int kWords = D_ / 32;          // 32-channel slices
    static constexpr int kPairs = D_ / 8;           // pairs of accumulators of a lane and row tile
    static constexpr int kRing = kStages * kUnitBytes;      // of a warp
    static constexpr int kPieceO = NT_ * kPairs * 32 * 8;   // a warp's outputs of one head, and
    static constexpr int kPiece = kPieceO + NT_ * 64;       // its running maxima and sums
    static_assert(kPiece <= kRing, "the last piece goes where the ring was");
    static constexpr int kSmem = kWarps * (kRing + kPiece);
};

// Length of sequence b, 0 (and a status) if the table or the accounts cannot hold it.
__device__ __forceinline__ int length_of(const DecParams& p, int b) {
    const int len = __ldcg(p.lengths + b);  // from L2: the joining kernel reads it before it has waited
    if (len < 0 || len > p.pages.capacity() || (p.weights_out != nullptr && len > p.slots)) {
        report(kStatusBadSeqlen);
        return 0;
    }
    return len;
}

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Places on the line that a head of sequence b takes.  (The whole line has fewer
// than 2^31: checked on the host for the table's capacity.)
template <int TOKENS>
__device__ __forceinline__ int places_of(int len) {
    return len > 0 ? (len + TOKENS - 1) / TOKENS + kStart : 0;
}
// Places of one head of all sequences, and of those before sequence `upto`; per warp.
template <int TOKENS>
__device__ __forceinline__ void count_places(const DecParams& p, int lane, int upto, int& all, int& before) {
    all = before = 0;
    for (int b = lane; b < p.B; b += 32) {
        const int n = places_of<TOKENS>(length_of(p, b));
        all += n;
        if (b < upto) before += n;
    }
    all = warp_sum(all);
    before = warp_sum(before);
}
// The line: every (sequence, head, row block) of n > 0 units takes n + kStart
// places, the first ones for the cost of starting it.  A warp's share of them.
__device__ __forceinline__ int share_of(const DecParams& p, int places) {
    const unsigned warps = static_cast<unsigned>(p.n_cta) * kWarps;
    return static_cast<int>(max((static_cast<unsigned>(places) + warps - 1) / warps, 1u));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// C = A B for bf16 A (16 x 16) and B (16 x 8), and for A (16 x 8) and B (8 x 8).
__device__ __forceinline__ void mma_bf16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes from global to shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^k as the product of two fp32 numbers, |k| <= 250.
__device__ __forceinline__ float2 pow2_parts(int k) {
    const int a = k / 2;
    return make_float2(__int_as_float((a + 127) << 23), __int_as_float((k - a + 127) << 23));
}

// The larger magnitude of each half; its sign means nothing.  A NaN gives way.
__device__ __forceinline__ uint32_t larger_of(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
// (2^14 / inv, 2^27 / inv), inv a power of two of 2^-112 to 2^114; the second at most 2^127.
__device__ __forceinline__ uint32_t range_of(float inv) {
    const uint32_t most = (268u << 7) - (__float_as_uint(inv) >> 16);
    return most | min(most + (13u << 7), 254u << 7) << 16;
}
__device__ __forceinline__ uint32_t smaller_of(uint32_t x, uint32_t y) {
    const __nv_bfloat162 r = __hmin2(as_bf2(x), as_bf2(y));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// N 32-bit words from shared memory in one load.
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&x)[N]) {
    static_assert(N == 1 || N == 2 || N == 4);
    if constexpr (N == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[0]) : "r"(addr));
    if constexpr (N == 2) asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(addr));
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(addr));
}

// A stretch of units of one (sequence, head, row block) inside a warp's share.
struct Segment {
    int b, hr;     // hr = head * RB + row block
    int u0, u1;    // units of the sequence
    int n, len;    // units and tokens of the sequence
};
// What a warp leaves to be joined.
struct Piece {
    int head;        // b * heads * RB + hr, or -1
    int first, last; // whether it holds the head's first and last unit
};

// Token of row r (0..7) of a fragment: any order serves, as K and V agree; this
// one puts neighbouring rows of K and the four rows of one V load on different
// halves of the banks.
__device__ __forceinline__ int token_of(int r) { return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1; }

template <int D, int G, int NT, bool SCORES>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) fa_kv4_decode_kernel(DecParams p) {
    using C = Cfg<D, G, NT>;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g4 = lane >> 2, j = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * C::kRing;
    // where piece y (0: a warp's first, 1: its last) of warp w is left
    auto piece_at = [&](int w, int y) -> unsigned char* {
        return smem + (y ? w * C::kRing : kWarps * C::kRing + w * C::kPiece);
    };
    __shared__ Piece s_piece[kWarps][2];
    const int HR = p.pages.heads * p.RB;

    wait_for_stream();
    if (lane == 0) s_piece[warp][0].head = s_piece[warp][1].head = -1;

    // this warp's share of the line; from place `skip` of its first head on
    Segment seg{0, 0, 0, 0, 0, 0};
    int left = 0;
    if (p.by_head) {
        seg.b = blockIdx.x / HR;
        seg.hr = blockIdx.x - seg.b * HR;
        seg.len = length_of(p, seg.b);
        seg.n = (seg.len + C::kTokens - 1) / C::kTokens;
        const int share = (seg.n + kWarps - 1) / kWarps;
        seg.u0 = min(seg.n, warp * share);
        seg.u1 = min(seg.n, seg.u0 + share);
        if (seg.n == 0) {  // no tokens
            const long long row = (static_cast<long long>(seg.b) * p.pages.heads + seg.hr / p.RB) * p.R + seg.hr % p.RB * NT * 8;
            const int rows = min(NT * 8, p.R - seg.hr % p.RB * NT * 8);
            for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads)
                reinterpret_cast<uint32_t*>(p.o + row * D)[i] = 0;
            if (threadIdx.x < rows) p.lse[row + threadIdx.x] = -INFINITY;
        }
    } else {
        int all, unused;
        count_places<C::kTokens>(p, lane, 0, all, unused);
        const int total = all * HR, share = share_of(p, total);
        const long long start = (blockIdx.x * static_cast<long long>(kWarps) + warp) * share;
        const int first = static_cast<int>(min(start, static_cast<long long>(total)));
        const int first_row = first / HR;  // the place's head ends behind this place of the one-head line
        int base = 0;                      // places of one head before the chunk of sequences
        for (int b0 = 0; b0 < p.B && first < total; b0 += 32) {
            const int b = b0 + lane;
            const int len = b < p.B ? length_of(p, b) : 0;
            const int n = places_of<C::kTokens>(len);
            int sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + sum > first_row);
            if (hit != 0) {
                const int src = __ffs(hit) - 1;
                const int places = __shfl_sync(0xffffffffu, n, src);
                const int rem = first - (base + __shfl_sync(0xffffffffu, sum, src) - places) * HR;
                seg.b = b0 + src;
                seg.len = __shfl_sync(0xffffffffu, len, src);
                seg.n = places - kStart;
                seg.hr = rem / places;
                const int place = rem - seg.hr * places;
                left = min(share, total - first);
                seg.u0 = max(place - kStart, 0);
                seg.u1 = min(seg.n, place + left - kStart);
                left -= min(left, places - place);
                break;
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    // the head after `s` and its places in what is left of the share; false at the end
    auto advance = [&](Segment& s) -> bool {
        if (left <= 0) return false;
        s.u0 = 0;
        if (++s.hr == HR) {
            s.hr = 0;
            do {
                if (++s.b >= p.B) return false;
                s.len = length_of(p, s.b);
                s.n = places_of<C::kTokens>(s.len) - kStart;
            } while (s.n < 0);
        }
        s.u1 = min(s.n, left - kStart);
        left -= min(left, s.n + kStart);
        return s.u1 > 0;
    };
    // a share may begin with the place of a head's start alone
    bool working = seg.u1 > seg.u0;
    if (!working && left > 0) working = advance(seg);

    // The next block to be copied, walked page by page, so that a table entry is
    // read once a page.  (Bulk copies, one per block and with a barrier per
    // stage, cost three times these instructions: their operands are uniform, so
    // two lanes' copies are a loop.)
    const int per_page = p.pages.blocks_page;
    const uint64_t policy = p.RB == 1 ? l2_policy_evict_first() : l2_policy_unchanged();
    int walk_left = 0, walk_in = 0, walk_head = 0;  // blocks left; block in the page; key/value head
    const int* walk_entry = nullptr;                // of that page; inside the sequence's row of the table while blocks are left
    const unsigned char* walk_from = nullptr;       // that block of the head, this lane's 16 bytes; null: no page
    auto look_up = [&]() {
        walk_from = nullptr;
        if (walk_left > 0) {
            const int page = *walk_entry;
            if (page >= 0 && page < p.pages.num_pages)
                walk_from = p.pages.pool + (page * static_cast<long long>(p.pages.heads) + walk_head) * p.pages.head_bytes() + lane * 16;
        }
    };
    auto walk_to = [&](const Segment& s) {
        const int block = s.u0 * C::UB, page = block / per_page;
        walk_left = (s.len + 15) / 16 - block;
        walk_in = block - page * per_page;
        walk_entry = p.pages.table + static_cast<long long>(s.b) * p.pages.width + page;
        walk_head = s.hr / p.RB;
        look_up();
        if (walk_from != nullptr) walk_from += walk_in * C::kBlock;
    };
    // copies a unit into a stage of this warp's ring; returns the blocks that have a page
    auto issue = [&](int stage) -> uint32_t {
        uint32_t valid = 0;
        uint32_t dst = ring + stage * C::kUnitBytes + lane * 16;
#pragma unroll
        for (int ub = 0; ub < C::UB; ++ub, dst += C::kBlock) {
            if (walk_left > 0) {
                if (walk_from != nullptr) {
                    valid |= 1u << ub;
#pragma unroll
                    for (int x = 0; x < C::kBlock; x += 512)
                        if (x + 512 <= C::kBlock || lane * 16 < C::kBlock - x) copy16(dst + x, walk_from + x, policy);
                    walk_from += C::kBlock;
                } else if (lane == 0) {
                    report(kStatusBadPage);
                }
                --walk_left;
                if (++walk_in == per_page) {
                    walk_in = 0;
                    ++walk_entry;
                    look_up();
                }
            }
        }
        return valid;
    };
    uint32_t masks = 0;  // 8 bits of each stage: its blocks with a page
    int stage = 0;       // of the next unit to be used
    // the first units of a segment; one group of copies per stage, empty or not
    auto prologue = [&](const Segment& s) {
        walk_to(s);
        masks = 0;
        stage = 0;
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            if (s.u0 + i < s.u1) masks |= issue(i) << (8 * i);
            copy_commit();
        }
    };
    const int tokA = token_of(g4), tokB = 8 + tokA;
    bool fresh = true;  // the first segment, whose copies are yet to be started
    while (working) {
        const int head = seg.hr / p.RB, rb = seg.hr % p.RB;
        const int bh = seg.b * p.pages.heads + head;
        const int row0 = rb * NT * 8;

        // ---- queries: operand fragments, group sums and score factors
        uint4 raw[NT][C::kWords];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = row0 + nt * 8 + g4;
#pragma unroll
            for (int w = 0; w < C::kWords; ++w) {
                raw[nt][w] = make_uint4(0, 0, 0, 0);
                if (row < p.R)
                    raw[nt][w] = *reinterpret_cast<const uint4*>(p.q + (static_cast<long long>(bh) * p.R + row) * D +
                                                                 32 * w + 8 * j);
            }
        }
        if (fresh) prologue(seg);  // while the queries are on their way
        uint32_t qf[NT][C::kWords][4];
        uint32_t qs[NT][(C::kGroups + 1) / 2];
        float factor[NT][2];
        uint32_t far = 0;  // rows whose scores take a further factor of 2^40: bit 4 row + tile
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            __nv_bfloat162 most = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::kWords; ++w) {
                const uint32_t word[4] = {raw[nt][w].x, raw[nt][w].y, raw[nt][w].z, raw[nt][w].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&word[e])));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) most = __hmax2_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float top = fmaxf(__low2float(most), __high2float(most));
            // 2^e <= top < 2^(e+1) goes to 2^14 (rows below 2^-113, to less)
            const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            const int up_e = min(14 - e, 127);
            const float up = p.sl2 == 0.f ? 0.f : copysignf(__int_as_float((up_e + 127) << 23), p.sl2);
            float group[C::kGroups];
#pragma unroll
            for (int g = 0; g < C::kGroups; ++g) group[g] = 0.f;
#pragma unroll
            for (int w = 0; w < C::kWords; ++w) {
                const uint32_t word[4] = {raw[nt][w].x, raw[nt][w].y, raw[nt][w].z, raw[nt][w].w};
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = __uint_as_float(word[i] << 16) * up;
                    x[2 * i + 1] = __uint_as_float(word[i] & 0xffff0000u) * up;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) group[w * 32 / G] += x[i];
                qf[nt][w][0] = pack_f16(x[0], x[4]);
                qf[nt][w][1] = pack_f16(x[1] * 0.0625f, x[5] * 0.0625f);
                qf[nt][w][2] = pack_f16(x[2], x[6]);
                qf[nt][w][3] = pack_f16(x[3] * 0.0625f, x[7] * 0.0625f);
            }
            // A positive factor: its sign went into q, and a scale of 0 made q zero.  (A row that is
            // not finite has a NaN among the pieces of its sums below, so that all of its scores
            // are, but for the tokens that it does not see.)
            float2 down = pow2_parts(24 - up_e);
            float back = p.sl2 == 0.f ? 1.f : fabsf(p.sl2) * down.x * down.y;
            const bool big = back > 0x1p100f;  // the factor alone might overflow where the score does not
            if (big) {
                down = pow2_parts(24 - 40 - up_e);
                back = fminf(fabsf(p.sl2) * down.x * down.y, FLT_MAX);
            }
            far |= (__ballot_sync(0xffffffffu, big) & 0x11111111u) << nt;
#pragma unroll
            for (int g = 0; g < C::kGroups; ++g) {
                float s = group[g];
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                s *= 5.9604644775390625e-8f;  // 2^-24, the codes' unit
                // the lane's piece of it: three bf16 pieces hold all 24 bits, lane j = 0, 1, 2 one each
                const float hi = __bfloat162float(__float2bfloat16_rn(s)), rest = s - hi;
                const float mid = __bfloat162float(__float2bfloat16_rn(rest));
                group[g] = j == 0 ? hi : j == 1 ? mid : j == 2 ? rest - mid : 0.f;
            }
            if constexpr (C::kGroups == 1) qs[nt][0] = pack_bf16x2(group[0], 0.f);
            else
#pragma unroll
                for (int g = 0; g < C::kGroups; g += 2) qs[nt][g / 2] = pack_bf16x2(group[g], group[g + 1]);
            factor[nt][0] = __shfl_sync(0xffffffffu, back, 8 * j);
            factor[nt][1] = __shfl_sync(0xffffffffu, back, 8 * j + 4);
        }
        const int all_see = p.causal ? seg.len - (p.Tq - 1) : seg.len;  // tokens every row sees

        float acc[NT][C::kWords][2][4];     // O^T: channels 32 w + 4 r + {0,1}, {2,3}
        float om[NT][C::kGroups][2], l[NT][2], ref[NT][2];
        // A row's outputs are held in units of 1 / inv, a power of two: 2^14 over one at or
        // above every value scale and 2^-13 of every minimum that the row saw (a group of two
        // bf16 numbers or more has a step above 2^-13 of its minimum, so that the minima of
        // flat groups alone take part).  P times a scale is then at most 2^14 and no sum
        // overflows, whatever bf16 numbers the cache stands for.  At the start, the format's
        // least scale's.  Rows differ in the units with tokens that some do not see only.
        float inv[NT][2];
        uint32_t range = range_of(0x1p114f);  // the scales and minima that inv is for, at most
        uint32_t lowest = 0x7f807f80u;        // the least step but 0 so far of this lane's share of them, in the low half
        float deepest = 1.f;  // the last band's factor; units take all bands from the first that needs another on
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int w = 0; w < C::kWords; ++w)
#pragma unroll
                for (int x = 0; x < 8; ++x) acc[nt][w][x >> 2][x & 3] = 0.f;
#pragma unroll
            for (int g = 0; g < C::kGroups; ++g) om[nt][g][0] = om[nt][g][1] = 0.f;
            l[nt][0] = l[nt][1] = 0.f;
            ref[nt][0] = ref[nt][1] = -INFINITY;
            inv[nt][0] = inv[nt][1] = 0x1p114f;
        }

        // One unit in the ring at `unit`.  some_hidden: a token of it is not there or not
        // seen by every row, its scales take several bands or a row a further factor.  The
        // other units have none of those tests, and return true, with nothing added, where
        // the scales take several bands.
        auto use = [&](auto some_hidden, uint32_t unit, uint32_t valid, int t0) -> bool {
            constexpr bool edge = decltype(some_hidden)::value;
            int seen[NT][2];  // tokens that a row sees
            if constexpr (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = row0 + nt * 8 + 2 * j + c;
                        seen[nt][c] = p.causal ? seg.len - (p.Tq - 1 - r % p.Tq) : seg.len;
                    }
            }
            // ---- S^T = K q^T
            float s[C::UB][NT][4];
#pragma unroll
            for (int ub = 0; ub < C::UB; ++ub) {
                const uint32_t blk = unit + ub * C::kBlock;
                uint32_t xa[C::kWords], xb[C::kWords], pa[C::kGroups], pb[C::kGroups];
                lds(blk + C::kKeyCodes + tokA * C::kRow + j * (C::kWords * 4), xa);
                lds(blk + C::kKeyCodes + tokB * C::kRow + j * (C::kWords * 4), xb);
                lds(blk + C::kKeyScales + tokA * C::kScaleRow, pa);
                lds(blk + C::kKeyScales + tokB * C::kScaleRow, pb);
                // the minima: sum_g m_tg sum(q_g), slots of the product: lane j's piece of the sums
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (C::kGroups == 1)
                        mma_bf16_zero(s[ub][nt], pa[0] >> 16, pb[0] >> 16, qs[nt][0]);
                    else if constexpr (C::kGroups == 2)
                        mma_bf16_zero(s[ub][nt], __byte_perm(pa[0], pa[1], 0x7632), __byte_perm(pb[0], pb[1], 0x7632),
                                      qs[nt][0]);
                    else
                        mma_bf16_zero(s[ub][nt], __byte_perm(pa[0], pa[1], 0x7632), __byte_perm(pb[0], pb[1], 0x7632),
                                      __byte_perm(pa[2], pa[3], 0x7632), __byte_perm(pb[2], pb[3], 0x7632), qs[nt][0],
                                      qs[nt][1]);
                }
#pragma unroll
                for (int g = 0; g < C::kGroups; ++g) {
                    float d[NT][4];
#pragma unroll
                    for (int w = g * (G / 32); w < (g + 1) * (G / 32); ++w) {
                        const uint32_t ya = xa[w] >> 8, yb = xb[w] >> 8;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (w == g * (G / 32))
                                mma_f16_zero(d[nt], xa[w] & 0x000f000fu, xb[w] & 0x000f000fu, xa[w] & 0x00f000f0u,
                                             xb[w] & 0x00f000f0u, qf[nt][w][0], qf[nt][w][1]);
                            else
                                mma_f16(d[nt], xa[w] & 0x000f000fu, xb[w] & 0x000f000fu, xa[w] & 0x00f000f0u,
                                        xb[w] & 0x00f000f0u, qf[nt][w][0], qf[nt][w][1]);
                            mma_f16(d[nt], ya & 0x000f000fu, yb & 0x000f000fu, ya & 0x00f000f0u, yb & 0x00f000f0u,
                                    qf[nt][w][2], qf[nt][w][3]);
                        }
                    }
                    const float sa = kv4_scale(pa[g]).x, sb = kv4_scale(pb[g]).x;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[ub][nt][c] = fmaf(c < 2 ? sa : sb, d[nt][c], s[ub][nt][c]);
                }
                if constexpr (edge) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (far >> (8 * j + 4 * (c & 1) + nt) & 1) s[ub][nt][c] *= 0x1p40f;
                    const bool here = valid >> ub & 1;
                    const int ta = t0 + ub * 16 + tokA, tb = ta + 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (!here || (c < 2 ? ta : tb) >= seen[nt][c & 1]) s[ub][nt][c] = -INFINITY;
                }
                if constexpr (SCORES) {
                    const int ta = t0 + ub * 16 + tokA, tb = ta + 8;
                    const int width = p.RB * NT * 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float* to = p.scores + (static_cast<long long>(bh) * p.cap + ta) * width + row0 + nt * 8 + 2 * j;
                        if (ta < seg.len)
                            *reinterpret_cast<float2*>(to) =
                                make_float2(s[ub][nt][0] * factor[nt][0], s[ub][nt][1] * factor[nt][1]);
                        if (tb < seg.len)
                            *reinterpret_cast<float2*>(to + 8LL * width) =
                                make_float2(s[ub][nt][2] * factor[nt][0], s[ub][nt][3] * factor[nt][1]);
                    }
                }
            }

            // ---- running maxima, of the value scales too
            // the value scales of a block's two tokens of this lane, 0 where no token is
            auto value_scales = [&](int ub, uint32_t (&va)[C::kGroups], uint32_t (&vb)[C::kGroups]) {
                const uint32_t blk = unit + ub * C::kBlock + C::kValueScales;
                lds(blk + tokA * C::kScaleRow, va);
                lds(blk + tokB * C::kScaleRow, vb);
                if constexpr (edge) {
                    const int ta = t0 + ub * 16 + tokA, tb = ta + 8;
#pragma unroll
                    for (int g = 0; g < C::kGroups; ++g) {
                        if (!(valid >> ub & 1) || ta >= seg.len) va[g] = 0;
                        if (!(valid >> ub & 1) || tb >= seg.len) vb[g] = 0;
                    }
                }
            };
            // what the outputs' unit goes by, the largest of a row's (s, 2^-13 m), and the least s
            auto size_of = [](uint32_t pair) {
                const float2 x = kv4_scale(pair);
                return fmaxf(fabsf(x.x), fabsf(x.y) * 0x1p-13f);
            };
            auto step_of = [](uint32_t pair) {  // a step of 0 adds nothing (2^-100 is the format's least)
                const float s = kv4_scale(pair).x;
                return s >= 0x1p-101f ? s : INFINITY;
            };
            auto pair_of_step = [](float s) { return __float_as_uint(s) >> 16 | 0x7f800000u; };
            float vtop[NT][2];
            uint32_t least = 0;
            bool more = false;  // the scales leave the range that the outputs' unit is for
            if constexpr (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) vtop[nt][c] = 0.f;
                float low = step_of(lowest);
#pragma unroll 1
                for (int ub = 0; ub < C::UB; ++ub) {
                    uint32_t v[2][C::kGroups];
                    value_scales(ub, v[0], v[1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t most = 0;
#pragma unroll
                        for (int g = 0; g < C::kGroups; ++g) {
                            most = larger_of(most, v[x][g]);
                            low = fminf(low, step_of(v[x][g]));
                        }
                        const float top = size_of(most);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (t0 + ub * 16 + tokA + 8 * x < seen[nt][c]) vtop[nt][c] = fmaxf(vtop[nt][c], top);
                    }
                }
                lowest = pair_of_step(low);
            } else {  // every row sees every token: the lanes share the unit's pairs
                constexpr int kBlocks = C::kGroups == 1 ? 2 : 1;  // a load's
                constexpr int kPairs = 16 * C::kGroups * kBlocks / 32;
                const uint32_t at = unit + C::kValueScales +
                                    (kBlocks == 2 ? (lane >> 4) * C::kBlock + (lane & 15) * 4 : lane * (4 * kPairs));
                uint32_t most = 0;
                least = lowest;  // and steps of 0
#pragma unroll
                for (int ub = 0; ub < C::UB; ub += kBlocks) {
                    uint32_t pairs[kPairs];
                    lds(at + ub * C::kBlock, pairs);
#pragma unroll
                    for (int x = 0; x < kPairs; ++x) {
                        most = larger_of(most, pairs[x]);
                        least = smaller_of(least, pairs[x]);
                    }
                }
                vtop[0][0] = size_of(most);
                const uint32_t floor = (range - (16u << 7) & 0xffffu) | 0xff800000u;  // (kLeast / inv, -infinity)
                more = !__hble2(as_bf2(most & 0x7fff7fffu), as_bf2(range)) || !__hbge2(as_bf2(least), as_bf2(floor));
            }
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    mx[nt][c] = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
                    for (int ub = 1; ub < C::UB; ++ub)
                        mx[nt][c] = fmaxf(mx[nt][c], fmaxf(s[ub][nt][c], s[ub][nt][c + 2]));
                    mx[nt][c] *= factor[nt][c];
                    more = more || mx[nt][c] > ref[nt][c];
                    if constexpr (edge)
                        more = more || vtop[nt][c] * inv[nt][c] > 16384.f || step_of(lowest) * (inv[nt][c] * deepest) < kLeast;
                }
            if (__any_sync(0xffffffffu, more)) {
                if constexpr (!edge) {
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) vtop[0][0] = fmaxf(vtop[0][0], __shfl_xor_sync(0xffffffffu, vtop[0][0], o));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) vtop[nt][0] = vtop[nt][1] = vtop[0][0];
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float alpha[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            mx[nt][c] = fmaxf(mx[nt][c], __shfl_xor_sync(0xffffffffu, mx[nt][c], o));
                        const float now = mx[nt][c] > ref[nt][c] ? mx[nt][c] + kAhead : ref[nt][c];
                        alpha[c] = ref[nt][c] == -INFINITY ? 0.f : ex2_approx(ref[nt][c] - now);
                        // nothing seen so far leaves NaN sums (a NaN score) as they are
                        if (now == -INFINITY) alpha[c] = 1.f;
                        ref[nt][c] = now;
                        l[nt][c] *= alpha[c];
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            vtop[nt][c] = fmaxf(vtop[nt][c], __shfl_xor_sync(0xffffffffu, vtop[nt][c], o));
                        if (vtop[nt][c] * inv[nt][c] > 16384.f) {
                            // 2^13 over the power of two at or above it
                            const int now = (267 << 23) - ((__float_as_int(vtop[nt][c]) + 0x007fffff) & 0x7f800000);
                            alpha[c] *= __int_as_float(max(0x3f800000 + now - __float_as_int(inv[nt][c]), 0));
                            inv[nt][c] = __int_as_float(now);
                        }
#pragma unroll
                        for (int g = 0; g < C::kGroups; ++g) om[nt][g][c] *= alpha[c];
                    }
#pragma unroll
                    for (int w = 0; w < C::kWords; ++w)
#pragma unroll
                        for (int x = 0; x < 8; ++x) acc[nt][w][x >> 2][x & 3] *= alpha[x & 1];
                }
                range = range_of(inv[0][0]);
                if constexpr (edge) {
                    float low = step_of(lowest);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
                    lowest = pair_of_step(low);
                    for (; deepest < kLastBand; deepest *= kBand) {
                        bool below = false;
#pragma unroll
                        for (int x = 0; x < 2 * NT; ++x) below = below || low * (inv[x >> 1][x & 1] * deepest) < kLeast;
                        if (!__any_sync(0xffffffffu, below)) break;
                    }
                } else if (__any_sync(0xffffffffu, kv4_scale(least).x * inv[0][0] < kLeast)) {  // or steps of 0
                    float low = step_of(lowest);
                    for (int x = lane; x < C::UB * 16 * C::kGroups; x += 32) {
                        uint32_t pair[1];
                        lds(unit + x / (16 * C::kGroups) * C::kBlock + C::kValueScales + x % (16 * C::kGroups) * 4, pair);
                        low = fminf(low, step_of(pair[0]));
                    }
                    lowest = least = pair_of_step(low);
                    if (__any_sync(0xffffffffu, low * inv[0][0] < kLeast)) return true;
                }
            }
            if constexpr (!edge) lowest = least;

            // ---- P, and O^T += V^T P^T
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float r0 = ref[nt][0] == -INFINITY ? 0.f : ref[nt][0];
                const float r1 = ref[nt][1] == -INFINITY ? 0.f : ref[nt][1];
#pragma unroll
                for (int ub = 0; ub < C::UB; ++ub) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        s[ub][nt][c] = ex2_approx(fmaf(s[ub][nt][c], factor[nt][c & 1], c & 1 ? -r1 : -r0));
                    l[nt][0] += s[ub][nt][0] + s[ub][nt][2];
                    l[nt][1] += s[ub][nt][1] + s[ub][nt][3];
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[ub][nt][c] *= inv[nt][c & 1];
                }
            }
            float boost = 1.f;  // of the band
            for (;;) {
#pragma unroll
                for (int ub = 0; ub < C::UB; ++ub) {
                    const uint32_t blk = unit + ub * C::kBlock + C::kValueCodes + g4 * (C::kWords * 2);
                    uint32_t va[C::kGroups], vb[C::kGroups];
                    value_scales(ub, va, vb);
                    uint32_t b0[C::kGroups][NT], b1[C::kGroups][NT];
#pragma unroll
                    for (int g = 0; g < C::kGroups; ++g) {
                        const float2 wa = kv4_scale(va[g]), wb = kv4_scale(vb[g]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float* q = s[ub][nt];
                            float w0 = q[0] * wa.x, w1 = q[1] * wa.x, w2 = q[2] * wb.x, w3 = q[3] * wb.x;
                            if constexpr (!edge) {
                                om[nt][g][0] = fmaf(q[0], wa.y, fmaf(q[2], wb.y, om[nt][g][0]));
                                om[nt][g][1] = fmaf(q[1], wa.y, fmaf(q[3], wb.y, om[nt][g][1]));
                            } else {
                                // a token hidden from a row adds nothing to it, whatever its scales hold
                                const int ta = t0 + ub * 16 + tokA, tb = ta + 8;
                                const auto add = [&](float& w, float q, float2 x, int at, int c) {
                                    const bool sees = at < seen[nt][c];
                                    w = sees ? q * x.x : 0.f;
                                    if (sees && boost == 1.f) om[nt][g][c] = fmaf(q, x.y, om[nt][g][c]);
                                    if (boost != deepest && w < kLeast) w = 0.f;                // a later band's
                                    if (boost != 1.f && !(w < kLeast * kBand)) w = 0.f;  // an earlier one's
                                };
                                add(w0, q[0], wa, ta, 0);
                                add(w1, q[1], wa, ta, 1);
                                add(w2, q[2], wb, tb, 0);
                                add(w3, q[3], wb, tb, 1);
                            }
                            b0[g][nt] = transpose8(pack_f16(w0, w1));
                            b1[g][nt] = transpose8(pack_f16(w2, w3));
                        }
                    }
                    uint32_t x0[C::kWords / 2], x1[C::kWords / 2], x2[C::kWords / 2], x3[C::kWords / 2];
                    lds(blk + token_of(2 * j) * C::kRow, x0);
                    lds(blk + token_of(2 * j + 1) * C::kRow, x1);
                    lds(blk + (8 + token_of(2 * j)) * C::kRow, x2);
                    lds(blk + (8 + token_of(2 * j + 1)) * C::kRow, x3);
#pragma unroll
                    for (int g = 0; g < C::kGroups; ++g) {
#pragma unroll
                        for (int w = g * (G / 32); w < (g + 1) * (G / 32); ++w) {
                            const uint32_t sel = w & 1 ? 0x7632u : 0x5410u;
                            const uint32_t z0 = __byte_perm(x0[w / 2], x1[w / 2], sel);
                            const uint32_t z1 = __byte_perm(x2[w / 2], x3[w / 2], sel);
                            const uint32_t y0 = z0 >> 8, y1 = z1 >> 8;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma_f16(acc[nt][w][0], z0 & 0x000f000fu, z0 & 0x00f000f0u, z1 & 0x000f000fu,
                                        z1 & 0x00f000f0u, b0[g][nt], b1[g][nt]);
                                mma_f16(acc[nt][w][1], y0 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x000f000fu,
                                        y1 & 0x00f000f0u, b0[g][nt], b1[g][nt]);
                            }
                        }
                    }
                }
                if (!edge || boost == deepest) break;
                boost *= kBand;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int w = 0; w < C::kWords; ++w)
#pragma unroll
                        for (int x = 0; x < 8; ++x) acc[nt][w][x >> 2][x & 3] *= kBand;
#pragma unroll
                    for (int ub = 0; ub < C::UB; ++ub)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[ub][nt][c] *= kBand;
                }
            }
            if (edge && boost != 1.f) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int w = 0; w < C::kWords; ++w)
#pragma unroll
                        for (int x = 0; x < 8; ++x) acc[nt][w][x >> 2][x & 3] *= 1.f / boost;
            }
            return false;
        };
        for (int u = seg.u0; u < seg.u1; ++u) {
            copy_wait<kStages - 1>();
            __syncwarp();
            const uint32_t unit = ring + stage * C::kUnitBytes;
            const uint32_t valid = masks >> (8 * stage) & 0xffu;
            const int t0 = u * C::kTokens;
            if (t0 + C::kTokens > all_see || valid != (1u << C::UB) - 1 || deepest != 1.f || far != 0 ||
                use(std::false_type{}, unit, valid, t0))
                use(std::true_type{}, unit, valid, t0);
            __syncwarp();  // every lane has read the stage
            if (u + kStages < seg.u1) masks = (masks & ~(0xffu << (8 * stage))) | issue(stage) << (8 * stage);
            copy_commit();
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }

        // ---- sums over the lanes; the next head's first copies run meanwhile
        Segment next = seg;
        working = advance(next);
        if (working) prologue(next);
        const bool first = seg.u0 == 0, last = seg.u1 == seg.n;
        // a head that ends here and began before, or goes on behind this warp's share
        Piece* piece = &s_piece[warp][working ? 0 : 1];
        float2* out = reinterpret_cast<float2*>(piece_at(warp, working ? 0 : 1));
        float* ml = reinterpret_cast<float*>(piece_at(warp, working ? 0 : 1) + C::kPieceO);
        if (!(first && last) && lane == 0) {
            piece->head = seg.b * HR + seg.hr;
            piece->first = first;
            piece->last = last;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], o);
#pragma unroll
                for (int g = 0; g < C::kGroups; ++g)
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) om[nt][g][c] += __shfl_xor_sync(0xffffffffu, om[nt][g][c], o);
            }
            const int row = row0 + nt * 8 + 2 * j;
            const float n0 = l[nt][0] == 0.f ? 0.f : 1.f / l[nt][0], n1 = l[nt][1] == 0.f ? 0.f : 1.f / l[nt][1];
            float unit_o[2];  // 1 / inv
#pragma unroll
            for (int c = 0; c < 2; ++c) unit_o[c] = __int_as_float((254 << 23) - __float_as_int(inv[nt][c]));
#pragma unroll
            for (int w = 0; w < C::kWords; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float k = i & 1 ? 0x1p20f : 0x1p24f;  // the codes' unit
                    const float x0 = fmaf(acc[nt][w][i >> 1][2 * (i & 1)], k, om[nt][w * 32 / G][0]);
                    const float x1 = fmaf(acc[nt][w][i >> 1][2 * (i & 1) + 1], k, om[nt][w * 32 / G][1]);
                    if (first && last) {
                        __nv_bfloat16* to = p.o + (static_cast<long long>(bh) * p.R + row) * D + 32 * w + 4 * g4 + i;
                        if (row < p.R) to[0] = __float2bfloat16_rn(x0 * n0 * unit_o[0]);
                        if (row + 1 < p.R) to[D] = __float2bfloat16_rn(x1 * n1 * unit_o[1]);
                    } else {
                        out[(nt * C::kPairs + w * 4 + i) * 32 + lane] =
                            make_float2(x0 * kPieceUnit * unit_o[0], x1 * kPieceUnit * unit_o[1]);
                    }
                }
            if (g4 == 0) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (!(first && last)) {
                        ml[nt * 16 + 2 * j + c] = ref[nt][c];
                        ml[nt * 16 + 8 + 2 * j + c] = l[nt][c];
                    } else if (row + c < p.R) {
                        p.lse[static_cast<long long>(bh) * p.R + row + c] =
                            l[nt][c] == 0.f ? -INFINITY : (ref[nt][c] + __log2f(l[nt][c])) * kLn2;
                    }
                }
            }
        }
        seg = next;
        fresh = false;
    }
    // ---- join the pieces that this CTA's warps share: they stand in the line's order
    __syncthreads();
    constexpr int kMost = 2 * kWarps;
    static_assert(kMost <= 32, "a lane for every piece");
    // the pieces of a head are neighbours; lane y looks at piece y
    const Piece mine = s_piece[(lane % kMost) >> 1][lane & 1];
    unsigned open = __ballot_sync(0xffffffffu, lane < kMost && mine.head >= 0);
    const unsigned peers = __match_any_sync(0xffffffffu, mine.head) & open;
    const int heads = __popc(__ballot_sync(0xffffffffu, (peers & ((2u << lane) - 1)) == 1u << lane));
    // With many heads a warp joins one by itself, or two, from its own pieces alone; with
    // few all warps join each, a part of the channels a warp.  (1920 heads of about 52
    // tokens and 16 rows take 41 us for both kernels; it was 39 against 61 with all warps
    // at each of a CTA's 8 heads and a block a head in the second kernel.  The second path
    // costs 8 long sequences 1 us of 221.)
    const bool alone = heads > kWarps / 2;
    for (int turn = 0; open != 0; ++turn) {
        const int y0 = __ffs(open) - 1;
        const int at = __shfl_sync(0xffffffffu, mine.head, y0);
        const unsigned group = __ballot_sync(0xffffffffu, mine.head == at) & open;
        const bool whole = __shfl_sync(0xffffffffu, mine.first, y0) && __shfl_sync(0xffffffffu, mine.last, 31 - __clz(group));
        open &= ~group;
        if (alone && turn % kWarps != warp) continue;
        const int hr = at % HR;
        const long long bh = static_cast<long long>(at / HR) * p.pages.heads + hr / p.RB;
        const long long slot = blockIdx.x + static_cast<long long>(at);
        auto put = [&](int nt, int pr, int row, float2 o, float2 sum) {
            if (!whole) {
                p.part_o[((slot * NT + nt) * C::kPairs + pr) * 32 + lane] = o;
            } else {
                const int ch = 32 * (pr >> 2) + 4 * g4 + (pr & 3);
                __nv_bfloat16* to = p.o + (bh * p.R + row) * D + ch;
                if (row < p.R) to[0] = __float2bfloat16_rn(sum.x == 0.f ? 0.f : o.x / sum.x * (1.f / kPieceUnit));
                if (row + 1 < p.R) to[D] = __float2bfloat16_rn(sum.y == 0.f ? 0.f : o.y / sum.y * (1.f / kPieceUnit));
            }
        };
        auto put_sums = [&](int nt, int row, float2 top, float2 sum) {
            if (!whole) {
                float2* ml = reinterpret_cast<float2*>(p.part_ml + (slot * NT + nt) * 16) + j;
                ml[0] = top;
                ml[4] = sum;
            } else {
                if (row < p.R) p.lse[bh * p.R + row] = sum.x == 0.f ? -INFINITY : (top.x + __log2f(sum.x)) * kLn2;
                if (row + 1 < p.R) p.lse[bh * p.R + row + 1] = sum.y == 0.f ? -INFINITY : (top.y + __log2f(sum.y)) * kLn2;
            }
        };
        if (__builtin_expect(alone, 0)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = (hr % p.RB) * NT * 8 + nt * 8 + 2 * j;
                float2 o[C::kPairs], top = make_float2(-INFINITY, -INFINITY), sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int pr = 0; pr < C::kPairs; ++pr) o[pr] = make_float2(0.f, 0.f);
                for (unsigned m = group; m != 0; m &= m - 1) {
                    const int y = __ffs(m) - 1;
                    const float2* ml = reinterpret_cast<const float2*>(piece_at(y >> 1, y & 1) + C::kPieceO) + nt * 8 + j;
                    if (ml[4].x != 0.f) top.x = fmaxf(top.x, ml[0].x);
                    if (ml[4].y != 0.f) top.y = fmaxf(top.y, ml[0].y);
                }
                for (unsigned m = group; m != 0; m &= m - 1) {
                    const int y = __ffs(m) - 1;
                    const unsigned char* piece = piece_at(y >> 1, y & 1);
                    const float2* ml = reinterpret_cast<const float2*>(piece + C::kPieceO) + nt * 8 + j;
                    const float2 f = make_float2(ex2_approx(ml[0].x - top.x), ex2_approx(ml[0].y - top.y)), lw = ml[4];
                    if (lw.x != 0.f) sum.x = fmaf(f.x, lw.x, sum.x);
                    if (lw.y != 0.f) sum.y = fmaf(f.y, lw.y, sum.y);
#pragma unroll
                    for (int pr = 0; pr < C::kPairs; ++pr) {
                        const float2 v = reinterpret_cast<const float2*>(piece)[(nt * C::kPairs + pr) * 32 + lane];
                        if (lw.x != 0.f) o[pr].x = fmaf(f.x, v.x, o[pr].x);
                        if (lw.y != 0.f) o[pr].y = fmaf(f.y, v.y, o[pr].y);
                    }
                }
#pragma unroll
                for (int pr = 0; pr < C::kPairs; ++pr) put(nt, pr, row, o[pr], sum);
                if (g4 == 0) put_sums(nt, row, top, sum);
            }
            continue;
        }
        // A head has last pieces of neighbouring warps, and at most one first piece, its
        // end.  All warps' last pieces are read, of this head or not, and every warp
        // computes all factors, so that no load waits for another and nothing is passed
        // round (a loop over the members took three times as long, a table of factors
        // and its barrier 1 us).
        const int first_piece = (group & 0x55555555u) != 0 ? __ffs(group & 0x55555555u) - 1 : 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = (hr % p.RB) * NT * 8 + nt * 8 + 2 * j;
            float2 f[kWarps + 1], lw[kWarps + 1], top = make_float2(-INFINITY, -INFINITY), sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int y = 0; y <= kWarps; ++y) {
                const float2* ml = reinterpret_cast<const float2*>(
                    piece_at(y < kWarps ? y : first_piece >> 1, y < kWarps) + C::kPieceO) + nt * 8 + j;
                f[y] = ml[0];
                lw[y] = ml[4];
                if (!(group >> (y < kWarps ? 2 * y + 1 : first_piece) & 1)) lw[y] = make_float2(0.f, 0.f);
                if (lw[y].x != 0.f) top.x = fmaxf(top.x, f[y].x);
                if (lw[y].y != 0.f) top.y = fmaxf(top.y, f[y].y);
            }
#pragma unroll
            for (int y = 0; y <= kWarps; ++y) {
                f[y].x = lw[y].x == 0.f ? 0.f : ex2_approx(f[y].x - top.x);
                f[y].y = lw[y].y == 0.f ? 0.f : ex2_approx(f[y].y - top.y);
                if (lw[y].x != 0.f) sum.x = fmaf(f[y].x, lw[y].x, sum.x);
                if (lw[y].y != 0.f) sum.y = fmaf(f[y].y, lw[y].y, sum.y);
            }
#pragma unroll
            for (int xi = 0; xi < C::kPairs / kWarps; ++xi) {
                const int pr = xi * kWarps + warp;
                float2 o = make_float2(0.f, 0.f);
#pragma unroll
                for (int y = 0; y <= kWarps; ++y) {
                    const float2 v = reinterpret_cast<const float2*>(
                        piece_at(y < kWarps ? y : first_piece >> 1, y < kWarps))[(nt * C::kPairs + pr) * 32 + lane];
                    // (a factor of 0 too: a NaN that the piece saw stays one)
                    if (lw[y].x != 0.f) o.x = fmaf(f[y].x, v.x, o.x);
                    if (lw[y].y != 0.f) o.y = fmaf(f[y].y, v.y, o.y);
                }
                put(nt, pr, row, o, sum);
            }
            if (warp == 0 && g4 == 0) put_sums(nt, row, top, sum);
        }
    }
}

// Which parts a head was cut into: CTAs c0 .. c1 hold some of its n units; `before` are
// the places of one head before its sequence, `share` those of a CTA.
__device__ __forceinline__ void cut_of(int before, int HR, int hr, int n, unsigned share, unsigned& c0, unsigned& c1) {
    const unsigned first = before * HR + hr * (n + kStart) + kStart;  // the first unit's place
    c0 = first / share;
    c1 = n == 0 ? c0 : (first + n - 1) / share;
}
template <class C>
__device__ __forceinline__ void parts_of(const DecParams& p, int lane, int b, int hr, int& n, unsigned& c0, unsigned& c1) {
    const int HR = p.pages.heads * p.RB;
    if (p.by_head) {
        n = (length_of(p, b) + C::kTokens - 1) / C::kTokens;
        c0 = c1 = 0;
        return;
    }
    int all, before;
    count_places<C::kTokens>(p, lane, b, all, before);
    n = max(places_of<C::kTokens>(length_of(p, b)) - kStart, 0);
    cut_of(before, HR, hr, n, static_cast<unsigned>(share_of(p, all * HR)) * kWarps, c0, c1);
}

// A running maximum, sum and output pair, and more of the same head.
struct Joined {
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, o[2] = {0.f, 0.f};
    __device__ __forceinline__ void take(float2 m, float2 l, float2 x) {
        const float ms[2] = {m.x, m.y}, ls[2] = {l.x, l.y}, xs[2] = {x.x, x.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (ls[e] == 0.f) continue;
            const float now = fmaxf(top[e], ms[e]);
            const float base = now == -INFINITY ? 0.f : now;  // NaN sums of rows that saw only NaN
            const float a = sum[e] == 0.f ? 0.f : ex2_approx(top[e] - base), f = ex2_approx(ms[e] - base);
            sum[e] = sum[e] * a + ls[e] * f;
            o[e] = o[e] * a + xs[e] * f;
            top[e] = now;
        }
    }
    __device__ __forceinline__ float lse2(int e) const { return sum[e] == 0.f ? -INFINITY : top[e] + __log2f(sum[e]); }
};

// Joins the parts of a head, CTAs c0 .. c1's; n is its units, none of them a row of zeros.
template <class C, int NT, int SPLIT>
__device__ __forceinline__ void join_head(const DecParams& p, int b, int hr, int n, unsigned c0, unsigned c1, int y,
                                          float2 (&sm)[3][8][32]) {
    constexpr int D = C::D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g4 = lane >> 2, j = lane & 3;
    const int head_row = b * p.pages.heads * p.RB + hr;
    const long long bh = static_cast<long long>(b) * p.pages.heads + hr / p.RB;
    const int pair = y * (8 / SPLIT) + warp / SPLIT, sub = warp % SPLIT;
    const int nt = pair / C::kPairs, i = pair % C::kPairs;
    const int row = (hr % p.RB) * NT * 8 + nt * 8 + 2 * j, ch = 32 * (i >> 2) + 4 * g4 + (i & 3);
    Joined all;
    if (n > 0) {
#pragma unroll 4
        for (unsigned c = c0 + sub; c <= c1; c += SPLIT) {
            const long long slot = static_cast<long long>(head_row) + c;
            const float* ml = p.part_ml + (slot * NT + nt) * 16 + 2 * j;
            all.take(*reinterpret_cast<const float2*>(ml), *reinterpret_cast<const float2*>(ml + 8),
                     p.part_o[((slot * NT + nt) * C::kPairs + i) * 32 + lane]);
        }
    }
    if constexpr (SPLIT > 1) {
        sm[0][warp][lane] = make_float2(all.top[0], all.top[1]);
        sm[1][warp][lane] = make_float2(all.sum[0], all.sum[1]);
        sm[2][warp][lane] = make_float2(all.o[0], all.o[1]);
        __syncthreads();
        if (sub != 0) return;
#pragma unroll
        for (int x = 1; x < SPLIT; ++x) all.take(sm[0][warp + x][lane], sm[1][warp + x][lane], sm[2][warp + x][lane]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (row + e >= p.R) continue;
        p.o[(bh * p.R + row + e) * D + ch] =
            __float2bfloat16_rn(all.sum[e] == 0.f ? 0.f : all.o[e] / all.sum[e] * (1.f / kPieceUnit));
        if (i == 0 && g4 == 0) p.lse[bh * p.R + row + e] = all.lse2(e) * kLn2;
    }
}

// Joins the parts of the heads that are cut between CTAs, and writes those that
// have no tokens.  A CTA takes 8 / SPLIT pairs of accumulators of each of `each`
// heads (sequence, head, row block) in a row, SPLIT warps to a pair taking the parts
// in turn.  (A CTA a head: 38 us for 1920 heads, most of them whole.)
template <class C, int NT, int SPLIT>
__device__ __forceinline__ void join_parts(const DecParams& p, int x, int y, int each, float2 (&sm)[3][8][32]) {
    const int lane = threadIdx.x & 31;
    const int HR = p.pages.heads * p.RB, heads = p.B * HR;
    int head_row = x * each;
    int b = head_row / HR, hr = head_row - b * HR, all, before;
    count_places<C::kTokens>(p, lane, b, all, before);
    int n = max(places_of<C::kTokens>(length_of(p, b)) - kStart, 0);
    const unsigned share = static_cast<unsigned>(share_of(p, all * HR)) * kWarps;
    unsigned c0, c1;
    cut_of(before, HR, hr, n, share, c0, c1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (const int end = min(head_row + each, heads);;) {
        if (n == 0 || c0 != c1) join_head<C, NT, SPLIT>(p, b, hr, n, c0, c1, y, sm);
        if (++head_row == end) break;
        if (++hr == HR) {
            hr = 0;
            before += n == 0 ? 0 : n + kStart;
            n = max(places_of<C::kTokens>(length_of(p, ++b)) - kStart, 0);
        }
        cut_of(before, HR, hr, n, share, c0, c1);
    }
}

// weights_out = weights + the sum over the rows of P, slot by slot, for a head's
// tokens from 256 x on, `step` apart.
template <class C, int NT>
__device__ __forceinline__ void add_weights(const DecParams& p, int bh, int x, int step, float* sm_lse) {
    const int b = bh / p.pages.heads, head = bh % p.pages.heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = length_of(p, b);
    int n;
    unsigned c0, c1;
    parts_of<C>(p, lane, b, head * p.RB, n, c0, c1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (static_cast<long long>(x) * 256 >= len) return;
    // the rows' log-sum-exp: from the head's CTA, or from the parts again, as nothing
    // says that their join is done; a warp takes a pair of rows, its lanes the parts
    const int width = p.RB * NT * 8;
    for (int pr = warp; pr < width / 2; pr += 8) {
        const int rb = pr / (NT * 4), nt = pr / 4 % NT, j = pr % 4;
        if (rb > 0) parts_of<C>(p, lane, b, head * p.RB + rb, n, c0, c1);
        if (c0 == c1) {
            if (lane < 2 && 2 * pr + lane < p.R) sm_lse[2 * pr + lane] = p.lse[static_cast<long long>(bh) * p.R + 2 * pr + lane] * kLog2e;
            continue;
        }
        Joined all;
        for (unsigned c = c0 + lane; c <= c1; c += 32) {
            const float* ml = p.part_ml + ((static_cast<long long>(bh) * p.RB + rb + c) * NT + nt) * 16 + 2 * j;
            all.take(*reinterpret_cast<const float2*>(ml), *reinterpret_cast<const float2*>(ml + 8), make_float2(0.f, 0.f));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float2 m = make_float2(__shfl_xor_sync(0xffffffffu, all.top[0], o), __shfl_xor_sync(0xffffffffu, all.top[1], o));
            const float2 l = make_float2(__shfl_xor_sync(0xffffffffu, all.sum[0], o), __shfl_xor_sync(0xffffffffu, all.sum[1], o));
            all.take(m, l, make_float2(0.f, 0.f));
        }
        if (lane == 0) {
            sm_lse[2 * pr] = all.lse2(0);
            sm_lse[2 * pr + 1] = all.lse2(1);
        }
    }
    __syncthreads();
    for (long long t = x * 256LL + threadIdx.x; t < len; t += step * 256LL) {
        const float4* s = reinterpret_cast<const float4*>(p.scores + (bh * p.cap + t) * width);
        float sum = 0.f;
        for (int r = 0; r < p.R; r += 4) {
            const float4 v = s[r >> 2];
            const float vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < p.R && vs[e] != -INFINITY) sum += ex2_approx(vs[e] - sm_lse[r + e]);
        }
        const long long at = bh * p.slots + t;
        p.weights_out[at] = (p.weights != nullptr ? p.weights[at] : 0.f) + sum;
    }
}

// What is left when the line is done: the first `joins` blocks join parts, D / 8 NT
// SPLIT / 8 of them in a row the same heads' channels, and the others add weights.
template <int D, int G, int NT, int SPLIT, bool WEIGHTS>
__global__ void __launch_bounds__(256) fa_kv4_finish_kernel(DecParams p, int joins, int each) {
    using C = Cfg<D, G, NT>;
    __shared__ float2 sm[3][8][32];
    static_assert(sizeof(sm) >= 1024 * sizeof(float), "the log-sum-exps of 1024 rows");
    // The lengths may be read at once: this kernel is scheduled when every CTA of the
    // decoding kernel has waited for the kernels before it, so their writes are in L2.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kY = D / 8 * NT * SPLIT / 8;
    const int x = blockIdx.x;
    if (x < joins) {
        join_parts<C, NT, SPLIT>(p, x / kY, x % kY, each, sm);
    } else if constexpr (WEIGHTS) {
        const int heads = p.B * p.pages.heads;
        add_weights<C, NT>(p, (x - joins) % heads, (x - joins) / heads, (gridDim.x - joins) / heads, reinterpret_cast<float*>(sm));
    }
}

// Row tiles of a CTA: one for up to 8 query rows, two above.  Two tiles take 255
// registers, so one CTA of 8 warps an SM, but read and unpack the cache once for 16
// rows: 57.5 us on 8 sequences of 16384 tokens with 16 rows a head, against 72 with
// one tile twice.  (Before the bands, 10 or 12 warps with 168 registers spilled: 66 and 68
// where two tiles took 59.)
int tiles_of(int R) { return R <= 8 ? 1 : 2; }
int ctas_of(int nt, int num_sms) { return nt == 1 ? 2 * num_sms : num_sms; }

struct Sizes {
    size_t part_o, part_ml, scores;
};
// Whether a CTA takes a head by itself (kByHead): short caches whose heads find room in
// two rounds of CTAs.  The others are cut like long ones: 1408 heads of 16 rows on 152
// CTAs take 23 us so and 62 with a CTA each, 1920 take 41 and 99; 512 heads on 304 take
// 16.9 and 16.5.
bool by_head(const Kv4Shape& c, size_t heads, int n_cta) {
    const int tokens = c.D == 128 ? Cfg<128, 64, 1>::kTokens : Cfg<64, 64, 1>::kTokens;
    return heads <= 2 * static_cast<size_t>(n_cta) &&
           static_cast<long long>(c.width) * c.page_size <= static_cast<long long>(kByHead) * kWarps * tokens;
}
Sizes sizes_of(const Kv4Shape& c, int Hq, int Tq, bool weights, int num_sms) {
    const int R = Hq / c.Hkv * Tq, nt = tiles_of(R);
    const size_t RB = (R + 8 * nt - 1) / (8 * nt), bh = static_cast<size_t>(c.B) * c.Hkv;
    const int n_cta = ctas_of(nt, num_sms);
    const size_t slots = by_head(c, bh * RB, n_cta) ? 0 : n_cta + bh * RB;
    return {slots * nt * c.D * 8 * 4, slots * nt * 16 * 4,
            weights ? bh * c.width * c.page_size * RB * nt * 8 * 4 : 0};
}

template <int D, int G, int NT, int SPLIT>
int launch_finish(const DecParams& p, cudaStream_t stream, int bh, int num_sms) {
    // More heads than CTAs are joined several to a block, in two ranges an SM (with 4 blocks
    // to a range, what is resident at once): at most a head a CTA is cut.
    constexpr int kY = D / 8 * NT * SPLIT / 8;
    const int heads = bh * p.RB, each = SPLIT > 1 ? 1 : (heads + 2 * num_sms - 1) / (2 * num_sms);
    const int joins = p.by_head ? 0 : (heads + each - 1) / each * kY;
    // Blocks to a head, sharing its tokens: what is resident at once (5 an SM).  (8 an SM, two
    // rounds: 92 us instead of 89 for 2 sequences of 32768 tokens, 59 instead of 57.5 for 24 ragged ones.)
    long long adds = 0;
    if (p.weights_out != nullptr) {
        const long long most = (p.cap + 255) / 256, want = (5LL * num_sms + bh - 1) / bh;
        adds = most < want ? most : want;
    }
    if (joins + adds == 0) return 0;
    const dim3 grid(static_cast<unsigned>(joins + adds * bh));
    return launch_chained(adds > 0 ? fa_kv4_finish_kernel<D, G, NT, SPLIT, true> : fa_kv4_finish_kernel<D, G, NT, SPLIT, false>,
                          grid, 256, 0, stream, p, joins, each);
}

template <int D, int G, int NT>
int launch(DecParams p, cudaStream_t stream, int num_sms, int bh, bool weights) {
    using C = Cfg<D, G, NT>;
    static_assert(C::kSmem + 2 * kWarps * static_cast<int>(sizeof(Piece)) + 1024 <= (NT == 1 ? 233472 / 2 : 232448), "shared memory of the resident CTAs");
    const auto kernel = weights ? fa_kv4_decode_kernel<D, G, NT, true> : fa_kv4_decode_kernel<D, G, NT, false>;
    static std::atomic<unsigned long long> allowed[2];
    if (!allow_shared_memory(kernel, C::kSmem, allowed[weights])) return -5;
    if (launch_chained(kernel, dim3(p.n_cta), kThreads, C::kSmem, stream, p) != 0) return -5;
    // Warps to a pair: a head has about n_cta / heads parts, more if few of the heads
    // are long.  (Eight warps to each of 64 heads with 2 to 4 parts: 45 us instead of 41.)
    const long long heads = static_cast<long long>(bh) * p.RB;
    return heads * 8 >= p.n_cta ? launch_finish<D, G, NT, 1>(p, stream, bh, num_sms)
                                : launch_finish<D, G, NT, 8>(p, stream, bh, num_sms);
}

}  // namespace

size_t kv4_decode_workspace(const Kv4Shape& c, int Hq, int Tq, bool weights, int num_sms) {
    const Sizes s = sizes_of(c, Hq, Tq, weights, num_sms);
    return s.part_o + s.part_ml + s.scores;
}

bool kv4_decode_fits(const Kv4Shape& c, int Hq, int Tq) {
    const int R = Hq / c.Hkv * Tq, nt = tiles_of(R);
    const double places = (static_cast<double>(c.width) * c.page_size / 32 + 1 + kStart) * c.B * c.Hkv * ((R + 8 * nt - 1) / (8 * nt));
    return places + 4096.0 * kWarps < 2147483647.0;
}

int launch_kv4_decode(const Kv4Shape& c, const void* pool, const int* table, const int* lengths, const void* q,
                      void* o, float* lse, int Hq, int Tq, float scale, bool causal, const float* weights,
                      float* weights_out, long long slots, void* workspace, cudaStream_t stream, int num_sms) {
    DecParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.pages = kv4_pages(static_cast<unsigned char*>(const_cast<void*>(pool)), table, c.width, c.num_pages, c.Hkv,
                        c.page_size, c.D, c.group);
    p.lengths = lengths;
    p.B = c.B;
    p.R = Hq / c.Hkv * Tq;
    const int nt = tiles_of(p.R);
    p.RB = (p.R + 8 * nt - 1) / (8 * nt);
    p.Tq = Tq;
    p.causal = causal;
    p.n_cta = ctas_of(nt, num_sms);
    p.by_head = by_head(c, static_cast<size_t>(c.B) * c.Hkv * p.RB, p.n_cta);
    if (p.by_head) p.n_cta = c.B * c.Hkv * p.RB;
    p.cap = static_cast<long long>(c.width) * c.page_size;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.weights = weights;
    p.weights_out = weights_out;
    p.slots = slots;
    p.sl2 = scale * kLog2e;
    const int bh = c.B * c.Hkv;
    const bool w = weights_out != nullptr;
    const Sizes s = sizes_of(c, Hq, Tq, w, num_sms);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    p.part_o = reinterpret_cast<float2*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + s.part_o);
    p.scores = w ? reinterpret_cast<float*>(ws + s.part_o + s.part_ml) : nullptr;
    if (c.D == 64) {
        if (c.group == 32)
            return nt == 1 ? launch<64, 32, 1>(p, stream, num_sms, bh, w) : launch<64, 32, 2>(p, stream, num_sms, bh, w);
        return nt == 1 ? launch<64, 64, 1>(p, stream, num_sms, bh, w) : launch<64, 64, 2>(p, stream, num_sms, bh, w);
    }
    if (c.group == 32)
        return nt == 1 ? launch<128, 32, 1>(p, stream, num_sms, bh, w) : launch<128, 32, 2>(p, stream, num_sms, bh, w);
    return nt == 1 ? launch<128, 64, 1>(p, stream, num_sms, bh, w) : launch<128, 64, 2>(p, stream, num_sms, bh, w);
}

int kv4_decode_take_status() {
    int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_kv4_decode, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_kv4_decode, &z, sizeof(int)) != cudaSuccess) return -5;
    return h;
}

}  // namespace fa
