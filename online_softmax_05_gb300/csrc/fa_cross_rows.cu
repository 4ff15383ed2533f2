// fa_cross_rows.cu -- cross attention of a few query rows over many keys on sm_103a.
//
// The rows of one key/value head, its group's heads times their Tq queries, are packed into
// tiles of 128 (row = head in the group x Tq + query), so that K and V are read once
// whatever the grouping, and the keys of a ragged batch are cut over the CTAs by fa_split.cuh,
// their pieces joined by a second kernel.
//
// Per CTA: warps 0-3 softmax (a TMEM lane is a row), warp 4 loads (TMA, K and V tiles of 128
// keys in one ring), warp 5 issues tcgen05.mma: S = Q K^T, then O += P V with P, in bf16, in the
// S columns.  A CTA's chain per tile is serial (S, softmax, P V): two CTAs share an SM
// and fill each other's gaps, and the ring keeps loads in flight meanwhile.  K's and V's bytes
// bound it; the tensor cores' 128-row tiles are mostly padding then.
//
// Measured: 256 heads' 5 rows over 32768 keys of 128 channels 581 us, 7.4 TB/s (reads alone are faster than
// the copy's 6.8); a token of 32 sequences of 0 to 3000 keys 45 us, 4.3 TB/s, as units end unevenly (all
// of 3000: 66 us, 5.9 TB/s); a lone token's 8 heads over 1500 keys 9.6 us, all of it latency.
// 168 registers a thread, spilled bytes (stores, loads): 68 and 116 at 128 channels, 16 and 20 at 64.
#include <cuda_runtime.h>

#include "fa_check.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_split.cuh"
#include "fa_tmap.h"
#include "fa_wait.cuh"

namespace fa {

static __device__ int g_status_cross_rows;

namespace {

constexpr int kThreads = 192;
constexpr int kKeys = 128;   // of a tile
constexpr int kRows = 128;   // of a unit
constexpr int kLeast = 1;    // tiles that are not worth cutting (12 tiles in pieces of 1, 2, 4: 9.6, 10.3, 12.4 us)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct RowsCfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtomBytes = 128 * 128;
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kStages = D == 128 ? 2 : 5;  // two CTAs an SM
    static constexpr int kRingOff = kTileBytes;       // Q first
    static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
    // kv_full[], kv_empty[], q_full, s_full, p_full, o_full, mma_done
    static constexpr int kNumBars = 2 * kStages + 5;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8 + 8;
    static constexpr int kSmemBytes = kMiscOff + 16 + sizeof(SplitItem) + 1024;  // + tensor memory's address, abort flag; alignment
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");
    static_assert(kBarOff >= 128 * D * 4, "a CTA's scaled rows go where Q and the ring were");
    // 256 TMEM columns: S (P over its first half), O
    static constexpr uint32_t kS = 0, kO = 128;
    static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kKeys, false, false);
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
};

struct RowsParams {
    CrossTensor q, o;
    __nv_bfloat16* o_rest;
    float* lse;
    const int* key_lengths;
    SplitPlan plan;
    SplitParts parts;
    int Hq, Hkv, group, Tq, Tk, R, row_tiles;
    float sl2, sl2_eff;
    int prescale;
    unsigned long long timeout_ns;
    int inject;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    fa_cross_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         RowsParams p) {
    using C = RowsCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem), ring = sQ + C::kRingOff, bars = sQ + C::kBarOff;
    auto kv_full = [&](int s) { return bars + 8u * s; };
    auto kv_empty = [&](int s) { return bars + 8u * (C::kStages + s); };
    const uint32_t q_full = bars + 8u * (2 * C::kStages), s_full = q_full + 8, p_full = q_full + 16,
                   o_full = q_full + 24, mma_done = q_full + 32;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
    const WaitCtl ctl{abort_flag, &g_status_cross_rows, p.timeout_ns};
    SplitItem* s_item = reinterpret_cast<SplitItem*>(smem + C::kMiscOff + 16);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 5) {
        tmem_alloc(smem_u32(tmem_slot), 256);
        tmem_relinquish();
    }
    wait_for_stream();
    auto keys_of = [&](int b) {
        const int keys = p.key_lengths != nullptr ? __ldg(p.key_lengths + b) : p.Tk;
        if (keys >= 0 && keys <= p.Tk) return keys;
        atomicCAS(&g_status_cross_rows, 0, kStatusBadSeqlen);
        return 0;
    };
    if (warp == 0) {
        const SplitItem it =
            split_item(p.plan, blockIdx.x, lane, [&](int b) { return (keys_of(b) + kKeys - 1) / kKeys; });
        if (lane == 0) *s_item = it;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    const SplitItem item = *s_item;
    if (item.unit < 0) {  // more CTAs than pieces
        if (warp == 5) tmem_dealloc(tmem, 256);
        return;
    }
    const int b = item.b, tile = item.unit % p.row_tiles, hk = item.unit / p.row_tiles, bh = b * p.Hkv + hk;
    const int rows = min(kRows, p.R - tile * kRows);  // of this tile
    const int active = (rows + 31) / 32;              // softmax warps with rows
    const int keys = keys_of(b), j0 = item.j0, n = item.n;  // this CTA's key tiles
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        mbar_init(q_full, 4);
        mbar_init(s_full, 1);
        mbar_init(p_full, active);
        mbar_init(o_full, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();

    // a softmax thread's row: its state, and whether it is one
    const int r = 32 * warp + lane;
    const int row = tile * 128 + r, head = hk * p.group + row / p.Tq, tok = row % p.Tq;
    float m = -INFINITY, l = 0.f;
    const uint32_t lane_base = tmem + ((32u * (warp & 3)) << 16);

    if (warp == 4) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_first();
            int fills = 0;
            for (int i = 0; i < 2 * n; ++i) {
                const int slot = i % C::kStages;
                const bool is_v = i & 1;
                const int j = j0 + i / 2;
                if (p.inject == 4 && blockIdx.x == 0 && i == 0) continue;  // a test's: its waits run out
                if (!wait_one(kv_empty(slot), ((i / C::kStages) & 1) ^ 1, ctl) ||
                    !FA_CHECK(j >= 0 && j * kKeys < keys, &g_status_cross_rows, abort_flag))
                    break;
                mbar_arrive_expect_tx(kv_full(slot), C::kTileBytes);
                fills = i + 1;
                for (int a = 0; a < C::kAtoms; ++a)
                    tma_load_4d_hint(ring + slot * C::kTileBytes + a * C::kAtomBytes, is_v ? &tm_v : &tm_k, kv_full(slot),
                                     64 * a, j * kKeys, hk, b, policy);
            }
            for (int f = max(0, fills - C::kStages); f < fills; ++f)
                drain(kv_full(f % C::kStages), (f / C::kStages) & 1, ctl);
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------------ matrix instructions
        const bool leader = elect_one_sync();
        const SDesc dQ = sdesc_make(sQ, 16, 1024), dK = sdesc_make(ring, 16, 1024),
                    dV = sdesc_make(ring, C::kAtomBytes, 1024);
        constexpr uint32_t kTile16 = C::kTileBytes >> 4;
        int i = 0;  // ring fills used
        if (n > 0 && wait_warp(q_full, 0, ctl)) {
            tc_fence_after();
            for (int j = 0; j < n; ++j) {
                const int ks = i % C::kStages;
                if (!wait_warp(kv_full(ks), (i / C::kStages) & 1, ctl)) break;
                ++i;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = ((s >> 2) * C::kAtomBytes + (s & 3) * 32) >> 4;
                    if (leader) mma_ss_d(tmem + C::kS, dQ, off, dK, ks * kTile16 + off, C::kIdescS, s > 0);
                }
                if (leader) {
                    mma_commit(s_full);
                    mma_commit(kv_empty(ks));
                }
                const int vs = i % C::kStages;
                if (!wait_warp(kv_full(vs), (i / C::kStages) & 1, ctl)) break;
                ++i;
                // what lies past the keys must not meet P = 0 as NaN (past the tensor, TMA has filled zeros)
                const int left = keys - (j0 + j) * kKeys;
                if (left < kKeys && keys < p.Tk) zero_tail_rows(ring + vs * C::kTileBytes, C::kAtoms, left, lane);
                if (!wait_warp(p_full, j & 1, ctl)) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < kKeys / 16; ++s)
                    if (leader)
                        mma_ts_d(tmem + C::kO, tmem + C::kS + s * 8, dV, vs * kTile16 + s * (2048 >> 4), C::kIdescPV,
                                 (j > 0 || s > 0) ? 1u : 0u);
                if (leader) mma_commit(kv_empty(vs));
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
        {
            uint4 x[D / 8];
            const bool there = r < rows;
            const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q.ptr) + b * p.q.b +
                                                               head * p.q.h + tok * p.q.t);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) x[c] = there ? __ldg(from + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                st_shared_v4(sQ + (c >> 3) * C::kAtomBytes + sw128_off(r, c & 7), x[c].x, x[c].y, x[c].z, x[c].w);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const uint32_t tS = lane_base + C::kS, tO = lane_base + C::kO;
        const float eff = p.sl2_eff;
        for (int j = 0; j < n && warp < active; ++j) {
            if (!wait_warp(s_full, j & 1, ctl)) break;
            tc_fence_after();
            uint32_t sr[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, sr + 32 * c);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) reg_fence32(sr + 32 * c);
            float* s = reinterpret_cast<float*>(sr);
            if (p.prescale) {
#pragma unroll
                for (int c = 0; c < 128; ++c) s[c] *= p.sl2;
            }
            const int left = keys - (j0 + j) * kKeys;
            if (left < kKeys) {
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (c >= left) s[c] = -INFINITY;
            }
            float mx8[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) mx8[c] = fmaxf(s[c], s[c + 8]);
#pragma unroll
            for (int c = 16; c < 128; c += 16)
#pragma unroll
                for (int a = 0; a < 8; ++a) mx8[a] = fmax3(mx8[a], s[c + a], s[c + 8 + a]);
            const float mx =
                fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * eff;
            // the reference is the running maximum itself: the dominant weight is then 1, exact in bf16
            const bool grows = j > 0 && mx > m;
            const float m_new = fmaxf(m, mx);
            const float alpha = grows ? ex2_approx(m - m_new) : 1.f;
            l *= alpha;
            m = m_new;
            const uint64_t eff2 = f2(eff, eff), neg2 = f2(-m, -m);
            uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
            auto weights = [&](int c0) {  // of 64 keys, packed into sr[c0 / 2 ..]
#pragma unroll
                for (int c = c0 / 2; c < c0 / 2 + 32; ++c) {
                    float x0, x1;
                    f2_split(fma2(f2(s[2 * c], s[2 * c + 1]), eff2, neg2), x0, x1);
                    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                    sum[c & 3] = add2(sum[c & 3], f2(p0, p1));
                    sr[c] = pack_bf16x2(p0, p1);
                }
                tmem_st32(tS + c0 / 2, sr + c0 / 2);
            };
            weights(0);
            if (__any_sync(0xffffffffu, grows)) {  // in the registers that half of the scores have left
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t* o = sr;
                    tmem_ld32(tO + 32 * c, o);
                    tmem_ld_wait();
                    reg_fence32(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tmem_st32(tO + 32 * c, o);
                }
            }
            weights(64);
            float s0, s1;
            f2_split(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
            l += s0 + s1;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
        }
        wait_warp(o_full, 0, ctl);
        tc_fence_after();
    }

    // ------------------------------------------------------------ outputs
    // (o_full and the loads' drain are behind every thread: Q and the ring are free)
    const bool whole = item.pieces == 1;
    // this item's piece, and its unit's entry, lie inside the workspace
    const bool room = (whole || FA_CHECK(item.part >= 0 && item.part + item.k < p.parts.count, &g_status_cross_rows,
                                         abort_flag)) &&
                      FA_CHECK(bh * p.row_tiles + tile < p.plan.B * p.plan.per_seq, &g_status_cross_rows, abort_flag);
    __syncthreads();
    if (warp < active) {
        // rows times their factors: fp32 into shared memory, 16-byte chunks turned by the row against conflicts
        const float factor = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            if (n > 0) {
                tmem_ld32(lane_base + C::kO + 32 * c, o);
                tmem_ld_wait();
                reg_fence32(o);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = n > 0 ? __float_as_uint(__uint_as_float(o[e]) * factor) : 0u;
#pragma unroll
            for (int g = 0; g < 8; ++g)
                st_shared_v4(sQ + r * (D * 4) + (((8 * c + g) ^ (r & (D / 4 - 1))) << 4), o[4 * g], o[4 * g + 1],
                             o[4 * g + 2], o[4 * g + 3]);
        }
        if (r < rows) {
            const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
            if (whole) p.lse[(static_cast<size_t>(b) * p.Hq + head) * p.Tq + tok] = lse2 * kLn2;
            else if (room) p.parts.lse[static_cast<size_t>(item.part + item.k) * p.parts.rows + r] = lse2;
        }
    }
    if (p.parts.units != nullptr && tid == 0 && item.k == 0 && room)
        p.parts.units[bh * p.row_tiles + tile] = make_int2(item.part, item.pieces);
    __syncthreads();
    for (int i = tid; i < rows * (D / 8); i += kThreads) {
        const int rr = i / (D / 8), c = i % (D / 8);
        float x[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 y =
                *reinterpret_cast<const float4*>(smem + rr * (D * 4) + (((2 * c + h) ^ (rr & (D / 4 - 1))) << 4));
            x[4 * h] = y.x;
            x[4 * h + 1] = y.y;
            x[4 * h + 2] = y.z;
            x[4 * h + 3] = y.w;
        }
        if (!whole) {
            if (!room) break;
            float4* to = reinterpret_cast<float4*>(p.parts.o + (static_cast<size_t>(item.part + item.k) * p.parts.rows + rr) * D + c * 8);
            to[0] = make_float4(x[0], x[1], x[2], x[3]);
            to[1] = make_float4(x[4], x[5], x[6], x[7]);
            continue;
        }
        const int at = tile * 128 + rr, hq = hk * p.group + at / p.Tq, t = at % p.Tq;
        uint32_t w[4], e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
            e[k] = pack_bf16x2(x[2 * k] - __uint_as_float(w[k] << 16), x[2 * k + 1] - __uint_as_float(w[k] & 0xffff0000u));
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o.ptr) + b * p.o.b + hq * p.o.h + t * p.o.t + c * 8) =
            make_uint4(w[0], w[1], w[2], w[3]);
        if (p.o_rest != nullptr)
            *reinterpret_cast<uint4*>(p.o_rest + ((static_cast<size_t>(b) * p.Hq + hq) * p.Tq + t) * D + c * 8) =
                make_uint4(e[0], e[1], e[2], e[3]);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int D>
int launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const RowsParams& p, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed{0};
    auto kern = fa_cross_rows_kernel<D>;
    if (!allow_shared_memory(kern, RowsCfg<D>::kSmemBytes, allowed)) return -5;
    return launch_chained(kern, dim3(p.plan.items), kThreads, RowsCfg<D>::kSmemBytes, stream, tk, tv, p);
}

struct RowUnits {
    int R, row_tiles, rows;  // of a head; most rows of a unit
    long long units;
    SplitPlan plan;          // items == units: nothing is cut
};
RowUnits units_of(const CrossShape& s, int num_sms) {
    RowUnits u;
    u.R = s.Hq / s.Hkv * s.Tq;
    u.row_tiles = (u.R + kRows - 1) / kRows;
    u.rows = u.R < kRows ? u.R : kRows;
    u.units = static_cast<long long>(s.B) * s.Hkv * u.row_tiles;
    // Many units keep the memory busy by themselves, but for the longest, which end late; a piece costs its join.
    // 256 units of 0 to 24 tiles with 4, 64 and 128 rows, us, cut above 5, 7 and 10 fourths of a slot's part:
    // 47.9, 57.1, 68.6; 44.8, 51.3, 58.9; 48.0, 53.2, 58.7 (none is cut).  192 of them: 39.3, 34.3, 40.4; 512 alike.
    // Few units are better cut (64: 18 us, whole 40).
    u.plan = split_plan(s.B, u.units, 2 * num_sms, kLeast, 7);
    if (s.Tk <= kLeast * kKeys) u.plan.items = static_cast<int>(u.units);
    return u;
}

}  // namespace

// One tile of rows a head, or too few pairs of query tiles for the kernel of whole tiles to have one on half
// the SMs (8 heads of 1024 rows over 8192 keys: 44 us here, 57 there; 16 of 512 over 4096, D = 64: 25 and 28).
// With more, that kernel shares each key tile between two of rows (64 heads of 2048 rows over 0 to 3000 keys,
// D = 64: 59 us there, 117 here).
bool cross_rows_wanted(const CrossShape& s, int num_sms) {
    const long long group = s.Hq / s.Hkv, heads = static_cast<long long>(s.B) * s.Hq;
    const long long pairs = group % 2 == 0 ? heads / 2 * ((s.Tq + 127) / 128) : heads * ((s.Tq + 255) / 256);
    return group * s.Tq <= kRows || 2 * pairs <= num_sms;
}

size_t cross_rows_workspace(const CrossShape& s, int num_sms) {
    if (!cross_rows_wanted(s, num_sms)) return 0;
    const RowUnits u = units_of(s, num_sms);
    return split_workspace(u.plan, u.rows, s.D);
}

int launch_cross_rows(const CrossShape& s, const CrossTensor& q, const CrossTensor& k, const CrossTensor& v,
                      const CrossTensor& o, void* o_rest, float* lse, float scale, void* workspace, cudaStream_t stream,
                      const DebugKnobs& dbg, int num_sms) {
    CUtensorMap tk, tv;
    if (!make_tmap_strided(&tk, {k.ptr, k.b, k.h, k.t}, s.B, s.Hkv, s.Tk, s.D, kKeys) ||
        !make_tmap_strided(&tv, {v.ptr, v.b, v.h, v.t}, s.B, s.Hkv, s.Tk, s.D, kKeys))
        return -5;
    const RowUnits u = units_of(s, num_sms);
    RowsParams p{};
    p.q = q;
    p.o = o;
    p.o_rest = static_cast<__nv_bfloat16*>(o_rest);
    p.lse = lse;
    p.key_lengths = s.key_lengths;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.group = s.Hq / s.Hkv;
    p.Tq = s.Tq;
    p.Tk = s.Tk;
    p.R = u.R;
    p.row_tiles = u.row_tiles;
    p.plan = u.plan;
    p.parts = split_parts(workspace, u.plan, u.rows, s.D);
    p.sl2 = scale * kLog2e;
    p.prescale = p.sl2 > 0.f ? 0 : 1;
    p.sl2_eff = p.prescale ? 1.f : p.sl2;
    p.timeout_ns = dbg.timeout_ns;
    p.inject = dbg.inject;
    const int rc = s.D == 64 ? launch_t<64>(tk, tv, p, stream) : launch_t<128>(tk, tv, p, stream);
    if (rc != 0 || u.plan.items == u.units) return rc;
    SplitOut out{};
    out.o = o;
    out.rest = p.o_rest;
    out.lse = lse;
    out.Hkv = s.Hkv;
    out.group = p.group;
    out.T = s.Tq;
    out.R = u.R;
    out.row_units = u.row_tiles;
    out.unit_rows = kRows;
    return launch_split_join(p.parts, out, s.B, s.D, u.plan.items, stream);
}

int cross_rows_take_status() {
    int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_cross_rows, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_cross_rows, &z, sizeof(int)) != cudaSuccess) return -5;
    return h;
}

}  // namespace fa
