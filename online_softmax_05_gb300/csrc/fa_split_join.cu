// fa_split_join.cu -- joins the pieces of units whose keys were cut over CTAs (fa_split.cuh):
//   M = max lse_k,  w_k = 2^(lse_k - M),  O = sum w_k O_k / sum w_k,  LSE = M + log2 sum w_k.
// A warp takes a row (two rows of 64 channels), or with many pieces a unit a block takes it, its
// warps an eighth of the pieces each.  Bound by latency: the launch hides behind the first
// kernel's end, then the unit's entry and the pieces, eight of a warp in flight at once.
#include <cuda_runtime.h>

#include "fa_check.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_split.cuh"

namespace fa {

#ifdef FA_DEBUG
static __device__ int g_status_split_join;  // only checks record anything here
#endif

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, int WARPS>  // warps to a row
__global__ void __launch_bounds__(kThreads) fa_split_join_kernel(SplitParts parts, SplitOut out, long long n_rows) {
    constexpr int kLanes = D / 4, kRows = 32 / kLanes, kTeams = kThreads / 32 / WARPS;
    __shared__ float s_state[2][WARPS][kRows];   // of a row's warps: maxima, sums
    __shared__ float4 s_acc[WARPS][32];
    [[maybe_unused]] __shared__ int s_failed;  // a check's flag: nothing is in flight that would be given up
    wait_for_stream();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % kLanes, mine = warp % WARPS;
    const long long at = (static_cast<long long>(blockIdx.x) * kTeams + warp / WARPS) * kRows + lane / kLanes;
    const bool row_there = at < n_rows;
    if (WARPS == 1 && !row_there) return;
    const long long bhl = row_there ? at / out.R : 0;
    const int bh = static_cast<int>(bhl), r = static_cast<int>(row_there ? at - bhl * out.R : 0);
    const int unit = bh * out.row_units + r / out.unit_rows, local = r % out.unit_rows;
    int2 pieces = __ldcg(parts.units + unit);
    // A unit of one piece was finished by its CTA: its entry names no piece that was written, behind the last
    // cut unit not even one that the workspace holds.  (Its warps stay for the barriers.)
    if (!row_there || pieces.y <= 1) pieces.y = 0;
    if (WARPS == 1 && pieces.y == 0) return;
    if (pieces.y > 0 && !FA_CHECK(pieces.x >= 0 && pieces.x + pieces.y <= parts.count, &g_status_split_join, &s_failed))
        pieces.y = 0;
    const float* lse = parts.lse + static_cast<size_t>(pieces.x) * parts.rows + local;
    const float* o = parts.o + (static_cast<size_t>(pieces.x) * parts.rows + local) * D + 4 * sub;
    const size_t step = static_cast<size_t>(parts.rows);
    auto load = [&](int k0, float (&l)[kAtOnce]) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = (k0 + k) * WARPS + mine;
            l[k] = i < pieces.y ? __ldcg(lse + i * step) : -INFINITY;
        }
    };
    float4 x[kAtOnce];  // of the first pieces, on their way while the log-sum-exps are joined
    auto fetch = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = (k0 + k) * WARPS + mine;
            x[k] = i < pieces.y ? __ldcg(reinterpret_cast<const float4*>(o + i * step * D)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    const int n = (pieces.y + WARPS - 1) / WARPS;  // of a warp, at most
    fetch(0);
    float top = -INFINITY, sum = 0.f, l[kAtOnce];
    for (int k0 = 0; k0 < n; k0 += kAtOnce) {
        load(k0, l);
        float now = top;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) now = fmaxf(now, l[k]);
        sum *= top == now ? 1.f : ex2_approx(top - now);
        top = now;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (l[k] != -INFINITY) sum += ex2_approx(l[k] - top);  // (-inf: saw nothing)
    }
    if constexpr (WARPS > 1) {
        if (sub == 0) {
            s_state[0][mine][lane / kLanes] = top;
            s_state[1][mine][lane / kLanes] = sum;
        }
        __syncthreads();
        float all = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (s_state[1][w][lane / kLanes] != 0.f) all = fmaxf(all, s_state[0][w][lane / kLanes]);
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float s = s_state[1][w][lane / kLanes];
            if (s != 0.f) sum += s * ex2_approx(s_state[0][w][lane / kLanes] - all);
        }
        top = all;
    }
    // each weight divided by their sum first: pieces near the largest number must not overflow in between
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < n; k0 += kAtOnce) {
        if (n > kAtOnce) load(k0, l);
        if (k0 > 0) fetch(k0);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (l[k] == -INFINITY) continue;
            const float w = ex2_approx(l[k] - top) * inv;
            y[0] = fmaf(w, x[k].x, y[0]);
            y[1] = fmaf(w, x[k].y, y[1]);
            y[2] = fmaf(w, x[k].z, y[2]);
            y[3] = fmaf(w, x[k].w, y[3]);
        }
    }
    if constexpr (WARPS > 1) {
        s_acc[mine][lane] = make_float4(y[0], y[1], y[2], y[3]);
        __syncthreads();
        if (mine != 0 || pieces.y == 0) return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            const float4 z = s_acc[w][lane];
            y[0] += z.x;
            y[1] += z.y;
            y[2] += z.z;
            y[3] += z.w;
        }
    }
    const int b = bh / out.Hkv, h = bh % out.Hkv * out.group + r / out.T, t = r % out.T;
    const uint32_t w0 = pack_bf16x2(y[0], y[1]), w1 = pack_bf16x2(y[2], y[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out.o.ptr) + b * out.o.b + h * out.o.h + t * out.o.t + 4 * sub) =
        make_uint2(w0, w1);
    const size_t row = (static_cast<size_t>(b) * out.Hkv * out.group + h) * out.T + t;
    if (out.rest != nullptr)
        *reinterpret_cast<uint2*>(out.rest + row * D + 4 * sub) =
            make_uint2(pack_bf16x2(y[0] - __uint_as_float(w0 << 16), y[1] - __uint_as_float(w0 & 0xffff0000u)),
                       pack_bf16x2(y[2] - __uint_as_float(w1 << 16), y[3] - __uint_as_float(w1 & 0xffff0000u)));
    if (sub == 0) out.lse[row] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

template <int D, int WARPS>
int launch_t(const SplitParts& parts, const SplitOut& out, long long n, cudaStream_t stream) {
    constexpr int kRows = kThreads / 32 / WARPS * (128 / D);
    return launch_chained(fa_split_join_kernel<D, WARPS>, dim3(static_cast<unsigned>((n + kRows - 1) / kRows)), kThreads, 0,
                          stream, parts, out, n);
}

}  // namespace

int launch_split_join(const SplitParts& parts, const SplitOut& out, int B, int D, int items, cudaStream_t stream) {
    const long long n = static_cast<long long>(B) * out.Hkv * out.R;
    const long long units = static_cast<long long>(B) * out.Hkv * out.row_units;
    const bool wide = items >= 2 * kAtOnce * units;  // pieces of a unit, if its share is fair
    if (D == 64) return wide ? launch_t<64, 8>(parts, out, n, stream) : launch_t<64, 1>(parts, out, n, stream);
    return wide ? launch_t<128, 8>(parts, out, n, stream) : launch_t<128, 1>(parts, out, n, stream);
}

int split_join_take_status() {
    int h = 0;
#ifdef FA_DEBUG
    const int z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_split_join, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_split_join, &z, sizeof(int)) != cudaSuccess) return -5;
#endif
    return h;
}

}  // namespace fa
