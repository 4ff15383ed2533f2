// fa_kv4_decode.cu -- attention of a few query rows over the 4-bit paged cache.
//
// With k = s n + m and v = s n + m per group g of channels (fa_kv4.cuh),
//   S_t = scale sum_g ( s_tg (q_g . n_tg) + m_tg sum(q_g) ),  P = softmax(S),
//   O_c = sum_t P_t (s_tg n_tc + m_tg).
// The tokens of each sequence are split over CTAs, each keeping a running
// maximum and sum, and a second kernel joins the parts, as in fa_decode.cu.
// With weights, the scores are kept as well and a third kernel adds every
// slot's attention weight, summed over the query rows, to its account.
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

__device__ int g_status_kv4_decode = 0;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWarps = 4;
constexpr int kRows = 8;  // query rows of one CTA

struct DecParams {
    const __nv_bfloat16* q;
    Kv4Pages pages;
    const int* lengths;
    float* part_m;    // [B Hkv][n_split][R]
    float* part_l;
    float* part_acc;  // [B Hkv][n_split][R][D]
    float* scores;    // [B Hkv][R][cap] in log2 units, or null
    __nv_bfloat16* o;
    float* lse;
    const float* weights;
    float* weights_out;
    long long slots, cap;
    int R, Tq, causal, n_split;
    float sl2;  // scale log2(e)
};

// Length of sequence b, 0 (and a status) if the table or the accounts cannot hold it.
__device__ __forceinline__ int length_of(const DecParams& p, int b) {
    const int len = p.lengths[b];
    if (len < 0 || len > p.pages.capacity() || (p.weights_out != nullptr && len > p.slots)) {
        atomicCAS(&g_status_kv4_decode, 0, kStatusBadSeqlen);
        return 0;
    }
    return len;
}
// Tokens that query row r sees.
__device__ __forceinline__ int seen_by(const DecParams& p, int r, int len) {
    return p.causal ? max(0, len - (p.Tq - 1 - r % p.Tq)) : len;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Code of channel c in a row of key or value codes.
template <int D>
__device__ __forceinline__ float key_code(const unsigned char* row, int c) {
    const int n = 8 * ((c % 32) / 8 * (D / 32) + c / 32) + c % 8;
    return static_cast<float>(row[n >> 1] >> (4 * (n & 1)) & 15);
}
template <int D>
__device__ __forceinline__ float value_code(const unsigned char* row, int c) {
    const int n = 4 * ((c % 32) / 4 * (D / 32) + c / 32) + c % 4;
    return static_cast<float>(row[n >> 1] >> (4 * (n & 1)) & 15);
}

// One warp takes one token at a time, lane = D/32 channels.
template <int D, int G>
__global__ void __launch_bounds__(kWarps * 32) fa_kv4_decode_kernel(DecParams p) {
    using L = Kv4<D, G>;
    constexpr int E = D / 32;
    const int split = blockIdx.x, bh = blockIdx.y, r0 = blockIdx.z * kRows;
    const int b = bh / p.pages.heads, h = bh % p.pages.heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = min(kRows, p.R - r0);
    const int len = length_of(p, b);
    const int chunk = (len + p.n_split - 1) / p.n_split;
    const int t0 = split * chunk, t1 = min(len, t0 + chunk);
    float q[kRows][E], m[kRows], l[kRows], acc[kRows][E];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[r][e] = r < rows ? __bfloat162float(p.q[(static_cast<long long>(bh) * p.R + r0 + r) * D + e * 32 + lane]) : 0.f;
            acc[r][e] = 0.f;
        }
    }
    for (int t = t0 + warp; t < t1; t += kWarps) {
        const long long at = p.pages.block_of(b, t >> 4);
        if (at < 0) {
            if (lane == 0) atomicCAS(&g_status_kv4_decode, 0, kStatusBadPage);
            if (p.scores != nullptr && lane < rows)
                p.scores[(static_cast<long long>(bh) * p.R + r0 + lane) * p.cap + t] = -INFINITY;
            continue;
        }
        const unsigned char* block = p.pages.pool + at + h * p.pages.head_bytes();
        const int i = t & 15;
        float kf[E], vf[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = e * 32 + lane, g = c / G;
            const float2 ks = kv4_scale(reinterpret_cast<const uint32_t*>(block + L::kKeyScales + i * L::kScaleRow)[g]);
            const float2 vs = kv4_scale(reinterpret_cast<const uint32_t*>(block + L::kValueScales + i * L::kScaleRow)[g]);
            kf[e] = fmaf(key_code<D>(block + L::kKeyCodes + i * L::kRow, c), ks.x, ks.y);
            vf[e] = fmaf(value_code<D>(block + L::kValueCodes + i * L::kRow, c), vs.x, vs.y);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= rows) break;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(q[r][e], kf[e], s);
            s = warp_sum(s) * p.sl2;
            if (t >= seen_by(p, r0 + r, len)) s = -INFINITY;
            if (p.scores != nullptr && lane == 0)
                p.scores[(static_cast<long long>(bh) * p.R + r0 + r) * p.cap + t] = s;
            if (s == -INFINITY) continue;
            const float m_new = fmaxf(m[r], s);
            const float alpha = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - m_new);
            const float w = ex2_approx(s - m_new);
            l[r] = l[r] * alpha + w;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[r][e] = fmaf(acc[r][e], alpha, w * vf[e]);
            m[r] = m_new;
        }
    }
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    __shared__ float sm_acc[kWarps][kRows][D];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (lane == 0) {
            sm_m[warp][r] = m[r];
            sm_l[warp][r] = l[r];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sm_acc[warp][r][e * 32 + lane] = acc[r][e];
    }
    __syncthreads();
    for (int r = warp; r < rows; r += kWarps) {
        float mm = -INFINITY, ll = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = sm_l[w][r] == 0.f ? 0.f : ex2_approx(sm_m[w][r] - mm);
            ll = fmaf(f[w], sm_l[w][r], ll);
        }
        const long long at = (static_cast<long long>(bh) * p.n_split + split) * p.R + r0 + r;
        for (int d = lane; d < D; d += 32) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) a = fmaf(f[w], sm_acc[w][r][d], a);
            p.part_acc[at * D + d] = a;
        }
        if (lane == 0) {
            p.part_m[at] = mm;
            p.part_l[at] = ll;
        }
    }
}

// One warp per query row: join the parts.
template <int D>
__global__ void __launch_bounds__(128) fa_kv4_merge_kernel(DecParams p, int n_rows) {
    const int row = (blockIdx.x * 128 + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (row >= n_rows) return;
    const int bh = row / p.R, r = row % p.R;
    auto at = [&](int s) { return (static_cast<long long>(bh) * p.n_split + s) * p.R + r; };
    float mm = -INFINITY, ll = 0.f;
    for (int s = 0; s < p.n_split; ++s) mm = fmaxf(mm, p.part_m[at(s)]);
    for (int s = 0; s < p.n_split; ++s)
        if (p.part_l[at(s)] != 0.f) ll = fmaf(ex2_approx(p.part_m[at(s)] - mm), p.part_l[at(s)], ll);
    for (int d = lane; d < D; d += 32) {
        float a = 0.f;
        for (int s = 0; s < p.n_split; ++s)
            if (p.part_l[at(s)] != 0.f) a = fmaf(ex2_approx(p.part_m[at(s)] - mm), p.part_acc[at(s) * D + d], a);
        p.o[static_cast<long long>(row) * D + d] = __float2bfloat16_rn(ll == 0.f ? 0.f : a / ll);
    }
    if (lane == 0) p.lse[row] = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * kLn2;
}

// weights_out = weights + the sum over the rows of P, slot by slot.
__global__ void __launch_bounds__(256) fa_kv4_weights_kernel(DecParams p) {
    const int bh = blockIdx.y, b = bh / p.pages.heads;
    const int len = length_of(p, b);
    for (long long t = blockIdx.x * 256 + threadIdx.x; t < len; t += gridDim.x * 256) {
        float sum = 0.f;
        for (int r = 0; r < p.R; ++r) {
            const float lse = p.lse[static_cast<long long>(bh) * p.R + r];
            if (t < seen_by(p, r, len))
                sum += ex2_approx(p.scores[(static_cast<long long>(bh) * p.R + r) * p.cap + t] - lse * kLog2e);
        }
        const long long at = bh * p.slots + t;
        p.weights_out[at] = (p.weights != nullptr ? p.weights[at] : 0.f) + sum;
    }
}

int splits_of(const Kv4Shape& c, int num_sms) {
    const long long bh = static_cast<long long>(c.B) * c.Hkv, cap = static_cast<long long>(c.width) * c.page_size;
    long long n = (16LL * num_sms + bh - 1) / bh;
    const long long most = (cap + 255) / 256;
    if (n > most) n = most;
    return n < 1 ? 1 : static_cast<int>(n);
}

}  // namespace

size_t kv4_decode_workspace(const Kv4Shape& c, int Hq, int Tq, bool weights, int num_sms) {
    const size_t rows = static_cast<size_t>(c.B) * Hq * Tq;
    return rows * splits_of(c, num_sms) * (c.D + 2) * 4 +
           (weights ? rows * static_cast<size_t>(c.width) * c.page_size * 4 : 0);
}

int launch_kv4_decode(const Kv4Shape& c, const void* pool, const int* table, const int* lengths, const void* q,
                      void* o, float* lse, int Hq, int Tq, float scale, bool causal, const float* weights,
                      float* weights_out, long long slots, void* workspace, cudaStream_t stream, int num_sms) {
    DecParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.pages.pool = static_cast<unsigned char*>(const_cast<void*>(pool));
    p.pages.table = table;
    p.pages.width = c.width;
    p.pages.num_pages = c.num_pages;
    p.pages.heads = c.Hkv;
    p.pages.blocks_page = c.page_size / 16;
    p.pages.block_bytes = 16LL * (c.D + 8 * c.D / c.group);
    p.lengths = lengths;
    p.R = Hq / c.Hkv * Tq;
    p.Tq = Tq;
    p.causal = causal;
    p.n_split = splits_of(c, num_sms);
    p.cap = static_cast<long long>(c.width) * c.page_size;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.weights = weights;
    p.weights_out = weights_out;
    p.slots = slots;
    p.sl2 = scale * kLog2e;
    const int bh = c.B * c.Hkv;
    const size_t parts = static_cast<size_t>(bh) * p.n_split * p.R;
    p.part_acc = static_cast<float*>(workspace);
    p.part_m = p.part_acc + parts * c.D;
    p.part_l = p.part_m + parts;
    p.scores = weights_out != nullptr ? p.part_l + parts : nullptr;
    const dim3 grid(p.n_split, bh, (p.R + kRows - 1) / kRows);
    if (c.D == 64) {
        if (c.group == 32) fa_kv4_decode_kernel<64, 32><<<grid, kWarps * 32, 0, stream>>>(p);
        else fa_kv4_decode_kernel<64, 64><<<grid, kWarps * 32, 0, stream>>>(p);
    } else {
        if (c.group == 32) fa_kv4_decode_kernel<128, 32><<<grid, kWarps * 32, 0, stream>>>(p);
        else fa_kv4_decode_kernel<128, 64><<<grid, kWarps * 32, 0, stream>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) return -5;
    const int rows = bh * p.R, blocks = (rows + 3) / 4;
    if (c.D == 64) fa_kv4_merge_kernel<64><<<blocks, 128, 0, stream>>>(p, rows);
    else fa_kv4_merge_kernel<128><<<blocks, 128, 0, stream>>>(p, rows);
    if (cudaGetLastError() != cudaSuccess) return -5;
    if (weights_out != nullptr) {
        long long n = (p.cap + 255) / 256;
        const long long most = (16LL * num_sms + bh - 1) / bh;
        fa_kv4_weights_kernel<<<dim3(static_cast<unsigned>(n < most ? n : most), bh), 256, 0, stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) return -5;
    }
    return 0;
}

int kv4_decode_take_status() {
    int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_kv4_decode, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_kv4_decode, &z, sizeof(int)) != cudaSuccess) return -5;
    return h;
}

}  // namespace fa
