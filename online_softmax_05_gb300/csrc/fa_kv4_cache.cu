// fa_kv4_cache.cu -- writing to the 4-bit paged key/value cache, reading it
// back, and evicting from it (layout: fa_kv4.cuh).
#include <cuda_runtime.h>

#include <climits>

#include "fa_internal.h"
#include "fa_kv4.cuh"

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

// Sequence of packed row t: the last b with cu[b] <= t, or -1.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int t) {
    if (t < cu[0] || t >= cu[B]) return -1;
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Channel c of a key row at position `pos`, rotated and rounded to bf16.
__device__ __forceinline__ float rotated(const AppendParams& p, const __nv_bfloat16* row, int c, long long pos) {
    const float x = __bfloat162float(row[c]);
    if (c >= p.R) return x;
    const int half = p.R >> 1;
    const int pair = p.interleaved ? c >> 1 : (c < half ? c : c - half);
    const bool first = p.interleaved ? (c & 1) == 0 : c < half;
    const int other = p.interleaved ? c ^ 1 : (first ? c + half : c - half);
    const float y = __bfloat162float(row[other]);
    const unsigned long long turn = static_cast<unsigned long long>(pos) * p.freq[pair];
    float s, co;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &s, &co);  // 2^-31
    s *= p.amp;
    co *= p.amp;
    return __bfloat162float(__float2bfloat16_rn(first ? x * co - y * s : x * co + y * s));
}

// One thread quantises 8 channels of one key or value row; the G/8 threads of
// a group find its range with shuffles.
template <int D, int G>
__global__ void __launch_bounds__(256) fa_kv4_append_kernel(AppendParams p) {
    using L = Kv4<D, G>;
    constexpr int kOct = D / 8;
    const long long item = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int oct = static_cast<int>(item % kOct);
    const int is_v = static_cast<int>(item / kOct) & 1;
    const long long th = item / (2 * kOct);
    const int h = static_cast<int>(th % p.pages.heads);
    const long long t_long = th / p.pages.heads;
    const int t = static_cast<int>(t_long < p.total ? t_long : p.total - 1);
    bool live = t_long < p.total;
    const int b = sequence_of(p.cu_new, p.B, t);
    live = live && b >= 0;
    long long slot = 0, pos = 0;
    unsigned char* block = nullptr;
    if (live) {
        const int n = p.cu_new[b + 1] - p.cu_new[b];
        slot = static_cast<long long>(p.lengths[b]) - n + (t - p.cu_new[b]);
        if (slot < 0 || slot >= p.pages.capacity() || (p.slots != 0 && slot >= p.slots)) {
            report(kStatusBadSeqlen);
            live = false;
        } else {
            const long long at = p.pages.block_of(b, static_cast<int>(slot >> 4));
            if (at < 0) {
                report(kStatusBadPage);
                live = false;
            } else {
                block = p.pages.pool + at + h * p.pages.head_bytes();
            }
            pos = slot;
            if (p.positions != nullptr)
                pos = p.pos64 ? static_cast<const long long*>(p.positions)[t]
                              : static_cast<long long>(static_cast<const int*>(p.positions)[t]);
        }
    }
    const __nv_bfloat16* row = is_v ? p.v + t * p.v_t + h * p.v_h : p.k + t * p.k_t + h * p.k_h;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!is_v && p.freq != nullptr) x[i] = rotated(p, row, oct * 8 + i, pos);
        else x[i] = __bfloat162float(row[oct * 8 + i]);
    }
    float lo = x[0], hi = x[0];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        nan = nan || isnan(x[i]);
    }
    if (nan) hi = INFINITY;  // makes the range infinite
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const float range = __fsub_rn(hi, lo);
    float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(range, 15.f)));
    const bool bad = !(range <= 3.402823466e38f);
    if (s < 7.888609052210118e-31f) s = 0.f;  // 2^-100
    uint32_t word = 0;
    if (!bad && s > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = fminf(rintf(__fdiv_rn(__fsub_rn(x[i], lo), s)), 15.f);
            word |= static_cast<uint32_t>(c) << (4 * i);
        }
    }
    if (!live) return;
    const int r = static_cast<int>(slot & 15), g = oct >> 2, j = oct & 3;
    if (is_v) {
        unsigned short* codes = reinterpret_cast<unsigned short*>(block + L::kValueCodes + r * L::kRow);
        codes[(2 * j) * (D / 32) + g] = static_cast<unsigned short>(word);
        codes[(2 * j + 1) * (D / 32) + g] = static_cast<unsigned short>(word >> 16);
    } else {
        reinterpret_cast<uint32_t*>(block + L::kKeyCodes + r * L::kRow)[j * (D / 32) + g] = word;
    }
    if (oct % (G / 8) == 0) {
        const __nv_bfloat162 sm = bad ? __floats2bfloat162_rn(NAN, NAN) : __floats2bfloat162_rn(s, lo);
        *reinterpret_cast<__nv_bfloat162*>(block + (is_v ? L::kValueScales : L::kKeyScales) + r * L::kScaleRow +
                                           oct / (G / 8) * 4) = sm;
    }
    if (is_v == 0 && oct == 0) {
        const long long at = (static_cast<long long>(b) * p.pages.heads + h) * p.slots + slot;
        if (p.weights != nullptr) p.weights[at] = 0.f;
        if (p.slot_positions != nullptr) p.slot_positions[at] = static_cast<int>(pos);
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
    long long items;
};

// One thread restores 8 channels of a token's key and value.
template <int D, int G>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(ReadParams p) {
    using L = Kv4<D, G>;
    constexpr int kOct = D / 8;
    const long long item = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (item >= p.items) return;
    const int oct = static_cast<int>(item % kOct);
    const long long row = item / kOct;
    const int i = static_cast<int>(row % p.count);
    const long long bh = row / p.count;
    const int h = static_cast<int>(bh % p.pages.heads), b = static_cast<int>(bh / p.pages.heads);
    const long long slot = (p.start != nullptr ? static_cast<long long>(p.start[b]) : 0) + i;
    uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (slot < p.lengths[b]) {
        long long at = -1;
        if (slot < 0 || slot >= p.pages.capacity()) {
            report(kStatusBadSeqlen);
        } else {
            at = p.pages.block_of(b, static_cast<int>(slot >> 4));
            if (at < 0) report(kStatusBadPage);
        }
        if (at >= 0) {
            const unsigned char* block = p.pages.pool + at + h * p.pages.head_bytes();
            const int r = static_cast<int>(slot & 15), g = oct >> 2, j = oct & 3;
            const uint32_t kw = reinterpret_cast<const uint32_t*>(block + L::kKeyCodes + r * L::kRow)[j * (D / 32) + g];
            const unsigned short* vc = reinterpret_cast<const unsigned short*>(block + L::kValueCodes + r * L::kRow);
            const uint32_t vw = vc[2 * j * (D / 32) + g] | static_cast<uint32_t>(vc[(2 * j + 1) * (D / 32) + g]) << 16;
            const int so = r * L::kScaleRow + oct / (G / 8) * 4;
            const float2 ks = kv4_scale(*reinterpret_cast<const uint32_t*>(block + L::kKeyScales + so));
            const float2 vs = kv4_scale(*reinterpret_cast<const uint32_t*>(block + L::kValueScales + so));
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t word = w ? vw : kw;
                const float2 sm = w ? vs : ks;
                uint32_t pk[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(
                        fmaf(static_cast<float>(word >> (8 * e) & 15u), sm.x, sm.y),
                        fmaf(static_cast<float>(word >> (8 * e + 4) & 15u), sm.x, sm.y));
                    pk[e] = *reinterpret_cast<const uint32_t*>(&y);
                }
                out[w] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
        }
    }
    reinterpret_cast<uint4*>(p.k)[item] = out[0];
    reinterpret_cast<uint4*>(p.v)[item] = out[1];
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
    Kv4Pages x;
    x.pool = static_cast<unsigned char*>(pool);
    x.table = table;
    x.width = c.width;
    x.num_pages = c.num_pages;
    x.heads = c.Hkv;
    x.blocks_page = c.page_size / 16;
    x.block_bytes = 16LL * (c.D + 8 * c.D / c.group);
    return x;
}

int last_error() { return cudaGetLastError() == cudaSuccess ? 0 : -5; }

}  // namespace

int launch_kv4_append(const Kv4Shape& c, void* pool, const int* table, const void* k, const void* v, long long k_t,
                      long long k_h, long long v_t, long long v_h, const int* lengths, const int* cu_new, int total,
                      const void* positions, int pos64, const void* freq, int R, int interleaved, float amplitude,
                      float* weights, int* slot_positions, long long slots, cudaStream_t stream) {
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
    const long long items = static_cast<long long>(total) * c.Hkv * (c.D / 4);
    const unsigned blocks = static_cast<unsigned>((items + 255) / 256);
    if (c.D == 64) {
        if (c.group == 32) fa_kv4_append_kernel<64, 32><<<blocks, 256, 0, stream>>>(p);
        else fa_kv4_append_kernel<64, 64><<<blocks, 256, 0, stream>>>(p);
    } else {
        if (c.group == 32) fa_kv4_append_kernel<128, 32><<<blocks, 256, 0, stream>>>(p);
        else fa_kv4_append_kernel<128, 64><<<blocks, 256, 0, stream>>>(p);
    }
    return last_error();
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
    p.items = static_cast<long long>(c.B) * c.Hkv * count * (c.D / 8);
    const unsigned blocks = static_cast<unsigned>((p.items + 255) / 256);
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
