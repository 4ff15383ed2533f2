// fa_kv4_keep.cu -- after a model has run over a tree of drafted tokens: which of them
// stand (fa_tree_accept), and keeping those in the 4-bit paged cache (fa_kv4_keep).
//
// Accepting: place i stands if every token on its way from a root is what the model picked
// behind the one before it.  A warp a sequence: the ways as 64-bit masks (fa_tree.cuh), the mismatches
// as one more, a maximum of depth and place.
//
// Keeping: the codes and scales of the accepted places of a key/value head move to the first
// of the tree's slots.  A block a head reads all of them into registers and then writes: 64
// records of 144 or 160 bytes are at most ten words a thread.  Both are bound by latency, a launch and three
// or four dependent loads: 32 sequences of 8 heads and 16 places, 5.5 and 5.9 us from cold caches; both
// and a read back 11 us in a row.
#include <cuda_runtime.h>

#include "fa_check.cuh"
#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_tree.cuh"

namespace fa {

static __device__ int g_status_kv4_keep;

namespace {

constexpr int kAcceptWarps = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kAcceptWarps)
    fa_tree_accept_kernel(const int* parents, const T* tokens, const T* picks, const T* first, int B, int N, int* path,
                          int* counts, T* next) {
    wait_for_stream();
    const int b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= B) return;
    const long long row = static_cast<long long>(b) * N;
    unsigned long long up[2], wrong = 0;
    tree_ancestors(parents + row, N, lane, up);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        bool differs = false;
        if (i < N && up[x] != 0) {
            const unsigned long long before = up[x] & ~(1ull << i);  // its parent is the highest of them
            if (before != 0)
                differs = tokens[row + i] != picks[row + 63 - __clzll(static_cast<long long>(before))];
            else
                differs = first != nullptr && tokens[row + i] != first[b];
        }
        wrong |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, differs)) << (32 * x);
    }
    int best = -1;  // the deepest, then the lowest place
#pragma unroll
    for (int x = 0; x < 2; ++x)
        if (up[x] != 0 && (up[x] & wrong) == 0) best = max(best, __popcll(up[x]) * 64 + 63 - (lane + 32 * x));
    best = __reduce_max_sync(0xffffffffu, best);
    unsigned long long way = 0;
    const int end = 63 - (best & 63);
    if (best >= 0) {
        const unsigned long long a = __shfl_sync(0xffffffffu, up[0], end & 31),
                                 c = __shfl_sync(0xffffffffu, up[1], end & 31);
        way = end >= 32 ? c : a;
    }
    const int count = __popcll(way);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        if (i < N && i >= count) path[row + i] = -1;
        if (way >> i & 1) path[row + __popcll(way & ((1ull << i) - 1))] = i;
    }
    if (lane == 0) {
        counts[b] = count;
        next[b] = count > 0 ? picks[row + end] : first != nullptr ? first[b] : static_cast<T>(-1);
    }
}

constexpr int kKeepThreads = 256;

template <int D, int G>
__global__ void __launch_bounds__(kKeepThreads)
    fa_kv4_keep_kernel(Kv4Pages pages, const int* lengths, const int* path, int N, int* lengths_out, float* weights,
                       int* slot_positions, long long slots) {
    using L = Kv4<D, G>;
    constexpr int kCodeWords = L::kRow / 4, kScaleWords = L::kScaleRow / 4, kHalf = kCodeWords + kScaleWords;
    constexpr int kMost = (kTreePlaces * 2 * kHalf + kKeepThreads - 1) / kKeepThreads;
    __shared__ long long s_from[kTreePlaces], s_to[kTreePlaces];  // byte offsets of a token's row in its block, or -1
    __shared__ int s_path[kTreePlaces];
    [[maybe_unused]] __shared__ int s_failed;  // a check's flag: nothing is in flight that would be given up
    wait_for_stream();
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int len = __ldg(lengths + b);
    const long long room = weights != nullptr || slot_positions != nullptr ? min(slots, pages.capacity()) : pages.capacity();
    bool bad = len < 0 || len > room || (len > 0 && len < N);

    // every warp reads the path: n places, rising, up to the first -1
    int place[2], n = 0;
    bool wrong = false;
    unsigned long long ends = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        place[x] = i < N ? __ldg(path + static_cast<long long>(b) * N + i) : -1;
        ends |= static_cast<unsigned long long>(__ballot_sync(0xffffffffu, place[x] == -1)) << (32 * x);
    }
    n = ends != 0 ? __ffsll(static_cast<long long>(ends)) - 1 : kTreePlaces;
    const int last0 = __shfl_sync(0xffffffffu, place[0], 31);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x, up = __shfl_up_sync(0xffffffffu, place[x], 1);
        const int before = i == 0 ? -1 : lane == 0 ? last0 : up;
        wrong = wrong || (i < n && (place[x] <= before || place[x] >= N));
    }
    if (__any_sync(0xffffffffu, wrong) && len != 0) bad = true;
    if (bad || len == 0) {  // the sequence stays as it is
        if (h == 0 && tid == 0) {
            if (bad) atomicCAS(&g_status_kv4_keep, 0, kStatusBadSeqlen);
            lengths_out[b] = len;
        }
        return;
    }
    const int ctx = len - N;
    if (h == 0 && tid == 0) lengths_out[b] = ctx + n;
    if (tid < 32)
#pragma unroll
        for (int x = 0; x < 2; ++x) s_path[lane + 32 * x] = place[x];
    __syncthreads();
    if (tid < n) {
        const int from = ctx + s_path[tid], to = ctx + tid;
        const long long f = pages.block_of(b, from >> 4), t = pages.block_of(b, to >> 4);
        if (f < 0 || t < 0) atomicCAS(&g_status_kv4_keep, 0, kStatusBadPage);
        const long long bytes = static_cast<long long>(pages.num_pages) * pages.heads * pages.head_bytes();
        const bool moves = f >= 0 && t >= 0 && from != to &&
                           FA_CHECK(max(f, t) + h * pages.head_bytes() + L::kBlock <= bytes, &g_status_kv4_keep, &s_failed);
        s_from[tid] = moves ? f : -1;
        s_to[tid] = t;
    }
    __syncthreads();
    unsigned char* mine = pages.pool + h * pages.head_bytes();
    // word w of a token's record: of the keys' codes, their scales, the values' codes, their scales
    auto offset = [&](int w, int token) {
        const int part = w >= kHalf, v = w - part * kHalf;
        return part * L::kValueCodes + (v < kCodeWords ? token * L::kRow + v * 4
                                                       : L::kKeyScales + token * L::kScaleRow + (v - kCodeWords) * 4);
    };
    uint32_t held[kMost];
    float weight = 0.f;
    int position = 0;
    const bool account = tid < n && s_from[tid] >= 0;  // as the codes: one whose page is bad is left out of both
    const long long at = (static_cast<long long>(b) * pages.heads + h) * slots + ctx;
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int x = tid + k * kKeepThreads, i = x / (2 * kHalf), w = x - i * (2 * kHalf);
        if (i < n && s_from[i] >= 0)
            held[k] = *reinterpret_cast<const uint32_t*>(mine + s_from[i] + offset(w, (ctx + s_path[i]) & 15));
    }
    if (account && weights != nullptr) weight = weights[at + s_path[tid]];
    if (account && slot_positions != nullptr) position = slot_positions[at + s_path[tid]];
    __syncthreads();  // all is read
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int x = tid + k * kKeepThreads, i = x / (2 * kHalf), w = x - i * (2 * kHalf);
        if (i < n && s_from[i] >= 0)
            *reinterpret_cast<uint32_t*>(mine + s_to[i] + offset(w, (ctx + i) & 15)) = held[k];
    }
    if (account && weights != nullptr) weights[at + tid] = weight;
    if (account && slot_positions != nullptr) slot_positions[at + tid] = position;
}

template <int D, int G>
int launch_keep_t(const Kv4Pages& pages, int B, const int* lengths, const int* path, int N, int* lengths_out,
                  float* weights, int* slot_positions, long long slots, cudaStream_t stream) {
    return launch_chained(fa_kv4_keep_kernel<D, G>, dim3(pages.heads, B), kKeepThreads, 0, stream, pages, lengths, path, N,
                          lengths_out, weights, slot_positions, slots);
}

}  // namespace

int launch_tree_accept(const int* parents, const void* tokens, const void* picks, const void* first, int tokens64, int B,
                       int N, int* path, int* counts, void* next, cudaStream_t stream) {
    const dim3 grid((B + kAcceptWarps - 1) / kAcceptWarps);
    if (tokens64)
        return launch_chained(fa_tree_accept_kernel<long long>, grid, 32 * kAcceptWarps, 0, stream, parents,
                              static_cast<const long long*>(tokens), static_cast<const long long*>(picks),
                              static_cast<const long long*>(first), B, N, path, counts, static_cast<long long*>(next));
    return launch_chained(fa_tree_accept_kernel<int>, grid, 32 * kAcceptWarps, 0, stream, parents,
                          static_cast<const int*>(tokens), static_cast<const int*>(picks), static_cast<const int*>(first),
                          B, N, path, counts, static_cast<int*>(next));
}

int launch_kv4_keep(const Kv4Shape& c, void* pool, const int* table, const int* lengths, const int* path, int N,
                    int* lengths_out, float* weights, int* slot_positions, long long slots, cudaStream_t stream) {
    const Kv4Pages pages = kv4_pages(static_cast<unsigned char*>(pool), table, c.width, c.num_pages, c.Hkv, c.page_size,
                                     c.D, c.group);
    const auto launch = c.D == 64 ? (c.group == 32 ? launch_keep_t<64, 32> : launch_keep_t<64, 64>)
                                  : (c.group == 32 ? launch_keep_t<128, 32> : launch_keep_t<128, 64>);
    return launch(pages, c.B, lengths, path, N, lengths_out, weights, slot_positions, slots, stream);
}

int kv4_keep_take_status() {
    int h = 0, z = 0;
    if (cudaMemcpyFromSymbol(&h, g_status_kv4_keep, sizeof(int)) != cudaSuccess) return -5;
    if (cudaMemcpyToSymbol(g_status_kv4_keep, &z, sizeof(int)) != cudaSuccess) return -5;
    return h;
}

}  // namespace fa
