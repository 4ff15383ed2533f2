// fa_internal.h -- declarations shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace fa {

struct DebugKnobs {
    unsigned long long timeout_ns;  // bound of every in-kernel wait
    int inject;                     // fault-injection mode (0 = off)
    cudaEvent_t ev[5];              // measurement hook: fwd begin/end; bwd: before dK/dV, between, after dQ (may be null)
    int deterministic;              // 1: the backward never sums into global memory (two-kernel form at every D)
};

// Status word values written by kernels (mirror of fa_status).
constexpr int kStatusTimeout = -7;
constexpr int kStatusBadSeqlen = -11;
constexpr int kStatusSmemAlign = -4;  // a kernel's dynamic shared-memory window was not 1024-byte aligned
constexpr int kStatusDebugCheck = -12;  // debug build: a run-time index failed its bounds check
constexpr int kStatusBadPage = -13;     // a page table names no page of the pool where a token lies

// Launchers: arguments already validated by the C-ABI layer.
// Hq query heads share Hkv key/value heads (Hq % Hkv == 0; Hkv == Hq is plain attention).
int launch_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int T,
               int D, float scale, bool causal, cudaStream_t stream, const DebugKnobs& dbg, int num_sms);
int launch_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
               void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int T, int D, float scale, bool causal,
               cudaStream_t stream, const DebugKnobs& dbg, int num_sms);

// Forward over a packed variable-length batch: (total, H, D) tensors, LSE (H, total).
int launch_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_seqlens,
                      int n_seq, int max_seqlen, int total, int H, int D, float scale, bool causal,
                      cudaStream_t stream, const DebugKnobs& dbg, int num_sms);

// Backward over a packed variable-length batch (the same layout; dq, dk, dv (total, H, D)).
int launch_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                      void* dq, void* dk, void* dv, const int* cu_seqlens, int n_seq, int max_seqlen, int total,
                      int H, int D, float scale, bool causal, cudaStream_t stream, const DebugKnobs& dbg,
                      int num_sms);

// Split-K decoding forward (fa_decode.cu).
int launch_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Tq, int Tk,
                  int D, float scale, cudaStream_t stream, int num_sms);

// Cross attention: Tq queries over Tk keys, key_lengths[b] (null: Tk) of them there, (B, heads, T, D)
// tensors by their strides in elements.
struct CrossShape {
    int B, Hq, Hkv, Tq, Tk, D;
    const int* key_lengths;
};
struct CrossTensor {
    void* ptr;
    long long b, h, t;
};
int launch_cross_fwd(const CrossShape& s, const CrossTensor& q, const CrossTensor& k, const CrossTensor& v,
                     const CrossTensor& o, void* o_rest, float* lse, float scale, cudaStream_t stream,
                     const DebugKnobs& dbg, int num_sms);
// The same for few rows a key/value head (fa_cross_rows.cu): whether it is the one to take, and its launch.
bool cross_rows_wanted(const CrossShape& s, int num_sms);
int launch_cross_rows(const CrossShape& s, const CrossTensor& q, const CrossTensor& k, const CrossTensor& v,
                      const CrossTensor& o, void* o_rest, float* lse, float scale, void* workspace,
                      cudaStream_t stream, const DebugKnobs& dbg, int num_sms);
size_t cross_rows_workspace(const CrossShape& s, int num_sms);  // 0 where they are not wanted
int cross_rows_take_status();
int split_join_take_status();  // of the debug build's checks
size_t cross_bwd_workspace(const CrossShape& s, bool deterministic, int num_sms);
int launch_cross_bwd(const CrossShape& s, const CrossTensor& q, const CrossTensor& k, const CrossTensor& v,
                     const CrossTensor& o, const void* o_rest, const CrossTensor& dO, const float* lse, const CrossTensor& dq,
                     const CrossTensor& dk, const CrossTensor& dv, float scale, void* workspace, cudaStream_t stream,
                     const DebugKnobs& dbg, int num_sms);

// Backward with the library's fixed device scratch buffer instead of an
// allocation; returns -10 if the problem does not fit, without launching.
size_t bwd_scratch_bytes(int B, int H, int T, int D);
// Whether fa_bwd sums dQ inside the dK/dV kernel for this shape on a GPU with num_sms SMs.
bool bwd_fuses_host(int B, int Hkv, int T, int D, int num_sms, bool deterministic);
int launch_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                       void* dq, void* dk, void* dv, int B, int H, int T, int D, float scale, bool causal,
                       cudaStream_t stream, const DebugKnobs& dbg, int num_sms);

// Rotary positions (fa_rope.cu).  One tensor (B, T, heads, D) by its strides in elements.
struct RopeTensor {
    const void* in;
    void* out;
    long long heads, in_b, in_t, in_h, out_b, out_t, out_h;
};
int launch_rope(const RopeTensor* tensors, int n_tensors, const void* positions, int pos64, long long pos_b,
                const void* freq, int B, int T, int D, int R, int interleaved, float amplitude, int inverse,
                int dtype, cudaStream_t stream, int num_sms);

// 4-bit paged key/value cache (fa_kv4_cache.cu, fa_kv4_decode.cu; layout in fa_kv4.cuh).
struct Kv4Shape {
    int B, Hkv, D, group, page_size, num_pages, width;
};
int launch_kv4_append(const Kv4Shape& c, void* pool, const int* table, const void* k, const void* v, long long k_t,
                      long long k_h, long long v_t, long long v_h, const int* lengths, const int* cu_new, int total,
                      const void* positions, int pos64, const void* freq, int R, int interleaved, float amplitude,
                      float* weights, int* slot_positions, long long slots, cudaStream_t stream, int num_sms);
int launch_kv4_read(const Kv4Shape& c, const void* pool, const int* table, const int* lengths, const int* start,
                    int count, void* k, void* v, cudaStream_t stream);
size_t kv4_evict_workspace(int B, int Hkv, int budget);
int launch_kv4_evict(const Kv4Shape& c, void* pool, const int* table, const int* lengths, const float* weights,
                     const int* slot_positions, long long slots, int budget, int recent, float* weights_out,
                     int* positions_out, int* lengths_out, int* source, void* workspace, cudaStream_t stream,
                     int num_sms);
size_t kv4_decode_workspace(const Kv4Shape& c, int Hq, int Tq, bool weights, int num_sms);
bool kv4_decode_fits(const Kv4Shape& c, int Hq, int Tq);  // whether the kernel's 32-bit line of units holds the shape
int launch_kv4_decode(const Kv4Shape& c, const void* pool, const int* table, const int* lengths, const void* q,
                      void* o, float* lse, int Hq, int Tq, float scale, bool causal, const float* weights,
                      float* weights_out, long long slots, void* workspace, cudaStream_t stream, int num_sms);
int launch_kv4_tree(const Kv4Shape& c, const void* pool, const int* table, const int* lengths, const int* parents,
                    const void* q, void* o, float* lse, int Hq, int N, float scale, void* workspace, cudaStream_t stream,
                    const DebugKnobs& dbg, int num_sms);
size_t kv4_tree_workspace(const Kv4Shape& c, int Hq, int N, int num_sms);
int launch_tree_accept(const int* parents, const void* tokens, const void* picks, const void* first, int tokens64, int B,
                       int N, int* path, int* counts, void* next, cudaStream_t stream);
int launch_kv4_keep(const Kv4Shape& c, void* pool, const int* table, const int* lengths, const int* path, int N,
                    int* lengths_out, float* weights, int* slot_positions, long long slots, cudaStream_t stream);
int kv4_tree_take_status();
int kv4_keep_take_status();
int kv4_cache_take_status();
int kv4_decode_take_status();

// Launches a kernel that may be scheduled while the one before it in the stream
// still runs: it hides the launch, and the kernel's first act is
// wait_for_stream(), which returns when that one is done and its writes are seen.
template <typename... Params, typename... Args>
inline int launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                          Args... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? 0 : -5;
}
#ifdef __CUDACC__
// Every thread of a chained kernel calls this before it reads or writes anything
// in global memory; the next chained kernel may be scheduled from here on.
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// Allows a kernel its dynamic shared memory, once per device (a microsecond a call otherwise).
template <typename Kernel>
inline bool allow_shared_memory(Kernel kernel, int bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Read and clear the device status word of each translation unit on the
// current device (caller synchronises first).  Return 0 or a negative code.
int fwd_take_status();
int bwd_take_status();

}  // namespace fa
