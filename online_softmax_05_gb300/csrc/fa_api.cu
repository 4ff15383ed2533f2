// fa_api.cu -- the C ABI of libfa.so (declared in include/fa.h): argument
// validation, device checks and dispatch to the kernel launchers.  Every
// argument check runs before the first CUDA call, so a rejected call enqueues
// nothing and needs no GPU.
#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa.h"
#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_sched.h"

namespace {

std::atomic<unsigned long long> g_timeout_ns{2000000000ull};
std::atomic<int> g_inject{0};
std::atomic<int> g_deterministic{0};
std::atomic<void*> g_events[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};

constexpr int kMaxDevices = 64;
std::once_flag g_dev_once[kMaxDevices];
int g_dev_sms[kMaxDevices];
int g_dev_arch_ok[kMaxDevices];

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_shape(int B, int H, int T, int D, float scale, int causal) {
    if (B < 1 || H < 1 || T < 1) return FA_ERR_SHAPE;
    const long long rows = static_cast<long long>(B) * H * T;
    if (rows > INT_MAX || static_cast<long long>(B) * H > (1 << 30)) return FA_ERR_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if (causal != 0 && causal != 1) return FA_ERR_ARG;
    if (!std::isfinite(scale)) return FA_ERR_ARG;
    return FA_OK;
}

struct Range {
    uintptr_t lo, hi;
};
Range range_of(const void* p, size_t bytes) {
    uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Resolve the current device, its SM count and whether it is sm_103.
int current_device(int* dev_out, int* sms_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
    std::call_once(g_dev_once[dev], [dev] {
        int major = 0, minor = 0, sms = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        g_dev_sms[dev] = sms;
        g_dev_arch_ok[dev] = (major == 10 && minor == 3) ? 1 : 0;
    });
    if (!g_dev_arch_ok[dev]) return FA_ERR_ARCH;
    *dev_out = dev;
    *sms_out = g_dev_sms[dev] > 0 ? g_dev_sms[dev] : 1;
    return FA_OK;
}

fa::DebugKnobs knobs() {
    fa::DebugKnobs k{g_timeout_ns.load(), g_inject.load(), {}, g_deterministic.load()};
    for (int i = 0; i < 5; ++i) k.ev[i] = static_cast<cudaEvent_t>(g_events[i].load());
    return k;
}

}  // namespace

extern "C" {

int fa_version(void) { return 100; }

const char* fa_strerror(int status) {
    switch (status) {
        case FA_OK: return "ok";
        case FA_ERR_NULL: return "a required pointer is NULL";
        case FA_ERR_SHAPE: return "B, H and T (Tq, Tk) must be >= 1 and B*H*T must fit in a 32-bit index";
        case FA_ERR_UNSUPPORTED: return "head dimension D must be 64 or 128 (and fa_decode takes at most 8 query rows)";
        case FA_ERR_ALIGN: return "tensor base pointers must be 16-byte aligned";
        case FA_ERR_CUDA: return "a CUDA runtime or driver call failed";
        case FA_ERR_NOMEM: return "stream-ordered workspace allocation failed";
        case FA_ERR_DEVICE_TIMEOUT: return "a kernel's bounded wait ran out (pipeline stall); outputs are invalid";
        case FA_ERR_ARG: return "causal must be 0 or 1, scale finite, and outputs must not overlap other buffers (or another argument is out of its range)";
        case FA_ERR_ARCH: return "the current device is not compute capability 10.3 (sm_103a)";
        case FA_ERR_SEQLEN: return "a cu_seqlens length is negative or above max_seqlen, or a cache's length, slot or position is outside its block table or accounts (recorded by the kernel)";
        case FA_ERR_SCRATCH: return "fa_bwd_noalloc: the problem needs more than the fixed 64 MiB scratch buffer";
        case FA_ERR_PAGE: return "a block table names no page of the pool where a token lies (recorded by the kernel)";
        case FA_ERR_DEBUG_CHECK: return "debug library: a kernel's run-time index failed its bounds check (access skipped)";
        default: return "unknown fa_status";
    }
}

}  // extern "C"

namespace {

// Shared checks and dispatch of the forward; Hq query heads over Hkv K/V heads.
int fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int T, int D,
             float scale, int causal, void* stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
    if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return FA_ERR_SHAPE;
    int rc = check_shape(B, Hq, T, D, scale, causal);
    if (rc != FA_OK) return rc;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_ALIGN;
    const size_t nq = static_cast<size_t>(B) * Hq * T * D * 2, nk = static_cast<size_t>(B) * Hkv * T * D * 2;
    const size_t nl = static_cast<size_t>(B) * Hq * T * 4;
    const Range rq = range_of(q, nq), rk = range_of(k, nk), rv = range_of(v, nk), ro = range_of(o, nq),
                rl = range_of(lse, nl);
    if (overlap(ro, rq) || overlap(ro, rk) || overlap(ro, rv) || overlap(ro, rl) || overlap(rl, rq) ||
        overlap(rl, rk) || overlap(rl, rv))
        return FA_ERR_ARG;
    int dev = 0, sms = 0;
    rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_fwd(q, k, v, o, lse, B, Hq, Hkv, T, D, scale, causal != 0, static_cast<cudaStream_t>(stream),
                          knobs(), sms);
}

// Shared checks and dispatch of the backward.
int bwd_impl(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse, void* dq,
             void* dk, void* dv, int B, int Hq, int Hkv, int T, int D, float scale, int causal, void* stream) {
    if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return FA_ERR_NULL;
    if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0) return FA_ERR_SHAPE;
    int rc = check_shape(B, Hq, T, D, scale, causal);
    if (rc != FA_OK) return rc;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) || !aligned16(lse) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return FA_ERR_ALIGN;
    const size_t nq = static_cast<size_t>(B) * Hq * T * D * 2, nk = static_cast<size_t>(B) * Hkv * T * D * 2;
    const size_t nl = static_cast<size_t>(B) * Hq * T * 4;
    const Range ins[6] = {range_of(q, nq), range_of(k, nk), range_of(v, nk), range_of(o, nq), range_of(dO, nq),
                          range_of(lse, nl)};
    const Range outs[3] = {range_of(dq, nq), range_of(dk, nk), range_of(dv, nk)};
    for (int a = 0; a < 3; ++a) {
        for (int b = 0; b < 6; ++b)
            if (overlap(outs[a], ins[b])) return FA_ERR_ARG;
        for (int b = a + 1; b < 3; ++b)
            if (overlap(outs[a], outs[b])) return FA_ERR_ARG;
    }
    int dev = 0, sms = 0;
    rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, T, D, scale, causal != 0,
                          static_cast<cudaStream_t>(stream), knobs(), sms);
}

}  // namespace

extern "C" {

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int T, int D, float scale,
           int causal, void* stream) {
    return fwd_impl(q, k, v, o, lse, B, H, H, T, D, scale, causal, stream);
}

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse, void* dq,
           void* dk, void* dv, int B, int H, int T, int D, float scale, int causal, void* stream) {
    return bwd_impl(q, k, v, o, dO, lse, dq, dk, dv, B, H, H, T, D, scale, causal, stream);
}

int fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int T,
               int D, float scale, int causal, void* stream) {
    return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, T, D, scale, causal, stream);
}

int fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse, void* dq,
               void* dk, void* dv, int B, int Hq, int Hkv, int T, int D, float scale, int causal, void* stream) {
    return bwd_impl(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, T, D, scale, causal, stream);
}

int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_seqlens, int n_seq,
                  int max_seqlen, int total, int H, int D, float scale, int causal, void* stream) {
    if (!q || !k || !v || !o || !lse || !cu_seqlens) return FA_ERR_NULL;
    if (n_seq < 1 || max_seqlen < 1 || total < 1 || H < 1) return FA_ERR_SHAPE;
    if (static_cast<long long>(total) * H > INT_MAX || static_cast<long long>(n_seq) * H > (1 << 30))
        return FA_ERR_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if (causal != 0 && causal != 1) return FA_ERR_ARG;
    if (!std::isfinite(scale)) return FA_ERR_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
        (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
        return FA_ERR_ALIGN;
    const size_t n = static_cast<size_t>(total) * H * D * 2, nl = static_cast<size_t>(total) * H * 4;
    const Range rq = range_of(q, n), rk = range_of(k, n), rv = range_of(v, n), ro = range_of(o, n),
                rl = range_of(lse, nl), rc_ = range_of(cu_seqlens, static_cast<size_t>(n_seq + 1) * 4);
    if (overlap(ro, rq) || overlap(ro, rk) || overlap(ro, rv) || overlap(ro, rl) || overlap(rl, rq) ||
        overlap(rl, rk) || overlap(rl, rv) || overlap(ro, rc_) || overlap(rl, rc_))
        return FA_ERR_ARG;
    int dev = 0, sms = 0;
    int rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_fwd_varlen(q, k, v, o, lse, cu_seqlens, n_seq, max_seqlen, total, H, D, scale, causal != 0,
                                 static_cast<cudaStream_t>(stream), knobs(), sms);
}

int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                  void* dq, void* dk, void* dv, const int* cu_seqlens, int n_seq, int max_seqlen, int total, int H,
                  int D, float scale, int causal, void* stream) {
    if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv || !cu_seqlens) return FA_ERR_NULL;
    if (n_seq < 1 || max_seqlen < 1 || total < 1 || H < 1) return FA_ERR_SHAPE;
    if (static_cast<long long>(total) * H > INT_MAX || static_cast<long long>(n_seq) * H > (1 << 30) ||
        static_cast<long long>(n_seq) * H * ((max_seqlen + 127) / 128) > INT_MAX)
        return FA_ERR_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if (causal != 0 && causal != 1) return FA_ERR_ARG;
    if (!std::isfinite(scale)) return FA_ERR_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) || !aligned16(lse) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
        return FA_ERR_ALIGN;
    const size_t n = static_cast<size_t>(total) * H * D * 2, nl = static_cast<size_t>(total) * H * 4;
    const Range ins[7] = {range_of(q, n),   range_of(k, n),   range_of(v, n),
                          range_of(o, n),   range_of(dO, n),  range_of(lse, nl),
                          range_of(cu_seqlens, static_cast<size_t>(n_seq + 1) * 4)};
    const Range outs[3] = {range_of(dq, n), range_of(dk, n), range_of(dv, n)};
    for (int a = 0; a < 3; ++a) {
        for (int b = 0; b < 7; ++b)
            if (overlap(outs[a], ins[b])) return FA_ERR_ARG;
        for (int b = a + 1; b < 3; ++b)
            if (overlap(outs[a], outs[b])) return FA_ERR_ARG;
    }
    int dev = 0, sms = 0;
    int rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_bwd_varlen(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, n_seq, max_seqlen, total, H, D, scale,
                                 causal != 0, static_cast<cudaStream_t>(stream), knobs(), sms);
}

int fa_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Tq, int Tk, int D,
              float scale, void* stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
    if (B < 1 || H < 1 || Tq < 1 || Tk < 1) return FA_ERR_SHAPE;
    if (static_cast<long long>(B) * H > (1 << 30) || static_cast<long long>(B) * H * Tk > INT_MAX) return FA_ERR_SHAPE;
    if (Tq > 8) return FA_ERR_UNSUPPORTED;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return FA_ERR_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_ALIGN;
    const size_t nq = static_cast<size_t>(B) * H * Tq * D * 2, nk = static_cast<size_t>(B) * H * Tk * D * 2;
    const size_t nl = static_cast<size_t>(B) * H * Tq * 4;
    const Range rq = range_of(q, nq), rk = range_of(k, nk), rv = range_of(v, nk), ro = range_of(o, nq),
                rl = range_of(lse, nl);
    if (overlap(ro, rq) || overlap(ro, rk) || overlap(ro, rv) || overlap(ro, rl) || overlap(rl, rq) ||
        overlap(rl, rk) || overlap(rl, rv))
        return FA_ERR_ARG;
    int dev = 0, sms = 0;
    int rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_decode(q, k, v, o, lse, B, H, Tq, Tk, D, scale, static_cast<cudaStream_t>(stream), sms);
}

// Same checks as fa_bwd, then the fixed-scratch backward (see include/fa.h:
// for callers that cannot allocate device memory at call time).
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                   void* dq, void* dk, void* dv, int B, int H, int T, int D, float scale, int causal, void* stream) {
    if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return FA_ERR_NULL;
    int rc = check_shape(B, H, T, D, scale, causal);
    if (rc != FA_OK) return rc;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) || !aligned16(lse) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return FA_ERR_ALIGN;
    const size_t n = static_cast<size_t>(B) * H * T * D * 2, nl = static_cast<size_t>(B) * H * T * 4;
    const Range ins[6] = {range_of(q, n), range_of(k, n), range_of(v, n), range_of(o, n), range_of(dO, n),
                          range_of(lse, nl)};
    const Range outs[3] = {range_of(dq, n), range_of(dk, n), range_of(dv, n)};
    for (int a = 0; a < 3; ++a) {
        for (int b = 0; b < 6; ++b)
            if (overlap(outs[a], ins[b])) return FA_ERR_ARG;
        for (int b = a + 1; b < 3; ++b)
            if (overlap(outs[a], outs[b])) return FA_ERR_ARG;
    }
    if (fa::bwd_scratch_bytes(B, H, T, D) > FA_BWD_NOALLOC_SCRATCH_BYTES) return FA_ERR_SCRATCH;
    int dev = 0, sms = 0;
    rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, T, D, scale, causal != 0,
                                  static_cast<cudaStream_t>(stream), knobs(), sms);
}

int fa_get_device_status(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
    int a = fa::fwd_take_status();
    int b = fa::bwd_take_status();
    int c = fa::kv4_cache_take_status();
    int d = fa::kv4_decode_take_status();
    if (a == -5 || b == -5 || c == -5 || d == -5) return FA_ERR_CUDA;
    return a != 0 ? a : b != 0 ? b : c != 0 ? c : d;
}

}  // extern "C"

namespace {

// Whether rows of D elements lie apart: by rising stride, each dimension's step clears what
// the dimensions within it span.
struct Dim {
    long long size, stride;
};
bool rows_apart(std::array<Dim, 3> dims, int D) {
    std::sort(dims.begin(), dims.end(), [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    long long span = D;
    for (const Dim& d : dims) {
        if (d.size == 1) continue;
        if (d.stride < span || d.stride > (LLONG_MAX - span) / (d.size - 1)) return false;
        span += (d.size - 1) * d.stride;
    }
    return true;
}

}  // namespace

extern "C" {

int fa_rope(const fa_rope_tensor* tensors, int n_tensors, const void* positions, int positions_64, long long positions_b,
            const void* freq, int B, int T, int D, int rotary, int interleaved, float amplitude, int inverse, int dtype,
            void* stream) {
    if (!tensors || !freq) return FA_ERR_NULL;
    if (n_tensors < 1 || n_tensors > 2) return FA_ERR_ARG;
    if (B < 1 || T < 1 || D < 2 || D > FA_ROPE_MAX_D) return FA_ERR_SHAPE;
    if (static_cast<long long>(B) * T > INT_MAX) return FA_ERR_SHAPE;
    if (rotary < 2 || rotary > D || rotary % 2 != 0) return FA_ERR_UNSUPPORTED;
    if (dtype < FA_BF16 || dtype > FA_FP32) return FA_ERR_UNSUPPORTED;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) ||
        (positions_64 != 0 && positions_64 != 1) || !std::isfinite(amplitude))
        return FA_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(freq) & 7u) ||
        (reinterpret_cast<uintptr_t>(positions) & (positions_64 ? 7u : 3u)))
        return FA_ERR_ALIGN;
    const int size = dtype == FA_FP32 ? 4 : 2;
    Range in[2], out[2];
    bool in_place[2];
    fa::RopeTensor x[2];
    for (int i = 0; i < n_tensors; ++i) {
        const fa_rope_tensor& t = tensors[i];
        if (!t.in || !t.out) return FA_ERR_NULL;
        if (t.heads < 1 || t.heads > (1 << 20)) return FA_ERR_SHAPE;
        if ((reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out)) & (size - 1)) return FA_ERR_ALIGN;
        if (t.in_b < 0 || t.in_t < 0 || t.in_h < 0 || t.out_b < 0 || t.out_t < 0 || t.out_h < 0) return FA_ERR_ARG;
        // an output element is written once: no two rows of it may share one
        if (!rows_apart({{{B, t.out_b}, {T, t.out_t}, {t.heads, t.out_h}}}, D)) return FA_ERR_ARG;
        in[i] = range_of(t.in, ((B - 1) * static_cast<size_t>(t.in_b) + (T - 1) * static_cast<size_t>(t.in_t) +
                                (t.heads - 1) * static_cast<size_t>(t.in_h) + D) * size);
        out[i] = range_of(t.out, ((B - 1) * static_cast<size_t>(t.out_b) + (T - 1) * static_cast<size_t>(t.out_t) +
                                  (t.heads - 1) * static_cast<size_t>(t.out_h) + D) * size);
        in_place[i] = t.in == t.out && t.in_b == t.out_b && t.in_t == t.out_t && t.in_h == t.out_h;
        if (!in_place[i] && overlap(in[i], out[i])) return FA_ERR_ARG;
        x[i] = {t.in, t.out, t.heads, t.in_b, t.in_t, t.in_h, t.out_b, t.out_t, t.out_h};
    }
    if (n_tensors == 2) {
        // two views of one projection interleave, which only rotating both in place keeps apart
        const bool views = in_place[0] && in_place[1] && tensors[0].in != tensors[1].in;
        if (!views && (overlap(out[0], out[1]) || overlap(out[0], in[1]) || overlap(out[1], in[0]))) return FA_ERR_ARG;
    }
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_rope(x, n_tensors, positions, positions_64, positions_b, freq, B, T, D, rotary, interleaved,
                           amplitude, inverse, dtype, static_cast<cudaStream_t>(stream), sms);
}

}  // extern "C"

namespace {

int check_kv4(const fa_kv4_cache* c) {
    if (!c) return FA_ERR_NULL;
    if (!c->pool || !c->block_table || !c->lengths) return FA_ERR_NULL;
    if (c->B < 1 || c->Hkv < 1 || c->num_pages < 1 || c->width < 1 || c->page_size < 16) return FA_ERR_SHAPE;
    if (static_cast<long long>(c->B) * c->Hkv > 65535) return FA_ERR_SHAPE;
    if (static_cast<long long>(c->width) * c->page_size > INT_MAX - 65536) return FA_ERR_SHAPE;
    if (static_cast<long long>(c->B) * c->width > INT_MAX) return FA_ERR_SHAPE;
    if (c->D != 64 && c->D != 128) return FA_ERR_UNSUPPORTED;
    if ((c->group != 32 && c->group != 64) || c->page_size % 16 != 0 || c->page_size > 65536)
        return FA_ERR_UNSUPPORTED;
    if (!aligned16(c->pool) || (reinterpret_cast<uintptr_t>(c->block_table) & 3u) ||
        (reinterpret_cast<uintptr_t>(c->lengths) & 3u))
        return FA_ERR_ALIGN;
    return FA_OK;
}
fa::Kv4Shape kv4_shape(const fa_kv4_cache* c) {
    return {c->B, c->Hkv, c->D, c->group, c->page_size, c->num_pages, c->width};
}
Range kv4_pool_range(const fa_kv4_cache* c) {
    return range_of(c->pool, static_cast<size_t>(c->num_pages) * c->Hkv * c->page_size * (c->D + 8 * c->D / c->group));
}
// Ranges of what a call only reads besides its own inputs.
Range kv4_table_range(const fa_kv4_cache* c) {
    return range_of(c->block_table, static_cast<size_t>(c->B) * c->width * 4);
}
Range kv4_lengths_range(const fa_kv4_cache* c) { return range_of(c->lengths, static_cast<size_t>(c->B) * 4); }
bool overlaps_any(Range a, const Range* r, int n) {
    for (int i = 0; i < n; ++i)
        if (overlap(a, r[i])) return true;
    return false;
}

// The caller's workspace, or one taken stream-ordered for the call.
struct Workspace {
    void* ptr = nullptr;
    bool mine = false;
    cudaStream_t stream;
    int take(void* given, size_t given_bytes, size_t need, cudaStream_t st) {
        stream = st;
        if (need == 0) return FA_OK;
        if (given != nullptr) {
            if (given_bytes < need) return FA_ERR_SCRATCH;
            if (!aligned16(given)) return FA_ERR_ALIGN;
            ptr = given;
            return FA_OK;
        }
        if (cudaMallocAsync(&ptr, need, st) != cudaSuccess) {
            cudaGetLastError();
            return FA_ERR_NOMEM;
        }
        mine = true;
        return FA_OK;
    }
    int release(int rc) {
        if (mine && cudaFreeAsync(ptr, stream) != cudaSuccess && rc == FA_OK) return FA_ERR_CUDA;
        return rc;
    }
};

}  // namespace

extern "C" {

int fa_kv4_append(const fa_kv4_cache* cache, const void* k, const void* v, long long k_t, long long k_h, long long v_t,
                  long long v_h, const int* cu_new, int total, const void* positions, int positions_64,
                  const void* freq, int rotary, int interleaved, float amplitude, float* weights, int* slot_positions,
                  long long slots, void* stream) {
    int rc = check_kv4(cache);
    if (rc != FA_OK) return rc;
    if (!k || !v || !cu_new) return FA_ERR_NULL;
    if (total < 1 || static_cast<long long>(total) * cache->Hkv > INT_MAX) return FA_ERR_SHAPE;
    if (k_t < 0 || k_h < 0 || v_t < 0 || v_h < 0) return FA_ERR_ARG;
    if (freq && (rotary < 2 || rotary > cache->D || rotary % 2 != 0)) return FA_ERR_UNSUPPORTED;
    if (freq && ((interleaved != 0 && interleaved != 1) || !std::isfinite(amplitude))) return FA_ERR_ARG;
    if (positions_64 != 0 && positions_64 != 1) return FA_ERR_ARG;
    if ((weights || slot_positions) && slots < 1) return FA_ERR_SHAPE;
    // a dimension of one element may have any stride
    if (!aligned16(k) || !aligned16(v) || (total > 1 && (k_t % 8 || v_t % 8)) || (cache->Hkv > 1 && (k_h % 8 || v_h % 8)) ||
        (reinterpret_cast<uintptr_t>(cu_new) & 3u) || (reinterpret_cast<uintptr_t>(freq) & 7u) ||
        (reinterpret_cast<uintptr_t>(positions) & (positions_64 ? 7u : 3u)) ||
        (reinterpret_cast<uintptr_t>(weights) & 3u) || (reinterpret_cast<uintptr_t>(slot_positions) & 3u))
        return FA_ERR_ALIGN;
    const int D = cache->D, H = cache->Hkv;
    const size_t n_slots = static_cast<size_t>(cache->B) * H * (slots > 0 ? slots : 0) * 4;
    const Range ins[6] = {
        range_of(k, ((total - 1) * static_cast<size_t>(k_t) + (H - 1) * static_cast<size_t>(k_h) + D) * 2),
        range_of(v, ((total - 1) * static_cast<size_t>(v_t) + (H - 1) * static_cast<size_t>(v_h) + D) * 2),
        kv4_table_range(cache), kv4_lengths_range(cache), range_of(cu_new, (cache->B + 1) * static_cast<size_t>(4)),
        range_of(positions, positions ? static_cast<size_t>(total) * (positions_64 ? 8 : 4) : 0)};
    const Range pool = kv4_pool_range(cache), rw = range_of(weights, weights ? n_slots : 0),
                rp = range_of(slot_positions, slot_positions ? n_slots : 0);
    if (overlaps_any(pool, ins, 6) || overlaps_any(rw, ins, 6) || overlaps_any(rp, ins, 6) || overlap(pool, rw) ||
        overlap(pool, rp) || overlap(rw, rp))
        return FA_ERR_ARG;
    int dev = 0, sms = 0;
    rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_kv4_append(kv4_shape(cache), cache->pool, cache->block_table, k, v, k_t, k_h, v_t, v_h,
                                 cache->lengths, cu_new, total, positions, positions_64, freq, rotary, interleaved,
                                 amplitude, weights, slot_positions, (weights || slot_positions) ? slots : 0,
                                 static_cast<cudaStream_t>(stream), sms);
}

int fa_kv4_read(const fa_kv4_cache* cache, const int* start, int count, void* k, void* v, void* stream) {
    int rc = check_kv4(cache);
    if (rc != FA_OK) return rc;
    if (!k || !v) return FA_ERR_NULL;
    if (count < 1 || static_cast<long long>(cache->B) * cache->Hkv * count > INT_MAX) return FA_ERR_SHAPE;
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(start) & 3u)) return FA_ERR_ALIGN;
    const size_t n = static_cast<size_t>(cache->B) * cache->Hkv * count * cache->D * 2;
    const Range rk = range_of(k, n), rv = range_of(v, n);
    const Range ins[4] = {kv4_pool_range(cache), kv4_table_range(cache), kv4_lengths_range(cache),
                          range_of(start, start ? cache->B * static_cast<size_t>(4) : 0)};
    if (overlap(rk, rv) || overlaps_any(rk, ins, 4) || overlaps_any(rv, ins, 4)) return FA_ERR_ARG;
    int dev = 0, sms = 0;
    rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::launch_kv4_read(kv4_shape(cache), cache->pool, cache->block_table, cache->lengths, start, count, k, v,
                               static_cast<cudaStream_t>(stream));
}

long long fa_kv4_decode_workspace(int B, int Hq, int Hkv, int Tq, int D, int slots, int weights) {
    if (B < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || Tq < 1 || slots < 16 || slots % 16 != 0) return FA_ERR_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    const fa::Kv4Shape c{B, Hkv, D, 64, 16, 1, slots / 16};
    return static_cast<long long>(fa::kv4_decode_workspace(c, Hq, Tq, weights != 0, sms));
}

int fa_kv4_decode(const fa_kv4_cache* cache, const void* q, void* o, float* lse, int Hq, int Tq, float scale,
                  int causal, const float* weights, float* weights_out, long long slots, void* workspace,
                  long long workspace_bytes, void* stream) {
    int rc = check_kv4(cache);
    if (rc != FA_OK) return rc;
    if (!q || !o || !lse || (weights && !weights_out)) return FA_ERR_NULL;
    if (Hq < 1 || Hq % cache->Hkv != 0 || Tq < 1) return FA_ERR_SHAPE;
    if (static_cast<long long>(cache->B) * Hq * Tq > INT_MAX) return FA_ERR_SHAPE;
    if (Tq > 8) return FA_ERR_UNSUPPORTED;
    if (Hq / cache->Hkv * Tq > 1024) return FA_ERR_UNSUPPORTED;
    if (!fa::kv4_decode_fits(kv4_shape(cache), Hq, Tq)) return FA_ERR_SHAPE;
    if (causal != 0 && causal != 1) return FA_ERR_ARG;
    if (!std::isfinite(scale)) return FA_ERR_ARG;
    if (weights_out && slots < 1) return FA_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || (reinterpret_cast<uintptr_t>(weights) & 3u) ||
        (reinterpret_cast<uintptr_t>(weights_out) & 3u))
        return FA_ERR_ALIGN;
    const size_t nq = static_cast<size_t>(cache->B) * Hq * Tq * cache->D * 2;
    const size_t nl = static_cast<size_t>(cache->B) * Hq * Tq * 4;
    const size_t nw = weights_out ? static_cast<size_t>(cache->B) * cache->Hkv * slots * 4 : 0;
    const fa::Kv4Shape shape = kv4_shape(cache);
    // the weights may be added to in place; nothing else is shared
    const Range ins[5] = {range_of(q, nq), kv4_pool_range(cache), kv4_table_range(cache), kv4_lengths_range(cache),
                          range_of(weights, weights && weights != weights_out ? nw : 0)};
    const Range outs[3] = {range_of(o, nq), range_of(lse, nl), range_of(weights_out, nw)};
    for (int i = 0; i < 3; ++i) {
        if (overlaps_any(outs[i], ins, 5)) return FA_ERR_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j])) return FA_ERR_ARG;
    }
    int dev = 0, sms = 0;
    rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    const size_t need = fa::kv4_decode_workspace(shape, Hq, Tq, weights_out != nullptr, sms);
    if (workspace) {
        const Range ws = range_of(workspace, need);
        if (overlaps_any(ws, ins, 5) || overlaps_any(ws, outs, 3)) return FA_ERR_ARG;
    }
    Workspace ws;
    rc = ws.take(workspace, static_cast<size_t>(workspace_bytes > 0 ? workspace_bytes : 0), need,
                 static_cast<cudaStream_t>(stream));
    if (rc != FA_OK) return rc;
    rc = fa::launch_kv4_decode(shape, cache->pool, cache->block_table, cache->lengths, q, o, lse, Hq, Tq, scale,
                               causal != 0, weights, weights_out, slots, ws.ptr, static_cast<cudaStream_t>(stream),
                               sms);
    return ws.release(rc);
}

long long fa_kv4_evict_workspace(int B, int Hkv, int budget) {
    if (B < 1 || Hkv < 1 || budget < 1) return FA_ERR_SHAPE;
    return static_cast<long long>(fa::kv4_evict_workspace(B, Hkv, budget));
}

int fa_kv4_evict(const fa_kv4_cache* cache, const float* weights, const int* slot_positions, long long slots,
                 int budget, int recent, float* weights_out, int* positions_out, int* lengths_out, int* source,
                 void* workspace, long long workspace_bytes, void* stream) {
    int rc = check_kv4(cache);
    if (rc != FA_OK) return rc;
    if (!weights || !slot_positions || !weights_out || !positions_out || !lengths_out || !source) return FA_ERR_NULL;
    if (slots < 1 || slots > INT_MAX - 65536 || budget < 1 || budget > (1 << 30)) return FA_ERR_SHAPE;
    if (recent < 0 || recent > budget) return FA_ERR_ARG;
    const void* words[6] = {weights, slot_positions, weights_out, positions_out, lengths_out, source};
    for (const void* w : words)
        if (reinterpret_cast<uintptr_t>(w) & 3u) return FA_ERR_ALIGN;
    const size_t heads = static_cast<size_t>(cache->B) * cache->Hkv, n = heads * slots * 4;
    const size_t need = fa::kv4_evict_workspace(cache->B, cache->Hkv, budget);
    const Range ins[4] = {range_of(weights, n), range_of(slot_positions, n), kv4_table_range(cache),
                          kv4_lengths_range(cache)};
    const Range outs[6] = {kv4_pool_range(cache),       range_of(weights_out, n),
                           range_of(positions_out, n),  range_of(lengths_out, cache->B * static_cast<size_t>(4)),
                           range_of(source, heads * budget * 4), range_of(workspace, workspace ? need : 0)};
    for (int i = 0; i < 6; ++i) {
        if (overlaps_any(outs[i], ins, 4)) return FA_ERR_ARG;
        for (int j = i + 1; j < 6; ++j)
            if (overlap(outs[i], outs[j])) return FA_ERR_ARG;
    }
    int dev = 0, sms = 0;
    rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    Workspace ws;
    rc = ws.take(workspace, static_cast<size_t>(workspace_bytes > 0 ? workspace_bytes : 0), need,
                 static_cast<cudaStream_t>(stream));
    if (rc != FA_OK) return rc;
    rc = fa::launch_kv4_evict(kv4_shape(cache), cache->pool, cache->block_table, cache->lengths, weights,
                              slot_positions, slots, budget, recent, weights_out, positions_out, lengths_out, source,
                              ws.ptr, static_cast<cudaStream_t>(stream), sms);
    return ws.release(rc);
}

long long fa_kv4_block_offset(const int* block_table, int width, int Hkv, int D, int group, int page_size,
                              int num_pages, int b, int h, int slot) {
    if (!block_table) return FA_ERR_NULL;
    if (width < 1 || Hkv < 1 || num_pages < 1 || page_size < 16 || b < 0 || h < 0 || h >= Hkv || slot < 0)
        return FA_ERR_SHAPE;
    if ((D != 64 && D != 128) || (group != 32 && group != 64) || page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
    const fa::Kv4Pages p = fa::kv4_pages(nullptr, block_table, width, num_pages, Hkv, page_size, D, group);
    const long long at = p.block_of(b, slot / 16);
    return at < 0 ? static_cast<long long>(FA_ERR_PAGE) : at + h * p.head_bytes();
}

int fa_sched_tile_rows(int D, int* bm_fwd, int* bn, int* bm_bwd) {
    if (!bm_fwd || !bn || !bm_bwd) return FA_ERR_NULL;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    *bm_fwd = fa::kFwdBM;
    *bn = fa::kBN;
    *bm_bwd = fa::bwd_bm(D);
    return FA_OK;
}

int fa_sched_fwd_tile_class(int T, int causal, int qt, int kt) {
    if (T < 1 || qt < 0 || kt < 0) return FA_ERR_SHAPE;
    return fa::fwd_tile_class(T, causal != 0, qt, kt);
}

int fa_sched_bwd_tile_class(int T, int D, int causal, int qt, int kt) {
    if (T < 1 || qt < 0 || kt < 0) return FA_ERR_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    return fa::bwd_tile_class(T, causal != 0, fa::bwd_bm(D), qt, kt);
}

int fa_sched_fwd_keep(int T, int causal, int i, int j) {
    if (T < 1 || i < 0 || j < 0) return FA_ERR_SHAPE;
    return fa::fwd_keep(T, causal != 0, i, j) ? 1 : 0;
}

int fa_sched_bwd_keep(int T, int D, int causal, int i, int j) {
    if (T < 1 || i < 0 || j < 0) return FA_ERR_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    return fa::bwd_keep(T, causal != 0, fa::bwd_bm(D), i, j) ? 1 : 0;
}

int fa_debug_set_wait_timeout_ns(unsigned long long ns) {
    if (ns == 0) return FA_ERR_ARG;
    g_timeout_ns.store(ns);
    return FA_OK;
}

int fa_set_timing_events(void* fwd_begin, void* fwd_end, void* bwd_begin, void* bwd_mid, void* bwd_end) {
    g_events[0].store(fwd_begin);
    g_events[1].store(fwd_end);
    g_events[2].store(bwd_begin);
    g_events[3].store(bwd_mid);
    g_events[4].store(bwd_end);
    return FA_OK;
}

int fa_bwd_sums_dq_in_place(int B, int Hkv, int T, int D) {
    if (B < 1 || Hkv < 1 || T < 1) return FA_ERR_SHAPE;
    if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != FA_OK) return rc;
    return fa::bwd_fuses_host(B, Hkv, T, D, sms, g_deterministic.load() != 0) ? 1 : 0;
}

int fa_set_deterministic(int on) {
    if (on != 0 && on != 1) return FA_ERR_ARG;
    g_deterministic.store(on);
    return FA_OK;
}

int fa_debug_checks_enabled(void) {
#ifdef FA_DEBUG
    return 1;
#else
    return 0;
#endif
}

int fa_debug_inject(int mode) {
    if (mode < 0 || mode > 3) return FA_ERR_ARG;
    g_inject.store(mode);
    return FA_OK;
}

}  // extern "C"
