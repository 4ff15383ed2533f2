/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact-attention library (libfa.so).
 *
 * What it computes (pages: "Lab 06 - Attention kernels: online softmax ->
 * FlashAttention -> Triton", sections 3 and 4; "Triton FlashAttention-2
 * forward", section "The kernel"; "Flash Attention and Kernel Optimization",
 * sections "Running softmax state", "Causal masking", "Output and saved
 * state"):
 *
 *   forward   S = Q K^T * scale, key j visible to query i iff j <= i when
 *             causal; O = softmax(S) V; LSE_i = log sum_j exp(S_ij)
 *             (natural log of the scaled scores), computed tile by tile
 *             with the online-softmax recurrence, never forming S in memory.
 *   backward  D_i = rowsum(dO o O); P = exp(S - LSE) recomputed per tile;
 *             dV = P^T dO; dP = dO V^T; dS = P o (dP - D);
 *             dQ = dS K * scale; dK = dS^T Q * scale.
 *
 * Layout.  Every tensor is contiguous (B, H, T, D) in bf16
 * (__nv_bfloat16, passed as void*), row stride D elements, head stride T*D.
 * LSE is contiguous (B, H, T) float32.  D must be 64 or 128.  T_q = T_k = T.
 *
 * Memory and ownership.  All tensor pointers are DEVICE pointers on the
 * current CUDA device, allocated and owned by the caller; the library keeps
 * no pointer after a call returns.  Base pointers must be 16-byte aligned
 * (the kernels move tiles with TMA).  Outputs must not overlap inputs.
 *
 * Streams.  `stream` is a cudaStream_t passed as void* (NULL = legacy default
 * stream).  Calls are asynchronous: they enqueue kernels on `stream` and
 * return without synchronising.  fa_bwd takes its workspace (two vectors of
 * B*H*T_pad floats, T_pad = T rounded up to 128: D and log2-scaled LSE, plus
 * 256 bytes for a work counter)
 * stream-ordered with cudaMallocAsync on `stream` and releases it with
 * cudaFreeAsync on the same stream before returning.  Nothing on these paths
 * synchronises, so every compute entry point may be called while `stream` is
 * being captured into a CUDA graph (the workspace becomes allocation nodes,
 * the backward's overlapped second kernel a programmatic dependency); a
 * replay reads the input buffers as they are at replay time.
 * fa_get_device_status synchronises and must not be captured.
 *
 * Errors.  Every entry point validates its arguments before launching
 * anything; on a validation error nothing is enqueued.  Return value 0
 * (FA_OK) or a negative fa_status.  A kernel that detects a stalled pipeline
 * (a bounded wait that ran out) records FA_ERR_DEVICE_TIMEOUT in a device
 * status word and exits cleanly; read it with fa_get_device_status.
 */
#ifndef FA_H_
#define FA_H_

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fa_status {
    FA_OK = 0,
    FA_ERR_NULL = -1,            /* a required pointer is NULL */
    FA_ERR_SHAPE = -2,           /* B, H, T (Tq, Tk) out of range, or a size overflows the index types */
    FA_ERR_UNSUPPORTED = -3,     /* D is not 64 or 128 */
    FA_ERR_ALIGN = -4,           /* a base pointer is not 16-byte aligned, or a stride no multiple of 8 elements */
    FA_ERR_CUDA = -5,            /* a CUDA runtime / driver call failed (launch, attribute, tensor map) */
    FA_ERR_NOMEM = -6,           /* stream-ordered workspace allocation failed */
    FA_ERR_DEVICE_TIMEOUT = -7,  /* a kernel's bounded wait ran out (pipeline stall); outputs invalid */
    FA_ERR_ARG = -8,             /* causal not 0/1, or scale not finite */
    FA_ERR_ARCH = -9,            /* current device is not compute capability 10.3 (sm_103a) */
    FA_ERR_SCRATCH = -10,        /* fa_bwd_noalloc: problem needs more than its fixed scratch buffer; or a given workspace is too small */
    FA_ERR_SEQLEN = -11,         /* recorded by a kernel: a cu_seqlens length is negative or above max_seqlen,
                                    a key length is outside its tensor, or a cache's length, slot or position is outside its block table or accounts */
    FA_ERR_DEBUG_CHECK = -12,    /* debug library only: a kernel's run-time index failed its bounds check */
    FA_ERR_PAGE = -13            /* recorded by a kernel: a block table names no page of the pool where a token lies */
} fa_status;

/*
 * Forward pass.
 *   q, k, v  in : (B, H, T, D) bf16
 *   o        out: (B, H, T, D) bf16, O = softmax(Q K^T scale [+ causal mask]) V
 *   lse      out: (B, H, T) float32, natural-log log-sum-exp of the scaled,
 *                 masked scores of each row (the only statistic the backward
 *                 needs: "Lab 06", section 4 and "Check yourself" item 3)
 *   scale       : finite float multiplying Q K^T (usually 1/sqrt(D))
 *   causal      : 0 = full attention, 1 = key j visible to query i iff j <= i
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
           int B, int H, int T, int D, float scale, int causal, void* stream);

/*
 * Backward pass.
 *   q, k, v, o, dO in : (B, H, T, D) bf16 (o from fa_fwd on the same inputs)
 *   lse            in : (B, H, T) float32 from fa_fwd
 *   dq, dk, dv     out: (B, H, T, D) bf16 gradients of sum(dO o O) with
 *                       respect to q, k, v (overwritten, not accumulated)
 *   B, H, T, D, scale, causal: as in fa_fwd.
 * dq is accumulated in float32 across key tiles and rounded to bf16 once:
 *   D = 128: in a second kernel that walks the key tiles of each query tile;
 *     no global-memory reductions, so the result is deterministic.
 *   D = 64, when the dk/dv grid (one CTA per 128-key tile and key/value
 *     head) has at least one CTA per SM: by the same kernel that computes
 *     dk and dv (key tiles outer, as "Lab 06", section 4 orders the loops),
 *     which adds each key tile's contribution into a float32 accumulator in
 *     the workspace with reduce-adds; the order of those additions varies
 *     from run to run, so dq may differ in its last bits between runs (dk
 *     and dv do not).  Smaller grids use the two-kernel form.
 *     fa_set_deterministic(1) selects the two-kernel form at D = 64 always.
 * Workspace: stream-ordered with cudaMallocAsync on `stream`, released before
 * returning: two vectors of B*H*T_pad floats plus 256 bytes (T_pad = T
 * rounded up to 128), and when dq is summed by reduce-adds (above) the
 * float32 dq accumulator, B*H*T_pad*D floats.  FA_ERR_NOMEM if it cannot be
 * had.
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
           const float* lse, void* dq, void* dk, void* dv,
           int B, int H, int T, int D, float scale, int causal, void* stream);

/*
 * Backward pass that allocates nothing.  The pages have no counterpart to
 * this entry point: it exists for callers that cannot allocate device memory
 * at call time, for example code running inside a memory pool that must not
 * grow, or a runtime whose allocator is not reachable from the calling
 * thread.  fa_bwd takes its workspace with cudaMallocAsync; this variant
 * instead uses a fixed scratch buffer compiled into the library
 * (FA_BWD_NOALLOC_SCRATCH_BYTES = 64 MiB of device memory, reserved on every
 * GPU that loads the library's backward module, held until the process
 * exits).  It calls no cudaMalloc, cudaFree or other allocating routine.
 *
 * Same arguments, layout, results and asynchrony as fa_bwd.  The caller
 * still owns every input and output.
 * Limit: 8 * B*H*T_pad + 256 bytes (each of the two vectors rounded up to
 *   256 bytes) must not exceed the scratch size, where T_pad is T rounded up
 *   to a multiple of 128 (B*H*T_pad just under 8 M rows); larger problems
 *   return FA_ERR_SCRATCH and nothing is enqueued.
 * Set-up: the first call on each device looks up the buffer's device
 *   address (cudaGetSymbolAddress) in the context current at that moment and
 *   keeps it for the rest of the process; make that first call before any
 *   stream capture.  The kept address belongs to that context: after
 *   cudaDeviceReset, or from another (non-primary) context on the same
 *   device, it is stale, so do not call fa_bwd_noalloc there.
 * Sharing: every call uses the same buffer, which keeps the previous call's
 *   contents (the backward rewrites all of it before reading it).  Calls whose
 *   work overlaps on the GPU (different streams, or different host threads
 *   without ordering) race on the buffer and corrupt each other's results;
 *   serialise them.
 */
#define FA_BWD_NOALLOC_SCRATCH_BYTES (64ull << 20)
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO,
                   const float* lse, void* dq, void* dk, void* dv,
                   int B, int H, int T, int D, float scale, int causal, void* stream);

/*
 * Grouped-query attention ("Lab 06 - Attention kernels", "Check yourself"
 * item 7): Hq query heads share Hkv key/value heads, Hq % Hkv == 0, query
 * head h using key/value head h / (Hq / Hkv).  Same computation, layout,
 * asynchrony and errors as fa_fwd / fa_bwd with
 *   q, o, dO, dq : (B, Hq, T, D) bf16;  lse : (B, Hq, T) float32
 *   k, v, dk, dv : (B, Hkv, T, D) bf16
 * dk and dv sum the contributions of every query head of the group.  The
 * forward pairs two query heads of one group on the same rows in a CTA, so
 * each K/V tile loaded into shared memory serves both; the backward walks the
 * query tiles of the whole group per key tile.  Hkv == Hq is plain attention.
 * FA_ERR_SHAPE if Hq or Hkv < 1 or Hq % Hkv != 0.
 */
int fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
               int B, int Hq, int Hkv, int T, int D, float scale, int causal, void* stream);
int fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dO,
               const float* lse, void* dq, void* dk, void* dv,
               int B, int Hq, int Hkv, int T, int D, float scale, int causal, void* stream);

/*
 * Forward over a packed batch of variable-length sequences ("Triton
 * FlashAttention-2 forward", "Exercises": a cu_seqlens index packs requests of
 * different lengths into one launch).  Sequence s occupies rows
 * cu_seqlens[s] .. cu_seqlens[s+1]-1 of the packed tensors and attends only
 * to itself (causal alignment relative to its own first token).
 *   q, k, v    in : (total, H, D) bf16, packed
 *   o          out: (total, H, D) bf16
 *   lse        out: (H, total) float32
 *   cu_seqlens in : DEVICE int32[n_seq + 1], cu_seqlens[0] = 0, non-decreasing,
 *                   cu_seqlens[n_seq] = total (lengths may be 0)
 *   max_seqlen    : an upper bound on every length (the caller knows it; the
 *                   library does not read cu_seqlens on the host)
 * A length above max_seqlen (or negative) is detected by the kernel and
 * reported as FA_ERR_SEQLEN by fa_get_device_status; those outputs are invalid.
 * Other arguments and errors as in fa_fwd.  No workspace.
 */
int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                  const int* cu_seqlens, int n_seq, int max_seqlen, int total, int H, int D,
                  float scale, int causal, void* stream);

/*
 * Backward of fa_fwd_varlen over the same packed batch ("Triton
 * FlashAttention-2 forward", "Exercises": the cu_seqlens packing; the
 * gradients as in fa_bwd, "Lab 06 - Attention kernels", section 4).  Each
 * sequence's gradients involve only its own rows.
 *   q, k, v, o, dO in : (total, H, D) bf16, packed; o and lse from fa_fwd_varlen
 *   lse            in : (H, total) float32
 *   dq, dk, dv     out: (total, H, D) bf16
 *   cu_seqlens, n_seq, max_seqlen, total: as in fa_fwd_varlen
 * Workspace: like fa_bwd's, stream-ordered with cudaMallocAsync on `stream`:
 * two vectors of H * n_seq * T_pad floats (T_pad = max_seqlen rounded up to
 * 128) plus 256 bytes, released before returning.
 * A length above max_seqlen (or negative) is reported as FA_ERR_SEQLEN by
 * fa_get_device_status; that sequence's gradients are left unwritten.
 * FA_ERR_ARG if an output overlaps an input or another output; other
 * arguments and errors as in fa_fwd_varlen and fa_bwd.
 */
int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dO,
                  const float* lse, void* dq, void* dk, void* dv, const int* cu_seqlens,
                  int n_seq, int max_seqlen, int total, int H, int D, float scale, int causal,
                  void* stream);

/*
 * Decoding forward, split over the keys ("Lab 06 - Attention kernels",
 * "Check yourself" item 2 and "Stretch": a few new query rows against a long
 * key/value cache).  Each of the Tq query rows of a head attends to ALL Tk
 * keys of the same head (no mask).  The keys are split into chunks processed
 * in parallel, each producing a partial (m, l, acc); a second kernel merges
 * them with the online-softmax rescaling rule.
 *   q       in : (B, H, Tq, D) bf16, 1 <= Tq <= 8
 *   k, v    in : (B, H, Tk, D) bf16, Tk >= 1
 *   o       out: (B, H, Tq, D) bf16
 *   lse     out: (B, H, Tq) float32, natural-log log-sum-exp of the scaled scores
 *   scale, stream: as in fa_fwd.  D must be 64 or 128.
 * Workspace: the partials (B*H*n_chunks*Tq*(D + 2) floats) are taken with
 * cudaMallocAsync on `stream` and released before returning.
 */
int fa_decode(const void* q, const void* k, const void* v, void* o, float* lse,
              int B, int H, int Tq, int Tk, int D, float scale, void* stream);

/*
 * Cross attention: Tq queries of a sequence over the Tk keys and values of another
 * (an encoder's states), grouped heads as in fa_fwd_gqa, no causal mask.
 *   S = Q K^T scale over the keys j < key_lengths[b], O = softmax(S) V,
 *   LSE = log sum exp(S);  the backward is fa_bwd's over the same keys.
 * A sequence without keys gives O = 0, LSE = -infinity and gradients of 0.
 *   q, o, dO, dq    : (B, Hq, Tq, D) bf16;  k, v, dk, dv: (B, Hkv, Tk, D) bf16,
 *                     each by its strides b, h, t in elements, positive
 *                     multiples of 8 where the dimension is more than one, channels
 *                     contiguous: heads may lie behind or before tokens, and
 *                     tensors may be views of a fused projection
 *   key_lengths  in : DEVICE int32[B], 0 .. Tk, or NULL: Tk everywhere.  Keys and
 *                     values past the length are not used, whatever they hold
 *                     (NaN and infinities too); dk and dv are 0 there.  Another length
 *                     is recorded as FA_ERR_SEQLEN and counts as 0.
 *   lse             : (B, Hq, Tq) float32, contiguous
 *   o_rest          : (B, Hq, Tq, D) bf16, contiguous, or NULL: what rounding o to
 *                     bf16 took off, written by the forward for the backward, whose
 *                     rowsum(dO o O) is then of O to 16 bits.  Without it dq is less exact where
 *                     keys have a mean.
 *   workspace       : fa_cross_fwd_workspace / fa_cross_bwd_workspace(B, Hq, Hkv, Tq,
 *                     Tk, D) bytes (0 for a forward that cuts no keys), 16-byte and
 *                     256-byte aligned, used until the call's work on `stream` is done; or
 *                     NULL: taken with cudaMallocAsync.  FA_ERR_SCRATCH if
 *                     workspace_bytes is too small.
 * B * Hq * Tq and B * Hkv * Tk within int32, Tk at most 2^31 - 128.  FA_ERR_ALIGN for a base that is not
 * 16-byte aligned or a stride that is no multiple of 8; FA_ERR_ARG for a stride
 * below 1, an output whose rows may share elements, or one whose range of addresses
 * meets another tensor's.  fa_set_deterministic holds as for fa_bwd: at D = 64, with
 * at least one CTA per SM, dq's last bits may otherwise vary.
 */
typedef struct fa_cross_shape {
    int B, Hq, Hkv, Tq, Tk, D;
    const int* key_lengths;
} fa_cross_shape;
typedef struct fa_cross_tensor {
    void* ptr;              /* not written through where the tensor is an input */
    long long b, h, t;      /* strides in elements */
} fa_cross_tensor;
int fa_cross_fwd(const fa_cross_shape* shape, const fa_cross_tensor* q, const fa_cross_tensor* k,
                 const fa_cross_tensor* v, const fa_cross_tensor* o, void* o_rest, float* lse, float scale,
                 void* workspace, long long workspace_bytes, void* stream);
long long fa_cross_fwd_workspace(int B, int Hq, int Hkv, int Tq, int Tk, int D);
long long fa_cross_bwd_workspace(int B, int Hq, int Hkv, int Tq, int Tk, int D);
int fa_cross_bwd(const fa_cross_shape* shape, const fa_cross_tensor* q, const fa_cross_tensor* k,
                 const fa_cross_tensor* v, const fa_cross_tensor* o, const void* o_rest,
                 const fa_cross_tensor* dO, const float* lse,
                 const fa_cross_tensor* dq, const fa_cross_tensor* dk, const fa_cross_tensor* dv, float scale,
                 void* workspace, long long workspace_bytes, void* stream);

/*
 * Rotary positions: turns pairs of channels of queries and keys by an angle
 * that grows with the position, before attention or before a cache.
 *   y1 = amplitude (x1 cos a - x2 sin a),  y2 = amplitude (x2 cos a + x1 sin a),
 * a = position * f_i for pair i, x1 and x2 the channels i and i + rotary/2, or
 * 2i and 2i + 1 when interleaved.  Channels from `rotary` on are copied.
 * inverse = 1 turns back (-sin) and is the gradient of the map.
 *   tensors      : n_tensors (1 or 2, e.g. queries and keys) (B, T, heads, D)
 *                  tensors, each with its own heads and its strides in
 *                  elements (channels are contiguous); in-place (out == in with
 *                  the same strides) is allowed, any other overlap is not.
 *                  Two in-place views of one buffer must not share elements.
 *   positions  in: DEVICE int32 (or int64 if positions_64) [B][T] with batch
 *                  stride positions_b (0: shared); NULL means 0 .. T-1.  May be
 *                  negative.
 *   freq       in: DEVICE uint64[rotary / 2], turns per position in units of
 *                  2^-64 (so the angle is exact modulo a turn at any position)
 *   rotary       : even, 2 .. D;  D: 2 .. FA_ROPE_MAX_D
 *   dtype        : FA_BF16, FA_FP16 or FA_FP32, of every tensor; cosine and
 *                  sine, products and sums are float32, each rounded to nearest,
 *                  the result rounded to the type
 * FA_ERR_UNSUPPORTED for rotary or dtype, FA_ERR_ARG for overlaps, negative
 * strides or an output whose rows may share elements (by rising stride, each of
 * its dimensions must step over all that those before it span).  No workspace.
 */
#define FA_BF16 0
#define FA_FP16 1
#define FA_FP32 2
#define FA_ROPE_MAX_D 1024
typedef struct fa_rope_tensor {
    const void* in;
    void* out;
    long long heads;
    long long in_b, in_t, in_h;    /* strides in elements */
    long long out_b, out_t, out_h;
} fa_rope_tensor;
int fa_rope(const fa_rope_tensor* tensors, int n_tensors, const void* positions, int positions_64,
            long long positions_b, const void* freq, int B, int T, int D, int rotary, int interleaved,
            float amplitude, int inverse, int dtype, void* stream);

/*
 * Key/value cache held in 4 bits, in pages.  A group of `group` channels of a
 * token and head is stored as m = min, s = bf16((max - min) / 15) (both bf16)
 * and the codes round((x - m) / s), ties to even, 0..15; it stands for
 * s * code + m.  s < 2^-100 is stored as 0.  A group that holds a NaN, or whose
 * range is not finite in float32, reads back as NaN.
 *   pool         : DEVICE bytes, num_pages * Hkv * page_size * (D + 8 D/group),
 *                  16-byte aligned: (num_pages, Hkv, page_size / 16) blocks of
 *                  16 tokens, each block key codes (16 rows of D/2 bytes), key
 *                  scales (16 rows of D/group pairs s, m), value codes, value
 *                  scales.  Key channel 32 g + 8 j + i is nibble i of the row's
 *                  32-bit word j D/32 + g; value channel 32 g + 4 r + i is
 *                  nibble i of its 16-bit half-word r D/32 + g.
 *   block_table in: DEVICE int32[B][width]: slot t of sequence b lies in page
 *                  block_table[b][t / page_size].  Entries behind the length
 *                  are not read.
 *   lengths    in: DEVICE int32[B], tokens held by each sequence (may be 0)
 *   D: 64 or 128; group: 32 or 64; page_size: a multiple of 16 up to 65536;
 *   B * Hkv <= 65535; width * page_size slots at most per sequence.
 * A length the table cannot hold (or negative) is recorded as FA_ERR_SEQLEN and
 * that sequence counts as empty; a table entry outside the pool, where a token
 * lies, is recorded as FA_ERR_PAGE and those tokens are left out (read with
 * fa_get_device_status; the outputs concerned are invalid).
 */
typedef struct fa_kv4_cache {
    void* pool;
    const int* block_table;
    const int* lengths;
    int B, Hkv, D, group, page_size, num_pages, width;
} fa_kv4_cache;

/*
 * Writes new tokens to the cache: rotates the keys if `freq` is given, rounds
 * them to bf16 as fa_rope does, quantises and stores.  cache->lengths counts
 * the new tokens already: sequence b's n = cu_new[b+1] - cu_new[b] tokens go to
 * slots lengths[b] - n .. lengths[b] - 1.
 *   k, v       in: packed (total, Hkv, D) bf16 with strides k_t, k_h, v_t, v_h
 *                  (elements, multiples of 8 where there is more than one token
 *                  or head; bases 16-byte aligned)
 *   cu_new     in: DEVICE int32[B + 1], non-decreasing; rows of k and v before
 *                  cu_new[0] and from cu_new[B] on are not used (n may be 0)
 *   positions  in: DEVICE int32 / int64 [total], NULL: the slot
 *   freq, rotary, interleaved, amplitude: as in fa_rope; freq NULL: no rotation
 *   weights   out: float32 [B][Hkv][slots] or NULL: 0 at the new slots
 *   slot_positions out: int32 [B][Hkv][slots] or NULL: the new slots' positions; one
 *                  that int32 cannot hold is recorded as FA_ERR_SEQLEN and stored as
 *                  the nearest that it can
 * A sequence without room for its tokens in the table (or in `slots`), or whose
 * length is below n, is recorded as FA_ERR_SEQLEN; none of its tokens is stored.
 */
int fa_kv4_append(const fa_kv4_cache* cache, const void* k, const void* v, long long k_t, long long k_h,
                  long long v_t, long long v_h, const int* cu_new, int total, const void* positions,
                  int positions_64, const void* freq, int rotary, int interleaved, float amplitude,
                  float* weights, int* slot_positions, long long slots, void* stream);

/*
 * Reads `count` slots of every sequence back, from start[b] (NULL: 0) on.
 *   k, v out: (B, Hkv, count, D) bf16, s * code + m rounded once, zeros for slots
 *             at or behind the length
 * A negative start is recorded as FA_ERR_SEQLEN and reads zeros.
 */
int fa_kv4_read(const fa_kv4_cache* cache, const int* start, int count, void* k, void* v, void* stream);

/*
 * Decoding over the 4-bit cache, grouped heads (query head h reads key/value
 * head h / (Hq / Hkv)), split over the tokens.
 *   q       in: (B, Hq, Tq, D) bf16, 1 <= Tq <= 8, Hq / Hkv * Tq <= 1024;
 *               B * Hkv * ceil(rows / 8) * width * page_size / 32 below 2^31
 *               (FA_ERR_SHAPE), with rows = Hq / Hkv * Tq
 *   o      out: (B, Hq, Tq, D) bf16
 *   lse    out: (B, Hq, Tq) float32, natural-log log-sum-exp of the scaled scores
 *   causal    : 1 = the queries are the last Tq tokens of the sequence, query i
 *               sees the slots below length - (Tq - 1 - i); 0 = all of them.
 *               A row that sees nothing gives o = 0 and lse = -infinity.
 *   weights in: float32 [B][Hkv][slots] or NULL (zeros); weights_out the same
 *               or NULL: weights_out = weights + each slot's attention weight,
 *               summed over the Hq / Hkv * Tq query rows that read the head.
 *               Slots at and behind the length are not written.  weights_out
 *               may be weights (added to in place).
 *   workspace : fa_kv4_decode_workspace(B, Hq, Hkv, Tq, D, width * page_size,
 *               weights_out != NULL) bytes, 16-byte aligned, used until the call's work
 *               on `stream` is done (with weights the scores of every slot that the table
 *               names, 4 bytes for each query row of a head, 8 or a multiple of 16 of
 *               them, whatever the lengths are); or NULL: taken with cudaMallocAsync.
 *               FA_ERR_SCRATCH if workspace_bytes is too small.
 * Sums, maxima and the softmax are float32.  A weight times a value's s is rounded to
 * fp16's 11 bits; a query's elements are exact down to 2^-28 of their row's largest,
 * what is smaller loses bits.  Within what a row sees, values whose s lies below 2^-110
 * of the largest s may count as their minimum.
 * A non-finite query row that sees a token gives NaN in its o and lse, and in the
 * accounts of the tokens that it sees.
 */
long long fa_kv4_decode_workspace(int B, int Hq, int Hkv, int Tq, int D, int slots, int weights);
int fa_kv4_decode(const fa_kv4_cache* cache, const void* q, void* o, float* lse, int Hq, int Tq, float scale,
                  int causal, const float* weights, float* weights_out, long long slots, void* workspace,
                  long long workspace_bytes, void* stream);

/*
 * Attention of a tree of drafted tokens over the 4-bit cache.  The last N slots of each
 * sequence (cache->lengths counts them) are the tree's places, written by
 * fa_kv4_append as any tokens.  Place i sees the context before the tree, its
 * ancestors and itself.
 *   q       in: (B, Hq, N, D) bf16, 1 <= N <= FA_TREE_MAX_PLACES; query head h reads
 *               key/value head h / (Hq / Hkv)
 *   parents in: DEVICE int32 [B][N]: the place of i's parent, below i, or -1 behind the
 *               context.  Any other value marks a place without a token: it, and what
 *               hangs on it, sees nothing and is seen by no other.
 *   o      out: (B, Hq, N, D) bf16;  lse out: (B, Hq, N) float32
 * A place without a token, or a sequence of length 0, gives o = 0 and lse = -infinity.
 * A length between 0 and N is recorded as FA_ERR_SEQLEN and counts as 0.  What a place does not
 * see does not touch its result, whatever the cache holds there.  Scores, sums and the
 * softmax are float32.  Keys are exact, and a query's elements down to 2^-25 of their row's
 * largest; what is smaller loses bits.  (Whole queries stay exact over tiles of 128
 * tokens with a key group whose s or m lies outside 2^-17 to 2^11.)  Weights and values go into
 * their product as bf16, each rounded once: a chain of drafted tokens is less exact than the same
 * tokens through fa_kv4_decode, which keeps the values' codes whole and rounds a weight times s to 11 bits.
 * No weights are accumulated for fa_kv4_evict, as fa_kv4_decode can: steps with drafts leave the accounts
 * as they are.
 *   workspace : fa_kv4_tree_workspace(B, Hq, Hkv, N, D, width * page_size) bytes, 16-byte
 *               aligned, used until the call's work on `stream` is done; or NULL: taken with
 *               cudaMallocAsync.  FA_ERR_SCRATCH if workspace_bytes is too small.
 */
#define FA_TREE_MAX_PLACES 64
long long fa_kv4_tree_workspace(int B, int Hq, int Hkv, int N, int D, int slots);
int fa_kv4_tree(const fa_kv4_cache* cache, const void* q, const int* parents, void* o, float* lse, int Hq, int N,
                float scale, void* workspace, long long workspace_bytes, void* stream);

/*
 * Which of a tree's tokens stand: place i does if it and every place on its way from a root
 * holds what the model picked behind the place before it (picks[b][parent], and for a root
 * first[b], the pick behind the context; first NULL: every root stands).  Kept is the way
 * to the deepest place that stands, to the lowest of equally deep ones.
 *   parents         in: DEVICE int32 [B][N], as in fa_kv4_tree
 *   tokens, picks   in: DEVICE int32 (int64 if tokens_64) [B][N]; first [B] or NULL
 *   path           out: int32 [B][N], the places on the way from the root on, -1 behind them
 *   counts         out: int32 [B], how many
 *   next           out: int32 / int64 [B], the pick behind the last of them (first[b], or -1
 *                       without first, where none stands)
 */
int fa_tree_accept(const int* parents, const void* tokens, const void* picks, const void* first, int tokens_64, int B,
                   int N, int* path, int* counts, void* next, void* stream);

/*
 * Keeps a path of the tree's places in the cache: token path[b][i] of the last N slots moves
 * to slot length - N + i, in every key/value head, and the rest is dropped.
 *   path        in: DEVICE int32 [B][N], rising places, up to the first -1
 *   lengths_out out: int32[B], length - N + the path's length; use it from then on
 *                    (cache->lengths is not changed); 0 for a sequence of length 0
 *   weights, slot_positions: float32 / int32 [B][Hkv][slots] or NULL: moved alike, in place
 * A path that does not rise or leaves the N places, a length between 0 and N or one that the
 * table or the accounts cannot hold is recorded as FA_ERR_SEQLEN: that sequence and its length stay as
 * they are.  Where the table names no page of the pool for a place on the path, or for the slot that it
 * goes to, FA_ERR_PAGE is recorded and that place is left out, its codes and its accounts: the length counts
 * it, its slot holds what it held.  The pages of the last N slots must be the sequence's own.
 */
int fa_kv4_keep(const fa_kv4_cache* cache, const int* path, int N, int* lengths_out, float* weights, int* slot_positions,
                long long slots, void* stream);

/*
 * Evicts down to `budget` tokens per sequence, for each key/value head by
 * itself.  Kept are the `recent` newest tokens (positions above the newest
 * minus recent) and the ones with the largest weights, ties to the lowest slot;
 * a NaN weight counts as the least.  A sequence of at most `budget` tokens
 * stays as it is.  Kept tokens below the new length stay in their slots; those
 * behind it move, in order, to the slots that fall free, so only what has to
 * move is moved (attention does not depend on the order of the slots).  The
 * pages of a sequence that loses tokens must be its own: what moves would move
 * under any other sequence whose table names them.
 *   weights, slot_positions in: [B][Hkv][slots] float32 / int32
 *   weights_out, positions_out out: the same after the eviction, 0 / -1 behind
 *                  the new length; buffers of their own
 *   lengths_out out: int32[B], min(length, budget)
 *   source     out: int32 [B][Hkv][budget]: the slot each kept token came from,
 *                  -1 behind the new length
 *   recent       : 0 .. budget (FA_ERR_ARG)
 *   workspace    : fa_kv4_evict_workspace(B, Hkv, budget) bytes, or NULL
 * cache->lengths is not changed: use lengths_out from then on.
 */
long long fa_kv4_evict_workspace(int B, int Hkv, int budget);
int fa_kv4_evict(const fa_kv4_cache* cache, const float* weights, const int* slot_positions, long long slots,
                 int budget, int recent, float* weights_out, int* positions_out, int* lengths_out, int* source,
                 void* workspace, long long workspace_bytes, void* stream);

/*
 * Host-only query (no GPU needed): the byte offset in the pool of the block
 * that holds `slot` of sequence b, head h, as the kernels look it up in a block
 * table, here a HOST int32[>= b + 1][width]; FA_ERR_PAGE where they refuse it.
 */
long long fa_kv4_block_offset(const int* block_table, int width, int Hkv, int D, int group, int page_size,
                              int num_pages, int b, int h, int slot);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* fa_strerror(int status);

/*
 * Synchronises `stream`, returns the device status word recorded by the
 * library's kernels on the current device since the last call (FA_OK,
 * FA_ERR_DEVICE_TIMEOUT, FA_ERR_SEQLEN or FA_ERR_PAGE), and clears it.  Returns FA_ERR_CUDA if the
 * synchronisation itself fails.
 */
int fa_get_device_status(void* stream);

/* Library ABI version (major * 100 + minor). */
int fa_version(void);

/*
 * Host-only schedule queries (no GPU needed).  They evaluate the exact index
 * logic the kernels use, so tests can compare it with a brute-force mask.
 *
 * fa_sched_fwd_tile_class / fa_sched_bwd_tile_class: class of the tile pair
 *   (query tile qt, key tile kt) as the forward / backward kernel sees it:
 *   0 = skipped (never loaded), 1 = full (no element mask), 2 = masked
 *   element by element.  The backward's query tile height depends on D.
 * fa_sched_fwd_keep / fa_sched_bwd_keep: 1 iff the kernel's composition of
 *   tile loop bounds, tile class and element mask keeps score (i, j).
 *   i and j may range over the padded extent (multiples of the tile sizes).
 * fa_sched_tile_rows: query tile height (fwd) or key tile height (bwd keys)
 *   and backward query tile height for head size D: writes bm_fwd, bn, bm_bwd.
 * Return negative fa_status on bad arguments.
 */
int fa_sched_fwd_tile_class(int T, int causal, int qt, int kt);
int fa_sched_bwd_tile_class(int T, int D, int causal, int qt, int kt);
int fa_sched_fwd_keep(int T, int causal, int i, int j);
int fa_sched_bwd_keep(int T, int D, int causal, int i, int j);
int fa_sched_tile_rows(int D, int* bm_fwd, int* bn, int* bm_bwd);

/*
 * Test hooks (host state, read at the next launch; default off).
 * fa_debug_set_wait_timeout_ns: bound of every in-kernel wait (default 2 s).
 * fa_debug_inject: 0 = off; 1 = the forward's load warp skips its first
 *   K/V tile copy; 2 = the load warp of the backward's first dK/dV CTA skips
 *   its third Q tile copy (its first when it has fewer); 3 = the load warp of
 *   the backward's first dQ CTA skips its first K tile copy; 4 = the load warp of the first CTA of cross
 *   attention's few-rows kernel skips its first K tile copy; 5 = the first CTA of fa_kv4_tree keeps its
 *   first tile of keys to itself.  The waits that depend on the missing copy
 *   run out, the CTA gives up (it waits, bounded, for its copies and MMAs in
 *   flight, frees its tensor memory and exits) and FA_ERR_DEVICE_TIMEOUT is
 *   reported instead of a hang; the outputs of that call are not valid.
 *   Used to test failure detection without faulting the GPU.  Other values
 *   return FA_ERR_ARG.
 */
int fa_debug_set_wait_timeout_ns(unsigned long long ns);
int fa_debug_inject(int mode);

/*
 * Backward determinism (host state, read by each fa_bwd / fa_bwd_gqa call;
 * default 0).  1: the backward never sums into global memory, so dq, dk and
 * dv are bitwise reproducible at every D (the two-kernel form; slower at
 * D = 64).  0: at D = 64 the backward computes dq in its dk/dv kernel and
 * sums the key tiles' contributions with float32 reduce-adds (see fa_bwd).
 * Returns FA_ERR_ARG unless on is 0 or 1.  fa_bwd_varlen and fa_bwd_noalloc
 * are always deterministic.
 */
int fa_set_deterministic(int on);

/*
 * Host query (no launch): 1 if fa_bwd / fa_bwd_gqa on this shape, on the
 * current device and in the current determinism mode, computes dq inside its
 * dk/dv kernel and sums it with reduce-adds (then its second kernel is the
 * conversion of the float32 accumulator to bf16 dq), 0 if it runs the
 * two-kernel form.  FA_ERR_SHAPE / FA_ERR_UNSUPPORTED for bad sizes,
 * FA_ERR_ARCH or FA_ERR_CUDA without a suitable current device.
 */
int fa_bwd_sums_dq_in_place(int B, int Hkv, int T, int D);

/*
 * 1 in the debug build of the library (compiled with FA_DEBUG), 0 in the
 * product build.  In the debug build the attention kernels check the tile
 * coordinates, ring stages, per-row vector offsets and tensor-memory columns
 * that they compute at run time before they use them (fa_decode, fa_rope and the other
 * fa_kv4_ calls but fa_kv4_tree and fa_kv4_keep have no such checks); a failed check skips the
 * access, makes the CTA give up through its bounded-wait exit path, and is
 * reported by fa_get_device_status as FA_ERR_DEBUG_CHECK.  Nothing traps.
 */
int fa_debug_checks_enabled(void);

/*
 * Measurement hook (default off; host state read by each call).  When the
 * pointers are non-NULL, later calls record these CUDA events (cudaEvent_t
 * passed as void*, created and owned by the caller) on the call's stream:
 * fwd_begin / fwd_end immediately around the forward kernel; bwd_begin
 * before the backward's dK/dV kernel, bwd_mid between it and the dQ kernel,
 * bwd_end after the dQ kernel (the preprocess is outside).  Pass NULLs to
 * turn it off.  Used to time the dominant kernels inside a timed region
 * without a profiler.
 */
int fa_set_timing_events(void* fwd_begin, void* fwd_end, void* bwd_begin, void* bwd_mid, void* bwd_end);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
