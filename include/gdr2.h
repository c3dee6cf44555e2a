/*
 * gdr2.h -- C ABI of the B200 (sm_100a) Gated Delta Rule-2 sequence-mixer library (libgdr2.so).
 *
 * The operation is the Gated Delta Rule-2 recurrence of "Gated DeltaNet-2: Decoupling Erase and
 * Write in Linear Attention" (Hatamizadeh, Choi, Kautz), Eq. 10, restated step by step in the
 * review page's section "The Gated Delta Rule-2 State Update" (Steps 1-5). Per (batch b, head h),
 * with an fp32 state S in R^{dk x dv} (row = key channel, column = value channel):
 *
 *     alpha_t = exp(log_alpha_t)                           (section "Gate Parameterization", Eq. 12)
 *     S_t = (I - k_t (b_t (.) k_t)^T) Diag(alpha_t) S_{t-1} + k_t (w_t (.) v_t)^T        (Eq. 10)
 *     o_t = S_t^T q_t                                      (Step 5: read of the updated state)
 *
 * log_alpha is the channel-wise log-decay (<= 0 in normal use), b the channel-wise erase gate on the
 * key axis (in [0,1], or [0,2] for the negative-eigenvalue variant of Eq. 11), w the channel-wise
 * write gate on the value axis. There is no query scale and no normalisation inside the mixer.
 *
 * Conventions shared by every entry point
 *   Pointers    : device pointers (memory of the current CUDA device) unless stated otherwise.
 *                 Every pointer must be 16-byte aligned.
 *   Layouts     : contiguous, row-major. Token tensors q, k, log_alpha, b, dq, dk, dlog_alpha, db
 *                 are [B, T, H, dk]; v, w, o, dv, dw, d_o are [B, T, H, dv]; states and their
 *                 gradients are [B, H, dk, dv]. Decode drops the T axis.
 *   dtype       : q, k, v, b, w, o and dq, dk, dv, db, dw, d_o are fp32 (GDR2_F32) or bf16
 *                 (GDR2_BF16). log_alpha, dlog_alpha, all states and state gradients are fp32
 *                 whatever the dtype (the pages keep the log-decay and the state in fp32).
 *   Sizes       : B, T, H >= 1; dk, dv in {64, 128} for the chunk entry points; decode takes dk in
 *                 {64, 128} and dv a multiple of 64 up to 256.
 *   Ownership   : the caller owns every buffer, workspaces included. The library never allocates,
 *                 frees or synchronises; all work is enqueued on `stream` (a cudaStream_t; NULL is
 *                 the legacy default stream) and results are valid once that stream reaches them.
 *                 Inputs are read only. Outputs must not overlap inputs or each other (except the
 *                 decode state, updated in place).
 *   Errors      : every function returns a status (GDR2_OK = 0) and never aborts or prints. Invalid
 *                 arguments are rejected before anything is launched. A failed launch returns
 *                 GDR2_ERR_CUDA. gdr2_status_string() names a status.
 *   Threads     : entry points are re-entrant; concurrent calls on different streams are safe if
 *                 their buffers (workspaces included) are distinct. The exception is
 *                 gdr2_chunk_fwd_noalloc, whose calls share one scratch array per device (see there).
 */
#ifndef GDR2_H
#define GDR2_H

#include <stddef.h>

#if defined(__GNUC__)
#define GDR2_API __attribute__((visibility("default")))
#else
#define GDR2_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDR2_F32 = 0, GDR2_BF16 = 1 } gdr2_dtype;

enum {
    GDR2_OK = 0,
    GDR2_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, non-positive size, bad dtype */
    GDR2_ERR_UNSUPPORTED = 2,  /* head dimensions the library has no kernel for */
    GDR2_ERR_WORKSPACE = 3,    /* workspace missing or smaller than gdr2_workspace_bytes() */
    GDR2_ERR_CUDA = 4,         /* a CUDA launch or device query failed */
    GDR2_ERR_TIMEOUT = 5,      /* a bounded device-side wait expired (reported by gdr2_check) */
    GDR2_ERR_RANGE = 6,        /* a chunk's cumulative log-decay left the supported range (gdr2_check) */
    GDR2_ERR_BOUNDS = 7        /* debug build only: an index check in a kernel failed (gdr2_check) */
};

/* Library version as 10000*major + 100*minor + patch. */
GDR2_API int gdr2_version(void);

/* Static text for a status code (never NULL). */
GDR2_API const char *gdr2_status_string(int status);

/*
 * Device-side status of the calls made so far. The kernels never trap: a bounded wait that gives up
 * (about 2^26 polls of an mbarrier) or an input the chunk form cannot represent sets a bit in a device
 * status word and the kernel finishes. gdr2_check synchronises `stream` (a cudaStream_t; NULL = the
 * legacy default stream), reads and clears those words, and returns
 *   GDR2_ERR_TIMEOUT  a bounded wait expired: the outputs of the calls since the last check are not valid;
 *   GDR2_ERR_RANGE    in some chunk a channel's cumulative log-decay G_C (the sum of log_alpha over the
 *                     chunk's 64 rows) left [-160, 160] on the tensor-core path (dtype GDR2_BF16 with
 *                     dk = dv = 128) or [-80, 80] on the fp32 path, or was NaN: the chunk form scales keys
 *                     and erase keys by exponentials of the in-chunk log-decay in fp32 (relative to the
 *                     mid-chunk value on the tensor-core path), which leave its normal range there, so the
 *                     outputs of those calls are not valid (a mean log_alpha of -2.5, resp. -1.25, per
 *                     token over a full chunk reaches the bound; decode steps have no such limit), or,
 *                     on the per-chain path (gdr2_set_chunk_path), an fp16 operand of the chunk form
 *                     (w (.) v, the WY factors, the state) exceeded 65504 in magnitude;
 *   GDR2_ERR_BOUNDS   (only in the debug build, libgdr2_debug.so, compiled with -DGDR2_DEBUG) an index check in
 *                     a kernel failed: a chunk, chain, tile row or column, TMEM column or output index outside
 *                     its range; this is a library bug, reported first;
 *   GDR2_ERR_CUDA     the synchronisation or the read failed;
 *   GDR2_OK           otherwise.
 * It blocks the host until `stream` is idle; call it where a synchronisation is acceptable.
 */
GDR2_API int gdr2_check(void *stream);

/*
 * Kernel path of the chunk entry points for bf16 operands with dk = dv = 128 (unpacked batches, one value
 * head per key head). Both paths compute the chunkwise algorithm of the review's section "Chunkwise
 * Parallel Training via WY Representation"; they differ in how the work is laid out on the GPU:
 *   1  per-chain: one CTA walks each (batch, head) chain's chunks in order, reading every input once and
 *      keeping every derived operand on chip; fastest when the B*H chains fill most of a wave of SMs;
 *   2  chunk-parallel: the chunk-local work runs over all chunks at once and the serial state passes
 *      read its intermediates from the workspace, with the chunk-level scan when B*H is small;
 *   0  automatic (default): path 1 when a cost model with the step times measured on B200 favours it (B*H from
 *      91 to 148 chains, from 181 to 296, ...), path 2 otherwise.
 * The setting is process-wide and read at each call: gdr2_workspace_bytes() reports the size for the
 * path in force, so query it after changing the path, and keep the same path for a gdr2_chunk_fwd_train /
 * gdr2_chunk_bwd_saved pair. Results agree within the library's tolerances, not bit for bit. Returns
 * GDR2_ERR_INVALID_ARG for a value outside {0, 1, 2}.
 */
GDR2_API int gdr2_set_chunk_path(int path);
GDR2_API int gdr2_get_chunk_path(void);

/*
 * Bytes of device workspace that gdr2_chunk_fwd (for_bwd = 0) or gdr2_chunk_bwd (for_bwd = 1)
 * needs for these sizes. Returns 0 for invalid sizes. The workspace holds per-chunk intermediates of
 * the chunkwise algorithm (section "Chunkwise Parallel Training via WY Representation"): the WY
 * factors of Eq. 20, the chunk-boundary states of Eq. 23 and, for the backward, their gradients. It
 * needs no initialisation and its contents are meaningless after the call.
 */
GDR2_API size_t gdr2_workspace_bytes(int B, int T, int H, int dk, int dv, int dtype, int for_bwd);

/*
 * Chunkwise-parallel forward, C = 64 (review sections "Chunkwise Parallel Training via WY
 * Representation", Steps 1-3, Eqs. 20-24, and Appendix C.2). Computes o_t for every token and the
 * state after the last token, exactly the Eq. 10 recurrence up to floating-point rounding.
 *   q, k, b        [B,T,H,dk] dtype     v, w  [B,T,H,dv] dtype     log_alpha [B,T,H,dk] fp32
 *   initial_state  [B,H,dk,dv] fp32, or NULL for a zero state
 *   o              [B,T,H,dv] dtype (written)
 *   final_state    [B,H,dk,dv] fp32 (written), or NULL when not wanted
 *   T may be any value >= 1; a partial last chunk behaves as identity transitions.
 */
GDR2_API int gdr2_chunk_fwd(const void *q, const void *k, const void *v, const float *log_alpha,
                   const void *b, const void *w, const float *initial_state,
                   void *o, float *final_state,
                   int B, int T, int H, int dk, int dv, int dtype,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gate-aware chunkwise backward (review section "Gate-Aware Backward Pass", Eqs. 64-65, the
 * triangular-inverse VJP, the gate gradients dB = dEbar*gamma*K, dW = dZ*V, dV = dZ*W, and the
 * in-chunk reverse cumulative sum for the log-decay). The forward inputs are passed again and the
 * forward is recomputed inside; nothing from a previous gdr2_chunk_fwd call is needed.
 *   d_o            [B,T,H,dv] dtype, or NULL for zero      d_final_state [B,H,dk,dv] fp32 or NULL
 *   dq, dk, db     [B,T,H,dk] dtype (written)              dv, dw [B,T,H,dv] dtype (written)
 *   dlog_alpha     [B,T,H,dk] fp32 (written)
 *   d_initial_state[B,H,dk,dv] fp32 (written), or NULL when not wanted
 * These are the gradients of L = <o, d_o> + <S_T, d_final_state> with respect to q, k, v,
 * log_alpha, b, w and the initial state.
 */
GDR2_API int gdr2_chunk_bwd(const void *q, const void *k, const void *v, const float *log_alpha,
                   const void *b, const void *w, const float *initial_state,
                   const void *d_o, const float *d_final_state,
                   void *dq, void *dk, void *dv, float *dlog_alpha, void *db, void *dw,
                   float *d_initial_state,
                   int B, int T, int H, int dk_, int dv_, int dtype,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Training pair: forward that keeps what the backward needs, and the backward that uses it.
 * gdr2_chunk_fwd_train computes exactly what gdr2_chunk_fwd computes (o, final_state) and, in the
 * same pass, fills `workspace` with the per-chunk intermediates of the chunkwise algorithm (WY
 * factors, decay-scaled operands and chunk-boundary states of Eqs. 20-24). The workspace must hold
 * gdr2_workspace_bytes(..., for_bwd = 1) bytes.
 * gdr2_chunk_bwd_saved then computes exactly what gdr2_chunk_bwd computes, reading those
 * intermediates instead of recomputing the forward. Its arguments are those of gdr2_chunk_bwd; the
 * inputs, sizes, dtype and workspace must be the ones of the gdr2_chunk_fwd_train call that filled
 * the workspace, with nothing else written to the workspace in between (the library cannot check
 * this; a mismatch gives wrong gradients, not an error).
 */
GDR2_API int gdr2_chunk_fwd_train(const void *q, const void *k, const void *v, const float *log_alpha,
                                  const void *b, const void *w, const float *initial_state,
                                  void *o, float *final_state,
                                  int B, int T, int H, int dk, int dv, int dtype,
                                  void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_bwd_saved(const void *q, const void *k, const void *v, const float *log_alpha,
                                  const void *b, const void *w, const float *initial_state,
                                  const void *d_o, const float *d_final_state,
                                  void *dq, void *dk, void *dv, float *dlog_alpha, void *db, void *dw,
                                  float *d_initial_state,
                                  int B, int T, int H, int dk_, int dv_, int dtype,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * Grouped value heads (review, "Headed architecture and grouped-value attention" and Appendix C.3):
 * Hv = G H value heads share each key head. The key-side tensors stay on the key-head axis and value
 * head j reads key head floor(j / G); v, w, o and the states live on the value-head axis:
 *   q, k, log_alpha, b and dq, dk, dlog_alpha, db   [B, T, H, dk]
 *   v, w, o, d_o and dv, dw                          [B, T, Hv, dv]
 *   initial_state, final_state, d_final_state, d_initial_state   [B, Hv, dk, dv] fp32
 * Value head j computes exactly the recurrence of Eq. 10 with q, k, log_alpha, b of key head j / G
 * (the key side "repeated across the value-head group"); the key-side gradients are the sums of the
 * group's value heads' gradients. The four calls mirror gdr2_chunk_fwd, gdr2_chunk_fwd_train,
 * gdr2_chunk_bwd and gdr2_chunk_bwd_saved; the key-side work of a chunk is done once per group.
 * Hv must be a positive multiple of H (Hv = H is the plain layout); GDR2_BF16 with dk = dv = 128
 * only (others return GDR2_ERR_UNSUPPORTED). gdr2_workspace_bytes_gva returns 0 for invalid or
 * unsupported sizes.
 */
GDR2_API size_t gdr2_workspace_bytes_gva(int B, int T, int H, int Hv, int dk, int dv, int dtype, int for_bwd);

GDR2_API int gdr2_chunk_fwd_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                const void *b, const void *w, const float *initial_state,
                                void *o, float *final_state,
                                int B, int T, int H, int Hv, int dk, int dv, int dtype,
                                void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_fwd_train_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                      const void *b, const void *w, const float *initial_state,
                                      void *o, float *final_state,
                                      int B, int T, int H, int Hv, int dk, int dv, int dtype,
                                      void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_bwd_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                const void *b, const void *w, const float *initial_state,
                                const void *d_o, const float *d_final_state,
                                void *dq, void *dk, void *dv, float *dlog_alpha, void *db, void *dw,
                                float *d_initial_state,
                                int B, int T, int H, int Hv, int dk_, int dv_, int dtype,
                                void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_bwd_saved_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                      const void *b, const void *w, const float *initial_state,
                                      const void *d_o, const float *d_final_state,
                                      void *dq, void *dk, void *dv, float *dlog_alpha, void *db, void *dw,
                                      float *d_initial_state,
                                      int B, int T, int H, int Hv, int dk_, int dv_, int dtype,
                                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * Packed variable-length batches (review, Appendix C.6: sequences of different lengths packed along
 * one token axis, the state reset at every sequence start). The token tensors are [T, H, d] (B = 1):
 * the N sequences lie back to back, sequence n on tokens [cu_seqlens[n], cu_seqlens[n+1]).
 *   cu_seqlens     int32 [N + 1] DEVICE array, 0 = c_0 <= c_1 <= ... <= c_N = T (read on the stream;
 *                  the host never looks at it). Empty sequences are allowed. Other contents are not
 *                  an error the host can see: sequence n then covers [max_{m<=n} c_m, max_{m<=n+1} c_m)
 *                  clamped to [0, T], and tokens outside every sequence keep unspecified outputs.
 *   initial_state, final_state, d_final_state, d_initial_state
 *                  [N, H, dk, dv] fp32: one state per sequence (initial_state NULL = zeros).
 * Each sequence is computed exactly as a batch of one by gdr2_chunk_fwd / gdr2_chunk_bwd: a sequence
 * whose length is not a multiple of 64 ends in a partial chunk, and no chunk spans two sequences.
 * The four calls mirror gdr2_chunk_fwd, gdr2_chunk_fwd_train, gdr2_chunk_bwd and
 * gdr2_chunk_bwd_saved (the training pair shares one workspace of
 * gdr2_workspace_bytes_varlen(..., for_bwd = 1) bytes; the saved backward must get the same
 * cu_seqlens contents). Supported: dtype GDR2_BF16 with dk = dv = 128 (others return
 * GDR2_ERR_UNSUPPORTED); N <= 65535.
 * gdr2_workspace_bytes_varlen depends on N, T and H only (room for T/64 + N chunks per head, the
 * chunk and sequence tables, and one staging tile per sequence and head for the outputs of its
 * partial last chunk); it returns 0 for invalid or unsupported sizes.
 */
GDR2_API size_t gdr2_workspace_bytes_varlen(int N, int T, int H, int dk, int dv, int dtype, int for_bwd);

GDR2_API int gdr2_chunk_fwd_varlen(const void *q, const void *k, const void *v, const float *log_alpha,
                                   const void *b, const void *w, const float *initial_state,
                                   void *o, float *final_state, const int *cu_seqlens,
                                   int N, int T, int H, int dk, int dv, int dtype,
                                   void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_fwd_train_varlen(const void *q, const void *k, const void *v, const float *log_alpha,
                                         const void *b, const void *w, const float *initial_state,
                                         void *o, float *final_state, const int *cu_seqlens,
                                         int N, int T, int H, int dk, int dv, int dtype,
                                         void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_bwd_varlen(const void *q, const void *k, const void *v, const float *log_alpha,
                                   const void *b, const void *w, const float *initial_state,
                                   const void *d_o, const float *d_final_state,
                                   void *dq, void *dk, void *dv, float *dlog_alpha, void *db, void *dw,
                                   float *d_initial_state, const int *cu_seqlens,
                                   int N, int T, int H, int dk_, int dv_, int dtype,
                                   void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_bwd_saved_varlen(const void *q, const void *k, const void *v, const float *log_alpha,
                                         const void *b, const void *w, const float *initial_state,
                                         const void *d_o, const float *d_final_state,
                                         void *dq, void *dk, void *dv, float *dlog_alpha, void *db, void *dw,
                                         float *d_initial_state, const int *cu_seqlens,
                                         int N, int T, int H, int dk_, int dv_, int dtype,
                                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * Packed variable-length batches with grouped value heads: the two layouts above together. The token
 * tensors q, k, b, log_alpha are [T, H, dk] and v, w, o (and dv, dw, d_o) are [T, Hv, dv] with
 * Hv = G H, value head j reading key head j / G; the states are [N, Hv, dk, dv], one per (sequence,
 * value head). cu_seqlens, the sequence semantics and the workspace rules are those of the packed
 * calls, with gdr2_workspace_bytes_varlen_gva(..., for_bwd) bytes. Each sequence is computed exactly as
 * a batch of one by the grouped-head calls. Supported: dtype GDR2_BF16 with dk = dv = 128, Hv a
 * multiple of H, N and Hv <= 65535 (others return GDR2_ERR_INVALID_ARG or GDR2_ERR_UNSUPPORTED).
 */
GDR2_API size_t gdr2_workspace_bytes_varlen_gva(int N, int T, int H, int Hv, int dk, int dv, int dtype,
                                                int for_bwd);

GDR2_API int gdr2_chunk_fwd_varlen_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                       const void *b, const void *w, const float *initial_state,
                                       void *o, float *final_state, const int *cu_seqlens,
                                       int N, int T, int H, int Hv, int dk, int dv, int dtype,
                                       void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_fwd_train_varlen_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                             const void *b, const void *w, const float *initial_state,
                                             void *o, float *final_state, const int *cu_seqlens,
                                             int N, int T, int H, int Hv, int dk, int dv, int dtype,
                                             void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_bwd_varlen_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                       const void *b, const void *w, const float *initial_state,
                                       const void *d_o, const float *d_final_state,
                                       void *dq, void *dk, void *dv, float *dlog_alpha, void *db, void *dw,
                                       float *d_initial_state, const int *cu_seqlens,
                                       int N, int T, int H, int Hv, int dk_, int dv_, int dtype,
                                       void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_chunk_bwd_saved_varlen_gva(const void *q, const void *k, const void *v, const float *log_alpha,
                                             const void *b, const void *w, const float *initial_state,
                                             const void *d_o, const float *d_final_state,
                                             void *dq, void *dk, void *dv, float *dlog_alpha, void *db,
                                             void *dw, float *d_initial_state, const int *cu_seqlens,
                                             int N, int T, int H, int Hv, int dk_, int dv_, int dtype,
                                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gate and normalisation prologue: the steps immediately upstream of the mixer ("Gated DeltaNet-2",
 * review page, section "Gate Parameterization", Eqs. 11-12, and "Block Design", steps 2-3). Per
 * (token, head), from the branch pre-activations:
 *     q = x_q / ||x_q||,  k = x_k / ||x_k||      (L2 norm over the head's dk channels; a zero
 *                                                 vector gives zero, with zero gradient)
 *     log_alpha = -exp(a) (.) softplus(x_f + delta)          computed and stored in fp32 (Eq. 12)
 *     b = sigmoid(x_b), or 2 sigmoid(x_b) when neg_eig != 0  (Eq. 11, negative-eigenvalue variant)
 *     w = sigmoid(x_w)                                       (Eq. 11)
 * The outputs are exactly the inputs gdr2_chunk_fwd / gdr2_decode_step take.
 *   xq, xk, xf, xb [B,T,H,dk] dtype     xw [B,T,H,dv] dtype     a, delta [H,dk] fp32
 *   q, k, b [B,T,H,dk] dtype (written)  w [B,T,H,dv] dtype      log_alpha [B,T,H,dk] fp32
 * gdr2_gate_prologue_bwd takes the same inputs and the gradients of those outputs (dq, dk, db
 * [B,T,H,dk] dtype, dlog_alpha [B,T,H,dk] fp32, dw [B,T,H,dv] dtype) and writes dxq, dxk, dxf, dxb
 * [B,T,H,dk], dxw [B,T,H,dv] (dtype) and da, ddelta [H,dk] fp32 (sums over every token; computed
 * in a fixed order, so repeated calls give identical bits). Its workspace holds per-block partial
 * sums: gdr2_gate_prologue_workspace_bytes(...) bytes. Sizes, dtypes and errors as for the chunk
 * entry points (dk, dv in {64, 128}).
 */
GDR2_API size_t gdr2_gate_prologue_workspace_bytes(int B, int T, int H, int dk, int dv, int dtype);

GDR2_API int gdr2_gate_prologue_fwd(const void *xq, const void *xk, const void *xf, const void *xb,
                                    const void *xw, const float *a, const float *delta, int neg_eig,
                                    void *q, void *k, float *log_alpha, void *b, void *w,
                                    int B, int T, int H, int dk, int dv, int dtype, void *stream);

GDR2_API int gdr2_gate_prologue_bwd(const void *xq, const void *xk, const void *xf, const void *xb,
                                    const void *xw, const float *a, const float *delta, int neg_eig,
                                    const void *dq, const void *dk, const float *dlog_alpha,
                                    const void *db, const void *dw,
                                    void *dxq, void *dxk, void *dxf, void *dxb, void *dxw,
                                    float *da, float *ddelta,
                                    int B, int T, int H, int dk_, int dv, int dtype,
                                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * One-token recurrent decode step (review, Appendix C.5 "Recurrent decoding kernel"): for every
 * (b, h) the fp32 state is decayed by exp(log_alpha), read along b (.) k, written with w (.) v along
 * k, and o = S^T q is returned from the updated state.
 *   q, k, b    [B,H,dk] dtype      v, w  [B,H,dv] dtype      log_alpha [B,H,dk] fp32
 *   state      [B,H,dk,dv] fp32, read and overwritten in place with the new state
 *   o          [B,H,dv] dtype (written)
 * Needs no workspace.
 */
GDR2_API int gdr2_decode_step(const void *q, const void *k, const void *v, const float *log_alpha,
                     const void *b, const void *w, float *state, void *o,
                     int B, int H, int dk, int dv, int dtype, void *stream);

/*
 * The attention half of the hybrid cell ("Gated DeltaNet-2", review page, hybrid design: the mixer alternates
 * with sliding-window softmax attention). Training and prefill take the query / key prologue; serving takes the
 * prologue that writes into a paged key-value cache, the attention of one new token over that cache, and the
 * cache's bookkeeping. The conventions at the top of this file hold, except that arrays of ints, the gains gq
 * and gk, dgq, dgk and lse need the alignment of their own type only.
 *
 * Sizes: d in {64, 128}; Hq, Hk from 1 to 65,535 (attention: Hq a multiple of Hk, at most 1,024 times as many; query
 * head j reads KV head j / (Hq / Hk)); any page_size >= 1. Counted in 32 bits, and GDR2_ERR_UNSUPPORTED beyond:
 *   P page_size (a sequence's tokens), R P (a table's entries), num_pages    at most 2^31 - 65,536 each
 *   attention      N Hq and Hk page_size below 2^31, Hk page_size num_pages (token rows of a pool) below 2^32
 *   kv_fork, kv_compact   with c = 2 Hk ceil(page_size d sizeof(dtype) / 4096), the pieces that a page is copied in:
 *                  c below 2^31, c num_pages below 2^32 - 65,536
 * Norms are formed in fp32: the sum of a row's squares has to stay below 2^128 (the row becomes 0 beyond) and, with
 * eps = 0, above 2^-126.
 */

/*
 * Frequencies of the rotary positions, in radians per position and 64 bits, written to HOST memory: freqs [rot / 2]
 * and, unless NULL, the magnitude mag of the rotated channels. Pair i turns by base^(-2 i / rot) a position;
 *   GDR2_ROPE_PLAIN   as it is;
 *   GDR2_ROPE_LINEAR  divided by factor (positions interpolated);
 *   GDR2_ROPE_BASE    with base * factor^(rot / (rot - 2)) for base (the slowest pair slows by factor, the first
 *                     keeps its pace; rot > 2);
 *   GDR2_ROPE_PARTS   pairs that make fewer than turns_low turns over the original context of orig_len positions
 *                     divided by factor, those with more than turns_high kept, a linear ramp in the number of
 *                     turns between; mag = 0.1 ln(factor) + 1.
 * rot even, base > 0, factor >= 1, 0 <= turns_low < turns_high; arguments a scaling does not use are ignored.
 */
enum { GDR2_ROPE_PLAIN = 0, GDR2_ROPE_LINEAR = 1, GDR2_ROPE_BASE = 2, GDR2_ROPE_PARTS = 3 };
GDR2_API int gdr2_rope_freqs(double *freqs, double *mag, int rot, double base, int scaling, double factor,
                             double orig_len, double turns_low, double turns_high);

/*
 * Query / key prologue of the attention layer. Per (token t, head), x the d channels of the projection:
 *     u = x / sqrt(mean(x^2) + eps) (.) g          (norm = 1; g = gq for queries, gk for keys, NULL = ones)
 *     u = x                                         (norm = 0; gq and gk have to be NULL)
 *     the first rot channels of u turned pairwise by pos[t] * freqs[i], i < rot / 2, and multiplied by mag; pair i
 *     is (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved != 0; the other channels pass unchanged.
 *   xq [T, Hq, d], xk [T, Hk, d] dtype   heads and channels contiguous, xq_stride / xk_stride elements from token to
 *                  token (multiples of 16 bytes; larger than H d for views of a fused projection). Batches are
 *                  flattened: T = B * sequence length.
 *   gq, gk [d] fp32   pos int32 [T] (any sign)   freqs fp64 [rot / 2], DEVICE memory; both may be NULL when rot = 0
 *   q [T, Hq, d], k [T, Hk, d] dtype (written, contiguous)
 * rot is a multiple of 16 of at most d. Angles are formed in 64 bits, norms and sums in fp32.
 * gdr2_attn_prologue_bwd takes the same inputs and dq, dk (contiguous, dtype) and writes dxq, dxk (with their own
 * token strides, so that they can be views of one gradient of a fused projection) and, unless NULL, dgq, dgk [d]
 * fp32: sums over every token and head, in a fixed order. Its workspace of
 * gdr2_attn_prologue_workspace_bytes(d) bytes is needed with dgq or dgk only.
 */
GDR2_API int gdr2_attn_prologue_fwd(const void *xq, const void *xk, const float *gq, const float *gk, int norm,
                                    float eps, const int *pos, const double *freqs, float mag, int rot,
                                    int interleaved, void *q, void *k, int T, int Hq, int Hk, int d, int dtype,
                                    long long xq_stride, long long xk_stride, void *stream);

GDR2_API size_t gdr2_attn_prologue_workspace_bytes(int d);

GDR2_API int gdr2_attn_prologue_bwd(const void *xq, const void *xk, const float *gq, const float *gk, int norm,
                                    float eps, const int *pos, const double *freqs, float mag, int rot,
                                    int interleaved, const void *dq, const void *dk, void *dxq, void *dxk, float *dgq,
                                    float *dgk, int T, int Hq, int Hk, int d, int dtype, long long xq_stride,
                                    long long xk_stride, long long dxq_stride, long long dxk_stride, void *workspace,
                                    size_t workspace_bytes, void *stream);

/*
 * The paged key-value cache: pools k_pages, v_pages [num_pages, Hk, page_size, d] dtype and a page table
 * int32 [R, P] in device memory. Entry (r, j) is the page that holds tokens [j page_size, (j + 1) page_size) of
 * sequence r; any value outside [0, num_pages) means that there is none.
 *
 * gdr2_attn_prologue_cache is the prologue for T new tokens of any of the cache's sequences (one each for a decode
 * step, whole prompts packed for a prefill): q is written as by gdr2_attn_prologue_fwd, the finished key and the value
 * row xv[t] go to the cache. Token t is token pos[t] of sequence seq[t].
 *   seq, pos int32 [T]     xv [T, Hk, d] dtype, xv_stride elements from token to token
 * A token whose seq is outside [0, R) is padding: nothing of it is written, its q row included. A token whose page is
 * not there (or whose pos is outside the table) gets its q row only. Two tokens for one place leave
 * it undefined.
 */
GDR2_API int gdr2_attn_prologue_cache(const void *xq, const void *xk, const void *xv, const float *gq, const float *gk,
                                      int norm, float eps, const int *seq, const int *pos, const double *freqs,
                                      float mag, int rot, int interleaved, void *q, void *k_pages, void *v_pages,
                                      const int *table, int T, int Hq, int Hk, int d, int R, int P, int page_size,
                                      int num_pages, int dtype, long long xq_stride, long long xk_stride,
                                      long long xv_stride, void *stream);

/*
 * Attention of one new token for each of N slots over the cache. Slot n reads sequence seq[n] (seq NULL: n, with
 * N <= R), tokens [max(0, len - window), len) with len = lens[seq[n]] (the new token included; held to
 * [0, P page_size]) and window = 0 for all of them; tokens whose page is not there are left out:
 *     s_i = scale q_j . k_i,   o_j = sum_i exp(s_i) v_i / sum_i exp(s_i),   lse_j = ln sum_i exp(s_i)
 *   q, o [N, Hq, d] dtype     lens int32 [R]     lse fp32 [N, Hq], or NULL when not wanted
 * With no token left o = 0 and lse = -inf. A slot whose seq is outside [0, R) is padding: its rows of o and lse are
 * left as they were. What lies in the pools outside the tokens read (NaN included) has no effect. Statistics and sums
 * are fp32; a finite v is assumed. Repeated calls give identical bits. The lengths are read on the stream, so a
 * captured call stays valid as sequences grow. The workspace query returns 0 for sizes that need none (short tables
 * or windows) and for invalid ones.
 */
GDR2_API size_t gdr2_attn_decode_workspace_bytes(int N, int Hq, int Hk, int d, int P, int page_size, int window,
                                                 int dtype);

GDR2_API int gdr2_attn_decode(const void *q, const void *k_pages, const void *v_pages, const int *table,
                              const int *lens, const int *seq, float scale, int window, void *o, float *lse, int N,
                              int Hq, int Hk, int d, int R, int P, int page_size, int num_pages, int dtype,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * Page bookkeeping, on the device and without the host's knowledge of any length. ref int32 [num_pages] counts the
 * table entries that name a page (a caller may add to it to pin one); a page with ref <= 0 is free. Free pages are
 * handed out lowest number first to entries in (r, j) order, so each call has exactly one result. Each call reads
 * table, lens and ref and writes the state after it to table_out, lens_out, ref_out; the workspace is
 * gdr2_kv_workspace_bytes(R, P, num_pages) bytes.
 *
 * gdr2_kv_reserve: pages for tokens [lens[r], want[r]) of every sequence: its entries j with
 * lens[r] / page_size <= j < ceil(want[r] / page_size) that have no page get one (want[r] = 0 asks for none). With
 * window > 0 the pages that lie wholly behind the window of the token at lens[r] are released first. missing (int32
 * [1]): how many pages were asked for and not found, past the table's end included, held to 2^31 - 1; their entries
 * stay empty.
 * table_out may be table and ref_out may be ref.
 *
 * gdr2_kv_fork: every sequence r takes over the content that sequence parent[r] had before the call: r itself (it
 * stays as it is), another one (a fork or a reordering), or, outside [0, R), none (its pages are released, its length
 * is 0). Full pages are shared. The last, partly filled page of a parent stays with one taker, together with pages
 * reserved beyond it: with the parent if it stays, else with the lowest r; every other taker gets the tokens of that
 * page copied to a fresh one (the rest of the fresh page is left as it was). missing: how many copies found no page;
 * those sequences end at their last full page. A length outside [0, P page_size] is taken over as it is; the pages then
 * follow as for the nearest length inside. table_out and lens_out must not be table and lens; ref_out may be ref.
 *
 * gdr2_kv_compact: the live pages end up in [0, live): those numbered live or above move, in order, to the free numbers
 * below. table_out and ref_out follow, live (int32 [1]) is written. table_out may be table and ref_out may be ref.
 * An entry that names a free page keeps its number.
 */
GDR2_API size_t gdr2_kv_workspace_bytes(int R, int P, int num_pages);

GDR2_API int gdr2_kv_reserve(const int *table, const int *lens, const int *want, const int *ref, int *table_out,
                             int *ref_out, int *missing, int R, int P, int page_size, int num_pages, int window,
                             void *workspace, size_t workspace_bytes, void *stream);

GDR2_API int gdr2_kv_fork(const int *table, const int *lens, const int *ref, const int *parent, int *table_out,
                          int *lens_out, int *ref_out, int *missing, void *k_pages, void *v_pages, int R, int P,
                          int Hk, int page_size, int d, int num_pages, int dtype, void *workspace,
                          size_t workspace_bytes, void *stream);

GDR2_API int gdr2_kv_compact(const int *table, const int *ref, int *table_out, int *ref_out, int *live, void *k_pages,
                             void *v_pages, int R, int P, int Hk, int page_size, int d, int num_pages, int dtype,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * The seven calls above with their arguments in one record: the parameters of each, in their order. For callers that
 * pay by the argument (through Python's ctypes a gdr2_attn_decode that the host bounds takes 13.2 us by its 22
 * arguments and 11.8 us by its record). args is aligned to 8 bytes, `bytes` is the record's size. The statuses are those of
 * the call itself.
 */
typedef struct {
    const void *xq; const void *xk; const float *gq; const float *gk; int norm; float eps; const int *pos;
    const double *freqs; float mag; int rot; int interleaved; void *q; void *k; int T; int Hq; int Hk; int d;
    int dtype; long long xq_stride; long long xk_stride; void *stream;
} gdr2_attn_prologue_fwd_args;

typedef struct {
    const void *xq; const void *xk; const float *gq; const float *gk; int norm; float eps; const int *pos;
    const double *freqs; float mag; int rot; int interleaved; const void *dq; const void *dk; void *dxq; void *dxk;
    float *dgq; float *dgk; int T; int Hq; int Hk; int d; int dtype; long long xq_stride; long long xk_stride;
    long long dxq_stride; long long dxk_stride; void *workspace; size_t workspace_bytes; void *stream;
} gdr2_attn_prologue_bwd_args;

typedef struct {
    const void *xq; const void *xk; const void *xv; const float *gq; const float *gk; int norm; float eps;
    const int *seq; const int *pos; const double *freqs; float mag; int rot; int interleaved; void *q;
    void *k_pages; void *v_pages; const int *table; int T; int Hq; int Hk; int d; int R; int P; int page_size;
    int num_pages; int dtype; long long xq_stride; long long xk_stride; long long xv_stride; void *stream;
} gdr2_attn_prologue_cache_args;

typedef struct {
    const void *q; const void *k_pages; const void *v_pages; const int *table; const int *lens; const int *seq;
    float scale; int window; void *o; float *lse; int N; int Hq; int Hk; int d; int R; int P; int page_size;
    int num_pages; int dtype; void *workspace; size_t workspace_bytes; void *stream;
} gdr2_attn_decode_args;

typedef struct {
    const int *table; const int *lens; const int *want; const int *ref; int *table_out; int *ref_out; int *missing;
    int R; int P; int page_size; int num_pages; int window; void *workspace; size_t workspace_bytes; void *stream;
} gdr2_kv_reserve_args;

typedef struct {
    const int *table; const int *lens; const int *ref; const int *parent; int *table_out; int *lens_out;
    int *ref_out; int *missing; void *k_pages; void *v_pages; int R; int P; int Hk; int page_size; int d;
    int num_pages; int dtype; void *workspace; size_t workspace_bytes; void *stream;
} gdr2_kv_fork_args;

typedef struct {
    const int *table; const int *ref; int *table_out; int *ref_out; int *live; void *k_pages; void *v_pages; int R;
    int P; int Hk; int page_size; int d; int num_pages; int dtype; void *workspace; size_t workspace_bytes;
    void *stream;
} gdr2_kv_compact_args;

enum {
    GDR2_CALL_ATTN_PROLOGUE_FWD = 0, GDR2_CALL_ATTN_PROLOGUE_BWD = 1, GDR2_CALL_ATTN_PROLOGUE_CACHE = 2,
    GDR2_CALL_ATTN_DECODE = 3, GDR2_CALL_KV_RESERVE = 4, GDR2_CALL_KV_FORK = 5, GDR2_CALL_KV_COMPACT = 6
};
GDR2_API int gdr2_attn_call(int call, const void *args, size_t bytes);

/*
 * gdr2_chunk_fwd for callers that cannot allocate device memory. The paper has no counterpart to
 * this entry point: it exists for callers that only receive input and output buffers -- plugins in a
 * host framework that owns all device memory through its own pool, or latency-critical loops where a
 * cudaMalloc (which may synchronise the device) is not allowed -- and so cannot pass the workspace
 * that gdr2_chunk_fwd needs.
 * Arguments and results are those of gdr2_chunk_fwd without the workspace pair; the computation is
 * the plain fp32-FMA chunkwise forward. Its scratch is one fixed 32 MiB array compiled into the
 * library, which every GPU that loads the library holds until the process exits.
 *   Limit   : B*H*ceil(T/64) * (6*64*dk + 2*64*dv + 2*64*64) * 4 bytes must not exceed 32 MiB, i.e.
 *             B*H*ceil(T/64) <= 113 (dk = dv = 128), 204 (dk = dv = 64), 170 (dk = 64, dv = 128) or
 *             128 (dk = 128, dv = 64). Larger problems (including sizes whose products would not fit
 *             in 64 bits) return GDR2_ERR_WORKSPACE before anything is launched.
 *   Set-up  : every call looks up the array's device address (cudaGetSymbolAddress, with the caller's
 *             device current), so the address stays right after a device reset or a rebuilt primary
 *             context. The first call on a device (and the first after such a reset) may load the
 *             library's device code; make it before any stream capture.
 *   Sharing : all calls in the process share the one array per device, which keeps the last call's
 *             contents (every scratch element is written before it is read, so nothing needs
 *             clearing). Calls whose kernels overlap on the GPU race on it: issue them on one stream
 *             or otherwise order them.
 * Allocates nothing: no cudaMalloc, cudaFree or allocating library routine is called.
 */
GDR2_API int gdr2_chunk_fwd_noalloc(const void *q, const void *k, const void *v, const float *log_alpha,
                                    const void *b, const void *w, const float *initial_state,
                                    void *o, float *final_state,
                                    int B, int T, int H, int dk, int dv, int dtype, void *stream);

/*
 * Benchmark support (not part of the method): per-kernel device time. gdr2_profile_enable(1) makes
 * every later kernel launch of this library record a CUDA event pair on its own stream (events come
 * from a pool created on first use; at most 8192 launches are held, later ones are counted in
 * *dropped). gdr2_profile_collect waits for the recorded events, writes up to max_entries distinct
 * kernel names (NUL-terminated, name_stride bytes apart in `names`) with their launch counts and summed
 * milliseconds, clears the records, and returns the number of entries (or minus a status code).
 * `names`, `launches`, `ms` and `dropped` are host pointers.
 */
GDR2_API int gdr2_profile_enable(int on);
GDR2_API int gdr2_profile_collect(char *names, int name_stride, int *launches, double *ms, int max_entries,
                                  int *dropped);

#ifdef __cplusplus
}
#endif

#endif /* GDR2_H */
