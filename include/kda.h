/*
 * kda.h -- C ABI of the GB300 (sm_103a) Kimi Delta Attention library, libkda.so.
 *
 * The operation.  Per (sequence, head) the library keeps a fixed-size state
 * S in R^{dk x dv} (fp32) and applies, for every token t, in this order
 * ("Kimi K3 Architecture Explained", section 3 "Kimi Delta Attention": decay
 * stale context first, then erase conflicting memory, then write):
 *
 *     S <- Diag(exp(g_t)) S               decay, per key channel
 *     S <- S - beta_t k_t (k_t^T S)        erase
 *     S <- S + beta_t k_t v_t^T            write
 *     o_t = S^T q_t                        read, after the update
 *
 * g is the caller's log-decay, normally g = -5 sigmoid(x) so that g lies in
 * (-5, 0) (Kimi K3 technical-report digest, section 2.1 (1): bounded scaled
 * sigmoid, g_min = -5).  There is no positional input and no 1/sqrt(d) scale.
 *
 * Layouts (all row-major, innermost index last, no padding):
 *   q, k : [T_tot, H, dk]   activation dtype (fp32 or bf16)
 *   v    : [T_tot, H, dv]   activation dtype
 *   out  : [T_tot, H, dv]   activation dtype
 *   g    : [T_tot, H, dk]   fp32
 *   beta : [T_tot, H]       fp32
 *   states (S0, S_final, S_inout, zero-initial states) : [.., dk, dv] fp32
 *   transfer matrices : [.., dk, dk] fp32
 * Sequences are packed along T_tot and delimited by cu_seqlens (device int32
 * [N+1], cu[0] = 0, non-decreasing, cu[N] = T_tot).
 *
 * Ownership and execution.  Every pointer except the descriptor is a DEVICE
 * pointer owned by the caller.  The library allocates no memory, never
 * synchronises the host, and launches only on the given stream (a
 * cudaStream_t passed as void*, NULL = the legacy default stream).  Results
 * are ready when that stream reaches them.  Outputs must not alias inputs,
 * except that S_final may equal S0.
 *
 * Errors.  Argument checks that the host can make return a status at once and
 * launch nothing.  Problems only the device can see (a malformed cu_seqlens, a
 * bounded wait that ran out) are written to *dev_status (device int32, may be
 * NULL; the first error sticks, 0 means no error) and the affected work is
 * skipped.  A failed launch returns KDA_ERR_CUDA.  Nothing aborts or throws.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1, /* null / misaligned pointer, bad size, bad cu_seqlens */
    KDA_ERR_UNSUPPORTED = 2, /* shape or dtype outside what the kernels cover      */
    KDA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required         */
    KDA_ERR_CUDA = 4,        /* a CUDA launch or runtime call failed               */
    KDA_ERR_TIMEOUT = 5      /* a bounded device-side wait gave up (dev_status)    */
} kda_status_t;

typedef enum { KDA_DTYPE_F32 = 0, KDA_DTYPE_BF16 = 1 } kda_dtype_t;

/* Problem description for the chunked prefill and the transfer pass. */
typedef struct {
    int32_t num_seqs;     /* N >= 0                                               */
    int32_t total_tokens; /* T_tot >= 0, equal to cu_seqlens[N]                   */
    int32_t num_heads;    /* H >= 1                                               */
    int32_t dk;           /* key / query width, 1..128                            */
    int32_t dv;           /* value width, 1..128                                  */
    int32_t act_dtype;    /* kda_dtype_t of q, k, v and out                       */
    int32_t chunk;        /* must be 16: the 16-token block of the digest, 2.1 (1) */
    int32_t num_segments; /* 0 = choose, 1 = one pass per (seq, head), S > 1 =     */
                          /* split every sequence into S chunk-aligned segments    */
                          /* joined by the transfer-matrix scan (digest 2.4 (1))   */
} kda_prefill_desc_t;

/*
 * Number of segments kda_prefill_chunked will use for desc (resolves
 * num_segments = 0 from the problem size and the current device's SM count).
 * Returns 0 for an invalid descriptor.
 */
int32_t kda_prefill_num_segments(const kda_prefill_desc_t *desc);

/*
 * Device workspace, in bytes, that kda_prefill_chunked needs for desc: zero
 * when it runs one pass, else room for N*H*S transfer matrices, zero-initial
 * states and segment start states (fp32), for BF16 at dk = dv = 128 also a BF16
 * copy of each start state laid out as a tensor-core operand (N*H*S x 128 x 128
 * x 2 bytes), and one dk-vector per token and head in the activation dtype;
 * each piece rounded up to 256 bytes.  Call with the same desc, on the same
 * device, as the prefill itself.
 */
size_t kda_prefill_workspace_size(const kda_prefill_desc_t *desc);

/*
 * Chunked prefill (the hot path): for every packed sequence and head, run the
 * recurrence above over its tokens starting from S0 (NULL = zeros), write o_t
 * for every token to out and, if S_final != NULL, the state after the last
 * token.  Chunked form: 16-token blocks, each turned into a WY/UT-transform
 * representation of its product of (I - beta k k^T) Diag(alpha) factors
 * ("intra-chunk parallel work"), then a sequential fp32 state step per block
 * ("cross-chunk state propagation"), overlapped as in the digest, section
 * 2.4 (1), FlashKDA.  With S > 1 segments every sequence is also split for
 * parallelism (digest 2.4 (1), KCP): kda_state_transfer on all S segments with
 * outputs (the zero-start outputs go straight to out), kda_state_compose (start
 * states and S_final), then kda_prefill_combine.  A zero-length sequence gives
 * S_final = S0.
 *
 *   desc            problem description (host pointer).
 *   q, k, v, g, beta, out   device arrays in the layouts above; q, k, v, g and
 *                   out 16-byte aligned, the rest 4-byte aligned.
 *   S0              [N, H, dk, dv] fp32 or NULL.
 *   cu_seqlens      [N+1] int32 (device).
 *   S_final         [N, H, dk, dv] fp32 or NULL; may equal S0.
 *   workspace       device buffer of workspace_bytes >= kda_prefill_workspace_size
 *                   (may be NULL when that is 0).  Contents on entry don't matter.
 *   dev_status      device int32 or NULL (see Errors).
 *   stream          cudaStream_t.
 */
kda_status_t kda_prefill_chunked(const kda_prefill_desc_t *desc, const void *q, const void *k,
                                 const void *v, const float *g, const float *beta,
                                 const float *S0, const int32_t *cu_seqlens, void *out,
                                 float *S_final, void *workspace, size_t workspace_bytes,
                                 int32_t *dev_status, void *stream);

/*
 * kda_prefill_chunked with stage timing, for measurement: identical launches
 * and results, and in addition records stage_events[0] (cudaEvent_t, created by
 * the caller) on the stream before the first launch, stage_events[1] after the
 * transfer pass (or the single output pass when the split is one segment),
 * stage_events[2] after the segment scan and stage_events[3] after the last
 * launch (with one segment 1, 2 and 3 follow each other).  Recording an event
 * between two launches keeps the next kernel from starting while the previous
 * one drains, so the call can take slightly longer than kda_prefill_chunked.
 * KDA_ERR_INVALID_ARG if stage_events or one of its four entries is NULL.
 */
kda_status_t kda_prefill_chunked_timed(const kda_prefill_desc_t *desc, const void *q,
                                       const void *k, const void *v, const float *g,
                                       const float *beta, const float *S0,
                                       const int32_t *cu_seqlens, void *out, float *S_final,
                                       void *workspace, size_t workspace_bytes,
                                       int32_t *dev_status, void *const *stage_events,
                                       void *stream);

/*
 * Fused gate prologue (digest, section 2.1 (1): g = -5 sigmoid(x), so g in
 * (-5, 0)): kda_prefill_chunked from the pre-activations, so the gates and the
 * normalised q, k are never written to memory.  The kernels take
 *     g = -5 sigmoid(x_g),  beta = sigmoid(x_beta),
 *     q <- q / ||q||,  k <- k / ||k||  per (token, head) over the key channels
 * (a zero row stays zero), in fp32, then run exactly as kda_prefill_chunked.
 * q, k [T_tot, H, dk] and v [T_tot, H, dv] as there (q, k not normalised); x_g
 * [T_tot, H, dk] in the activation dtype, 16-byte aligned; x_beta [T_tot, H]
 * fp32.  BF16 activations with dk = dv = 128 only (else KDA_ERR_UNSUPPORTED);
 * workspace as kda_prefill_workspace_size(desc).  HBM traffic per head-token
 * falls from 1540 to 1284 bytes at d = 128 (x_g in BF16 instead of fp32 g).
 */
kda_status_t kda_prefill_chunked_gated(const kda_prefill_desc_t *desc, const void *q,
                                       const void *k, const void *v, const void *x_g,
                                       const float *x_beta, const float *S0,
                                       const int32_t *cu_seqlens, void *out, float *S_final,
                                       void *workspace, size_t workspace_bytes,
                                       int32_t *dev_status, void *stream);

/*
 * Sparse state checkpoints during prefill (the fixed-size state is the unit of
 * the prefix cache: digest, section 2.4 (4)).  Everything kda_prefill_chunked
 * does, and in addition, for every sequence n and k = 0, 1, ... with
 * (k+1) * ckpt_interval <= len_n, the state after its first (k+1) * ckpt_interval
 * tokens is written to
 *     ckpt_states[(base_n + k) * H * dk * dv ...]   ([K, H, dk, dv] fp32),
 * base_n = sum over m < n of floor(len_m / ckpt_interval), K = that sum over all
 * sequences (the caller sizes ckpt_states for it; a checkpoint at a sequence's
 * last token equals its S_final).  ckpt_interval must be a positive multiple of
 * 16 (the block size), ckpt_states 4-byte aligned and not aliasing any other
 * argument.  With S > 1 segments the transfer pass also keeps the transfer matrix
 * so far at each checkpoint (floor(T_tot / ckpt_interval) * H * dk * dk fp32 of
 * extra workspace) and a last kernel adds its product with the segment's start
 * state once the scan has it.  Workspace: kda_prefill_ckpt_workspace_size(desc,
 * ckpt_interval) (0 on invalid arguments).  Errors as for kda_prefill_chunked;
 * a non-positive or unaligned interval returns KDA_ERR_INVALID_ARG.
 */
size_t kda_prefill_ckpt_workspace_size(const kda_prefill_desc_t *desc, int32_t ckpt_interval);
kda_status_t kda_prefill_chunked_ckpt(const kda_prefill_desc_t *desc, const void *q,
                                      const void *k, const void *v, const float *g,
                                      const float *beta, const float *S0,
                                      const int32_t *cu_seqlens, void *out, float *S_final,
                                      int32_t ckpt_interval, float *ckpt_states, void *workspace,
                                      size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * One decode step for `batch` independent sequences (one new token each): the
 * recurrence above applied once, in place on S_inout [batch, H, dk, dv] fp32,
 * with q, k [batch, H, dk], v, out [batch, H, dv] in act_dtype, g [batch, H,
 * dk] and beta [batch, H] fp32.  Streams each state through once.  dv must be
 * a multiple of 4 and S_inout 16-byte aligned (the others 4-byte aligned).
 * dev_status (device int32 or NULL, 4-byte aligned): KDA_ERR_TIMEOUT if a
 * bounded device-side wait gave up, in which case some states may not have
 * been stepped (S_inout is then partly old, partly new).
 */
kda_status_t kda_decode_step(int32_t batch, int32_t num_heads, int32_t dk, int32_t dv,
                             int32_t act_dtype, const void *q, const void *k, const void *v,
                             const float *g, const float *beta, float *S_inout, void *out,
                             int32_t *dev_status, void *stream);

/*
 * Transfer pass of the context-parallel split (digest, section 2.4 (1)): with
 * S = desc->num_segments >= 1, split every sequence into S chunk-aligned
 * segments (sequence n has c = ceil(len_n / 16) chunks; segment s takes chunks
 * [floor(s c / S), floor((s+1) c / S))) and compute for each (n, h, s)
 *     transfer        [N, H, S, dk, dk]  the matrix A with S_end = A S_start + B
 *     zero_init_state [N, H, S, dk, dv]  B, the state the segment reaches from 0.
 * Only segments s in [seg_begin, seg_end) are computed (0 <= seg_begin <=
 * seg_end <= S); the other slots are left untouched, so ranks or passes can
 * split the segments between them.  An empty segment gives A = I, B = 0.
 *
 * Outputs (optional: q, out_zero and out_transfer all NULL, or all given):
 * since S_t = A_t start + B_t inside a segment, o_t = B_t^T q_t + start^T (A_t^T
 * q_t).  The pass then also writes, for every token of those segments,
 *     out_zero     [T_tot, H, dv]  B_t^T q_t   (the output from a zero start)
 *     out_transfer [T_tot, H, dk]  A_t^T q_t
 * in the activation dtype; kda_prefill_combine adds the second term once the
 * start states are known.
 */
kda_status_t kda_state_transfer(const kda_prefill_desc_t *desc, int32_t seg_begin,
                                int32_t seg_end, const void *q, const void *k, const void *v,
                                const float *g, const float *beta, const int32_t *cu_seqlens,
                                float *transfer, float *zero_init_state, void *out_zero,
                                void *out_transfer, int32_t *dev_status, void *stream);

/*
 * Prefix scan that joins the segments (digest, section 2.4 (1)): for each of
 * `units` independent chains of `segments` (A_s, B_s) pairs,
 *     start_0 = S0 (NULL = zeros),  start_s = A_{s-1} start_{s-1} + B_{s-1},
 * written to seg_init_states [units, segments, dk, dv] (may be NULL), and
 * S_final [units, dk, dv] = A_{S-1} start_{S-1} + B_{S-1} (may be NULL; when it
 * is NULL the last pair is never read, so it need not have been computed).
 * transfer is [units, segments, dk, dk], zero_init_state [units, segments, dk,
 * dv]; all fp32, 16-byte aligned.  The scan is sequential over segments and
 * parallel over units and column blocks, in fp32.
 *
 * start_images (may be NULL; dk = dv = 128 only, else it must be NULL):
 * [units, segments, 128 * 128] BF16, 16-byte aligned, each start state rounded
 * to BF16 and laid out as the B operand of kda_prefill_combine's tensor-core
 * product (an internal layout: only kda_prefill_combine reads it).
 *
 * dev_status (device int32 or NULL, 4-byte aligned): KDA_ERR_TIMEOUT if a
 * bounded device-side wait of the scan gave up (its outputs are then
 * incomplete).
 */
kda_status_t kda_state_compose(int32_t units, int32_t segments, int32_t dk, int32_t dv,
                               const float *transfer, const float *zero_init_state,
                               const float *S0, float *seg_init_states, float *S_final,
                               void *start_images, int32_t *dev_status, void *stream);

/*
 * Output correction of the context-parallel split: for every token t of the
 * segments s in [first_segment, S) (S = desc->num_segments),
 *     out[t, h, :] += seg_init_states[n, h, s]^T out_transfer[t, h, :]
 * with seg_init_states [N, H, S, dk, dv] fp32 (from kda_state_compose) and
 * out_transfer [T_tot, H, dk] (from kda_state_transfer) in the activation
 * dtype.  out holds the zero-start outputs on entry and the outputs on exit.
 * first_segment = 1 skips the first segments' correction when they start from
 * zeros.  A dense product per segment on tensor cores for BF16 at d = 128: with
 * start_images (the BF16 images kda_state_compose wrote for the same states,
 * 16-byte aligned) through tcgen05, and seg_init_states may then be NULL;
 * without them from the fp32 states through mma.sync.  Other shapes: fp32 on
 * CUDA cores from seg_init_states.
 */
kda_status_t kda_prefill_combine(const kda_prefill_desc_t *desc, int32_t first_segment,
                                 const float *seg_init_states, const void *start_images,
                                 const void *out_transfer, const int32_t *cu_seqlens, void *out,
                                 int32_t *dev_status, void *stream);

/*
 * Output pass of the context-parallel split: with S = desc->num_segments >= 1
 * (segments as in kda_state_transfer), run segments [seg_begin, seg_end) of
 * every (sequence, head) from their given start states seg_init_states [N, H,
 * S, dk, dv] (as written by kda_state_compose; NULL = zeros), write o_t for
 * those segments' tokens to out and, if S_final != NULL and seg_end == S, the
 * state after the last segment.  With S = 1 and seg_init_states = S0 it is the
 * one-pass prefill; with S > 1 it is the alternative to kda_prefill_combine
 * (re-running every segment from its start state instead of correcting the
 * zero-start outputs).  Arguments otherwise as for kda_prefill_chunked.
 */
kda_status_t kda_prefill_segments(const kda_prefill_desc_t *desc, int32_t seg_begin,
                                  int32_t seg_end, const void *q, const void *k, const void *v,
                                  const float *g, const float *beta,
                                  const float *seg_init_states, const int32_t *cu_seqlens,
                                  void *out, float *S_final, int32_t *dev_status, void *stream);

/* Size of the device scratch compiled into the library for
 * kda_prefill_chunked_noalloc: 64 MiB, held on every GPU that loads it. */
#define KDA_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

/*
 * kda_prefill_chunked for callers that cannot allocate device memory (for
 * example an inference-engine plugin that may not call cudaMalloc while it
 * enqueues work, or a host whose device memory is all owned by another
 * framework's pool).  The source pages have no counterpart to this: it is a
 * convenience of this library.
 *
 * Same arguments and results as kda_prefill_chunked, minus the workspace: the
 * segment split's workspace comes from a fixed KDA_NOALLOC_SCRATCH_BYTES array
 * inside the library, and nothing is allocated.  A problem whose workspace
 * (kda_prefill_workspace_size) exceeds that returns KDA_ERR_WORKSPACE without
 * launching anything; pass desc->num_segments = 1 (no workspace) or a smaller
 * split instead.  The first call that needs the scratch on a device looks up
 * its address there (make that first call before any stream capture).  All
 * calls on a device share the one array and leave their data in it; nothing
 * has to be cleared between calls, but calls whose GPU work overlaps (e.g. on
 * two unordered streams) race on it and give wrong results.
 */
kda_status_t kda_prefill_chunked_noalloc(const kda_prefill_desc_t *desc, const void *q,
                                         const void *k, const void *v, const float *g,
                                         const float *beta, const float *S0,
                                         const int32_t *cu_seqlens, void *out, float *S_final,
                                         int32_t *dev_status, void *stream);

/*
 * Backward pass of the prefill ("Kimi K3 Architecture Explained", section 3: the
 * per-token recurrence, differentiated).  For the same inputs as
 * kda_prefill_chunked (q, k, v, g, beta, S0, cu_seqlens; q and k as the recurrence
 * uses them, i.e. already normalised) and the adjoints d_out [T_tot, H, dv] (the
 * activation dtype) and d_S_final [N, H, dk, dv] fp32 (NULL: zero), writes the
 * gradients of <d_out, o> + <d_S_final, S_final>:
 *     dq, dk, dg  [T_tot, H, dk] fp32,   dv [T_tot, H, dv] fp32,
 *     dbeta [T_tot, H] fp32,             dS0 [N, H, dk, dv] fp32 (NULL: skipped).
 * dg is the gradient with respect to the log-decay g (alpha = e^g).  All outputs
 * are overwritten; none may alias an input.
 *
 * BF16 activations at dk = dv = 128 take the chunked form on tensor cores (the
 * 16-token blocks of the prefill): the forward chain stores the BF16 state after
 * every 32 tokens, an adjoint chain runs every segment from its last block to its
 * first and stores the adjoint at every block end (BF16), and one CTA per SM then
 * walks the (block pair, head) items, forming every block's gradients from its
 * start state (stored, or one small product away inside the pair) and its end
 * adjoint, with no atomics.  q, k, v, g and d_out must then be 16-byte aligned
 * (KDA_ERR_INVALID_ARG otherwise).  Its results follow BF16 rounding of the
 * chain's operands and of the stored states (the BF16 tolerance of the prefill
 * applies).  Workspace: 32 KB per head and 32 tokens for the states and 32 KB per
 * head and 16 tokens (plus one block per sequence) for the adjoints, about 3 KB per
 * head-token, plus 256 KB per (sequence, head, segment) when segments are used,
 * part of it shared with the states.  Other dtypes and shapes take the token-level
 * form in fp32: one CTA per (sequence, head, 32 value columns) recomputes the
 * states from a checkpoint at every 4-token block start (16 KB of workspace per
 * head-token at d = 128); dq, dk, dg and dbeta are zeroed on the stream, then
 * accumulated.
 *
 * desc->num_segments (0: the library's choice, at most 64) splits every sequence
 * into segments run in parallel: each segment's transfer matrix A, zero-start
 * state and zero-end adjoint first, then scans for every segment's start state
 * and end adjoint (the adjoint map of a segment is A^T), then the chains per
 * segment.  The library's choice gives every SM one chain (chunked form: at least
 * 4 blocks per segment) or two (token-level form).  Workspace:
 * kda_prefill_backward_workspace_size(desc) (0 on invalid arguments).  A batch
 * too long for device memory is differentiated piece by piece, last piece first:
 * each piece from its start state (S0) with d_S_final = the next piece's dS0.
 * Pointers at least 4-byte aligned; KDA_ERR_INVALID_ARG on a missing or
 * misaligned pointer, KDA_ERR_WORKSPACE on a short workspace,
 * KDA_ERR_UNSUPPORTED as kda_prefill_chunked.
 */
size_t kda_prefill_backward_workspace_size(const kda_prefill_desc_t *desc);
/* Segments per sequence the backward pass uses for desc (0 on invalid arguments). */
int32_t kda_prefill_backward_num_segments(const kda_prefill_desc_t *desc);
kda_status_t kda_prefill_backward(const kda_prefill_desc_t *desc, const void *q, const void *k,
                                  const void *v, const float *g, const float *beta,
                                  const float *S0, const int32_t *cu_seqlens, const void *d_out,
                                  const float *d_S_final, float *dq, float *dk, float *dv,
                                  float *dg, float *dbeta, float *dS0, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------
 * Around the mixer: the norms, the token embedding and the loss of a model whose
 * mixer is the recurrence above, each with its gradient.  Same rules: device
 * pointers owned by the caller, nothing allocated or synchronised, launches on
 * the given stream only.  Activations (x, h, y, gate, tables, weights of the
 * loss, and their gradients) in act_dtype; norm weights and their gradients,
 * losses and row statistics fp32.  All arithmetic and every sum is in fp32,
 * rounded once on output.
 * ------------------------------------------------------------------------ */

typedef enum { KDA_GATE_NONE = 0, KDA_GATE_SIGMOID = 1, KDA_GATE_SILU = 2 } kda_gate_t;

/* Problem description of the norms. */
typedef struct {
    int64_t tokens;      /* T >= 0                                                   */
    int64_t x_stride;    /* elements from one token's x to the next's; 0 = heads x    */
    int64_t gate_stride; /* width.  The same for gate.  At least heads x width        */
    int32_t heads;       /* H >= 1 rows per token (1 for the residual norm)           */
    int32_t width;       /* D, 1..16384: the norm's row                              */
    int32_t act_dtype;   /* kda_dtype_t                                               */
    int32_t gate;        /* kda_gate_t (KDA_GATE_NONE for the residual norm)          */
    float eps;           /* > 0: r = 1 / sqrt(mean(x^2) + eps)                        */
} kda_norm_desc_t;

/*
 * The norm of a mixer's output with its gate: per row of D channels
 *     out = x r weight a(gate),  a = sigmoid, silu (z sigmoid(z)), or 1 without.
 *   x, gate   [T, H, D], tokens x_stride / gate_stride elements apart (a slice of a
 *             wider projection's output); gate NULL if and only if KDA_GATE_NONE.
 *   weight    [D] fp32, shared by all heads, or NULL (ones).
 *   out       [T, H, D] contiguous.
 * Pointers aligned to their element (16 bytes, with widths and strides of whole
 * 16-byte pieces, is the fast case), else KDA_ERR_INVALID_ARG.  dev_status (device
 * int32 or NULL), here and in the next three: KDA_ERR_TIMEOUT if a bounded wait of
 * the kernel gave up, its outputs being incomplete then.
 */
kda_status_t kda_gated_norm_forward(const kda_norm_desc_t *desc, const void *x, const void *gate,
                                    const float *weight, void *out, int32_t *dev_status,
                                    void *stream);

/*
 * Its gradients for the adjoint d_out [T, H, D] (contiguous): dx, d_gate [T, H, D]
 * (contiguous; d_gate NULL if and only if KDA_GATE_NONE) and d_weight [D] fp32
 * (may be NULL; zeros when T = 0), from the forward's inputs alone.  The sum over
 * rows behind d_weight has a fixed order.  Workspace (for d_weight):
 * kda_norm_backward_workspace_size(desc), 16-byte aligned (0 on invalid
 * arguments); KDA_ERR_WORKSPACE if it is short.
 */
size_t kda_norm_backward_workspace_size(const kda_norm_desc_t *desc);
kda_status_t kda_gated_norm_backward(const kda_norm_desc_t *desc, const void *d_out, const void *x,
                                     const void *gate, const float *weight, void *dx, void *d_gate,
                                     float *d_weight, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_status, void *stream);

/*
 * The residual stream between two blocks: the block's output y enters it scaled,
 * and the next block's input is its norm,
 *     h_out = h + scale y,   out = h_out r weight      (out from the unrounded sum)
 * over [T, D] (desc->heads = 1, KDA_GATE_NONE, strides 0).  y and h_out are both
 * NULL (the first block: out = norm of h) or both given; h_out may equal h.
 */
kda_status_t kda_residual_norm_forward(const kda_norm_desc_t *desc, const void *h, const void *y,
                                       const float *weight, float scale, void *h_out, void *out,
                                       int32_t *dev_status, void *stream);

/*
 * Its gradients, from h_out: with d_out for out and d_h_out (NULL: zero) for h_out,
 *     dh = d_h_out + (gradient through the norm),   dy = scale dh,
 * and d_weight [D] fp32 (may be NULL).  dy may be NULL (scale = 1: dy is dh).  dh may
 * equal d_h_out.  Workspace as kda_gated_norm_backward.
 */
kda_status_t kda_residual_norm_backward(const kda_norm_desc_t *desc, const void *d_out,
                                        const void *d_h_out, const void *h_out, const float *weight,
                                        float scale, void *dh, void *dy, float *d_weight,
                                        void *workspace, size_t workspace_bytes,
                                        int32_t *dev_status, void *stream);

typedef enum { KDA_ID_I32 = 0, KDA_ID_I64 = 1 } kda_id_dtype_t;

/* Problem description of the embedding. */
typedef struct {
    int32_t tokens;    /* T, 0..2^30                       */
    int32_t rows;      /* V, 1..2^30: the table's rows     */
    int32_t width;     /* D, 1..65536                      */
    int32_t act_dtype; /* kda_dtype_t of table, out, ...   */
    int32_t id_dtype;  /* kda_id_dtype_t of ids            */
    float scale;       /* finite                           */
} kda_embed_desc_t;

/*
 * Token embedding: out[t] = scale table[ids[t]], table [V, D], ids [T], out [T, D].
 * An id outside [0, V) gives a row of zeros and KDA_ERR_INVALID_ARG in dev_status.
 */
kda_status_t kda_embedding_forward(const kda_embed_desc_t *desc, const void *table, const void *ids,
                                   void *out, int32_t *dev_status, void *stream);

/*
 * The table's gradient, every row of d_table [V, D] (zeros for ids that do not
 * occur): d_table[v] = scale x sum of d_out[t] over the t with ids[t] = v.  The
 * tokens are sorted by id (stable), so the sum has a fixed order and needs no
 * floating-point atomics.  Ids outside [0, V) contribute nothing and are reported
 * as above.  Workspace: kda_embedding_backward_workspace_size(desc), 16-byte
 * aligned (0 on invalid arguments).
 */
size_t kda_embedding_backward_workspace_size(const kda_embed_desc_t *desc);
kda_status_t kda_embedding_backward(const kda_embed_desc_t *desc, const void *d_out,
                                    const void *ids, void *d_table, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Problem description of the cross entropy over a vocabulary. */
typedef struct {
    int64_t ignore_index; /* rows with this target have no loss and no gradient       */
    int32_t tokens;       /* T, 0..2^24                                              */
    int32_t vocab;        /* V, 1..2^24                                              */
    int32_t width;        /* D, 1..2^17                                              */
    int32_t act_dtype;    /* kda_dtype_t of x, weight and their gradients            */
    int32_t id_dtype;     /* kda_id_dtype_t of targets                               */
    int32_t piece;        /* backward: vocabulary columns per piece; 0 = choose      */
} kda_ce_desc_t;

/*
 * Softmax cross entropy of the logits z = x weight^T, x [T, D], weight [V, D],
 * which are never stored:
 *     lse[t] = log sum_v exp(z_tv),   loss[t] = lse[t] - z_{t, targets[t]}
 * (both [T] fp32; loss 0 where the target is ignore_index), and mean (one fp32, may
 * be NULL): the mean loss over the other rows, 0 if there are none.  A target
 * outside [0, V) other than ignore_index counts as ignored and is reported in
 * dev_status (KDA_ERR_INVALID_ARG).  BF16: products of BF16 on tensor cores with
 * fp32 accumulation; F32: each operand as three BF16 terms, six products, to
 * about fp32's own accuracy.  x and weight 16-byte aligned (tensor-map copies).
 * Workspace: kda_linear_ce_workspace_size(desc, 0), 16-byte aligned.
 */
size_t kda_linear_ce_workspace_size(const kda_ce_desc_t *desc, int32_t backward);
kda_status_t kda_linear_ce_forward(const kda_ce_desc_t *desc, const void *x, const void *weight,
                                   const void *targets, float *loss, float *lse, float *mean,
                                   void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                   void *stream);

/*
 * Its gradients for the adjoint d_loss [T] fp32 of loss (lse as the forward gave
 * it): dx [T, D] and d_weight [V, D] (either may be NULL), both overwritten.  Works
 * through the vocabulary in pieces of desc->piece columns (rounded up to 256; 0: 512 MiB
 * of dz, 4,096 columns at least): the piece's logits are computed again, dz = d_loss
 * (softmax - onehot) of the piece is held in BF16 (F32: three BF16 terms), and both
 * products read it.  BF16: dz's rounding is up to 2^-8 of a term; a factor that all rows'
 * d_loss share is not rounded.  Rows whose target is ignored have no part in d_weight
 * whatever x holds there (NaN, say), and dx 0.
 * Workspace: kda_linear_ce_workspace_size(desc, 1), 16-byte aligned: dz of a piece, a copy
 * of x and, whatever the piece, one of all of W where a tensor map cannot read it as it is
 * (F32 of more than 128 tokens, BF16 widths that are no multiples of 8).
 */
kda_status_t kda_linear_ce_backward(const kda_ce_desc_t *desc, const void *x, const void *weight,
                                    const void *targets, const float *lse, const float *d_loss,
                                    void *dx, void *d_weight, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------
 * A recurrent layer's parts beside the mixer: a linear recurrence whose state is
 * a vector, the gated feed-forward block, dropout.  Same rules as above.
 * ------------------------------------------------------------------------ */

/* What a token writes into the state: x itself, or (1 - e^g) x (a mean of the past
 * with weights that sum to 1, a GRU's update). */
typedef enum { KDA_WRITE_ADD = 0, KDA_WRITE_MIX = 1 } kda_write_t;

/* Problem description of the gated linear recurrence. */
typedef struct {
    int64_t x_stride;  /* elements from one token's x to the next's, 0 = channels: at   */
    int64_t g_stride;  /* least channels, at most 2^30.  The same for g                 */
    int32_t num_seqs;  /* N, 1..2^24                                                    */
    int32_t tokens;    /* T, 0..2^30                                                    */
    int32_t channels;  /* C, 1..2^20                                                    */
    int32_t act_dtype; /* kda_dtype_t of x, h and their adjoints                        */
    int32_t write;     /* kda_write_t                                                   */
} kda_recurrence_desc_t;

/*
 * The gated linear recurrence over packed sequences: every channel has a state,
 *     h_t = e^{g_t} h_{t-1} + w_t x_t,   w = 1 (KDA_WRITE_ADD) or 1 - e^{g_t} (KDA_WRITE_MIX),
 * from the sequence's h0 on.
 *   x           [T, C] act_dtype, tokens x_stride elements apart (a slice of a wider
 *               projection's output).
 *   g           [T, C] fp32 log-decays, normally <= 0 (-inf: the state starts anew; as by the
 *               formula, an infinite or NaN state does not).  Positive ones let a state grow:
 *               then the product of e^g over any run of tokens within 2,048 consecutive ones
 *               must stay between 2^-126 and 2^127.  Tokens are joined by such products, and
 *               beyond that range a state that is itself still finite may become infinite, NaN
 *               or zero.  (With g <= 0 a product below 2^-126 may count as zero.)  A state that
 *               has become infinite may be NaN from a later token on.
 *   h0          [N, C] fp32, or NULL (zero).
 *   cu_seqlens  int32 [N+1] as for the prefill (sequences may be empty), or NULL with
 *               N = 1: one sequence.
 *   h           [T, C] act_dtype: the state after every token, rounded once; the
 *               recurrence runs on in fp32.
 *   h_final     [N, C] fp32, or NULL: the state after each sequence's last token (h0
 *               where it has none); may equal h0.
 * A malformed cu_seqlens is reported in dev_status (KDA_ERR_INVALID_ARG) and nothing or
 * only part of the outputs is written; KDA_ERR_TIMEOUT there: a bounded wait gave up.
 * The results do not depend on how the work was spread over the GPU.
 * Workspace: kda_recurrence_workspace_size(desc, 0), 16-byte aligned (0 up to 256 tokens and
 * on invalid arguments).
 * Pointers aligned to their element; 64 channels or more, with strides and bases of whole 16
 * bytes, are the fast case.
 */
size_t kda_recurrence_workspace_size(const kda_recurrence_desc_t *desc, int32_t backward);
kda_status_t kda_recurrence_forward(const kda_recurrence_desc_t *desc, const void *x, const float *g,
                                    const float *h0, const int32_t *cu_seqlens, void *h,
                                    float *h_final, void *workspace, size_t workspace_bytes,
                                    int32_t *dev_status, void *stream);

/*
 * Its gradients for the adjoints d_h [T, C] (act_dtype) and d_h_final [N, C] fp32 (NULL:
 * zero), from x (read for KDA_WRITE_MIX only, may be NULL for KDA_WRITE_ADD), g, h0 and the
 * forward's h [T, C] (h_{t-1} is taken as it was rounded there), all but x and g contiguous:
 *     dx [T, C] act_dtype,  dg [T, C] fp32,  d_h0 [N, C] fp32 (NULL: skipped; may equal
 *     d_h_final).
 * Workspace: kda_recurrence_workspace_size(desc, 1), as above.
 */
kda_status_t kda_recurrence_backward(const kda_recurrence_desc_t *desc, const void *d_h,
                                     const void *x, const float *g, const void *h, const float *h0,
                                     const int32_t *cu_seqlens, const float *d_h_final, void *dx,
                                     float *dg, float *d_h0, void *workspace, size_t workspace_bytes,
                                     int32_t *dev_status, void *stream);

/*
 * One token of each of N sequences (desc->tokens = N): state_out = e^g state + w x [N, C]
 * fp32, h [N, C] the same in act_dtype.  state_out may equal state (in place).
 */
kda_status_t kda_recurrence_step(const kda_recurrence_desc_t *desc, const void *x, const float *g,
                                 const float *state, float *state_out, void *h, void *stream);

typedef enum { KDA_FFN_SIGMOID = 1, KDA_FFN_SILU = 2, KDA_FFN_GELU = 3 } kda_ffn_act_t;

/* Problem description of the gated feed-forward block. */
typedef struct {
    int32_t tokens;    /* T, 0..2^24                                              */
    int32_t width;     /* D, 1..2^17: the channels that it reads                  */
    int32_t hidden;    /* F, 1..2^20: the channels that it writes                 */
    int32_t act_dtype; /* kda_dtype_t of x, weight, h and their gradients         */
    int32_t act;       /* kda_ffn_act_t: sigmoid, silu, or gelu (with the error   */
                       /* function)                                               */
} kda_ffn_desc_t;

/*
 * The gated feed-forward block up to its last projection: with weight [2, F, D] (the
 * gate's projection, then the other one),
 *     h = act(x weight[0]^T) * (x weight[1]^T),   x [T, D], h [T, F];
 * the projections are never stored.  BF16: products of BF16 on tensor cores with fp32
 * accumulation; F32: each operand as three BF16 terms, six products, to about fp32's
 * own accuracy (of an infinite operand, or one that BF16 rounds to infinity, those terms are
 * NaN).  x and weight 16-byte aligned (tensor-map copies).  Workspace:
 * kda_gated_ffn_workspace_size(desc, 0), 16-byte aligned (may be NULL when that is 0).
 * dev_status, here and below: KDA_ERR_TIMEOUT if a bounded wait gave up.
 */
size_t kda_gated_ffn_workspace_size(const kda_ffn_desc_t *desc, int32_t backward);
kda_status_t kda_gated_ffn_forward(const kda_ffn_desc_t *desc, const void *x, const void *weight,
                                   void *h, void *workspace, size_t workspace_bytes,
                                   int32_t *dev_status, void *stream);

/*
 * Its gradients for the adjoint d_h [T, F]: dx [T, D] and d_weight [2, F, D] (either may
 * be NULL; d_weight zeros when T = 0).  The projections are computed again, in pieces of
 * the F channels whose adjoints (BF16; F32: three BF16 terms) take 1 GiB at most, or 512
 * channels.  BF16: those adjoints' rounding is up to 2^-8 of a term of dx and d_weight.
 * Workspace: kda_gated_ffn_workspace_size(desc, 1), 16-byte aligned.
 */
kda_status_t kda_gated_ffn_backward(const kda_ffn_desc_t *desc, const void *d_h, const void *x,
                                    const void *weight, void *dx, void *d_weight, void *workspace,
                                    size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Dropout whose mask is never stored: element (t, c) of a [T, D] array is kept where word
 * c mod 4 of Philox 4x32-10 (counter ((t ceil(D / 4) + c / 4) + site 2^48, offset), key
 * seed) is at least round(p 2^32), and kept values are divided by 1 - p (p as rounded). */
typedef struct {
    const int64_t *rng; /* device [2]: seed, offset; read when the kernel runs, so a captured */
                        /* graph drops other elements once they have changed                  */
    double p;           /* 0 <= p, and round(p 2^32) < 2^32                                   */
    int32_t site;       /* 0..65535: which of the dropouts that share rng this is             */
} kda_dropout_t;

/*
 * out = dropout of x, both [tokens, width] contiguous in act_dtype (tokens x width up to
 * 2^42); out may equal x.  Dropped elements are 0 whatever x holds there.  The gradient is
 * the same call on the adjoint of out.
 */
kda_status_t kda_dropout(const kda_dropout_t *dropout, int64_t tokens, int32_t width,
                         int32_t act_dtype, const void *x, void *out, void *stream);

/*
 * kda_residual_norm_forward with y (required) dropped out before it is added:
 *     h_out = h + scale dropout(y),   out = h_out r weight,
 * and kda_residual_norm_backward with the mask again: dy (required) = scale dropout(dh).
 * With p = 0 they give what the calls without dropout give.
 */
kda_status_t kda_residual_norm_dropout_forward(const kda_norm_desc_t *desc,
                                               const kda_dropout_t *dropout, const void *h,
                                               const void *y, const float *weight, float scale,
                                               void *h_out, void *out, int32_t *dev_status,
                                               void *stream);
kda_status_t kda_residual_norm_dropout_backward(const kda_norm_desc_t *desc,
                                                const kda_dropout_t *dropout, const void *d_out,
                                                const void *d_h_out, const void *h_out,
                                                const float *weight, float scale, void *dh, void *dy,
                                                float *d_weight, void *workspace,
                                                size_t workspace_bytes, int32_t *dev_status,
                                                void *stream);

/* Human-readable name of a status. Never NULL. */
const char *kda_status_string(kda_status_t status);

/* Build description (target architecture, library version). Never NULL. */
const char *kda_build_info(void);

/*
 * Self-test of the bounded device-side waits: one CTA waits, with a limit of
 * about limit_us microseconds of SM clocks, on an mbarrier that nothing arrives
 * on, then records KDA_ERR_TIMEOUT in dev_status (device int32, first error
 * wins) and returns, the same path every kernel takes when a wait gives up.
 * Nothing faults and the context stays usable.  limit_us in (0, 1e7].
 */
kda_status_t kda_selftest_wait_timeout(int32_t limit_us, int32_t *dev_status, void *stream);

/*
 * The same for a kernel whose blocks wait for one another: the linear recurrence of one
 * sequence (KDA_WRITE_ADD, no states; h NULL: its forward pass from x to out [T, C]; else its
 * gradient for the adjoint x, to out and dg) with no time to wait.  Of a long sequence some
 * block gives up in the middle of the work, the others with it, and dev_status (required) is
 * KDA_ERR_TIMEOUT; the outputs are then incomplete.  Workspace as for the call it stands for.
 */
kda_status_t kda_selftest_recurrence_timeout(const kda_recurrence_desc_t *desc, const void *x,
                                             const float *g, const void *h, void *out, float *dg,
                                             void *workspace, size_t workspace_bytes,
                                             int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
