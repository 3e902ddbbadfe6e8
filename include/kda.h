/*
 * kda.h - C ABI of the MI355X (gfx950) Kimi Delta Attention forward library.
 *
 * One call, kda_fwd(), runs the chunked KDA forward pass on the GPU: the
 * per-channel gated delta-rule recurrence over head dimension K = V = 128.
 * Per (sequence, head) chain and token t (state S is K x V, fp32):
 *
 *   a_t  = lower_bound * sigmoid(exp(A_log[h]) * (g_t + dt_bias[h,:]))
 *   S    = diag(exp(a_t)) S
 *   S    = S + sigmoid(beta_t) k_t (v_t - S^T k_t)^T
 *   o_t  = scale * S^T q_t
 *
 * Where each piece is defined (the FlashKDA pages):
 *   - the tensor contract, dtypes, shapes, contiguity, K = V = 128, the
 *     sigmoid on beta, the optional recurrent states and packed sequences:
 *     "FlashKDA Input Tensor Shapes and DTypes", all sections;
 *   - the gate, lower_bound in [-5, 0] and its log2 rescaling
 *     gate_scale = lower_bound * log2(e): "FlashKDA lower_bound Parameter",
 *     "Conversion to the Gate Scale Factor" and the FAQ on dt_bias;
 *   - the base-2 exponent: "Base-2 Exponent Optimization in FlashKDA",
 *     "Re-basing the Gate Activation";
 *   - chunks of 16 tokens and the 16x16 unit-triangular inverse:
 *     "How FlashKDA's CHUNK Size of 16 Improves Numerical Stability",
 *     "Efficient 16x16 Matrix Inversion".
 * The pages never write the delta-rule update or the place of A_log; the
 * library takes the reading above (A_log multiplies the biased gate inside
 * the sigmoid; decay, then write with the decayed state, then read).
 *
 * Ownership and threading: the caller owns every buffer.  All tensor
 * pointers are DEVICE pointers to contiguous row-major memory on the current
 * HIP device.  The library allocates nothing, reads no environment
 * variables, never synchronises and is safe to call from several host
 * threads; apart from kda_fwd_scan_static (one fixed scratch array per GPU,
 * shared by its calls, see there) it keeps no state between calls.  The
 * work is enqueued on `stream` (a hipStream_t; NULL = the default stream)
 * and completes asynchronously.
 */
#ifndef KDA_H
#define KDA_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes.  Every argument error is detected on the host, before any
 * work is enqueued, and leaves every buffer untouched. */
typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_NULL_POINTER = 1,  /* q, k, v, g, beta or out is NULL while T > 0,
                                  or a state pointer is given with dtype
                                  KDA_DTYPE_NONE */
    KDA_ERR_HEAD_DIM = 2,      /* K != 128 or V != 128 */
    KDA_ERR_LOWER_BOUND = 3,   /* lower_bound outside [-5, 0], or NaN */
    KDA_ERR_VARLEN_BATCH = 4,  /* cu_seqlens given with B != 1, or num_seqs < 0 */
    KDA_ERR_STATE_DTYPE = 5,   /* unknown state dtype, or initial_state and
                                  final_state both given with different dtypes */
    KDA_ERR_ALIAS = 6,         /* out or final_state overlaps an input, or
                                  final_state partly overlaps initial_state */
    KDA_ERR_SIZE = 7,          /* B < 1, H < 1, H > 65536, T < 0 or
                                  T > 2^31-1, sizes overflow int64, or more
                                  than 2^31-1 (sequence, head) chains; the
                                  layer operators: also rows < 0, gate_period
                                  < 1, a grid beyond 2^32 threads, T >= 2^31
                                  - 128 of kda_ssm_fwd and kda_delta_fwd,
                                  window < 0, or page tables for more than
                                  2^31 - 65537 tokens */
    KDA_ERR_SCALE = 8,         /* scale is not finite; the layer operators: eps is
                                  not finite or negative, or a scale is not 0
                                  or a normal number of fp32 */
    KDA_ERR_LAUNCH = 9,        /* the HIP runtime rejected the launch */
    KDA_ERR_WORKSPACE = 10,    /* kda_fwd_scan, kda_ssm_fwd, kda_delta_fwd,
                                  kda_paged_attention: workspace NULL, not
                                  16-byte aligned, smaller than the call's
                                  ..._workspace_bytes(), or overlapping a
                                  tensor argument */
    KDA_ERR_ALIGNMENT = 11,    /* a non-NULL pointer is misaligned: q, k, v,
                                  g, out, initial_state and final_state need
                                  16 bytes, beta 2, A_log and dt_bias 4,
                                  cu_seqlens 8 (allocator memory and whole
                                  token rows of it always are); the layer
                                  operators' other inputs: their element's
                                  size, residual_out 16 */
    KDA_ERR_OPTION = 12,       /* kda_options: an unknown value, a non-zero
                                  reserved field, or a kernel / inverse /
                                  sigmoid combination that no kernel of the
                                  library implements for this call; the layer
                                  operators: an unknown activation or flag, or
                                  a non-zero reserved field */
    KDA_ERR_SHAPE = 13,        /* layer operators: a width, head, state, group
                                  or norm size outside the supported ones */
    KDA_ERR_DTYPE = 14,        /* layer operators: a weight, gate or residual
                                  dtype that is neither bf16 nor fp32 */
    KDA_ERR_STRIDE = 15        /* layer operators: a negative stride, one
                                  whose extent overflows int64, a token
                                  stride beyond kda_ssm_fwd's or
                                  kda_delta_fwd's, or a cache to be written
                                  whose places share memory */
} kda_status;

/* Element type of initial_state / final_state (and of the layer operators'
 * weights, gates and residual streams). */
typedef enum kda_dtype {
    KDA_DTYPE_NONE = 0,
    KDA_DTYPE_BF16 = 1,
    KDA_DTYPE_FP32 = 2
} kda_dtype;

/*
 * Explicit choices for kda_fwd_ex and kda_fwd_scan (a NULL options pointer
 * means all defaults, which is what kda_fwd uses).  They change how the
 * same result is computed, never what is computed: the kernel, and two of
 * the pages' own design choices kept as ablations.
 *
 *   kernel   KDA_KERNEL_AUTO: decode-shaped calls (no cu_seqlens, at most
 *            16 tokens), where the state traffic dominates, take the token
 *            recurrence (at most 8 tokens) or the single-chunk kernel; all
 *            other calls the pipelined chunked kernel.  CHUNKED, RECURRENT
 *            and SINGLE force one kernel; SINGLE takes only calls without
 *            cu_seqlens of at most 16 tokens.
 *   inverse  how the chunked kernels form the unit lower-triangular 16x16
 *            inverse (I + A)^-1: fp32 forward substitution (default), or the
 *            fp16 Neumann-series product the chunk-size page describes under
 *            "Efficient 16x16 Matrix Inversion" (pipelined chunked kernel
 *            only).
 *   sigmoid  how the gate evaluates the logistic function: 1/(1 + 2^-x') with
 *            the hardware exp2 and reciprocal (default), or 1/2 + tanh(x/2)/2
 *            with a rational tanh, the tanh form the lower_bound page names
 *            (whole-chain calls of the chunked and single-chunk kernels,
 *            forward substitution only).
 *   reserved must be 0.
 *
 * With KDA_KERNEL_AUTO a non-default inverse or sigmoid restricts the choice
 * to the kernels that implement it; a forced kernel that does not implement
 * the requested combination, or cannot take the call, gives KDA_ERR_OPTION.
 */
typedef enum kda_kernel {
    KDA_KERNEL_AUTO = 0,
    KDA_KERNEL_CHUNKED = 1,
    KDA_KERNEL_RECURRENT = 2,
    KDA_KERNEL_SINGLE = 3
} kda_kernel;

typedef enum kda_inverse {
    KDA_INVERSE_SUBSTITUTION = 0,
    KDA_INVERSE_NEUMANN = 1
} kda_inverse;

typedef enum kda_sigmoid {
    KDA_SIGMOID_EXP2 = 0,
    KDA_SIGMOID_TANH = 1
} kda_sigmoid;

typedef struct kda_options {
    int32_t kernel;   /* kda_kernel */
    int32_t inverse;  /* kda_inverse */
    int32_t sigmoid;  /* kda_sigmoid */
    int32_t reserved; /* 0 */
} kda_options;

/*
 * kda_fwd - chunked KDA forward pass.
 *
 *   q, k, g      bf16 [B,T,H,K]; v bf16 [B,T,H,V]; channel index fastest.
 *   beta         bf16 [B,T,H], logits (the sigmoid is applied inside).
 *   scale        finite scalar applied to the read-out, o = scale * S^T q.
 *   out          bf16 [B,T,H,V], written (round to nearest even).  Rows of
 *                a packed batch that lie outside every sequence are not
 *                written.
 *   A_log        fp32 [H] or NULL (NULL acts as A_log = 0).
 *   dt_bias      fp32 [H,K] or NULL (NULL acts as 0).
 *   lower_bound  in [-5, 0]; 0 turns the decay off.
 *   initial_state  [N,H,V,K] of initial_state_dtype (bf16 or fp32), stored
 *                transposed: element [n,h,v,k] is S[k][v].  NULL = zero.
 *   final_state  [N,H,V,K] of final_state_dtype, written with the state
 *                after the last token of each sequence (bf16: round to
 *                nearest even).  NULL = not written.  It may be the same
 *                buffer as initial_state (in-place update) but must not
 *                partly overlap it.
 *   cu_seqlens   NULL for batch mode (N = B sequences of length T), or a
 *                device int64 [num_seqs+1] of sequence start offsets into
 *                the packed token axis (B must be 1; N = num_seqs).  Its
 *                contents are not read on the host: they should be
 *                nondecreasing from 0 to T; the kernels clamp every segment
 *                to [0, T], so bad contents give wrong results, never an
 *                out-of-bounds access.
 *   B, T, H      sizes; T may be 0 (then only final_state is written).
 *   K, V         head dimensions; must both be 128.
 *   stream       hipStream_t to enqueue on (NULL = default stream).
 *
 * Returns KDA_OK once the work is enqueued, or an error code (nothing
 * enqueued).  num_seqs is ignored in batch mode.
 */
kda_status kda_fwd(const void *q, const void *k, const void *v, const void *g,
                   const void *beta, double scale, void *out,
                   const float *A_log, const float *dt_bias, double lower_bound,
                   const void *initial_state, kda_dtype initial_state_dtype,
                   void *final_state, kda_dtype final_state_dtype,
                   const int64_t *cu_seqlens, int64_t num_seqs,
                   int64_t B, int64_t T, int64_t H, int64_t K, int64_t V,
                   void *stream);

/*
 * kda_fwd_ex - kda_fwd with explicit options (NULL = the defaults, which is
 * exactly kda_fwd).  Same arguments, results and errors as kda_fwd, plus
 * KDA_ERR_OPTION.
 */
kda_status kda_fwd_ex(const void *q, const void *k, const void *v, const void *g,
                      const void *beta, double scale, void *out,
                      const float *A_log, const float *dt_bias, double lower_bound,
                      const void *initial_state, kda_dtype initial_state_dtype,
                      void *final_state, kda_dtype final_state_dtype,
                      const int64_t *cu_seqlens, int64_t num_seqs,
                      int64_t B, int64_t T, int64_t H, int64_t K, int64_t V,
                      const kda_options *options, void *stream);

/*
 * kda_fwd_scan - the same forward pass as kda_fwd (same arguments, same
 * results up to rounding), computed with parallelism inside each sequence:
 * for workloads with few (sequence, head) chains, where kda_fwd leaves most
 * of the GPU idle.
 *
 * Each chain is cut into segments of seg_chunks chunks (16 tokens each).
 * The recurrence above is affine in the state, so a segment maps its start
 * state S to M S + b.  The call enqueues three steps on `stream`: one pass
 * that computes b for every segment but the last (segment 0 from the real
 * initial state, the others from zero) and M for the inner segments (the
 * state update with v set to zero, from an identity start), a combine step
 * that walks each chain's segments in order (start of segment s+1 =
 * M_s * start of s + b_s), and the output pass, every segment from its true
 * start state (two steps when no chain has more than two segments).  b and
 * the combined states stay fp32; M and the running state enter the combine
 * as hi + lo bf16 pairs (about 17 significant bits each), so the results
 * match kda_fwd's to within the rounding of the bf16 matrix operands both
 * forms use.  The first pass also keeps a copy of each chain's initial
 * state in the workspace, which the output pass reads: final_state may be
 * the initial_state buffer here too.
 *
 *   seg_chunks       chunks per segment, >= 1 (KDA_ERR_SIZE otherwise).  One
 *                    segment per chain (seg_chunks >= ceil(T / 16)) is exactly
 *                    kda_fwd.
 *   workspace        DEVICE scratch owned by the caller, 16-byte aligned, at
 *                    least kda_fwd_scan_workspace_bytes() bytes, not
 *                    overlapping any tensor argument.  Its contents on entry
 *                    are ignored and on return are unspecified; it must not be
 *                    used by other work until the call's work has completed
 *                    on `stream`.
 *   workspace_bytes  its size in bytes.
 *   options          as for kda_fwd_ex (NULL = defaults); the segmented
 *                    form runs the pipelined chunked kernel, so the kernel
 *                    must be AUTO or CHUNKED and the sigmoid EXP2
 *                    (KDA_ERR_OPTION otherwise).
 * Every other argument, the ownership rules and the error codes are those of
 * kda_fwd, plus KDA_ERR_WORKSPACE and KDA_ERR_OPTION.
 */
kda_status kda_fwd_scan(const void *q, const void *k, const void *v, const void *g,
                        const void *beta, double scale, void *out,
                        const float *A_log, const float *dt_bias, double lower_bound,
                        const void *initial_state, kda_dtype initial_state_dtype,
                        void *final_state, kda_dtype final_state_dtype,
                        const int64_t *cu_seqlens, int64_t num_seqs,
                        int64_t B, int64_t T, int64_t H, int64_t K, int64_t V,
                        int64_t seg_chunks, void *workspace, int64_t workspace_bytes,
                        const kda_options *options, void *stream);

/*
 * kda_fwd_scan_static - kda_fwd_scan without a workspace argument, for
 * callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation.  The scratch the
 * segmented form needs (kda_fwd_scan_workspace_bytes() for these sizes) is
 * taken from a fixed device array of the library, KDA_SCAN_STATIC_BYTES per
 * GPU, which each GPU the library runs on holds until the process ends; the
 * call itself allocates nothing.  Calls whose scratch would exceed it return
 * KDA_ERR_WORKSPACE (nothing enqueued); the automatic segment length of the
 * Python binding keeps about 256 (chain, segment) pairs, i.e. 32 MiB.
 * Every call on one GPU shares that GPU's array: calls that may overlap on
 * one GPU (different streams, or different host threads without ordering)
 * race on it and give wrong results; calls ordered on one stream are safe.
 * Nothing in the array needs to start at zero (each call writes every slab
 * before reading it).  Same arguments (minus the workspace), results and
 * other errors as kda_fwd_scan; KDA_ERR_LAUNCH if the array's device address
 * cannot be looked up on the current device.
 */
#define KDA_SCAN_STATIC_BYTES (32ll << 20)
kda_status kda_fwd_scan_static(const void *q, const void *k, const void *v, const void *g,
                               const void *beta, double scale, void *out,
                               const float *A_log, const float *dt_bias, double lower_bound,
                               const void *initial_state, kda_dtype initial_state_dtype,
                               void *final_state, kda_dtype final_state_dtype,
                               const int64_t *cu_seqlens, int64_t num_seqs,
                               int64_t B, int64_t T, int64_t H, int64_t K, int64_t V,
                               int64_t seg_chunks, const kda_options *options, void *stream);

/*
 * Bytes of workspace kda_fwd_scan needs for these sizes: two fp32 128x128
 * slabs per (chain, segment), with ceil(ceil(T/16) / seg_chunks) segments per
 * chain (every sequence has at most T tokens).  cu_seqlens is only tested for
 * NULL (batch mode: N = B chains per head) and never read.  Returns -1 for
 * seg_chunks < 1, negative sizes or overflow.
 */
int64_t kda_fwd_scan_workspace_bytes(const int64_t *cu_seqlens, int64_t num_seqs,
                                     int64_t B, int64_t T, int64_t H, int64_t seg_chunks);

/* Static, NUL-terminated description of a status code. */
const char *kda_status_string(kda_status status);

/*
 * Name of the kernel kda_fwd_ex runs for a call with T tokens per batch row
 * (varlen != 0: cu_seqlens given) and these options (NULL = defaults, i.e.
 * kda_fwd's choice): "recurrent" (the token recurrence itself), "single"
 * (the chunked stages for one chunk, one small workgroup per chain) or
 * "mfma" (the pipelined chunked kernel); see kda_options.  Returns NULL when
 * the options are invalid for such a call (kda_fwd_ex would return
 * KDA_ERR_OPTION).  A static string; pure host logic, no device work.
 * kda_fwd_scan always runs the chunked kernel.
 */
const char *kda_fwd_kernel(int64_t T, int varlen, const kda_options *options);

/* -------------------------------------------------------------------------
 * The layer operators: what surrounds a recurrent mixer in a layer, and KDA's
 * sibling with one decay per head, which takes the same states.  The rules
 * above hold for them too: device pointers on the current device, nothing
 * allocated, every check on the host before anything is enqueued, no state
 * between calls, asynchronous on `stream`.  Activations are bf16 with
 * fp32 arithmetic and one rounding to nearest even at the end.  The arguments
 * come in a struct whose unused fields are 0.  Outputs are contiguous; inputs
 * may be slices of wider rows, given by element strides of the batch row and
 * of the token (>= 0) with the channels of a token adjacent.  Token tensors
 * need no alignment beyond their element's; out and the states 16 bytes.
 * Outputs must not overlap inputs, except where it is said.  Norms hold for
 * rows of any size, also where fp32 does not hold their squares, and for any eps
 * >= 0 (with 0, a row of zeros is NaN).  Sizes whose grid
 * would pass 2^32 threads are KDA_ERR_SIZE (the norms take any number of rows).
 * ---------------------------------------------------------------------- */

typedef enum kda_activation {
    KDA_ACT_NONE = 0,
    KDA_ACT_SILU = 1,    /* v / (1 + e^-v) */
    KDA_ACT_SIGMOID = 2  /* 1 / (1 + e^-v) */
} kda_activation;

/*
 * kda_short_conv - the short causal depthwise convolution in front of a
 * mixer, with its activation and, for query and key heads, their L2 norm
 * (kda_fwd takes q and k as the caller normalised them):
 *
 *   y[t,c]   = act(bias[c] + sum_j weight[c,j] x[t - W + 1 + j, c])
 *   out[t,c] = y[t,c], or with l2norm = L > 0
 *              y[t,c] / sqrt(l2norm_eps + sum of y[t,.]^2 over the L channels
 *              of c's group), groups of L channels from channel 0 on
 *
 * Inputs before a sequence's first token are its initial_state's.
 *
 *   x              bf16 [B,T,D], strides x_stride_b, x_stride_t.
 *   weight, bias   [D,W] and [D] or NULL, both of weight_dtype.
 *   out            bf16 [B,T,D], contiguous.  Rows outside every packed
 *                  sequence are not written.
 *   initial_state, final_state
 *                  [N,W-1,D] of their dtypes (equal if both are given), the
 *                  last W - 1 inputs before / of the sequence, oldest first;
 *                  NULL = zeros / not written.  They may be one buffer.  A
 *                  sequence shorter than W - 1 keeps the newest inputs of its
 *                  initial state; an empty one passes it through.
 *   cu_seqlens, num_seqs, B, T   as for kda_fwd.
 *   D              channels, 1 <= D <= 2^24.
 *   W              taps, 1 <= W <= 8 (KDA_ERR_SHAPE otherwise).
 *   activation     KDA_ACT_NONE or KDA_ACT_SILU.
 *   l2norm         0, 64, 128 or 256, dividing D (KDA_ERR_SHAPE otherwise).
 *   l2norm_eps     finite, >= 0 (KDA_ERR_SCALE otherwise).
 */
typedef struct kda_conv_args {
    const void *x;
    int64_t x_stride_b, x_stride_t;
    const void *weight;
    const void *bias;
    void *out;
    const void *initial_state;
    void *final_state;
    const int64_t *cu_seqlens;
    int64_t num_seqs, B, T, D, W;
    int32_t weight_dtype, initial_state_dtype, final_state_dtype; /* kda_dtype */
    int32_t activation;                                           /* kda_activation */
    int64_t l2norm;
    double l2norm_eps;
    int64_t reserved;
} kda_conv_args;
kda_status kda_short_conv(const kda_conv_args *args, void *stream);

/*
 * kda_ssm_fwd - the selective state space scan with one decay per head, over
 * prompts and single tokens.  Per (sequence, head) and token (state S is
 * P x N, fp32):
 *
 *   dt_t = softplus(dt + dt_bias[h])     (dt + dt_bias[h] without softplus)
 *   S    = exp(-exp(A_log[h]) dt_t) S + dt_t x_t b_t^T
 *   y_t  = S c_t + D[h] x_t
 *   out_t = y_t silu(z_t)                (y_t without z)
 *
 *   x, z, out      bf16 [B,T,H,P]; z may be NULL.  out is contiguous.  For
 *                  more than 8 tokens, or packed ones, the token strides of
 *                  x, b and c are at most 2^27 elements and that of z 2^26
 *                  (KDA_ERR_STRIDE otherwise).
 *   dt             bf16 [B,T,H].
 *   b, c           bf16 [B,T,G,N]; heads h with the same h / (H / G) share a
 *                  group's b and c (G divides H).
 *   A_log, D, dt_bias  fp32 [H]; D and dt_bias may be NULL (0).
 *   softplus       1 or 0.  Without it a negative dt grows the state: by up to
 *                  2^100 from any token to a later one, beyond which results
 *                  may be infinite or NaN.
 *   initial_state, final_state  [N_seq,H,P,N] of their dtypes, as for
 *                  kda_fwd (they may be one buffer).
 *   cu_seqlens, num_seqs, B, T, H   as for kda_fwd, with T < 2^31 - 128
 *                  (KDA_ERR_SIZE otherwise).
 *   P              a multiple of 32, at most 256; N is 32, 64, 128 or 256
 *                  (KDA_ERR_SHAPE otherwise).
 *   seg_tokens     tokens a segment: sequences longer than that are cut into
 *                  segments that run in parallel, joined in fp32 (the state
 *                  at a segment's start is affine in the one before, by one
 *                  factor per head).  0 lets the library choose from the
 *                  sizes; otherwise a multiple of 32 (KDA_ERR_SHAPE).  Calls
 *                  without cu_seqlens of at most 8 tokens run token by token,
 *                  whatever seg_tokens is.
 *   workspace, workspace_bytes   DEVICE scratch, 16-byte aligned, at least
 *                  kda_ssm_workspace_bytes(args) bytes (which may be 0), as
 *                  for kda_fwd_scan (KDA_ERR_WORKSPACE otherwise).
 *
 * A non-finite x, dt, b or c reaches outputs from its own token on, never
 * earlier ones: those of its column (x), head (dt) or group's heads (b; c: at
 * its token alone), to the end of its sequence, or none after the state has
 * decayed by more than 2^-300.  It never reaches another sequence.  A step that
 * grows the state by 2^128 or more counts as non-finite, and so does an A_log
 * that is NaN.
 */
typedef struct kda_ssm_args {
    const void *x;
    const void *dt;
    const void *b;
    const void *c;
    const void *z;
    void *out;
    int64_t x_stride_b, x_stride_t, dt_stride_b, dt_stride_t, b_stride_b, b_stride_t;
    int64_t c_stride_b, c_stride_t, z_stride_b, z_stride_t;
    const float *A_log;
    const float *D;
    const float *dt_bias;
    const void *initial_state;
    void *final_state;
    const int64_t *cu_seqlens;
    int64_t num_seqs, B, T, H, P, G, N;
    int32_t initial_state_dtype, final_state_dtype; /* kda_dtype */
    int32_t softplus;
    int32_t reserved;
    int64_t seg_tokens;
    void *workspace;
    int64_t workspace_bytes;
} kda_ssm_args;
kda_status kda_ssm_fwd(const kda_ssm_args *args, void *stream);

/*
 * Bytes of workspace kda_ssm_fwd needs for these sizes, cu_seqlens (tested
 * for NULL, never read) and seg_tokens; the pointers to tensors are ignored.
 * -1 where the sizes are ones kda_ssm_fwd refuses.
 */
int64_t kda_ssm_workspace_bytes(const kda_ssm_args *args);

/*
 * kda_gated_norm - the norm of a mixer's output with its gate, over groups of
 * `group` channels (D / group of them in a row):
 *
 *   out = v / sqrt(eps + mean of v^2 over the group) * weight * act(gate),
 *         v = x                                     (gate_first = 0)
 *   out = v / sqrt(eps + mean of v^2 over the group) * weight,
 *         v = x * act(gate)                         (gate_first = 1)
 *
 *   x, gate        bf16 [rows, D], element strides x_stride, gate_stride of a
 *                  row; gate may be NULL (a plain norm).
 *   weight         [D] of weight_dtype.
 *   out            bf16 [rows, D], contiguous.
 *   group          divides D, 1 <= group <= 16384 (KDA_ERR_SHAPE otherwise).
 *   activation     KDA_ACT_SIGMOID or KDA_ACT_SILU (ignored without gate).
 *   eps            finite, >= 0 (KDA_ERR_SCALE otherwise).
 * rows = 0 does nothing.
 */
typedef struct kda_gated_norm_args {
    const void *x;
    const void *gate;
    const void *weight;
    void *out;
    int64_t x_stride, gate_stride, rows, D, group;
    int32_t weight_dtype; /* kda_dtype */
    int32_t activation;   /* kda_activation */
    int32_t gate_first;   /* 0 or 1 */
    int32_t reserved;
    double eps;
} kda_gated_norm_args;
kda_status kda_gated_norm(const kda_gated_norm_args *args, void *stream);

/*
 * kda_residual_norm - the residual update between two blocks with the norm
 * after the one, its gate and scales, and the norm before the next:
 *
 *   y = x, or x / sqrt(eps + mean x^2) * post_weight
 *   r = residual_scale * residual + block_scale * gate * y
 *   residual_out = r
 *   out = r / sqrt(eps + mean r^2) * weight       (from the unrounded r)
 *
 *   x              bf16 [rows, D], element stride x_stride of a row.
 *   residual       [rows, D] of residual_dtype, contiguous; NULL = 0.
 *   residual_out   [rows, D] of residual_out_dtype, contiguous; NULL = not
 *                  written.  It may be `residual`, if the dtypes are equal.
 *   post_weight    [D] of post_weight_dtype; NULL = no norm after the block.
 *   gate           of gate_dtype; row r reads the D values at
 *                  (r / gate_period) * gate_stride: one gate for all rows
 *                  (gate_stride 0), per sequence (gate_period = its rows) or
 *                  per row (gate_period 1).  NULL = 1.
 *   weight, out    [D] of weight_dtype and bf16 [rows, D], contiguous; both
 *                  NULL: no norm before the next block.
 *   D              1 <= D <= 16384 (KDA_ERR_SHAPE otherwise).
 *   residual_scale, block_scale  0, or normal numbers as fp32; eps finite, >= 0
 *                  (KDA_ERR_SCALE).
 * rows = 0 does nothing.
 */
typedef struct kda_residual_norm_args {
    const void *x;
    const void *residual;
    void *residual_out;
    const void *post_weight;
    const void *gate;
    const void *weight;
    void *out;
    int64_t x_stride, gate_stride, gate_period, rows, D;
    int32_t residual_dtype, residual_out_dtype, post_weight_dtype, gate_dtype, weight_dtype; /* kda_dtype */
    int32_t reserved;
    double residual_scale, block_scale, eps;
} kda_residual_norm_args;
kda_status kda_residual_norm(const kda_residual_norm_args *args, void *stream);

/*
 * kda_delta_fwd - the gated delta rule with one decay per head, over prompts
 * and single tokens.  Per (sequence, head) and token (state S is K x V, fp32):
 *
 *   S   = exp(-exp(A_log[h]) softplus(g_t + dt_bias[h])) S
 *   S   = S + sigmoid(beta_t) k_t (v_t - S^T k_t)^T
 *   o_t = scale * S^T q_t
 *
 * which is kda_fwd's recurrence with a decay that all channels of a head share
 * and that has no lower bound.
 *
 *   q, k           bf16 [B,T,G,K]; heads h with the same h / (H / G) share q
 *                  and k (G divides H).  The caller normalises them, as for
 *                  kda_fwd: a k longer than 1 can make the recurrence grow.
 *   v, out         bf16 [B,T,H,V]; out is contiguous.
 *   g, beta        bf16 [B,T,H], the raw decay and the logit of the write.
 *   A_log, dt_bias fp32 [H]; dt_bias may be NULL (0).
 *   scale          0 or a normal number of fp32.
 *   initial_state, final_state  [N,H,V,K] of their dtypes, stored as kda_fwd
 *                  stores them; they may be one buffer.
 *   cu_seqlens, num_seqs, B, T, H   as for kda_fwd, with T < 2^31 - 128
 *                  (KDA_ERR_SIZE otherwise).
 *   K              64, 128 or 256; V a multiple of 16, at most 512
 *                  (KDA_ERR_SHAPE otherwise).
 *   seg_tokens     tokens a segment: sequences longer than that are cut into
 *                  segments that run in parallel, joined in fp32 (a segment
 *                  maps the state it starts with to M S + b).  0 lets the
 *                  library choose from the sizes (it keeps many packed sequences
 *                  whole, also where one is far longer than the others);
 *                  otherwise a multiple of 64 (KDA_ERR_SHAPE).
 *   workspace, workspace_bytes   DEVICE scratch, 16-byte aligned, at least
 *                  kda_delta_workspace_bytes(args) bytes (which may be 0), as
 *                  for kda_fwd_scan (KDA_ERR_WORKSPACE otherwise).
 * Calls without cu_seqlens of at most 8 tokens run token by token, whatever
 * seg_tokens is, and packed ones of at most two a sequence on average unless
 * seg_tokens cuts them.  With cu_seqlens, or more than 8 tokens, token strides
 * are at most 2^24 elements (KDA_ERR_STRIDE otherwise).
 *
 * A non-finite q reaches its own token's output alone; a non-finite k, v, g or
 * beta reaches outputs of its head (k: its group's heads) from its own token
 * on, never earlier ones, and never another sequence.  Numbers on the way that
 * round to infinity as bf16 (from 3.39e38 on) count as non-finite.  Where the
 * recurrence itself overflows, which keys no longer than 1 keep it from, up to
 * 15 tokens before that may be lost, too.
 */
typedef struct kda_delta_args {
    const void *q;
    const void *k;
    const void *v;
    const void *g;
    const void *beta;
    void *out;
    int64_t q_stride_b, q_stride_t, k_stride_b, k_stride_t, v_stride_b, v_stride_t;
    int64_t g_stride_b, g_stride_t, beta_stride_b, beta_stride_t;
    const float *A_log;
    const float *dt_bias;
    const void *initial_state;
    void *final_state;
    const int64_t *cu_seqlens;
    int64_t num_seqs, B, T, H, G, K, V;
    int32_t initial_state_dtype, final_state_dtype; /* kda_dtype */
    int64_t reserved;
    double scale;
    int64_t seg_tokens;
    void *workspace;
    int64_t workspace_bytes;
} kda_delta_args;
kda_status kda_delta_fwd(const kda_delta_args *args, void *stream);

/*
 * Bytes of workspace kda_delta_fwd needs for these sizes, cu_seqlens (tested
 * for NULL, never read) and seg_tokens; the pointers to tensors are ignored.
 * -1 where the sizes are ones kda_delta_fwd refuses.
 */
int64_t kda_delta_workspace_bytes(const kda_delta_args *args);

/* -------------------------------------------------------------------------
 * The attention layers that a hybrid model alternates with recurrent ones:
 * queries and keys normalised and rotated, the paged cache and the attention
 * of one new token over it.  The layer operators' rules hold.
 *
 * A cache is bf16 [pages, page_size, Hk, D] with the channels adjacent and any
 * strides of page, token and head (elements, >= 0).  Slot s of it is token
 * s % page_size of page s / page_size.
 * ---------------------------------------------------------------------- */

/*
 * kda_qk_norm_rotary - RMS norm of every query and key head and the rotation
 * of its first R channels by the token's position, in one pass:
 *
 *   y = x / sqrt(eps + mean of x^2 over the head) * weight   (x without weight)
 *   the pair (y_i, y_j) of frequency f is turned by angle positions[t] inv_freq[f]:
 *     out_i = rotary_scale (y_i cos - y_j sin), out_j = rotary_scale (y_j cos + y_i sin)
 *   pairs: (f, f + R / 2), or interleaved (2 f, 2 f + 1); channels from R on stay y.
 *
 *   q, k           bf16 [B,T,Hq,D] and [B,T,Hk,D]; k may be NULL (Hk is 0 then).
 *   q_out, k_out   bf16, contiguous; each may be its input, where that is
 *                  contiguous.
 *   positions      int64 [B,T], contiguous; inv_freq fp32 [R/2].  Angles are
 *                  formed and reduced in 64 bits.  Both NULL: no rotation (R
 *                  is ignored).
 *   q_weight, k_weight   [D] of their dtypes; NULL = no norm.
 *   D              a multiple of 2, at most 512; R a multiple of 2, 2 <= R <= D
 *                  (KDA_ERR_SHAPE otherwise).
 *   eps, rotary_scale    eps finite, >= 0; rotary_scale 0 or a normal number of
 *                  fp32 (KDA_ERR_SCALE otherwise).
 */
typedef struct kda_rotary_args {
    const void *q;
    const void *k;
    void *q_out;
    void *k_out;
    int64_t q_stride_b, q_stride_t, k_stride_b, k_stride_t;
    const int64_t *positions;
    const float *inv_freq;
    const void *q_weight;
    const void *k_weight;
    int64_t B, T, Hq, Hk, D, R;
    int32_t q_weight_dtype, k_weight_dtype; /* kda_dtype */
    int32_t interleaved;                    /* 0 or 1 */
    int32_t reserved;
    double eps, rotary_scale;
} kda_rotary_args;
kda_status kda_qk_norm_rotary(const kda_rotary_args *args, void *stream);

/*
 * kda_append_kv - writes the keys and values of new tokens into their slots of
 * a paged cache, the keys normalised and rotated on the way as
 * kda_qk_norm_rotary does it.
 *
 *   k, v           bf16 [B,T,Hk,D].
 *   k_cache, v_cache   see above; no two places of a cache may share memory
 *                  (KDA_ERR_STRIDE).  Only the tokens' slots are written.
 *   slots          int64 [B,T], contiguous: the token's slot.  Tokens with a
 *                  slot outside [0, pages * page_size) are left out (a padded
 *                  token has -1).  Tokens that share a slot leave one of their
 *                  values in each element of it, which one is not defined.
 *   positions, inv_freq, weight, D, R, eps, rotary_scale
 *                  as for kda_qk_norm_rotary.
 */
typedef struct kda_append_args {
    const void *k;
    const void *v;
    void *k_cache;
    void *v_cache;
    int64_t k_stride_b, k_stride_t, v_stride_b, v_stride_t;
    int64_t k_cache_stride_page, k_cache_stride_token, k_cache_stride_head;
    int64_t v_cache_stride_page, v_cache_stride_token, v_cache_stride_head;
    const int64_t *slots;
    const int64_t *positions;
    const float *inv_freq;
    const void *weight;
    int64_t B, T, Hk, D, R, pages, page_size;
    int32_t weight_dtype; /* kda_dtype */
    int32_t interleaved;  /* 0 or 1 */
    int64_t reserved;
    double eps, rotary_scale;
} kda_append_args;
kda_status kda_append_kv(const kda_append_args *args, void *stream);

/*
 * kda_paged_attention - softmax attention of one new token per sequence over
 * its keys and values in a paged cache:
 *
 *   out[n,h] = sum_t p_t v_t,  p = softmax over t of scale * q[n,h] . k_t,
 *   lse[n,h] = log of the sum over t of exp(scale * q[n,h] . k_t)
 *
 * over the tokens t of sequence n that are visible: t < lengths[n], and with
 * window > 0 t >= lengths[n] - window.  Token t lies in page block_table[n,
 * t / page_size].  Query heads h with the same h / (Hq / Hk) share a key head.
 *
 *   q              bf16 [N,Hq,D], element stride q_stride of a sequence.
 *   block_table    int32 [N, table_width], element stride table_stride of a
 *                  sequence.  A page outside [0, pages) is not read: its
 *                  tokens are not visible.
 *   lengths        int32 [N]; clamped to [0, table_width * page_size].
 *   out            bf16 [N,Hq,D], contiguous.
 *   lse            fp32 [N,Hq], contiguous; NULL = not written.
 *                  Sequences without a visible token get out = 0, lse = -inf;
 *                  where every visible one's score is -inf, or one's inf,
 *                  out is NaN and lse that infinity.  A v that is infinite
 *                  makes out so, or NaN where its p is below 2^-112.
 *                  Tokens that are not visible may hold anything.
 *   D              a multiple of 16, at most 256; Hk divides Hq
 *                  (KDA_ERR_SHAPE otherwise).
 *   scale          0 or a normal number of fp32 (KDA_ERR_SCALE otherwise).
 *                  q . k and scores are formed in fp32: one that this does
 *                  not hold is infinite.
 *   window         >= 0; 0 = every token (KDA_ERR_SIZE otherwise).
 *   table_width    * page_size at most 2^31 - 65537 (KDA_ERR_SIZE otherwise).
 *   workspace, workspace_bytes   DEVICE scratch, 16-byte aligned, at least
 *                  kda_paged_attention_workspace_bytes(args) bytes (which may
 *                  be 0), as for kda_fwd_scan (KDA_ERR_WORKSPACE otherwise).
 * N = 0 does nothing.  The contents of block_table and lengths are not read on
 * the host; table_width bounds the work that is launched, and a sequence is split
 * by it: one far wider than the lengths need costs time (64 requests of 2000
 * tokens, 8 key heads of 128, with room for 2000 / 16000 / 128000: 118 / 157 / 945 us).
 */
typedef struct kda_attention_args {
    const void *q;
    const void *k_cache;
    const void *v_cache;
    const int32_t *block_table;
    const int32_t *lengths;
    void *out;
    float *lse;
    int64_t q_stride, table_stride;
    int64_t k_cache_stride_page, k_cache_stride_token, k_cache_stride_head;
    int64_t v_cache_stride_page, v_cache_stride_token, v_cache_stride_head;
    int64_t N, Hq, Hk, D, pages, page_size, table_width, window;
    int64_t reserved;
    double scale;
    void *workspace;
    int64_t workspace_bytes;
} kda_attention_args;
kda_status kda_paged_attention(const kda_attention_args *args, void *stream);

/*
 * Bytes of workspace kda_paged_attention needs for these sizes; pointers are
 * ignored.  -1 where the sizes are ones kda_paged_attention refuses.
 */
int64_t kda_paged_attention_workspace_bytes(const kda_attention_args *args);

/* ABI version of this header (bumped on any signature change). */
#define KDA_ABI_VERSION 6
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
