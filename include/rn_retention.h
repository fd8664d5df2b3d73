/*
 * rn_retention.h — C ABI of the multi-scale retention forward pass on MI355X (gfx950).
 *
 * Retention (RetNet, "Retentive Network") maps q, k, v to
 *     O_t = alpha * sum_{s<=t} gamma^(t-s) * Re[(q_t e^{i p_t theta})(k_s e^{i p_s theta})^dagger] v_s
 * (hwhale.com RetNet notes: closed form of O_n after diagonalising A; definition of
 * Q = (XW_Q) ⊙ Θ, K = (XW_K) ⊙ conj(Θ), D_nm = gamma^(n-m) for n >= m).
 * Three algebraically equal forms are exported — parallel, chunkwise and one
 * recurrent (decode) step — plus the per-head GroupNorm with the swish gate.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout (row-major, contiguous, the argument comments of the ParallelRetention /
 * RecurrentRetention / ChunkwiseRetention listings on the hwhale.com notes):
 *     q, k        [B, H, N, d_k]
 *     v, gate,out [B, H, N, d_v]
 *     state       [B, H, d_k, d_v]   always float32
 * Rotation: coordinates (2j, 2j+1) form one complex number (sdkjxy.cn walkthrough,
 * "Retention 機制": elements taken two by two as real and imaginary parts); pair j at
 * absolute position p is multiplied by e^{+i p theta_j}; k is conjugated in the
 * score. Positions are p_t = pos0 + t with 0-based t. The angle p*theta_j is formed
 * and reduced modulo 2*pi in float64 on the device before the float32 sine/cosine.
 * alpha (qk_scale) multiplies the score; it never enters the recurrent state, so
 * states are interchangeable between the chunkwise and recurrent entry points.
 *
 * Ownership: every tensor argument is a DEVICE pointer owned by the caller; the
 * library never allocates device memory on these paths (the chunkwise entry point
 * takes a caller-owned workspace). gamma and theta (in rn_desc) are HOST arrays
 * read during the call. gn_weight / gn_bias / gamma_pair are DEVICE arrays or NULL.
 * Asynchrony: each call enqueues kernels on `stream` (a hipStream_t; NULL = the
 * null stream) and returns without synchronising; device faults surface at the
 * caller's next synchronisation.
 * Errors: arguments are validated on the host before any HIP call, so an invalid
 * call launches nothing and touches no device memory. Return codes only (no
 * printing, no abort); rn_last_error() gives a thread-local message.
 * NaN/Inf in inputs propagate; they are never masked.
 * Overlapping calls that share a workspace or a state buffer race.
 */
#ifndef RN_RETENTION_H
#define RN_RETENTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t rn_status;
#define RN_OK               0
#define RN_ERR_INVALID_ARG (-1) /* null pointer, size < 1, odd d_k, chunk < 1, bad flags, eps < 0 ... */
#define RN_ERR_UNSUPPORTED (-2) /* valid but outside what is built: d_k > 256, d_v > 512, N > 2^30, H > 128 ... */
#define RN_ERR_HIP         (-3) /* HIP runtime / launch error; text via rn_last_error() */
#define RN_ERR_WORKSPACE   (-4) /* workspace NULL or smaller than rn_chunkwise_workspace_bytes() */
#define RN_ERR_EXCHANGE    (-5) /* reported by rn_chunkwise_check: a wait between the workgroups of
                                   the sequential chunkwise kernel hit its time limit (1 s); the
                                   call's out and state_out hold NaN where they were written */
#define RN_ERR_NONFINITE   (-6) /* reported by rn_chunkwise_check: a matrix-core chunkwise
                                   schedule produced a non-finite output or final state: a
                                   non-finite input, or a value beyond its half-precision operand
                                   range (see rn_retention_chunkwise) */

typedef int32_t rn_dtype;
#define RN_F32  0   /* IEEE float32 */
#define RN_BF16 1   /* bfloat16 (upper half of a float32) */
#define RN_E4M3 2   /* 8-bit float, 4 exponent and 3 mantissa bits, largest 448, no infinities (rn_rmsnorm_forward's out) */
#define RN_INT8 3   /* 8-bit integer (rn_rmsnorm_forward's out) */

/* flags */
#define RN_NORM_D_ROW (1u << 0) /* parallel only: D_nm / sqrt(sum_{i<=n} D_ni)  (hwhale notes, 2nd rescaling) */
#define RN_NORM_R_ROW (1u << 1) /* parallel only: R_nm / max(|sum_{i<=n} R_ni|, 1) (hwhale notes, 3rd rescaling) */
#define RN_EPI_GN     (1u << 2) /* per-(token, head) GroupNorm over d_v (hwhale notes, multi-head paragraph) */
#define RN_EPI_GATE   (1u << 3) /* out = GN(.) * swish(gate); requires RN_EPI_GN (m0nads notes, swish gate) */
#define RN_FORCE_GENERIC (1u << 8) /* take the kernels that read their operands through
                                      pointers with 64-bit offsets (no per-head size bound):
                                      plain float32 arithmetic for the forward forms; for the
                                      backward, float32 staging with half-operand MFMA
                                      products when the inputs are bf16. For testing and for
                                      shapes past the other kernels' bounds. */
#define RN_CHUNK_PARALLEL (1u << 9) /* chunkwise: the two-kernel chunk-parallel pair (state
                                       snapshots per 256 tokens, then all chunks' outputs in
                                       parallel) instead of the single sequential kernel; same
                                       result, another workspace size. Without any schedule flag
                                       it runs only for gamma_pair at d_k 256, d_v 512 (where the
                                       sequential kernel does not apply because gamma^32 < 2^-6,
                                       the segmented schedule runs) */
#define RN_CHUNK_SEGMENTED (1u << 10) /* chunkwise, bf16 with d_k 256, d_v 512 and one decay per
                                       head: the segmented schedule (segment-local states per
                                       2048 tokens, a scan over segments, then all chunks'
                                       outputs in parallel); same result, another workspace size,
                                       no limit on gamma. Elsewhere the flag is ignored. At most
                                       one of RN_CHUNK_PARALLEL and RN_CHUNK_SEGMENTED may be set. */
#define RN_TEST_FORCE_TIMEOUT (1u << 12) /* testing only: every cross-workgroup wait of the
                                       sequential chunkwise kernel gives up at once, as if its time
                                       limit had passed, so that the error path (NaN outputs,
                                       RN_ERR_EXCHANGE from rn_chunkwise_check) can be exercised
                                       while every kernel still ends normally; other paths ignore it */

typedef struct rn_desc {
    int32_t B;             /* batch, >= 1 */
    int32_t H;             /* heads, 1..128 */
    int32_t N;             /* tokens; must be 1 for rn_retention_recurrent_step */
    int32_t d_k;           /* query/key head dim: even, 2..256 */
    int32_t d_v;           /* value head dim: 1..512 */
    rn_dtype in_dtype;     /* dtype of q, k, v, gate */
    rn_dtype out_dtype;    /* dtype of out; accumulation is always float32 */
    uint32_t flags;        /* RN_* flags above */
    int64_t pos0;          /* absolute position of token 0 (the step's position for decode), >= 0 */
    float qk_scale;        /* alpha; finite */
    float gn_eps;          /* GroupNorm epsilon, >= 0 (used with RN_EPI_GN) */
    const float* gamma;    /* HOST [H]: per-head decay, 0 < gamma <= 1 (hwhale notes: one gamma per head) */
    const float* theta;    /* HOST [d_k/2]: one angle per coordinate pair, finite */
    const float* gn_weight;/* DEVICE [H*d_v] GroupNorm scale, or NULL (= 1) */
    const float* gn_bias;  /* DEVICE [H*d_v] GroupNorm shift, or NULL (= 0) */
    const float* gamma_pair;
    /* DEVICE [H * d_k/2] float32, 4-byte aligned, or NULL. When set, each head keeps
     * one decay per coordinate pair instead of one number: gamma_pair[h*d_k/2 + j]
     * decays pair j (state rows 2j and 2j+1) of head h, and `gamma` is not read (it may
     * be NULL). This is the form the pages state before simplifying the decay to a
     * scalar (hwhale notes: A diagonalised as Λ(γe^{iθ})Λ^{-1}; m0nads notes,
     * "Retention": γ and θ as two vectors), under which the score becomes
     *     s_ts = alpha * Re sum_j gamma_j^(t-s) zq_{t,j} conj(zk_{s,j}).
     * Values must lie in (0, 1]; they are read by the kernels, so the host cannot check
     * them (other values give unspecified numbers, never an access outside the
     * buffers). Accepted by the parallel form (not with RN_NORM_D_ROW, whose rescaling
     * is defined by the scalar decay), the chunkwise forms and the decode steps; the
     * chunkwise backward returns RN_ERR_UNSUPPORTED. */
} rn_desc;

/*
 * Bytes of device workspace rn_retention_parallel needs for `desc` (0 for an invalid
 * descriptor or when the call needs none). The MFMA path stores the rotated k and the
 * blocked, transposed v in half precision there: 2*B*H*ceil(N/64)*64*(d_k + d_v) bytes,
 * linear in N (q is rotated where it is read).
 */
size_t rn_parallel_workspace_bytes(const rn_desc* desc);

/*
 * Parallel form: O = ((alpha * Qh Kh^T) ⊙ D) V with the optional row rescalings,
 * then the optional GroupNorm / gate epilogue.
 * (hwhale notes: parallel-form equation, the ParallelRetention listing and the list
 * of three rescalings; rescalings are applied in the listed order as per-row
 * scalars: c_t = 1/sqrt(sum_{m<=t} gamma^m) for RN_NORM_D_ROW, then division by
 * max(|signed row sum of R|, 1) for RN_NORM_R_ROW.)
 * q, k: [B,H,N,d_k]; v: [B,H,N,d_v]; gate: [B,H,N,d_v] (required iff RN_EPI_GATE,
 * else ignored); out: [B,H,N,d_v] in out_dtype. No state: the parallel form starts
 * from S = 0. workspace: device buffer of at least rn_parallel_workspace_bytes(desc)
 * bytes, 256-byte aligned (may be NULL when that size is 0); contents ignored.
 * Precision and range. bf16 inputs with d_k = 256, d_v = 512 and N * 2048 < 2^31
 * (N below 1,048,576) take matrix-core products on IEEE-half operands with float32
 * accumulation: alpha*Qh, Kh, v and the decayed scores alpha*gamma^(t-s) Qh_t.Kh_s
 * must stay below 65504 in magnitude (no decay factor is folded into the operands
 * here); other inputs run float32 kernels.
 */
rn_status rn_retention_parallel(const rn_desc* desc, const void* q, const void* k,
                                const void* v, const void* gate, void* out,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace rn_retention_chunkwise needs for `desc` (independent of
 * N). Returns 0 for an invalid descriptor.
 */
size_t rn_chunkwise_workspace_bytes(const rn_desc* desc, int32_t chunk);

/*
 * Chunkwise recurrent form (hwhale notes: chunkwise equation with
 * xi_j = gamma^(j+1), and the ChunkwiseRetention listing; m0nads notes,
 * "Chunkwise representation"). For chunk i of length L (the last may be shorter):
 *   O_[i]   = alpha * ((Qh Kh^T ⊙ D) V + (Qh S_i) ⊙ xi),  xi_j = gamma^(j+1)
 *   S_{i+1} = gamma^L S_i + sum_j gamma^(L-1-j) Kh_j^T V_j
 * then the optional GroupNorm / gate epilogue per token. The result does not
 * depend on `chunk` beyond rounding (every chunk length gives the same O and
 * S_final); the kernels carry the state at a granularity of their own.
 * state_in:  [B,H,d_k,d_v] float32 initial state S_0, or NULL for zeros.
 * state_out: [B,H,d_k,d_v] float32 final state, or NULL to discard; may equal
 *            state_in (updated in place).
 * workspace: device buffer of at least rn_chunkwise_workspace_bytes(desc, chunk)
 *            bytes, 256-byte aligned; contents on entry are ignored.
 * RN_NORM_D_ROW / RN_NORM_R_ROW are rejected (parallel form only).
 * Precision and range. float32 inputs run float32 kernels. bf16 inputs with d_k = 256 and
 * d_v in {256, 512} (the sequential kernel, the default) or d_v = 512 (the segmented and
 * chunk-parallel schedules) take matrix-core products whose operands are rounded to IEEE
 * half with float32 accumulation: the rotated q and k, v, the decayed scores and the copy
 * of the state used by the cross term must stay below 65504 in magnitude. In the
 * sequential kernel the rotated rows also carry decay factors up to gamma^-32 (at most 64,
 * since that kernel takes gamma^32 >= 2^-6), so |alpha q|, |k| < 1000 and |state| < 2^15
 * keep every operand in range; RetNet-scaled data sits many orders of magnitude below.
 * Outside that range the result is not finite; rn_chunkwise_check then reports
 * RN_ERR_NONFINITE (all three matrix-core schedules keep the status word).
 */
rn_status rn_retention_chunkwise(const rn_desc* desc, int32_t chunk, const void* q,
                                 const void* k, const void* v, const void* gate,
                                 const float* state_in, float* state_out, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * rn_retention_chunkwise without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the workspace is a 32 MiB buffer the library keeps in device memory, one per
 * GPU, from the first call on that GPU until the process ends. The call allocates nothing.
 * Arguments, routing and results are those of rn_retention_chunkwise (chunkwise equation
 * of the hwhale notes, as above); a call whose rn_chunkwise_workspace_bytes exceeds 32 MiB
 * is rejected with RN_ERR_UNSUPPORTED before any launch (the default sequential kernel
 * with d_v = 512 needs at most 17 MiB, for any number of heads).
 * Every call on one GPU shares its buffer: calls that overlap on one GPU (on different
 * streams, or from several threads without ordering) race and their results are
 * undefined; calls ordered on one stream are safe. The buffer keeps the last call's
 * contents; the kernels clear what must start at zero themselves.
 */
rn_status rn_retention_chunkwise_noalloc(const rn_desc* desc, int32_t chunk, const void* q,
                                         const void* k, const void* v, const void* gate,
                                         const float* state_in, float* state_out, void* out,
                                         void* stream);

/*
 * Chunkwise form over a padded batch of sequences that start at positions of their own
 * and hold numbers of tokens of their own: the prompt (prefill) half of serving, whose
 * state_out the decode steps below continue from. (eepw translation, "inference cost"
 * section with Fig. 6: decoding runs on the recurrent representation, so its cost per
 * token does not grow with the length already processed; hwhale notes, chunkwise and
 * recurrent equations: the state after a prefix is all the recurrence needs.)
 * Sequence b takes rows [0, lengths[b]) of its [N, .] slices of q, k, v, gate and
 * out; token t of it sits at absolute position pos[b] + t. Everything else is as in
 * rn_retention_chunkwise, with N replaced by lengths[b] per sequence:
 *   out rows t >= lengths[b] are not written;
 *   state_out[b] is the state after lengths[b] tokens (state_in[b], or zeros, when
 *   lengths[b] == 0).
 * pos:     DEVICE int64 [B], 8-byte aligned, or NULL for desc->pos0 everywhere. The
 *          values are not checked (they move no memory access); angles are formed
 *          and reduced in float64 as for pos0, so |p| <= 2^40 keeps them accurate.
 * lengths: DEVICE int32 [B], 4-byte aligned, or NULL for N everywhere. Each value is
 *          clamped to [0, N] on the device, so no value can reach outside the padded
 *          buffers.
 * The same workspace size as rn_retention_chunkwise applies
 * (rn_chunkwise_workspace_bytes).
 */
rn_status rn_retention_chunkwise_varlen(const rn_desc* desc, int32_t chunk,
                                        const int64_t* pos, const int32_t* lengths,
                                        const void* q, const void* k, const void* v,
                                        const void* gate, const float* state_in,
                                        float* state_out, void* out, void* workspace,
                                        size_t workspace_bytes, void* stream);

/*
 * One recurrent (decode) step at absolute position desc->pos0 (desc->N must be 1):
 *   S <- gamma S + Kh^T v   (in place),   o = alpha Qh S,   optional GN / gate.
 * (hwhale notes: recurrent equations and the RecurrentRetention listing, which
 * includes the current token and sums over d_k.)
 * q, k: [B,H,1,d_k]; v, gate, out: [B,H,1,d_v]; state: [B,H,d_k,d_v] float32 in/out.
 */
rn_status rn_retention_recurrent_step(const rn_desc* desc, const void* q, const void* k,
                                      const void* v, const void* gate, float* state,
                                      void* out, void* stream);

/*
 * One recurrent (decode) step with a position per sequence: the token of sequence b
 * sits at pos[b] (batched decode of sequences of different lengths, e.g. continuing
 * from rn_retention_chunkwise_varlen with pos[b] = its pos[b] + lengths[b]).
 * Otherwise identical to rn_retention_recurrent_step; desc->pos0 is not used.
 * (eepw translation, "inference cost" section: batched decode on the recurrent
 * representation; hwhale notes, recurrent equations.)
 * pos: DEVICE int64 [B], 8-byte aligned, required; the values are not checked (they
 *      move no memory access); |p| <= 2^40 keeps the float64-reduced angles accurate.
 *      Keeping the positions on the device lets a decode loop advance them without
 *      host work.
 */
rn_status rn_retention_recurrent_step_at(const rn_desc* desc, const int64_t* pos,
                                         const void* q, const void* k, const void* v,
                                         const void* gate, float* state, void* out,
                                         void* stream);

/*
 * Bytes of device workspace rn_retention_chunkwise_backward needs for `desc`: the state
 * at every 256-token chunk start and the gradient reaching it (float32, d_k x d_v each,
 * per head), and the gradient of the pre-GroupNorm output (float32 [B,H,N,d_v]).
 * Returns 0 for an invalid descriptor.
 */
size_t rn_chunkwise_backward_workspace_bytes(const rn_desc* desc, int32_t chunk);

/*
 * Gradients of the chunkwise call (same descriptor, inputs and chunk as the forward call)
 * given the gradient of a loss with respect to its output and, optionally, its final
 * state: the chunkwise recurrence differentiated, the GroupNorm and gate included
 * (hwhale notes: chunkwise and recurrent equations, ChunkwiseRetention listing; GroupNorm
 * per head and swish gate of the multi-scale layer). Recomputes the forward pass
 * internally; nothing from the forward call is needed.
 * dout:       [B,H,N,d_v] in out_dtype; dstate_out: [B,H,d_k,d_v] float32 or NULL (zero).
 * dq, dk:     [B,H,N,d_k], dv: [B,H,N,d_v], in in_dtype (written).
 * dgate:      [B,H,N,d_v] in in_dtype, required iff RN_EPI_GATE (written).
 * dstate_in:  [B,H,d_k,d_v] float32 or NULL (not computed); gradient for state_in.
 * dgn_weight, dgn_bias: DEVICE float32 [H*d_v] or NULL, written when RN_EPI_GN (sums over
 *             the batch and the rows); ignored otherwise.
 * workspace:  at least rn_chunkwise_backward_workspace_bytes(desc, chunk), 256-byte aligned.
 * Arithmetic: float32 inputs take float32 products throughout.
 * bf16 inputs take matrix-core products (16x16x32 f16 MFMA, float32 accumulation): with
 * d_k and d_v multiples of 8, v, dv, dout, gate and dgate 16-byte aligned and q and k
 * 4-byte aligned, every operand is
 * rounded to IEEE half (so, as for the forward, operands must stay below 65504 in
 * magnitude); other bf16 shapes stage float32 operands and take the same products. Every
 * shape and dtype the forward accepts is accepted.
 */
rn_status rn_retention_chunkwise_backward(const rn_desc* desc, int32_t chunk, const void* q,
                                          const void* k, const void* v, const void* gate,
                                          const float* state_in, const void* dout,
                                          const float* dstate_out, void* dq, void* dk, void* dv,
                                          void* dgate, float* dstate_in, float* dgn_weight,
                                          float* dgn_bias, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * Gated multi-scale retention layer (m0nads notes and hwhale notes, "Gated Multi-Scale
 * Retention"; sdkjxy walkthrough, the MSR block):
 *     Q = X W_Q,  K = X W_K,  V = X W_V,  G = X W_G
 *     Y_h = GroupNorm_h(Retention_h(Q_h, K_h, V_h))      (chunkwise form, this desc)
 *     out = (swish(G) ⊙ Concat_h Y_h) W_O
 * where head h owns columns [h d_k, (h+1) d_k) of Q and K and [h d_v, (h+1) d_v) of V
 * and G. The pages state W_G and W_O as d x d; here they are d_model x (H d_v) and
 * (H d_v) x d_model, which is d x d when H d_v = d_model.
 * Arguments (DEVICE, row-major, caller-owned):
 *     x    [B, N, d_model] bf16            w_q, w_k [d_model, H*d_k] bf16
 *     w_v, w_g [d_model, H*d_v] bf16       w_o  [H*d_v, d_model] bf16
 *     out  [B, N, d_model] in desc->out_dtype (bf16 or float32)
 *     state_in / state_out [B, H, d_k, d_v] float32 or NULL, as for rn_retention_chunkwise.
 * desc: B, H, N, d_k, d_v, decays (gamma or gamma_pair), theta, pos0, qk_scale, GroupNorm
 * parameters and flags as for rn_retention_chunkwise; in_dtype must be RN_BF16 (else
 * RN_ERR_UNSUPPORTED); RN_EPI_GN applies the per-head GroupNorm, RN_EPI_GATE the gate
 * (w_g is then required; without the flag w_g is not read). d_v must be a multiple of 8.
 * The four projections and W_O run as rocBLAS GEMMs with bf16 operands and float32
 * accumulation; Q, K, V, G and the heads' outputs are held in bf16 in the workspace
 * (rn_msr_layer_workspace_bytes, linear in B*N), then the retention kernels run as in
 * rn_retention_chunkwise. The first call on a host thread and device creates a rocBLAS
 * handle, which keeps its own device memory for the life of the process.
 * Errors: as for rn_retention_chunkwise; a rocBLAS failure returns RN_ERR_HIP.
 */
size_t rn_msr_layer_workspace_bytes(const rn_desc* desc, int32_t d_model, int32_t chunk);
rn_status rn_msr_layer_forward(const rn_desc* desc, int32_t d_model, int32_t chunk,
                               const void* x, const void* w_q, const void* w_k,
                               const void* w_v, const void* w_g, const void* w_o,
                               const float* state_in, float* state_out, void* out,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Standalone per-head GroupNorm (+ swish gate):
 *   y = (x - mean) / sqrt(var + eps) * w + b over the d_v channels of each (b,h,t),
 *   out = y * g * sigmoid(g) if gate != NULL, else y.
 * (hwhale notes, multi-head paragraph: GroupNorm per head; m0nads notes, "Gated
 * Multi-Scale Retention": swish gate.) x, gate, out: [B,H,N,d_v]; x and gate in
 * in_dtype, out in out_dtype; w, b: DEVICE [H*d_v] or NULL. out may equal x when
 * both dtypes match.
 */
rn_status rn_groupnorm_gate(int32_t B, int32_t H, int32_t N, int32_t d_v,
                            rn_dtype in_dtype, rn_dtype out_dtype, const void* x,
                            const void* gate, const float* w, const float* b, float eps,
                            void* out, void* stream);

/*
 * Status of a completed rn_retention_chunkwise / rn_retention_chunkwise_varlen call (same
 * desc and chunk), read from its workspace: RN_OK; RN_ERR_EXCHANGE if a wait between the
 * workgroups of the sequential kernel hit its time limit (its outputs are then NaN);
 * RN_ERR_NONFINITE if the call's matrix-core schedule (sequential, segmented or
 * chunk-parallel) produced a non-finite output or final state. The float32 kernels
 * record nothing and give RN_OK.
 * workspace: the call's device workspace, in which case `stream` (the call's stream) is
 * synchronised and the status word copied to the host; or a host copy of at least its
 * first 256 bytes, read directly. Must be called before the workspace is reused.
 * (Host calls that cannot block until the GPU finishes should keep using the outputs'
 * own checks instead.)
 */
rn_status rn_chunkwise_check(const rn_desc* desc, int32_t chunk, const void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * ---- operators around retention -----------------------------------------------------------
 * Layer norm, rotary positions and linear attention with a decay per head and token. Same
 * conventions as above, except that tensors are described by strides (in elements; the last
 * axis is always contiguous), so that the rows of a projection's output need no copy.
 * Strides are >= 0 and at most 2^40; a stride of 0 repeats an input along that axis (outputs
 * must not overlap themselves). An output overlaps other operands only where that is allowed below;
 * the calls refuse what two tensors of one type and the same strides show of it, and of the rest the
 * caller has to take care.
 */

/*
 * Layer norm of rows of d values, with the residual sum before it (the norm in front of a
 * retention layer, whose input is the residual stream):
 *     h = x + residual        (h = x where residual is NULL)
 *     out = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias,   biased variance.
 * Statistics and the normalised values are formed in float32 from the float32 sum h; sum_out
 * receives h rounded to in_dtype (the next residual stream).
 */
typedef struct rn_norm_desc {
    int64_t rows;          /* 1 .. 2^40 */
    int32_t d;             /* 1 .. 16384 */
    rn_dtype in_dtype;     /* x, residual, sum_out; backward: x, dsum, dx */
    rn_dtype out_dtype;    /* out; backward: dout */
    float eps;             /* finite, >= 0 */
    int64_t x_stride;      /* elements between rows: x */
    int64_t res_stride;    /* residual; backward: dsum */
    int64_t sum_stride;    /* sum_out; backward: dx */
    int64_t out_stride;    /* out; backward: dout */
} rn_norm_desc;

/*
 * weight, bias: DEVICE float32 [d] or NULL (1 and 0). residual and sum_out: NULL, or rows of
 * in_dtype (sum_out needs no residual; it then receives a copy of x). sum_out may equal x or
 * residual with the same stride, out may equal x or residual where in_dtype == out_dtype and the
 * strides agree (out and sum_out must differ); outputs overlap nothing else.
 */
rn_status rn_layernorm_forward(const rn_norm_desc* desc, const void* x, const void* residual,
                               const float* weight, const float* bias, void* sum_out, void* out,
                               void* stream);

/* Bytes of device workspace rn_layernorm_backward needs (0 for an invalid descriptor). */
size_t rn_layernorm_backward_workspace_bytes(const rn_norm_desc* desc);

/*
 * Gradients of out = LN(x) with x the rows the forward call normalised (its sum_out where it
 * had a residual); statistics are recomputed, nothing else from the forward call is needed:
 *     g = dout * weight,  xh = (x - mean) / sqrt(var + eps)
 *     dx = (g - mean(g) - xh mean(g xh)) / sqrt(var + eps) + dsum
 *     dweight = sum over rows of dout xh,   dbias = sum over rows of dout.
 * dsum: the gradient reaching the residual sum by its other path, or NULL (0); dx is then the
 * gradient of both x and residual. dx: in_dtype, may equal x, dout or dsum where types and
 * strides agree, and overlaps nothing else. dweight, dbias: DEVICE float32 [d] or NULL, written (not
 * added to); their sums run in a fixed order (the same bits on every call). workspace: 256-byte aligned, at
 * least rn_layernorm_backward_workspace_bytes(desc); unused (may be NULL) when both dweight
 * and dbias are NULL.
 */
rn_status rn_layernorm_backward(const rn_norm_desc* desc, const void* dout, const void* x,
                                const float* weight, const void* dsum, void* dx, float* dweight,
                                float* dbias, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Root-mean-square norm of rows of d values, with the residual sum before it:
 *     h = x + residual        (h = x where residual is NULL)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 * formed in float32; out receives y in float32 or bf16, or in 8 bits with float32 scales, one for each
 * row or for each `group` columns of it (the last group may be shorter):
 *     scale = max(max|y| / most, 2^-126),    out = y / scale rounded to nearest even,
 * most = 448 (RN_E4M3) or 127 (RN_INT8); out * scale stands for y. Where a NaN or infinity is among the
 * values of a scale, the scale is NaN (and out is NaN in RN_E4M3, 0 in RN_INT8). sum_out receives h
 * rounded to in_dtype. The sum of squares is float32: where it passes float32's range (from values of
 * 1.8e19 / sqrt(d) on: 1.4e17 at d = 16384), y is zero, and gradients hold zeros or NaN; beside an eps near 0,
 * values below 1e-18 lose digits of it.
 */
typedef struct rn_rms_desc {
    int64_t rows;          /* 1 .. 2^40 */
    int32_t d;             /* 1 .. 16384 */
    rn_dtype in_dtype;     /* RN_F32, RN_BF16: x, residual, sum_out; backward: x, dsum, dx */
    rn_dtype out_dtype;    /* out: any; backward: dout, RN_F32 or RN_BF16 */
    int32_t group;         /* columns a scale: 32, 64 or 128; 0 = the whole row, and where out is not of 8 bits */
    float eps;             /* finite, >= 0 */
    int64_t x_stride;      /* elements between rows: x */
    int64_t res_stride;    /* residual; backward: dsum */
    int64_t sum_stride;    /* sum_out; backward: dx */
    int64_t out_stride;    /* out; backward: dout */
    int64_t scale_stride;  /* scale */
} rn_rms_desc;

/*
 * weight: DEVICE float32 [d] or NULL (1). residual, sum_out: NULL, or rows of in_dtype. scale: DEVICE
 * float32, rows of 1 or ceil(d / group) values; required where out is of 8 bits, else not read. sum_out
 * may equal x or residual with the same stride, out may equal x or residual where in_dtype == out_dtype
 * and the strides agree (out and sum_out must differ); outputs overlap nothing else.
 */
rn_status rn_rmsnorm_forward(const rn_rms_desc* desc, const void* x, const void* residual,
                             const float* weight, void* sum_out, void* out, float* scale,
                             void* stream);

/* Bytes of device workspace rn_rmsnorm_backward needs (0 for an invalid descriptor). */
size_t rn_rmsnorm_backward_workspace_bytes(const rn_rms_desc* desc);

/*
 * Gradients of y with x the rows the forward call normalised (its sum_out where it had a residual):
 *     g = dout * weight,  xh = x / sqrt(mean(x^2) + eps)
 *     dx = (g - xh mean(g xh)) / sqrt(mean(x^2) + eps) + dsum,    dweight = sum over rows of dout xh.
 * dsum, dx, dweight, workspace: as for rn_layernorm_backward (workspace unused where dweight is NULL).
 */
rn_status rn_rmsnorm_backward(const rn_rms_desc* desc, const void* dout, const void* x,
                              const float* weight, const void* dsum, void* dx, float* dweight,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rotary positions: coordinate pairs of the first `rot` of d coordinates of every head are
 * turned by the angle p * theta_j of their token's position p and scaled by `magnitude`:
 *     (a, b) -> magnitude * (a cos - b sin, a sin + b cos),
 * where pair j is coordinates (2j, 2j+1), or (j, j + rot/2) with RN_ROTARY_HALF. The other
 * coordinates are copied. RN_ROTARY_INVERSE turns by -p theta_j: the transpose, hence also
 * the gradient's way back (with the same magnitude). Angles are formed and reduced in float64.
 * Retention called with theta = 0 on tensors turned here equals retention with its own
 * rotation (interleaved pairs, rot = d_k, magnitude 1).
 */
#define RN_ROTARY_HALF      (1u << 0)
#define RN_ROTARY_INVERSE   (1u << 1)
#define RN_ROTARY_POS_TOKEN (1u << 2) /* pos is [B, N] (row-major): a position per token */

typedef struct rn_rotary_desc {
    int32_t B, N;          /* >= 1; B * N <= 2^31 - 1 */
    int32_t H_q, H_k;      /* heads of q (>= 1) and k (>= 0; 0 = no k); at most 65535 in all */
    int32_t d;             /* 2 .. 512 */
    int32_t rot;           /* even, 2 .. min(d, 256) */
    rn_dtype dtype;        /* of all four tensors */
    uint32_t flags;        /* RN_ROTARY_* */
    int64_t pos0;          /* position of token 0 where pos is NULL, in [0, 2^40] */
    float magnitude;       /* finite */
    const double* theta;   /* HOST [rot/2]: finite */
    int64_t q_stride[3];   /* elements between batch rows, heads, tokens */
    int64_t k_stride[3];
    int64_t q_out_stride[3];
    int64_t k_out_stride[3];
} rn_rotary_desc;

/*
 * q [B, H_q, N, d], k [B, H_k, N, d] (any strides) -> q_out, k_out. An output may be its own
 * input (same pointer and strides; the coordinates past `rot` are then not touched), and overlaps
 * nothing else.
 * pos: DEVICE int64, 8-byte aligned: NULL (token t of every row sits at pos0 + t), [B] (at
 * pos[b] + t), or [B, N] with RN_ROTARY_POS_TOKEN. Values are not checked (they move no
 * memory access); |p| <= 2^40 keeps the angles accurate.
 */
rn_status rn_rotary(const rn_rotary_desc* desc, const int64_t* pos, const void* q, const void* k,
                    void* q_out, void* k_out, void* stream);

/*
 * The rot/2 angles theta_j = base^(-2j/rot), and their forms for contexts `factor` times as
 * long as the `length` positions a model was trained on. Host only.
 *   RN_ROPE_PLAIN     theta_j
 *   RN_ROPE_LINEAR    theta_j / factor
 *   RN_ROPE_BASE      base replaced by base * factor^(rot/(rot-2)): the slowest pair is
 *                     stretched by factor, the fastest keeps its angle (rot >= 4)
 *   RN_ROPE_BY_PARTS  with n_j = length theta_j / (2 pi) turns over the trained length: pairs
 *                     with n_j >= fast keep theta_j, pairs with n_j <= slow take theta_j /
 *                     factor, those between are mixed in proportion to n_j; *magnitude
 *                     becomes 0.1 ln(factor) + 1 (1 for the other kinds).
 * factor >= 1; base > 1 and finite, the replaced one too; for BY_PARTS length >= 1 and 0 <= slow < fast.
 */
#define RN_ROPE_PLAIN    0
#define RN_ROPE_LINEAR   1
#define RN_ROPE_BASE     2
#define RN_ROPE_BY_PARTS 3
rn_status rn_rotary_frequencies(int32_t rot, double base, int32_t kind, double factor,
                                double length, double slow, double fast, double* theta,
                                float* magnitude);

/*
 * Linear attention with a decay per head and token (retention whose decay the tokens set):
 *     S_t = exp(g_t) S_{t-1} + k_t^T v_t,     o_t = qk_scale q_t S_t
 * with log decays g <= 0 (DEVICE float32; -inf clears the state before the token; NaN
 * propagates). No rotation is applied (see rn_rotary). Heads: H states and outputs; q, k and v
 * may have fewer, each dividing H: head h reads q head h / (H / H_q), and so on.
 *
 * Precision: prompts with bf16 inputs and a bf16 output run matrix products where d_k and d_v are
 * multiples of 8 and rows start on 16 bytes (strides multiples of 8, pointers 16-byte aligned):
 * scores and the state's copy read by the queries enter them in two bf16 parts (2^-16 relative, so
 * that an output is the float32 result rounded once), the state itself is carried in float32 from
 * products of three bf16 parts (float32 accuracy). All other calls run float32 arithmetic throughout.
 * Outputs must not overlap the inputs (states: see below).
 * A NaN or infinity in a token's q, k, v or decay reaches only outputs of that token and later
 * ones of its sequence, and the final state.
 */
#define RN_LINEAR_ZERO_REST (1u << 0)  /* chunked: rows of `out` behind each sequence (padded), or
                                          behind the last one (packed), are set to zero */
#define RN_LINEAR_GENERIC   (1u << 8)  /* take the float32 kernels (for testing) */

typedef struct rn_linear_desc {
    int32_t S;             /* sequences, 1 .. 65534 */
    int32_t N;             /* most tokens of a sequence, 1 .. 2^30; the step form needs 1 */
    int32_t H;             /* heads of the state, decays and output: 1 .. 65535 */
    int32_t H_q, H_k, H_v; /* heads of q, k, v: divisors of H */
    int32_t d_k;           /* 1 .. 256 */
    int32_t d_v;           /* 1 .. 512 */
    rn_dtype in_dtype;     /* q, k, v */
    rn_dtype out_dtype;    /* out */
    uint32_t flags;        /* RN_LINEAR_* */
    float qk_scale;        /* finite */
    int64_t T;             /* packed batches: token rows of the tensors, 1 .. 2^31 - 1; else 0 */
    int32_t n_slots;       /* states in state_in / state_out where slots are given */
    int64_t q_stride[3];   /* elements between sequences (ignored if packed), heads, tokens */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int64_t g_stride[3];
    int64_t out_stride[3];
} rn_linear_desc;

/* Bytes of device workspace rn_linear_attention_chunked needs (0 when it needs none, or for an
 * invalid descriptor). */
size_t rn_linear_attention_workspace_bytes(const rn_linear_desc* desc);

/*
 * Prompts: every sequence's tokens at once.
 * Padded (T = 0): sequence s holds lengths[s] tokens (DEVICE int32 [S], clamped to [0, N]; NULL
 * = N) at rows s of the tensors. Packed (T > 0): cu_seqlens, DEVICE int32 [S+1], holds each
 * sequence's first token row, 0 first; rows cu_seqlens[s] .. cu_seqlens[s+1]-1 are sequence s
 * (clamped to [0, T] and to N tokens). Rows of no sequence are not written (but see
 * RN_LINEAR_ZERO_REST).
 * state_in, state_out: float32 [S, H, d_k, d_v], or [n_slots, H, d_k, d_v] with slots (DEVICE
 * int32 [S]: the state of sequence s is slot slots[s]; one outside [0, n_slots) starts from
 * zeros and keeps no state; two sequences must not share a slot). 16-byte aligned; NULL = start
 * from zeros / discard; they may be the same buffer. A sequence without tokens passes its
 * state on. workspace: 256-byte aligned, rn_linear_attention_workspace_bytes(desc) bytes.
 */
rn_status rn_linear_attention_chunked(const rn_linear_desc* desc, const int32_t* cu_seqlens,
                                      const int32_t* lengths, const int32_t* slots, const void* q,
                                      const void* k, const void* v, const float* log_decay,
                                      const float* state_in, float* state_out, void* out,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token for each of S sequences; `state` is updated in place (layout and slots as above; a
 * sequence whose slot is outside [0, n_slots) is skipped and its output row set to zero).
 */
rn_status rn_linear_attention_step(const rn_linear_desc* desc, const int32_t* slots, const void* q,
                                   const void* k, const void* v, const float* log_decay,
                                   float* state, void* out, void* stream);

/*
 * ---- the short convolution and the selective scan ------------------------------------------
 * Batches of sequences. Padded (T = 0): sequence s holds lengths[s] tokens (DEVICE int32 [S], clamped
 * to [0, N]; NULL = N) at row s of tensors [S, N, D]. Packed (T > 0): cu_seqlens, DEVICE int32 [S+1],
 * holds each sequence's first token row, 0 first, of tensors [1, T, D]; rows cu_seqlens[s] ..
 * cu_seqlens[s+1]-1 are sequence s (clamped to [0, T] and to N tokens). Rows of no sequence are not
 * read, and not written but with RN_SEQ_ZERO_REST. Strides are (sequence, token), the sequence's being
 * ignored if packed; B and C, as heads, have (sequence, group, token).
 * States are addressed as linear attention's: [S, ...], or [n_slots, ...] with slots (DEVICE int32
 * [S]; one outside [0, n_slots) starts from zeros and keeps no state; two sequences must not share a
 * slot); NULL = start from zeros / discard; state_in and state_out may be the same buffer. A sequence
 * without tokens passes its state on. Outputs overlap no other operand.
 */
#define RN_SEQ_ZERO_REST (1u << 0)     /* rows of `out` (backward: of the token gradients) of no sequence
                                          are set to zero */
#define RN_CONV_SILU     (1u << 1)     /* out = u sigmoid(u) */
#define RN_SCAN_SOFTPLUS (1u << 1)     /* the step is softplus(dt + bias) */

/*
 * Short causal convolution of every channel with its own K weights:
 *     u_t = bias + sum_{j < K} weight_j x_{t-K+1+j},    out = u, or u sigmoid(u) with RN_CONV_SILU,
 * in float32. The K - 1 inputs before a sequence's first token are its state: rows of K - 1 tokens,
 * [K - 1, D] a sequence, in dtype (exact copies of x).
 */
typedef struct rn_conv_desc {
    int32_t S;             /* sequences, 1 .. 65534 */
    int32_t N;             /* most tokens of a sequence, 1 .. 2^30, S * N <= 2^31 - 1; the step form needs 1 */
    int32_t D;             /* channels, 1 .. 65536 */
    int32_t K;             /* 1 .. 8 */
    rn_dtype dtype;        /* RN_F32, RN_BF16: x, out, states; backward: x, dout, dx, state_in */
    uint32_t flags;        /* RN_SEQ_ZERO_REST, RN_CONV_SILU */
    int64_t T;             /* packed batches: token rows of the tensors, 1 .. 2^31 - 1; else 0 */
    int32_t n_slots;
    int64_t x_stride[2];   /* elements between sequences and tokens */
    int64_t out_stride[2]; /* out; backward: dout */
    int64_t dx_stride[2];  /* backward: dx */
} rn_conv_desc;

/* weight: DEVICE float32 [D, K]; bias: DEVICE float32 [D] or NULL (0). */
rn_status rn_short_conv(const rn_conv_desc* desc, const int32_t* cu_seqlens, const int32_t* lengths,
                        const int32_t* slots, const void* x, const float* weight, const float* bias,
                        const void* state_in, void* state_out, void* out, void* stream);

/* One token for each of S sequences; `state` is updated in place (a sequence whose slot is outside
 * [0, n_slots) is skipped and its output row set to zero). state may be NULL where K is 1. */
rn_status rn_short_conv_step(const rn_conv_desc* desc, const int32_t* slots, const void* x,
                             const float* weight, const float* bias, void* state, void* out,
                             void* stream);

/* Bytes of device workspace rn_short_conv_backward needs (0 for an invalid descriptor). */
size_t rn_short_conv_backward_workspace_bytes(const rn_conv_desc* desc);

/*
 * Gradients of rn_short_conv (states per sequence, without slots), u being recomputed:
 *     du = dout (the derivative of the output's form at u),   dx_t = sum_j weight_j du_{t+K-1-j},
 *     dweight_j = sum_t du_t x_{t-K+1+j},   dbias = sum_t du_t.
 * dstate_out: float32 [S, K - 1, D] or NULL (0): the gradient reaching the final state. dx: as out.
 * dstate_in: float32 [S, K - 1, D] or NULL. dweight [D, K], dbias [D]: float32 or NULL, written; sums in a
 * fixed order. workspace: 256-byte aligned; unused where dweight and dbias are NULL.
 */
rn_status rn_short_conv_backward(const rn_conv_desc* desc, const int32_t* cu_seqlens,
                                 const int32_t* lengths, const void* dout, const void* x,
                                 const float* weight, const float* bias, const void* state_in,
                                 const float* dstate_out, void* dx, float* dweight, float* dbias,
                                 float* dstate_in, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * Selective scan: a diagonal linear recurrence whose step, input and output the tokens set, n states a
 * channel:
 *     D_t = softplus(dt_t + bias)    (dt_t + bias without RN_SCAN_SOFTPLUS)
 *     h_t = exp(D_t A) h_{t-1} + D_t x_t B_t,     y_t = C_t h_t + skip x_t,
 *     out_t = y_t, or y_t z_t sigmoid(z_t) where z is given.
 * Channels come in G groups of D / G that share B and C. All arithmetic is float32. A NaN or infinity
 * at a token reaches only outputs of that token and later ones of its sequence, and its final state.
 * Decays are joined over many tokens: where D A is positive and exp of its sum over a sequence passes
 * float32's range, results may be infinite or NaN though the formula's are not; where an infinite state (or
 * gradient of one) meets joined decays below float32's range, results are NaN where the formula's are infinite.
 */
typedef struct rn_scan_desc {
    int32_t S;             /* sequences, 1 .. 65534 */
    int32_t N;             /* most tokens of a sequence, 1 .. 2^30, S * N <= 2^31 - 1; the step form needs 1 */
    int32_t D;             /* channels, 1 .. 65536 */
    int32_t n;             /* states a channel, 1 .. 64 */
    int32_t G;             /* groups of channels: a divisor of D */
    rn_dtype dtype;        /* RN_F32, RN_BF16: x, dt, B, C, z, out and their gradients */
    uint32_t flags;        /* RN_SEQ_ZERO_REST, RN_SCAN_SOFTPLUS */
    int32_t n_slots;
    int64_t T;             /* packed batches: token rows of the tensors, 1 .. 2^31 - 1; else 0 */
    int64_t x_stride[2];   /* elements between sequences and tokens */
    int64_t dt_stride[2];
    int64_t z_stride[2];
    int64_t out_stride[2]; /* out; backward: dout */
    int64_t b_stride[3];   /* elements between sequences, groups and tokens */
    int64_t c_stride[3];
} rn_scan_desc;

/* Bytes of device workspace rn_selective_scan_chunked needs (0 when it needs none, or for an invalid
 * descriptor). */
size_t rn_selective_scan_workspace_bytes(const rn_scan_desc* desc);

/*
 * Prompts. x, dt, z (or NULL), out [.., D]; B, C [.., G, .., n]; A: DEVICE float32 [D, n]; skip, bias:
 * DEVICE float32 [D] or NULL (0). States: float32 [D, n] a sequence, 16-byte aligned where n is a multiple
 * of 4. workspace: 256-byte aligned.
 */
rn_status rn_selective_scan_chunked(const rn_scan_desc* desc, const int32_t* cu_seqlens,
                                    const int32_t* lengths, const int32_t* slots, const void* x,
                                    const void* dt, const float* A, const void* B, const void* C,
                                    const float* skip, const float* bias, const void* z,
                                    const float* state_in, float* state_out, void* out,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* One token for each of S sequences; `state` is updated in place (a sequence whose slot is outside
 * [0, n_slots) is skipped and its output row set to zero). */
rn_status rn_selective_scan_step(const rn_scan_desc* desc, const int32_t* slots, const void* x,
                                 const void* dt, const float* A, const void* B, const void* C,
                                 const float* skip, const float* bias, const void* z, float* state,
                                 void* out, void* stream);

/* Strides of the gradients, as the inputs' own. */
typedef struct rn_scan_grad_desc {
    int64_t dx_stride[2];  /* elements between sequences and tokens */
    int64_t ddt_stride[2];
    int64_t dz_stride[2];
    int64_t db_stride[3];  /* elements between sequences, groups and tokens */
    int64_t dc_stride[3];
} rn_scan_grad_desc;

/* Bytes of device workspace rn_selective_scan_backward needs (0 for an invalid descriptor). */
size_t rn_selective_scan_backward_workspace_bytes(const rn_scan_desc* desc);

/*
 * Gradients of rn_selective_scan_chunked (states per sequence, without slots) given those of its output and,
 * optionally, of its final state (dstate_out: float32 [S, D, n] or NULL); the states are recomputed. With
 * dy = dout z sigmoid(z) (dout without z), g_t = C_t dy_t + exp(D_{t+1} A) g_{t+1} and
 * p_t = exp(D_t A) h_{t-1}:
 *     dC_t = sum_d dy_t h_t,    dB_t = sum_d g_t D_t x_t    (d: the channels of a group)
 *     dx_t = D_t sum_n g_t B_t + skip dy_t,    dz_t = dout_t y_t (z sigmoid(z))'
 *     ddt_t = (x_t sum_n g_t B_t + sum_n g_t p_t A) times the derivative of the step
 *     dA = sum_t g_t p_t D_t,    dskip = sum_t dy_t x_t,    dbias = sum_t ddt_t
 * dx, ddt, dB, dC and dz (NULL without z) in dtype; dA float32 [D, n]; dskip, dbias float32 [D] or NULL
 * (not wanted); dstate_in float32 [S, D, n] or NULL. All are written; sums run in a fixed order.
 * workspace: 256-byte aligned.
 */
rn_status rn_selective_scan_backward(const rn_scan_desc* desc, const rn_scan_grad_desc* grads,
                                     const int32_t* cu_seqlens, const int32_t* lengths,
                                     const void* dout, const void* x, const void* dt, const float* A,
                                     const void* B, const void* C, const float* skip,
                                     const float* bias, const void* z, const float* state_in,
                                     const float* dstate_out, void* dx, void* ddt, float* dA, void* dB,
                                     void* dC, float* dskip, float* dbias, void* dz, float* dstate_in,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* Static name of a status code. */
const char* rn_status_str(rn_status s);
/* Message describing the last failure on the calling thread ("" if none). */
const char* rn_last_error(void);
/* Library version, e.g. "0.1.0". */
const char* rn_version(void);

#ifdef __cplusplus
}
#endif
#endif /* RN_RETENTION_H */
