/*
 * kdn.h -- C ABI of the GB300 (sm_103a) uncertainty-tracked linear-attention
 * scans.  Plain pointers and sizes only; no C++ or framework types.
 *
 * The two scans:
 *
 *  kdn_diag_scan_fwd -- the diagonal metaplastic update of
 *    "Learning to Remember, Learn, and Forget in Attention-Based Models"
 *    (Metodologia 1: forget gate alpha_t = exp(-A d_t); Metodologia 2: the
 *    closed-form update of the importance I_t and the mean mu_t), per head a
 *    d_v x d_k state, with readout o_t = mu_t q_t (the posterior mean read by
 *    the query, "Kalman Linear Attention (KLA)", Metodologia 1, "Readout"):
 *        I_t  = alpha_t I_{t-1} + (1-alpha_t) I_prior + beta_t (x) k_t^2
 *        mu_t = alpha_t (I_{t-1}/I_t) . mu_{t-1} + (1/I_t) . [(beta_t . v_t) (x) k_t]
 *        o_t[i] = sum_j mu_t[i][j] q_t[j]
 *    with beta_t on the value axis: (beta (x) k^2)[i][j] = beta_i k_j^2 and
 *    ((beta . v) (x) k)[i][j] = beta_i v_i k_j.
 *
 *  kdn_mobius_scan -- the precision recursion of "Kalman Linear Attention
 *    (KLA)", Metodologia 2 ("Parallelizzazione tramite Trasformazioni di
 *    Moebius"):
 *        lambda_t = (a_t lambda_{t-1} + b_t) / (c_t lambda_{t-1} + d_t),
 *    computed as a parallel prefix scan of 2x2 matrix products.
 *
 * Beside them: the non-metaplastic limit, the backward pass and the one-token
 * step of the diagonal scan, a gated recurrence with one gate per channel
 * (forward, backward, step), the norm and position rotation that make the
 * scans' queries and keys (forward, backward), the gated delta rule (forward,
 * backward, step), and the residual's addition with its norm (forward,
 * backward).
 *
 * Conventions shared by every entry point:
 *  - All tensors are dense, row-major (C order) and contiguous.  Device
 *    pointers must point to memory of the current CUDA device; they are
 *    read/written asynchronously on `stream` (a cudaStream_t, or NULL for the
 *    legacy default stream).  The call returns as soon as the work is queued.
 *  - The caller owns every buffer.  Entry points may take short-lived
 *    stream-ordered scratch from the device's default memory pool
 *    (cudaMallocAsync / cudaFreeAsync on `stream`); the library holds no other
 *    device memory besides one error word per device, the fixed array of
 *    kdn_mobius_scan_noalloc and the pool of the host-buffer calls.
 *  - Errors detectable on the host (null pointers, bad sizes, unsupported
 *    head dimensions, misaligned pointers) are returned before anything is
 *    launched.  Launch failures return KDN_ERR_CUDA.  Errors found by a
 *    kernel (a bounded wait that ran out) are recorded in a per-device error
 *    word and reported by kdn_get_device_error().
 *  - Values are not checked: non-finite inputs or non-positive Moebius
 *    denominators propagate as IEEE inf/nan.
 */
#ifndef KDN_H_
#define KDN_H_

#if defined(__GNUC__) || defined(__clang__)
#define KDN_API __attribute__((visibility("default")))
#else
#define KDN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDN_OK = 0,
    KDN_ERR_INVALID_ARG = -1,  /* null pointer, size out of range, misalignment */
    KDN_ERR_UNSUPPORTED = -2,  /* head dimension or dtype not supported */
    KDN_ERR_CUDA = -3,         /* a CUDA runtime call or launch failed */
    KDN_ERR_TIMEOUT = -4,      /* a bounded device-side wait ran out */
    KDN_ERR_ALLOC = -5         /* scratch allocation failed */
} kdn_status;

typedef enum {
    KDN_F32 = 0,   /* IEEE binary32 */
    KDN_BF16 = 1,  /* bfloat16 */
    KDN_E4M3 = 2   /* 8-bit float, 4 exponent and 3 mantissa bits, largest value 448 (outputs that say so) */
} kdn_dtype;

/*
 * kdn_diag_scan_fwd -- forward diagonal metaplastic scan with readout.
 *
 *   q, k       [B,H,T,dk]  in_dtype   query and key of each token-head
 *   v, beta    [B,H,T,dv]  in_dtype   value and input-dependent importance
 *   d          [B,H,T]     in_dtype   gate input; alpha_t = exp(-A[h] d_t)
 *   A          [H]         fp32       per-head gate rate
 *   I_prior                fp32       prior importance (> 0)
 *   I0, mu0    [B,H,dv,dk] fp32 or NULL   initial importance and mean; both
 *                          NULL => I_0 = I_prior, mu_0 = 0.  If exactly one is
 *                          NULL, that one takes its default.
 *   out        [B,H,T,dv]  fp32       o_t = mu_t q_t (after the token's update)
 *   final_state [2,B,H,dv,dk] fp32 or NULL   mu_T then I_T; feeding them back
 *                          as mu0/I0 of a call on the following tokens gives
 *                          the same result as one call over all tokens.
 *   B >= 1, H >= 1, T >= 0.  T = 0 writes only final_state (= the initial
 *   state); q, k, v, beta, d, A and out are then not read and may be NULL.
 *   dk, dv in {16, 32, 64, 128}, B*H*T*max(dk,dv) < 2^62.
 *   Pointers must be 16-byte aligned.  in_dtype is KDN_F32 or KDN_BF16.
 *
 * Arithmetic: fp32 state and accumulation.  The library computes the same
 * recurrence in the equivalent information form eta = I . mu with exact
 * power-of-two rescaling (the kernel source documents the rescaling); results match the
 * fp64 definition to a few fp32 ulps times the sequence's conditioning.
 */
KDN_API kdn_status kdn_diag_scan_fwd(const void* q, const void* k, const void* v,
                             const void* beta, const void* d, const float* A,
                             float I_prior, const float* I0, const float* mu0,
                             float* out, float* final_state,
                             int B, int H, int T, int dk, int dv,
                             kdn_dtype in_dtype, void* stream);

/*
 * kdn_diag_mobius_scan_fwd -- kdn_diag_scan_fwd and, in the same launch, the
 * per-head precision recursion of "Kalman Linear Attention (KLA)",
 * Metodologia 2 ("Parallelizzazione tramite Trasformazioni di Moebius"):
 * one lambda sequence per head over the same T tokens,
 *     lambda_t = (a_t lambda_{t-1} + b_t) / (c_t lambda_{t-1} + d_t).
 *
 *   q ... final_state   as for kdn_diag_scan_fwd
 *   ma, mb, mc, md  [B*H, T] fp32   the coefficients a, b, c, d of each head
 *                   (row b*H + h)
 *   lambda0         [B*H]    fp32   lambda_0 of each head
 *   lambda_out      [B*H, T] fp32   lambda_1 .. lambda_T of each head
 *   Sizes and errors as for kdn_diag_scan_fwd; the Moebius pointers must be
 *   4-byte aligned and are required when T > 0.
 *
 * When T % 4 == 0 and ma, mb, mc, md, lambda_out are 16-byte aligned, the
 * lambda sequences are walked by extra CTAs of the diagonal scan's full-pass
 * grid, placed after the scan's CTAs so that they fill the CTA slots its last
 * wave leaves free; otherwise the Moebius scan runs as its own launch after
 * the scan (same results, same stream).  lambda equals kdn_mobius_scan on the
 * same coefficients (the same tile composition and sequential evaluation).
 */
KDN_API kdn_status kdn_diag_mobius_scan_fwd(const void* q, const void* k, const void* v,
                                    const void* beta, const void* d, const float* A,
                                    float I_prior, const float* I0, const float* mu0,
                                    float* out, float* final_state,
                                    const float* ma, const float* mb, const float* mc,
                                    const float* md, const float* lambda0, float* lambda_out,
                                    int B, int H, int T, int dk, int dv,
                                    kdn_dtype in_dtype, void* stream);

/*
 * kdn_lin_scan_fwd -- the non-metaplastic limit of kdn_diag_scan_fwd: the
 * importance is held at I_prior ("Learning to Remember, Learn, and Forget in
 * Attention-Based Models", Metodologia 4, Unificazione Teorica: Mamba2 is the
 * case I_t = I_prior), so per head and token
 *     mu_t = alpha_t mu_{t-1} + (beta_t . v_t) (x) k_t / I_prior,
 *     o_t[i] = sum_j mu_t[i][j] q_t[j],        alpha_t = exp(-A d_t)
 * (decayed linear attention with a per-token scalar decay).
 *
 *   q, k, v, beta, d, A, I_prior   as for kdn_diag_scan_fwd
 *   mu0       [B,H,dv,dk] fp32 or NULL (mu_0 = 0)
 *   out       [B,H,T,dv] fp32
 *   final_mu  [B,H,dv,dk] fp32 or NULL   mu_T (feeding it back as mu0 of a
 *             call on the following tokens gives one call's result)
 *   Sizes, alignment and errors as for kdn_diag_scan_fwd.
 *
 * Same kernels as the diagonal scan with the importance update and the
 * per-element division taken out (two FP32 FMA per state element and token:
 * the write and the readout); long sequences with few heads are split into
 * token parts the same way.
 */
KDN_API kdn_status kdn_lin_scan_fwd(const void* q, const void* k, const void* v,
                            const void* beta, const void* d, const float* A,
                            float I_prior, const float* mu0, float* out,
                            float* final_mu, int B, int H, int T, int dk, int dv,
                            kdn_dtype in_dtype, void* stream);

/*
 * kdn_diag_scan_bwd -- backward pass of kdn_diag_scan_fwd (the pages' kernels
 * serve training on GPUs: "Learning to Remember, Learn, and Forget in
 * Attention-Based Models", Contributi Chiave).  For the scalar
 *     L = sum grad_out . out + sum dmu_T . mu_T + sum dI_T . I_T
 * of the forward call with the same inputs, writes dL/d(input) for every
 * input.  The forward is recomputed inside the call (nothing from a forward
 * call is needed).
 *
 *   q, k, v, beta, d, A, I_prior, I0, mu0   as for kdn_diag_scan_fwd
 *   grad_out          [B,H,T,dv] fp32   dL/d out
 *   grad_final_state  [2,B,H,dv,dk] fp32 or NULL   dL/d mu_T then dL/d I_T
 *                                    (NULL: the final state is not used)
 *   grad_q, grad_k    [B,H,T,dk] fp32   written
 *   grad_v, grad_beta [B,H,T,dv] fp32   written
 *   grad_d            [B,H,T]    fp32   written
 *   grad_A            [H] fp32 or NULL  written: summed over the batch
 *   grad_init_state   [2,B,H,dv,dk] fp32 or NULL   written: dL/d mu_0 then
 *                     dL/d I_0 (of the initial state used, given or default)
 *   I_prior gets no gradient (a fixed hyperparameter).
 *
 *   B >= 1, H >= 1, T >= 0; dk, dv in {16, 32, 64, 128};
 *   B*H*T*max(dk,dv)^2 < 2^62.  Array pointers 16-byte aligned (d and A:
 *   element-aligned; grad_d, grad_A: 4-byte aligned).  With T = 0 only
 *   grad_init_state (= grad_final_state) and grad_A (= 0) are written.
 *
 * Scratch ("workspace"): kdn_diag_scan_bwd_workspace gives its size, about
 * B*H*T*dv*dk + 8*B*H*T*dv bytes (every 8th token's state, and per-column-
 * block row sums; 16*B*H*T*dv for the latter when so few heads that the call
 * takes 16-column blocks, B*H*dk/32*2 <= the current device's SM count).
 * With workspace == NULL the call takes it from the
 * stream-ordered allocator (cudaMallocAsync, freed on the stream before
 * return; KDN_ERR_ALLOC if it cannot be had); otherwise workspace is a
 * 256-byte aligned device buffer of at least that many bytes, owned by the
 * caller and in use until the call's work on the stream completes
 * (KDN_ERR_INVALID_ARG if smaller or unaligned).  Each CTA owns all of its
 * SM's tensor memory while it runs.  Arithmetic: fp32 (the information form
 * eta = I mu, J = I - I_prior); results are deterministic (fixed summation
 * order).
 */
KDN_API kdn_status kdn_diag_scan_bwd(const void* q, const void* k, const void* v,
                             const void* beta, const void* d, const float* A,
                             float I_prior, const float* I0, const float* mu0,
                             const float* grad_out, const float* grad_final_state,
                             float* grad_q, float* grad_k, float* grad_v,
                             float* grad_beta, float* grad_d, float* grad_A,
                             float* grad_init_state,
                             int B, int H, int T, int dk, int dv,
                             kdn_dtype in_dtype, void* workspace,
                             long long workspace_bytes, void* stream);

/* Bytes of workspace kdn_diag_scan_bwd needs for these sizes on the current
 * device (no GPU work; it reads the device's SM count). */
KDN_API kdn_status kdn_diag_scan_bwd_workspace(int B, int H, int T, int dk, int dv,
                                       long long* workspace_bytes);

/*
 * kdn_mobius_scan -- lambda_t = (a_t lambda_{t-1} + b_t) / (c_t lambda_{t-1} + d_t)
 * for N independent sequences.
 *
 *   a, b, c, d [N,T] fp32   coefficients of step t (index t = 0..T-1)
 *   lambda0    [N]   fp32   initial value of each sequence
 *   out        [N,T] fp32   lambda_1..lambda_T (lambda0 is not repeated)
 *   N >= 0, T >= 0, N*T < 2^62; pointers 4-byte aligned (16-byte alignment
 *   with T % 4 == 0 enables the vector path).
 *
 * Sequences are cut into tiles of 2048 steps.  With T % 4 == 0 and 16-byte
 * aligned buffers, multi-tile sequences normally run on persistent CTAs that
 * each own whole sequences, with no scratch.  A few long sequences (too few
 * to fill the GPU, each long enough that walking it tile by tile costs more
 * than a look-back) and unaligned rows instead chain the tiles of a sequence
 * by a cross-block look-back that uses stream-ordered scratch
 * (cudaMallocAsync; KDN_ERR_ALLOC if it cannot be had).  kdn_mobius_scan_plan
 * tells which for given sizes.
 */
KDN_API kdn_status kdn_mobius_scan(const float* a, const float* b, const float* c,
                           const float* d, const float* lambda0, float* out,
                           long long N, long long T, void* stream);

/*
 * kdn_diag_step -- one token of kdn_diag_scan_fwd's update for B x H heads
 * whose state is kept on the device between calls (batched decoding), the
 * state read and overwritten in place.  The same equations for T = 1:
 *     alpha = exp(-A d); I' = alpha I + (1 - alpha) I_prior + beta_i k_j^2;
 *     mu' = (alpha I mu + beta_i v_i k_j) / I';  o_i = sum_j mu'_ij q_j.
 *
 *   q, k     [B,H,dk]  in_dtype     v, beta [B,H,dv] in_dtype   d [B,H] in_dtype
 *   A        [H] fp32               I_prior scalar
 *   state    [2,B,H,dv,dk] fp32, 16-byte aligned: mu then I (the layout of
 *            kdn_diag_scan_fwd's final_state and of its mu0 / I0); read and
 *            overwritten with the state after the token
 *   out      [B,H,dv] fp32
 *
 * Equal to kdn_diag_scan_fwd with T = 1, mu0 = state[0], I0 = state[1] and
 * final_state = state, up to rounding.  The step reads and writes each state
 * element once (16 bytes) and is bound by HBM bandwidth.  Asynchronous on
 * `stream`; no scratch.
 */
KDN_API kdn_status kdn_diag_step(const void* q, const void* k, const void* v, const void* beta,
                                 const void* d, const float* A, float I_prior, float* state,
                                 float* out, int B, int H, int dk, int dv, kdn_dtype in_dtype,
                                 void* stream);

/*
 * kdn_diag_scan_fwd_host -- kdn_diag_scan_fwd with every tensor (inputs,
 * A, I0, mu0, out, final_state) in host memory: same arguments, layouts and
 * results; pointers need only their element alignment.  The call returns when
 * the results are in host memory.
 *
 * With B >= 4 the call is cut into about eight groups of whole batches,
 * pipelined over three device buffers: a group's inputs (contiguous in host
 * memory) are copied in on an internal stream, in group order, while
 * earlier groups are scanned on `stream`, and each group's out and final
 * state are copied back on another internal stream.  With B < 4 the tokens
 * are cut into about eight chunks (at least 512 tokens each) instead: later
 * chunks' inputs come in on internal streams while chunk c is scanned,
 * outputs go straight into page-locked 16-byte aligned host memory from the
 * scan (or are copied back), and the state passes from chunk to chunk on
 * the device.  Page-locked host buffers (cudaHostAlloc, cudaHostRegister,
 * pinned framework tensors) let the copies overlap the scan; pageable
 * buffers give the same results with serialised copies.  Device memory for
 * three groups or chunks (and, for chunks, the carried states and d) comes,
 * stream-ordered on `stream`, from a memory pool of the library's own (one
 * per device) that keeps freed memory for the next host-buffer call instead
 * of releasing it to CUDA: after a call the pool holds up to the largest
 * scratch a host-buffer call has needed (about three groups' inputs,
 * outputs and states; 0.31 GB for 8 x 16 heads x 4096 tokens at d = 128).
 * KDN_ERR_ALLOC if the memory cannot be had.
 */
KDN_API kdn_status kdn_diag_scan_fwd_host(const void* q, const void* k, const void* v,
                                          const void* beta, const void* d, const float* A,
                                          float I_prior, const float* I0, const float* mu0,
                                          float* out, float* final_state, int B, int H, int T,
                                          int dk, int dv, kdn_dtype in_dtype, void* stream);

/*
 * kdn_mobius_scan_host -- kdn_mobius_scan with a, b, c, d, lambda0 and out in
 * host memory; returns when out is written.  The sequences are cut into
 * groups (about eight, at least 16 MB of coefficients each) whose copies in
 * and out overlap the scans of their neighbours, as for
 * kdn_diag_scan_fwd_host; scratch from the same library pool.
 */
KDN_API kdn_status kdn_mobius_scan_host(const float* a, const float* b, const float* c,
                                        const float* d, const float* lambda0, float* out,
                                        long long N, long long T, void* stream);

/*
 * kdn_diag_scan_plan -- how kdn_diag_scan_fwd would run these sizes on the
 * current device, without launching anything: `parts` = token ranges the
 * sequence is split into (1 = no split), `kernels` = kernels one call
 * launches, `scratch_bytes` = stream-ordered scratch one call takes.  Any
 * output pointer may be NULL.  Needs a CUDA device (occupancy query).
 */
KDN_API kdn_status kdn_diag_scan_plan(int B, int H, int T, int dk, int dv, kdn_dtype in_dtype,
                                      int* parts, int* kernels, long long* scratch_bytes);

/*
 * kdn_mobius_scan_plan -- kernels one kdn_mobius_scan call launches and the
 * scratch bytes it takes (plus one cudaMemsetAsync of part of the scratch
 * when scratch_bytes > 0), for 16-byte aligned buffers on the current device
 * (the choice between the look-back and the sequence-per-CTA kernel depends
 * on the device's resident CTA count).
 */
KDN_API kdn_status kdn_mobius_scan_plan(long long N, long long T, int* kernels,
                                        long long* scratch_bytes);

/*
 * kdn_mobius_scan_noalloc -- kdn_mobius_scan for callers that must not
 * allocate device memory during a call (for instance a process whose
 * framework reserved the GPU's memory up front, or a latency-critical loop
 * where allocator calls are not allowed).  The pages have no counterpart:
 * this is an interface variant, not part of the method.
 *
 * Same arguments, layouts and results as kdn_mobius_scan.  The look-back
 * scratch lives in a fixed 1 MiB array inside the library's device image,
 * which every GPU that loads the library holds until the process exits; no
 * cudaMalloc/cudaMallocAsync/cudaFree is called.  Limit: a call that needs
 * look-back scratch may use at most 43690 tiles, N * ceil(T / 2048) <= 43690;
 * larger calls return KDN_ERR_INVALID_ARG without launching.  A call needs
 * look-back scratch when T > 2048 and the sequence-walk kernel does not take
 * it.  That kernel needs T % 4 == 0 and a, b, c, d, out 16-byte aligned (an
 * offset view of a larger tensor may not be); on such rows it is chosen when
 * the sequences fill the GPU, when a cost model prefers it, or when the
 * look-back would need more tiles than the array holds.  So only calls with
 * T % 4 != 0 or unaligned rows can meet the limit.  The cost model counts no
 * allocation for this entry point, so it may pick the look-back where
 * kdn_mobius_scan would walk (kdn_mobius_scan_plan reports the allocating
 * entry point's choice).
 * The first call on a device fetches the array's device address
 * (cudaGetSymbolAddress); make that first call before any stream capture.
 * All calls share the one array: calls whose executions overlap on the GPU
 * (for example on two streams) race and give wrong results; serialise them.
 */
KDN_API kdn_status kdn_mobius_scan_noalloc(const float* a, const float* b, const float* c,
                                           const float* d, const float* lambda0, float* out,
                                           long long N, long long T, void* stream);

/*
 * kdn_gated_scan_fwd -- gated linear recurrence with one gate per channel:
 *     alpha_t[c] = exp(-A[h][c] d_t[c]),
 *     h_t[c] = alpha_t[c] h_{t-1}[c] + w_t[c] x_t[c],
 * with w_t = 1 (leak = 0) or w_t = 1 - alpha_t (leak = 1: the state is a
 * running mean of x).  It is the affine recursion of "Kalman Linear Attention
 * (KLA)", Metodologia 2 (the information mean, an affine map per token after
 * the lambda path), with the gate of the diagonal scan (alpha = exp(-A d)) on
 * a vector state.
 *
 *   x, d      [B,H,T,C] in_dtype  input and gate input.  Consecutive tokens
 *             are x_ld and d_ld elements apart (>= C; C when dense), rows
 *             (b,h) T * ld: with H = 1 a tensor may be a column slice of a
 *             wider [B,T,ld] projection.
 *   A         [H,C] fp32          gate rate of each channel, at most 2^127 (A
 *             log2(e) has to be a float)
 *   h0        [B,H,C] fp32 or NULL (h_0 = 0)
 *   out       [B,H,T,C] out_dtype, dense: h_t
 *   final_state [B,H,C] fp32 or NULL: h_T (feeding it back as h0 of a call on
 *             the following tokens gives one call's result)
 *
 * Packed sequences: with offsets (nseq + 1 int32 values in device memory,
 * non-decreasing, within [0, T]) and B = 1, sequence n is tokens offsets[n]
 * to offsets[n+1] - 1 of every head; h0 and final_state are then
 * [nseq,H,C].  An empty sequence's final state is its initial one.  Tokens in
 * no sequence are neither read nor written.  offsets = NULL (nseq = 0): B
 * sequences of T tokens.  Offsets out of range are clamped to [0, T]; where
 * they decrease, which tokens belong to which sequence is unspecified.
 *
 *   B >= 1, H >= 1, 0 <= T <= 2^31 - 1 - 2^16, 1 <= C <= 2^28; x, d and out
 *   element-aligned (16-byte aligned rows, C and the lds multiples of 16
 *   bytes, take the widest path).  B*H*T*max(x_ld, d_ld) < 2^62.  T = 0 writes only final_state.
 *   out and final_state overlap no input.
 *
 * The state and every sum are fp32 whatever the types; out is rounded once.
 * A d >= 0 is expected (alpha <= 1).  An infinite state stays infinite; a
 * token whose own decay underflows fp32 (A d > 87) may make NaN of it.
 * Results are deterministic.  Long sequences of few channels take
 * stream-ordered scratch (KDN_ERR_ALLOC).
 */
KDN_API kdn_status kdn_gated_scan_fwd(const void* x, long long x_ld, const void* d, long long d_ld,
                                      const float* A, const float* h0, const int* offsets, int nseq,
                                      int leak, void* out, float* final_state, int B, int H, int T,
                                      int C, kdn_dtype in_dtype, kdn_dtype out_dtype, void* stream);

/*
 * kdn_gated_scan_bwd -- backward pass of kdn_gated_scan_fwd: for
 *     L = sum grad_out . out + sum grad_final_state . h_T
 * writes dL/d(x, d, A, h0), given the forward's out.
 *
 *   x         as for the forward; read only when leak = 1 (may be NULL else)
 *   d, A, h0, offsets, nseq, leak   as for the forward
 *   out       [B,H,T,C] out_dtype, dense: the forward's output (the states)
 *   grad_out  [B,H,T,C] out_dtype, dense
 *   grad_final_state [B,H,C] ([nseq,H,C]) fp32 or NULL
 *   grad_x, grad_d  [B,H,T,C] in_dtype, dense, written (tokens in no sequence
 *             are not)
 *   grad_A    [H,C] fp32 or NULL, written: summed over batch and tokens
 *   grad_h0   [B,H,C] ([nseq,H,C]) fp32 or NULL, written
 *   workspace as for kdn_diag_scan_bwd: at least kdn_gated_scan_bwd_workspace
 *             bytes, 256-byte aligned, or NULL (stream-ordered scratch).
 *
 * The outputs overlap no input.  The states enter dL/dd as given: with a bf16
 * out they carry its rounding, |A u_t| times up to 2^-8 |h_{t-1}| of dL/dd.
 * Sums in fp32, in a fixed order (deterministic).  T = 0 writes grad_h0 (=
 * grad_final_state) and grad_A (= 0).
 */
KDN_API kdn_status kdn_gated_scan_bwd(const void* x, long long x_ld, const void* d, long long d_ld,
                                      const float* A, const float* h0, const int* offsets, int nseq,
                                      int leak, const void* out, const void* grad_out,
                                      const float* grad_final_state, void* grad_x, void* grad_d,
                                      float* grad_A, float* grad_h0, int B, int H, int T, int C,
                                      kdn_dtype in_dtype, kdn_dtype out_dtype, void* workspace,
                                      long long workspace_bytes, void* stream);

/* Bytes of workspace kdn_gated_scan_bwd needs for these sizes on the current
 * device (no GPU work; it reads the device's SM count). */
KDN_API kdn_status kdn_gated_scan_bwd_workspace(int B, int H, int T, int C, int nseq,
                                                long long* workspace_bytes);

/*
 * kdn_gated_step -- one token of kdn_gated_scan_fwd for B x H rows whose
 * state is kept on the device (batched decoding).
 *
 *   x, d      [B,H,C] in_dtype, dense      A [H,C] fp32
 *   state     [B,H,C] fp32: h before the token
 *   new_state [B,H,C] fp32: h after it; may be state itself (in place), but
 *             may not overlap it otherwise
 *   out       [B,H,C] out_dtype
 *
 * Equal to kdn_gated_scan_fwd with T = 1, h0 = state, up to rounding.  No
 * scratch.
 */
KDN_API kdn_status kdn_gated_step(const void* x, const void* d, const float* A, int leak,
                                  const float* state, float* new_state, void* out, int B, int H,
                                  int C, kdn_dtype in_dtype, kdn_dtype out_dtype, void* stream);

typedef enum {
    KDN_NORM_NONE = 0,
    KDN_NORM_RMS = 1,   /* x / sqrt(mean(x^2) + eps) */
    KDN_NORM_L2 = 2     /* x / sqrt(sum(x^2) + eps) */
} kdn_norm;

/*
 * kdn_qk_norm_rope_fwd -- the queries and keys that the scans take, from the
 * rows of a projection: every head's dk elements are normalised, scaled by a
 * weight and rotated by the token's position, and written in the scans'
 * [B,H,T,dk] layout.
 *
 *   q, k      token (b,t) is row b*T + t of q_ld (k_ld) elements, head h its
 *             elements h*dk .. h*dk + dk - 1, in_dtype: a dense [B,T,H,dk]
 *             (ld = H*dk) or a column slice of a fused projection.  Hq or Hk
 *             may be 0 (that tensor, its weight, its output and its gradients
 *             are then not touched and may be NULL).
 *   wq, wk    [dk] fp32 or NULL (1)
 *   norm, eps the norm above; eps >= 0, unused with KDN_NORM_NONE
 *   rot       number of leading elements that rotate (even, 0 <= rot <= dk);
 *             the rest are only normalised.  Pair p (p < rot/2) is elements
 *             (p, p + rot/2), or (2p, 2p + 1) when interleaved != 0, and
 *             (y1, y2) becomes (y1 cos - y2 sin, y1 sin + y2 cos) with
 *             theta = pos * inv_freq[p].
 *   pos       [axes,B,T] int32 or NULL (every axis is t).  1 <= axes <= 4:
 *             one position per axis (for instance time, height, width).
 *   axis      [rot/2] int32 or NULL (all 0): the axis whose position pair p
 *             takes (values are clamped to [0, axes-1])
 *   inv_freq  [rot/2] fp32, finite
 *   q_out     [B,Hq,T,dk], k_out [B,Hk,T,dk]  out_dtype, dense
 *
 *   B >= 1, T >= 0, Hq, Hk >= 0 and not both 0, H*dk <= 2^30, dk in {16, 32,
 *   64, 128}.
 *   Tensors 16-byte aligned, lds multiples of 16 bytes.  Outputs overlap no
 *   input.
 *
 * The sum of squares is fp32 (|x| < 1e18; without eps, rows of 1e-18 and less
 * are lost in it).  Angles are taken in 64-bit fixed-point turns: for
 * |inv_freq| <= 2^40 an angle is within |pos| 2^-60 (2^-29 at the farthest
 * position), and cos and sin within 6 half steps of their values there, also
 * where they are small.
 */
KDN_API kdn_status kdn_qk_norm_rope_fwd(const void* q, long long q_ld, const void* k, long long k_ld,
                                        const float* wq, const float* wk, kdn_norm norm, float eps,
                                        const int* pos, int axes, const float* inv_freq,
                                        const int* axis, int rot, int interleaved, void* q_out,
                                        void* k_out, int B, int T, int Hq, int Hk, int dk,
                                        kdn_dtype in_dtype, kdn_dtype out_dtype, void* stream);

/*
 * kdn_qk_norm_rope_bwd -- backward pass of kdn_qk_norm_rope_fwd for
 *     L = sum grad_q_out . q_out + sum grad_k_out . k_out.
 *
 *   q ... interleaved   as for the forward (the forward's inputs)
 *   grad_q_out, grad_k_out  [B,H,T,dk] out_dtype, dense (the layout and type
 *             of kdn_diag_scan_bwd's grad_q and grad_k with KDN_F32)
 *   grad_q, grad_k  in_dtype, written in the projection's layout, rows of
 *             gq_ld (gk_ld) elements
 *   grad_wq, grad_wk  [dk] fp32 or NULL, written: summed over tokens and
 *             heads (of the weight used, given or 1)
 *   workspace as for kdn_diag_scan_bwd, at least
 *             kdn_qk_norm_rope_bwd_workspace bytes (needed only when grad_wq
 *             or grad_wk is written)
 *
 * The outputs overlap no input.  Deterministic.  T = 0 writes only grad_wq,
 * grad_wk (= 0).
 */
KDN_API kdn_status kdn_qk_norm_rope_bwd(const void* q, long long q_ld, const void* k, long long k_ld,
                                        const float* wq, const float* wk, kdn_norm norm, float eps,
                                        const int* pos, int axes, const float* inv_freq,
                                        const int* axis, int rot, int interleaved,
                                        const void* grad_q_out, const void* grad_k_out, void* grad_q,
                                        long long gq_ld, void* grad_k, long long gk_ld,
                                        float* grad_wq, float* grad_wk, int B, int T, int Hq, int Hk,
                                        int dk, kdn_dtype in_dtype, kdn_dtype out_dtype,
                                        void* workspace, long long workspace_bytes, void* stream);

/* Bytes of workspace kdn_qk_norm_rope_bwd needs for these sizes on the
 * current device (no GPU work; it reads the device's SM count). */
KDN_API kdn_status kdn_qk_norm_rope_bwd_workspace(int B, int T, int Hq, int Hk, int dk,
                                                  long long* workspace_bytes);

/*
 * kdn_delta_scan_fwd -- the gated delta rule: decayed linear attention that
 * writes what the state does not yet answer for a key.  Per head a d_v x d_k
 * state S, and per token
 *     r_t = v_t - alpha_t S_{t-1} k_t,           alpha_t = exp(-A[h] d_t),
 *     S_t = alpha_t S_{t-1} + beta_t r_t k_t^T,  o_t = S_t q_t,
 * with one beta per token and head.  The gate, the layouts and the readout are
 * kdn_lin_scan_fwd's, whose update writes beta_t v_t instead.
 *
 *   q, k      [B,H,T,dk] in_dtype     v [B,H,T,dv] in_dtype
 *   beta, d   [B,H,T]    in_dtype     A [H] fp32
 *   S0        [B,H,dv,dk] fp32 or NULL (S_0 = 0)
 *   out       [B,H,T,dv] out_dtype
 *   final_state [B,H,dv,dk] fp32 or NULL: S_T (feeding it back as S0 of a call
 *             on the following tokens gives one call's result)
 *
 * Packed sequences: offsets, nseq, S0 and final_state [nseq,H,dv,dk] as for
 * kdn_gated_scan_fwd (B = 1; sequence n is tokens offsets[n] to offsets[n+1] -
 * 1 of every head; an empty sequence's final state is its initial one; tokens
 * in no sequence are neither read nor written).
 *
 *   workspace at least kdn_delta_scan_fwd_workspace bytes, 256-byte aligned, or
 *             NULL (stream-ordered scratch), as for kdn_diag_scan_bwd.  Calls
 *             that overlap on the GPU need workspaces of their own.
 *
 *   B >= 1, H >= 1, 0 <= T <= 2^31 - 1 - 2^16; dk, dv in {16, 32, 64, 128};
 *   B*H*T*max(dk,dv) < 2^62.  A call has at most 2^31 - 1 chunks of 64 tokens,
 *   B*H*ceil(T/64) (packed: H*(ceil(T/64) + nseq + 1)), in the backward and on the
 *   tensor cores, and at most that many blocks of 32 state rows (64 for dk of 32
 *   and less).  Tensors 16-byte aligned (d, beta: element-aligned; A, offsets: 4).
 *   T = 0 writes only final_state.  Outputs overlap no input.
 *
 * The state and every sum are fp32; out is rounded once.  alpha_t <= 1 and
 * beta_t |k_t|^2 <= 2 are expected (the state grows otherwise).  Values that
 * are not finite spoil the outputs of their token and of those behind it (in v:
 * of their channel alone), and the final state; none before.  Deterministic.
 *
 * bf16 inputs with dk*dv of 64*64 or more (64*32 with few heads), and sequences
 * (T / nseq, of packed ones) of 64 tokens or more for heads of 128 (28 with more
 * than 64 heads in all), 48 to 112 for narrower ones, are taken in chunks of 64
 * tokens on the tensor cores, with operands of 22 bits: errors are those of fp32
 * arithmetic, relative to the largest terms of a chunk.  What is smaller than
 * 2^-24 of those has fewer bits of its own, below 2^-38 none: what strong decays
 * leave beside the rest of the chunk, and a token's query, key or gradient of out
 * beside its chunk's largest (token by token they keep theirs); nor has a chunk
 * whose keys, queries or gradients are all below 2^-74.  Few heads of long
 * sequences (not packed ones) are cut along the tokens.
 */
KDN_API kdn_status kdn_delta_scan_fwd(const void* q, const void* k, const void* v, const void* beta,
                                      const void* d, const float* A, const float* S0,
                                      const int* offsets, int nseq, void* out, float* final_state,
                                      int B, int H, int T, int dk, int dv, kdn_dtype in_dtype,
                                      kdn_dtype out_dtype, void* workspace,
                                      long long workspace_bytes, void* stream);

/* Bytes of workspace kdn_delta_scan_fwd needs for these sizes on the current
 * device (0: none; no GPU work). */
KDN_API kdn_status kdn_delta_scan_fwd_workspace(int B, int H, int T, int dk, int dv, int nseq,
                                                kdn_dtype in_dtype, long long* workspace_bytes);

/*
 * kdn_delta_scan_bwd -- backward pass of kdn_delta_scan_fwd: for
 *     L = sum grad_out . out + sum grad_final_state . S_T
 * writes dL/d(input) for every input.  The forward is recomputed inside.
 *
 *   q ... nseq  as for the forward
 *   grad_out  [B,H,T,dv] out_dtype
 *   grad_final_state [B,H,dv,dk] ([nseq,H,dv,dk]) fp32 or NULL
 *   grad_q, grad_k [B,H,T,dk], grad_v [B,H,T,dv], grad_beta, grad_d [B,H,T]
 *             in_dtype, written (tokens in no sequence are not)
 *   grad_A    [H] fp32 or NULL, written: summed over batch and tokens
 *   grad_S0   [B,H,dv,dk] ([nseq,H,dv,dk]) fp32 or NULL, written
 *   workspace at least kdn_delta_scan_bwd_workspace bytes (about B*H*T*dv*(dk/8
 *             + 8), where the tensor cores take the call 4.3 KB a token and head:
 *             each 64th token's state and its adjoint, two rows a token, and what
 *             the chunks' tokens say of one another), or NULL
 *
 * Sizes, alignment and rules as for the forward.  T = 0 writes grad_S0 (=
 * grad_final_state) and grad_A (= 0).  Sums in fp32, in a fixed order
 * (deterministic).  A decay's gradient is the sum of the terms that have this
 * decay as a factor, so a strong decay's keeps its digits, however small.  The tensor-core form takes bf16 inputs and grad_out with
 * dk*dv of 64*64 or more (64*32 with few heads), of any length.
 */
KDN_API kdn_status kdn_delta_scan_bwd(const void* q, const void* k, const void* v, const void* beta,
                                      const void* d, const float* A, const float* S0,
                                      const int* offsets, int nseq, const void* grad_out,
                                      const float* grad_final_state, void* grad_q, void* grad_k,
                                      void* grad_v, void* grad_beta, void* grad_d, float* grad_A,
                                      float* grad_S0, int B, int H, int T, int dk, int dv,
                                      kdn_dtype in_dtype, kdn_dtype out_dtype, void* workspace,
                                      long long workspace_bytes, void* stream);

/* Bytes of workspace kdn_delta_scan_bwd needs for these sizes on the current
 * device (no GPU work). */
KDN_API kdn_status kdn_delta_scan_bwd_workspace(int B, int H, int T, int dk, int dv, int nseq,
                                                kdn_dtype in_dtype, long long* workspace_bytes);

/*
 * kdn_delta_step -- one token of kdn_delta_scan_fwd for B x H heads whose state
 * is kept on the device (batched decoding).
 *
 *   q, k      [B,H,dk], v [B,H,dv], beta, d [B,H]  in_dtype     A [H] fp32
 *   state     [B,H,dv,dk] fp32: S before the token
 *   new_state [B,H,dv,dk] fp32: S after it; may be state itself (in place),
 *             but may not overlap it otherwise
 *   out       [B,H,dv] out_dtype
 *
 * Equal to kdn_delta_scan_fwd with T = 1, S0 = state, up to rounding.  Tensors
 * 16-byte aligned (d, beta, v, out: element-aligned; A: 4).  No scratch.
 */
KDN_API kdn_status kdn_delta_step(const void* q, const void* k, const void* v, const void* beta,
                                  const void* d, const float* A, const float* state,
                                  float* new_state, void* out, int B, int H, int dk, int dv,
                                  kdn_dtype in_dtype, kdn_dtype out_dtype, void* stream);

/*
 * kdn_add_rms_norm_fwd -- the residual's addition and its norm, before a
 * mixer's projection: for each row of C channels
 *     s = x + residual (rounded to res_dtype),  y = weight . s / sqrt(mean(s^2) + eps).
 *
 *   x         rows of C elements, x_ld >= C apart, x_dtype
 *   residual  [rows,C] res_dtype, or NULL (s = x; sum is then NULL too, and
 *             res_dtype is x_dtype)
 *   weight    [C] fp32 or NULL (1)           eps >= 0
 *   sum       [rows,C] res_dtype: s; may be residual itself (in place)
 *   y         [rows,C] y_dtype.  With KDN_E4M3 it is in 8 bits, y / scale
 *             rounded to nearest (ties to even), with
 *   scale     [rows, ceil(C/128)] fp32: for each group of 128 channels its
 *             largest |y| / 448, or 1 where that quotient is 0 in fp32.  (A
 *             subnormal quotient has few bits; y / scale is at most 448 all the
 *             same.)  NULL for other types.
 *
 *   0 <= rows < 2^31, 1 <= C <= 2^28, rows * x_ld < 2^60; element-aligned
 *   (16-byte aligned tensors, C and x_ld multiples of 8, take the widest path).
 *   Outputs overlap no input otherwise.  What is not finite stays in its row.
 *   The sum of squares is fp32 (|s| < 1e18; without eps, rows of 1e-18 and less
 *   are lost in it).
 */
KDN_API kdn_status kdn_add_rms_norm_fwd(const void* x, long long x_ld, const void* residual,
                                        const float* weight, float eps, void* sum, void* y,
                                        float* scale, long long rows, int C, kdn_dtype x_dtype,
                                        kdn_dtype res_dtype, kdn_dtype y_dtype, void* stream);

/*
 * kdn_add_rms_norm_bwd -- backward pass of kdn_add_rms_norm_fwd with y in bf16
 * or fp32: for L = sum grad_y . y + sum grad_sum . s, with s the forward's sum
 * (or x without a residual); x and residual have one gradient, dL/ds.
 *
 *   sum       [rows,C] res_dtype            weight, eps as for the forward
 *   grad_y    [rows,C] y_dtype
 *   grad_sum  [rows,C] res_dtype or NULL (0)
 *   grad_residual [rows,C] res_dtype or NULL, written; may be grad_sum itself
 *   grad_x    [rows,C] x_dtype or NULL, written (the same values in x's type)
 *   grad_weight [C] fp32 or NULL, written: summed over the rows (of the weight
 *             used, given or 1)
 *   workspace at least kdn_add_rms_norm_bwd_workspace bytes, as for
 *             kdn_diag_scan_bwd (needed only when grad_weight is written)
 *
 * Outputs overlap no input otherwise.  Deterministic.  rows = 0 writes only
 * grad_weight (= 0).
 */
KDN_API kdn_status kdn_add_rms_norm_bwd(const void* sum, const float* weight, float eps,
                                        const void* grad_y, const void* grad_sum,
                                        void* grad_residual, void* grad_x, float* grad_weight,
                                        long long rows, int C, kdn_dtype x_dtype,
                                        kdn_dtype res_dtype, kdn_dtype y_dtype, void* workspace,
                                        long long workspace_bytes, void* stream);

/* Bytes of workspace kdn_add_rms_norm_bwd needs for these sizes on the current
 * device (no GPU work; it reads the device's SM count). */
KDN_API kdn_status kdn_add_rms_norm_bwd_workspace(long long rows, int C, long long* workspace_bytes);

/* Human-readable name of a status code (static string). */
KDN_API const char* kdn_status_string(kdn_status s);

/*
 * kdn_get_device_error -- synchronises `stream`, then reads and clears the
 * current device's error word.  Returns KDN_OK if no kernel recorded an
 * error since the last call, else the recorded status (e.g.
 * KDN_ERR_TIMEOUT), or KDN_ERR_CUDA if synchronisation failed.
 */
KDN_API kdn_status kdn_get_device_error(void* stream);

/*
 * kdn_set_wait_limit_ns -- upper bound, in nanoseconds of GPU time, on any
 * single device-side wait of later launches (default 2e9).  A wait that runs
 * out records KDN_ERR_TIMEOUT and the kernel carries on without blocking.
 * Values <= 0 restore the default.
 */
KDN_API void kdn_set_wait_limit_ns(long long ns);

/*
 * kdn_debug_stall_mobius_tile -- fault injection for tests.  For the next
 * kdn_mobius_scan launches, the block that takes look-back tile `tile`
 * (0-based, in scheduling order) never publishes its result, so its
 * successor's wait must run out (KDN_ERR_TIMEOUT) instead of hanging.
 * A negative value (the default) disables the injection.
 */
KDN_API void kdn_debug_stall_mobius_tile(long long tile);

/*
 * kdn_debug_stall_gated_rank -- fault injection for tests.  In later
 * kdn_gated_scan_fwd / _bwd calls that run in clusters, the CTAs of this rank
 * send nothing to the others of their cluster, whose waits must run out
 * (KDN_ERR_TIMEOUT; each CTA waits once) instead of hanging.  A negative value
 * (the default) disables the injection.
 */
KDN_API void kdn_debug_stall_gated_rank(int rank);

/*
 * kdn_debug_stall_delta_chunk -- fault injection for tests.  In later
 * kdn_delta_scan_fwd / _bwd calls on the tensor cores, chunk `chunk` of 64
 * tokens (of a sequence, and of every walk over one or over a part of it) is
 * not announced to those that wait for it, whose waits must run out
 * (KDN_ERR_TIMEOUT; a CTA waits a few times at most) instead of hanging.  The
 * call's outputs are then unspecified.  A negative value (the default)
 * disables the injection.
 */
KDN_API void kdn_debug_stall_delta_chunk(int chunk);

/* Library version string, e.g. "kdn 0.1.0 sm_103a". */
KDN_API const char* kdn_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KDN_H_ */
