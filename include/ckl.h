/*
 * ckl.h -- C ABI of the fused chunked KL distillation loss for MI355X (gfx950).
 *
 * The loss compares a student's full-vocabulary distribution with an offline
 * cache of the teacher's top-K logits per position and returns the loss with
 * its gradients, without ever holding the student's vocabulary x sequence
 * logit grid: the sequence is processed in row chunks and each chunk's logits
 * are computed, turned into gradient and discarded before the next chunk
 * ("A New Trick Slashes the Cost of Shrinking Giant AI Models", sections
 * "What did the researchers change?" and "Does this matter for longer
 * documents?"; "Making Knowledge Distillation Cheap Enough to Run at Scale"
 * (aiphreaks.com), bullet "Fused Chunked KL Loss").
 *
 * Definition (the readings where the pages are silent are stated here):
 *   z_r      = H_r . W^T                        student logits of position r, length V
 *   log p_S  = z_r - logsumexp(z_r)             full-vocabulary log-softmax
 *   p_T      = softmax(T_r)                     over the K cached teacher logits only;
 *                                               the other V - K tokens get no mass
 *                                               (elseif.net page, limitations paragraph)
 *   KL_r     = sum_k p_T,k (log p_T,k - log p_S,id_k)
 *   loss     = (1 / n) sum_r mask_r KL_r,       n = number of valid positions
 *                                               (loss = 0 and all gradients 0 if n = 0)
 *   dL/dz_r  = (mask_r / n) (softmax(z_r) - scatter(p_T,r))
 *   dH       = G W,   dW = G^T H                with G the stacked dL/dz_r
 * Temperature 1.  Teacher ids within a row must be distinct and in [0, V).
 * The logit at each cached id is the very fp32 value the logits contraction
 * accumulated (copied out before any exponential), so log p_S at the ids is
 * that of the dense definition to fp32 rounding of the log-normaliser.
 *
 * Ids outside [0, V), and repeats within a row, are outside the supported
 * inputs: no kernel reads or writes at them (they are left out of the loss
 * and the gradient, so the result is not the definition's), and a device
 * flag records them.  With the environment variable CKL_DEBUG=1, each loss
 * call waits for its own kernels and then returns CKL_EINVAL if the flag is
 * set.
 *
 * Layout and ownership (every call):
 *   - all arrays are row-major and contiguous, in device memory of the device
 *     that is current on the calling thread, and `stream` belongs to it;
 *   - H, W, dH, dW must be 16-byte aligned; ids, logits, out_loss 4-byte;
 *   - the caller owns every buffer; the library keeps no pointer after the
 *     call returns.  Work is enqueued on `stream` with no host synchronisation,
 *     so inputs and outputs must stay alive until the stream has finished;
 *   - d must be a multiple of 8; 1 <= K <= min(V, 2048);
 *   - N = 0 is an empty batch: no row is read (H, ids, logits, mask, dH and
 *     the per-position arrays may be null), and a loss call writes 0 to
 *     out_loss and zeros to dW, the result for a batch with no valid
 *     position; ckl_plan gives chunk 0 and 0 bytes, ckl_topk does nothing;
 *   - the library holds one grow-only device workspace per (device, stream),
 *     sized by ckl_plan; ckl_release_workspace frees them all.
 *
 * Environment: CKL_WORKSPACE_BYTES (workspace budget, default 6 GiB);
 * CKL_DEBUG=1 (input checks reported by the call, see above); CKL_TRACE=1
 * (roctx ranges around every loss call and every chunk, for rocprofv3
 * --marker-trace; skipped if no roctx library can be opened).
 *
 * Errors: arguments that are invalid or not supported are reported before
 * anything is enqueued, and the outputs are untouched.  A HIP failure returns
 * CKL_EHIP or CKL_ENOMEM and leaves the outputs undefined; since every call
 * overwrites dW (it does not accumulate into it), the call can be repeated.
 * No C++ exception crosses this interface.
 */
#ifndef CKL_H_
#define CKL_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CKL_OK = 0,
  CKL_EINVAL = -1,       /* null or misaligned pointer, N < 0, d, V or K < 1, K > V, chunk < 0 */
  CKL_ENOMEM = -2,       /* device workspace allocation failed */
  CKL_EBUDGET = -3,      /* no chunk size fits the workspace budget (or the given chunk does not) */
  CKL_EHIP = -4,         /* a HIP runtime call failed */
  CKL_EUNSUPPORTED = -5  /* d % 8 != 0, K > 2048, V > 2^26, a chunk above 2^20 rows, or a size
                            beyond 32-bit grid limits */
} ckl_status;

typedef enum { CKL_DTYPE_BF16 = 0, CKL_DTYPE_F32 = 1 } ckl_dtype;

/* Fused forward + backward of the loss above (bf16 hidden states and weight).
 *   H          bf16 [N, d]   student final hidden states
 *   W          bf16 [V, d]   LM-head weight
 *   topk_idx   int32 [N, K]  cached teacher ids, distinct per row, in [0, V)
 *   topk_logit fp32 [N, K]   cached teacher logits
 *   mask       uint8 [N]     1 = position counts, 0 = ignored; NULL = all count
 *   chunk      rows per chunk; 0 lets ckl_plan choose under the workspace budget
 *              (environment CKL_WORKSPACE_BYTES, default 6 GiB)
 *   out_loss   fp32 device scalar
 *   dH         bf16 [N, d]   gradient of the loss with respect to H (overwritten)
 *   dW         fp32 [V, d]   gradient with respect to W (overwritten)
 * Masked positions contribute nothing and cost no GEMM work: with a mask,
 * each chunk's valid rows are gathered to the front of workspace buffers
 * before its contractions, so masked rows get no logits.  Their dH rows are
 * written as +0.
 * The pages' interface statement is that a training code only swaps in this
 * loss, fed by the precomputed top-K cache (elseif.net page, adoption paragraph). */
int ckl_fwd_bwd(const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
                const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk,
                float* out_loss, void* dH, float* dW, hipStream_t stream);

/* Same as ckl_fwd_bwd with H, W and dH in fp32 (fp32 matrix cores). */
int ckl_fwd_bwd_f32(const float* H, const float* W, const int32_t* topk_idx, const float* topk_logit,
                    const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk,
                    float* out_loss, float* dH, float* dW, hipStream_t stream);

/* ckl_fwd_bwd / ckl_fwd_bwd_f32 selected by `dtype` (ckl_dtype), with two
 * optional per-position outputs (device, caller-owned, may be NULL):
 *   row_kl   fp32 [N]  KL_r of each position (0 for masked positions)
 *   row_lse  fp32 [N]  logsumexp of the student logits of each position (0 for
 *                      masked positions)
 * The loss is the sum of row_kl divided by the valid count. */
int ckl_fwd_bwd_ex(int dtype, const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
                   const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk,
                   float* out_loss, void* dH, float* dW, float* row_kl, float* row_lse, hipStream_t stream);

/* Largest workspace ckl_fwd_bwd_noalloc can use, in bytes (256 MiB). */
#define CKL_NOALLOC_MAX_BYTES (256ull << 20)

/* ckl_fwd_bwd_ex for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, results and errors as ckl_fwd_bwd_ex, except that the
 * workspace is a fixed array of CKL_NOALLOC_MAX_BYTES in the library's own
 * device memory, which every GPU the library runs on holds until the process
 * ends; the call itself allocates and frees nothing.
 *   - The chunk planner runs with that size as its budget: a shape whose
 *     smallest workspace (or whose given chunk) does not fit returns
 *     CKL_EBUDGET before anything is enqueued.  The tiled copy of W alone
 *     takes V x d x (2 or 4) bytes, so this fits heads up to about
 *     V x d = 60 M elements in bf16 (e.g. d = 2048, V = 32,000), not the
 *     largest vocabularies.
 *   - Every call on one GPU shares that GPU's array and leaves its contents
 *     behind; nothing in it has to start at zero (each buffer is written
 *     before it is read within a call).  Calls that overlap on one GPU (on
 *     different streams, or from several threads) race on the array and give
 *     undefined results: the caller orders them.
 *   - With the same chunk, the results are bitwise those of ckl_fwd_bwd_ex. */
int ckl_fwd_bwd_noalloc(int dtype, const void* H, const void* W, const int32_t* topk_idx,
                        const float* topk_logit, const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K,
                        int64_t chunk, float* out_loss, void* dH, float* dW, float* row_kl, float* row_lse,
                        hipStream_t stream);

/* The two-pass form of the same loss, for a training code whose backward runs
 * apart from its forward: the forward keeps one number per position and the
 * backward recomputes each chunk's logits from H and W instead of storing them
 * ("A New Trick Slashes the Cost of Shrinking Giant AI Models", section "What
 * did the researchers change?": chunks are computed and discarded, and what the
 * backward pass needs is recomputed; the same page's table lists a
 * forward-chunked loss beside the fused one).  Together the two calls do four
 * d x V contractions per position instead of the fused call's three.
 *
 * ckl_fwd: loss and per-position log-normaliser, no gradients.
 *   dtype      ckl_dtype of H and W
 *   H, W, topk_idx, topk_logit, mask, N, d, V, K, chunk   as for ckl_fwd_bwd
 *   out_loss   fp32 device scalar
 *   row_lse    fp32 [N] (required)   logsumexp of each position's student logits
 *                                    (0 for masked positions)
 *   row_kl     fp32 [N] or NULL      KL_r (0 for masked positions)
 * With the same inputs and chunk, loss, row_lse and row_kl are bitwise equal
 * to those of ckl_fwd_bwd_ex (and they do not depend on the chunk).  No exp
 * values are kept, so the workspace per row is a small fraction of the fused
 * call's and the planner's chunk is correspondingly longer. */
int ckl_fwd(int dtype, const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
            const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk, float* out_loss,
            float* row_lse, float* row_kl, hipStream_t stream);

/* ckl_bwd: dH and dW of `grad_loss` x loss, recomputing every chunk's logits.
 *   row_lse    fp32 [N] (required)   the values ckl_fwd wrote for these inputs
 *   grad_loss  fp32 device scalar multiplying both gradients, or NULL for 1
 *   dH         [N, d] in dtype (overwritten);  dW  fp32 [V, d] (overwritten)
 * The log-normaliser is read from row_lse rather than recomputed.  With
 * grad_loss NULL and the same chunk, dH and dW are bitwise equal to those of
 * ckl_fwd_bwd. */
int ckl_bwd(int dtype, const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
            const uint8_t* mask, const float* row_lse, const float* grad_loss, int64_t N, int64_t d, int64_t V,
            int64_t K, int64_t chunk, void* dH, float* dW, hipStream_t stream);

typedef enum { CKL_PASS_FUSED = 0, CKL_PASS_FWD = 1, CKL_PASS_BWD = 2 } ckl_pass;

/* Offline top-K cache writer: the step that produces topk_idx / topk_logit from
 * the teacher's logits, run once per training corpus ("A New Trick...",
 * section "What did the researchers change?": the teacher is run once and only
 * its top 100 predictions per position are saved; elseif.net page,
 * offline-cache paragraph).
 *   dtype     ckl_dtype of logits
 *   logits    [N, V] row-major, bf16 or fp32 (2- or 4-byte aligned); no NaN
 *   ids_out   int32 [N, K]   token ids of the K largest logits of each row
 *   vals_out  fp32 [N, K]    those logits (exact conversion of the inputs)
 * Each row's K pairs are ordered by value descending; equal values (-0 equals
 * +0) by id ascending, so the result is unique.  1 <= K <= min(V, 2048),
 * V < 2^31.  Enqueued on `stream`; no workspace.  Errors as for the other
 * calls; nothing is enqueued on an error. */
int ckl_topk(int dtype, const void* logits, int64_t N, int64_t V, int64_t K, int32_t* ids_out, float* vals_out,
             hipStream_t stream);

/* Token embedding: the other end of the vocabulary table whose head gradient
 * the loss computes.
 *   out[n] = scale W[ids[n]], rounded once to W's type
 *   dtype     ckl_dtype of W and out
 *   ids       int32 [N]; an id outside [0, V) is a position without a token:
 *             its row of out is zeros
 *   W         [V, d], out [N, d], 16-byte aligned
 * N < 2^26, V <= 2^26, d % 8 == 0, d <= 2^20; CKL_EUNSUPPORTED also where a
 * launch would pass 2^24 - 1 workgroups (the last three N, for rows of more than
 * 512 bytes).  No workspace. */
int ckl_embed(int dtype, const int32_t* ids, const void* W, float scale, int64_t N, int64_t d, int64_t V, void* out,
              hipStream_t stream);

/* Gradient of ckl_embed with respect to W:
 *   dW[v] (+)= scale (sum of dY[n] over the positions n with ids[n] = v)
 *   dtype       ckl_dtype of dY [N, d]
 *   accumulate  0: dW is overwritten, rows of absent tokens with zeros;
 *               1: the sums are added to dW and rows of absent tokens are left
 *               alone (tied weights: dW as a loss call wrote it)
 *   dW          fp32 [V, d], 16-byte aligned
 *   workspace   device buffer of at least ckl_embed_bwd_workspace bytes,
 *               256-byte aligned; it need not be cleared, and no two calls
 *               that may overlap may share it
 * Sums are fp32 in a fixed order, so the result depends on the inputs alone.
 * Positions without a token contribute nothing.  N = 0: dW = 0, or nothing.
 * Shapes as for ckl_embed; CKL_EUNSUPPORTED also where a launch would pass
 * 2^24 - 1 workgroups. */
int ckl_embed_bwd(int dtype, const int32_t* ids, const void* dY, float scale, int64_t N, int64_t d, int64_t V,
                  int accumulate, float* dW, void* workspace, uint64_t workspace_bytes, hipStream_t stream);
int ckl_embed_bwd_workspace(int64_t N, int64_t d, int64_t V, uint64_t* bytes_out);

/* Settings of ckl_sample: one value for all rows or, where the array is not
 * NULL, the row's value from a device array [N].  Single values outside their
 * range are CKL_EINVAL; array values are taken as stated. */
typedef struct ckl_sampling {
  double temperature; /* >= 0; 0 (in an array also below 0 or NaN): the largest logit, lowest id first */
  int64_t top_k;      /* 0 (in an array also below 0) or >= V: no limit */
  double top_p;       /* [0, 1]; 1 (in an array also above 1 or NaN): no limit */
  double min_p;       /* [0, 1]; 0 (in an array also below 0 or NaN): no limit; above 1 as 1 */
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
} ckl_sampling;

/* One token per row of logits from given random numbers.  In a row the tokens
 * are ordered as ckl_topk orders them (logit descending, equal logits by id
 * ascending).  With e_j = exp((l_j - l_max) / temperature), the kept prefix is
 * the shortest of
 *   the first top_k tokens,
 *   the shortest prefix whose mass reaches top_p x the mass of those,
 *   the tokens with e_j >= min_p,
 * and never empty.  The token is the first of the order at which the
 * cumulative mass exceeds u x the kept mass S: its probability is e / S.
 *   logits    [N, V], rows row_stride >= 0 elements apart, elements of a row
 *             adjacent, aligned to an element.  -inf and NaN are tokens that
 *             cannot be drawn; where +inf occurs, its tokens share the row
 *   u         fp32 [N] in [0, 1) (NaN and below 0 as 0, from 1 on as the
 *             largest value below 1)
 *   how       NULL: temperature 1, no limit
 *   ids_out   int32 [N]; -1 for a row without a token that can be drawn
 *   logp_out  fp32 [N] or NULL: log(e / S) of the drawn token (-inf for -1)
 * Masses and borders are computed in 64 bits, so the token is that of the
 * formulas except where a border is within about 1e-13 + V / 2^62 of the total
 * (1.4e-13 at 201,088 tokens, 1.5e-11 at 2^26); tokens whose e is below 2^-64
 * count as 0.  V <= 2^26, N < 2^22.
 *   workspace NULL, or a device buffer of at least ckl_sample_workspace bytes
 *             (0 for most shapes), 256-byte aligned, not shared by calls that
 *             may overlap: with it, long rows of a small batch are split over
 *             several workgroups.  The results are the same bits either way. */
int ckl_sample(int dtype, const void* logits, int64_t N, int64_t V, int64_t row_stride, const float* u,
               const ckl_sampling* how, int32_t* ids_out, float* logp_out, void* workspace,
               uint64_t workspace_bytes, hipStream_t stream);
int ckl_sample_workspace(int dtype, int64_t N, int64_t V, uint64_t* bytes_out);

/* Matrix product in 8-bit floating point (OCP e4m3) with an fp32 scale per
 * block of 128, for a head whose weight is held in 8 bits (a teacher's logits
 * for ckl_topk, a served student's for ckl_sample).  A value is q x its
 * block's scale.
 *   rows    [R, C] with block_rows = 1: scales [ceil(C / 128), R], one per
 *           1 x 128 block, blocks of columns outermost
 *   weight  [R, C] with block_rows = 128: scales [ceil(R / 128), ceil(C / 128)]
 * ckl_quantize_fp8: scale = amax / 448 of the block's finite values (1 for a
 * block of zeros, at least 2^-126), q = the fp32 quotient x / scale rounded to
 * nearest even; values that are not finite become NaN, and only they.
 *   dtype     ckl_dtype of x (16-byte aligned, as q_out)
 *   C         a multiple of 16, at most 2^20; the last block of 128 columns
 *             and of 128 rows may be short */
int ckl_quantize_fp8(int dtype, const void* x, int64_t R, int64_t C, int64_t block_rows, uint8_t* q_out,
                     float* scales_out, hipStream_t stream);

/* out[m][v] = sum over blocks kb of xs[kb][m] ws[v / 128][kb]
 *             (sum over k of block kb of xq[m][k] wq[v][k]),
 * block sums and the sum over blocks in fp32, rounded once to out_dtype.  The
 * two scales are multiplied first, in fp32: a product of theirs below 2^-126
 * loses bits, one past fp32's range is inf.  For
 * bf16 results the products of a group of 8 k are aligned to the group's
 * largest and what lies 14 bits and more below it may be dropped (less than
 * 7 x 2^-13 of that product a group); fp32 results keep fp32's bits.  Up to 16
 * rows with V < 16,384, and one or two with V d > 2^28, go by a kernel that keeps
 * them for bf16 results too; all other calls give a row the same bits whatever
 * the rows beside it.
 *   xq, xs    [M, d] and [ceil(d / 128), M], as ckl_quantize_fp8 writes rows
 *   wq, ws    [V, d] and [ceil(V / 128), ceil(d / 128)], as it writes a weight
 *   out       [M, V] in out_dtype (overwritten)
 * xq and wq 16-byte aligned; d a multiple of 16, at most 2^20; V and M at most
 * 2^26, and at most 2^26 tiles of 64 x 64.  No workspace, no gradient. */
int ckl_matmul_fp8(int out_dtype, const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, int64_t M,
                   int64_t V, int64_t d, void* out, hipStream_t stream);

/* Log-probabilities of given tokens, entropy and the most likely alternatives of
 * rows of logits.  Of a row z, with M its largest logit and L = log sum exp(z - M):
 *   logp[t]  = z[ids[t]] - M - L      entropy = -sum p log p, p = exp(z - M - L)
 *   top      the `top` largest logits, ordered as ckl_topk orders them, with their
 *            log-probabilities
 *   dtype      ckl_dtype of logits
 *   logits     [N, V], rows row_stride >= 0 elements apart, elements of a row
 *              adjacent, aligned to an element.  -inf has probability 0 and adds
 *              nothing to the entropy; a row of nothing else has entropy 0 and
 *              log-probabilities -inf.  NaN or +inf makes its row's logp, entropy,
 *              stats (L) and top_logp NaN
 *   ids        int32 [N, T]; an id outside [0, V) is an entry without a token: its
 *              logp is 0.  NULL with T = 0
 *   mask       uint8 [N], 0 = the row is not read: its outputs are 0 and its
 *              top_ids -1; NULL: every row counts
 *   logp       fp32 [N, T];  entropy fp32 [N]
 *   stats      fp32 [2, N]: M and L, for the gradient (M + L is the log-normaliser)
 *   top_ids    int32 [N, top], top_logp fp32 [N, top]; -1 and -inf where a row has
 *              fewer logits above -inf (NaN is never one).  NULL with top = 0
 *   workspace  NULL, or at least ckl_logprobs_workspace bytes (0 for most shapes),
 *              256-byte aligned, not shared by calls that may overlap: with it,
 *              rows of a small batch are split over several workgroups
 * T <= 2048, top <= min(V, 512), V <= 2^26, N < 2^22.  Sums are fp32, with or
 * without a workspace in an order of their own. */
int ckl_logprobs(int dtype, const void* logits, int64_t N, int64_t V, int64_t row_stride, const int32_t* ids, int64_t T,
                 const uint8_t* mask, int64_t top, float* logp, float* entropy, float* stats, int32_t* top_ids,
                 float* top_logp, void* workspace, uint64_t workspace_bytes, hipStream_t stream);
int ckl_logprobs_workspace(int64_t N, int64_t V, int64_t top, uint64_t* bytes_out);

/* Gradient of sum_t dlogp[t] logp[t] + dentropy entropy with respect to the logits:
 *   dz_j = (sum of dlogp over the entries with id j) - p_j (W + dentropy (log p_j + entropy)),
 * W the sum of dlogp over the row's entries with a token.  logits, ids, mask, stats
 * and entropy are the forward call's.
 *   dlogp     fp32 [N, T], NULL with T = 0;  dentropy fp32 [N] or NULL for zeros
 *             (entropy may then be NULL)
 *   dlogits   [N, V] in dtype, rows out_stride >= V elements apart; may be logits
 *             with the same stride.  Masked rows and rows without a logit above
 *             -inf are zeros
 * The same id may be given several times.  N, V and T as above, and N x (V in runs
 * of 8,192) below 2^24.  No workspace. */
int ckl_logprobs_bwd(int dtype, const void* logits, int64_t N, int64_t V, int64_t row_stride, const int32_t* ids,
                     int64_t T, const uint8_t* mask, const float* stats, const float* entropy, const float* dlogp,
                     const float* dentropy, void* dlogits, int64_t out_stride, hipStream_t stream);

/* The same from hidden states, for logits z = H W^T that are never held: rows go in
 * chunks, as in the loss calls.
 *   dtype      ckl_dtype of H [N, d] and W [V, d], 16-byte aligned
 *   ids, mask, logp, entropy, stats   as for ckl_logprobs (masked rows cost no
 *              contraction)
 *   chunk      rows per chunk, 0 = what ckl_head_logprobs_plan chooses
 *   workspace  at least the bytes that ckl_head_logprobs_plan gives for this call,
 *              256-byte aligned, need not be cleared, not shared by calls that may
 *              overlap
 * d % 8 == 0, d <= 2^20, V <= 2^26, N T <= 2^26, N <= 2^26. */
int ckl_head_logprobs(int dtype, const void* H, const void* W, const int32_t* ids, const uint8_t* mask, int64_t N,
                      int64_t d, int64_t V, int64_t T, int64_t chunk, float* logp, float* entropy, float* stats,
                      void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/* Its gradient, recomputing the logits: dH = G W and dW = G^T H with G = dz above in
 * dtype (rounded once for bf16), sums in fp32.
 *   logp, entropy, stats   the forward call's outputs (entropy as for ckl_logprobs_bwd)
 *   dH         [N, d] in dtype, 16-byte aligned; zeros for masked rows
 *   dW         [V, d], 16-byte aligned: fp32 (dw_dtype CKL_DTYPE_F32), overwritten, or
 *              added to with accumulate = 1 (as a loss call wrote it); or bf16 with a
 *              bf16 W, rounded once after the last chunk (accumulate = 0)
 * N = 0: dW = 0, or nothing. */
int ckl_head_logprobs_bwd(int dtype, const void* H, const void* W, const int32_t* ids, const uint8_t* mask, int64_t N,
                          int64_t d, int64_t V, int64_t T, int64_t chunk, const float* logp, const float* entropy,
                          const float* stats, const float* dlogp, const float* dentropy, void* dH, int dw_dtype,
                          int accumulate, void* dW, void* workspace, uint64_t workspace_bytes, hipStream_t stream);

/* Rows per chunk and workspace bytes of the two calls (pure host computation):
 * backward = 0 or 1, dw_dtype as for ckl_head_logprobs_bwd (ignored for the forward
 * call), chunk > 0 checks that many rows against the budget, budget_bytes 0 =
 * CKL_WORKSPACE_BYTES or 6 GiB.  Returns as ckl_plan_pass does. */
int ckl_head_logprobs_plan(int backward, int dtype, int dw_dtype, int64_t N, int64_t d, int64_t V, int64_t chunk,
                           uint64_t budget_bytes, int64_t* chunk_out, uint64_t* workspace_bytes_out);

/* Dropout whose mask is never stored.  Element i of a tensor takes 16 bits of
 * Philox4x32-10 under the key `seed`: with the counter (i / 8, offset), bits
 * 16 (j % 2) .. + 15 of word j / 2, j = i % 8.  It goes if they are below
 * border = floor(65536 p + 0.5), and is multiplied by 65536 / (65536 - border)
 * if not, so the mean is kept whatever p rounds to.  The same seed, offset and
 * shape give the same mask, in every call that takes a ckl_drop and in their
 * gradients.
 *   p           [0, 1]; below 2^-17 nothing goes, at 1 everything
 *   offset_dev  NULL, or a device int64 (8-byte aligned) added to offset when
 *               the call's kernels run: a captured step that moves it on draws
 *               another mask in every replay */
typedef struct ckl_drop {
  double p;
  uint64_t seed;
  uint64_t offset;
  const int64_t* offset_dev;
} ckl_drop;

/* out[i] = x[i] x 65536 / (65536 - border), or 0 where element i goes (also where
 * x[i] is not finite), in fp32, rounded once to dtype.  It is its own gradient:
 * dx is the call on dout with the same ckl_drop.  out may be x.
 *   x, out   [n] of ckl_dropout's dtype, aligned to an element; n < 2^37 */
int ckl_dropout(int dtype, const void* x, int64_t n, const ckl_drop* how, void* out, hipStream_t stream);

/* The residual's norms around a block:
 *   u  = w_post y / rms(y)            u = y without w_post; rms(v) = sqrt(mean(v^2) + eps) over a row
 *   r' = r + scale gate u             u's elements dropped as ckl_dropout drops them, element index n d + j
 *   x  = w_pre r' / rms(r')
 * in fp32, r' and x each rounded once: x is that of the fp32 r'.  The last
 * block's x is the H of the loss calls.
 *   dtype     ckl_dtype of y, r, w_post, w_pre, gate, r_out and x
 *   w_post    [d] or NULL;  w_pre [d], or NULL: x (then NULL) is not computed
 *   gate      [d], or [N, d] with gate_rows = 1, or NULL for 1
 *   drop      NULL: nothing is dropped
 *   r_out     [N, d], may be r (a gradient needs r as it was); x [N, d], not r_out
 *   stats     fp32 [2, N] or NULL: 1 / rms(y) and 1 / rms(r') (1 where not
 *             computed), for the gradient
 * d % 8 == 0, d <= 16384, N <= 2^31; arrays aligned to an element.  A row of
 * zeros with eps = 0 gives NaN, as the formula does. */
typedef struct ckl_norm {
  const void* w_post;
  const void* w_pre;
  const void* gate;
  int gate_rows;
  float scale;
  float eps; /* >= 0 */
  const ckl_drop* drop;
} ckl_norm;
int ckl_add_norm(int dtype, const void* y, const void* r, const ckl_norm* how, int64_t N, int64_t d, void* r_out,
                 void* x, float* stats, hipStream_t stream);

/* Its gradient.  `how` (the same arrays, numbers and drop), y, r and stats are the
 * forward call's.
 *   dx, dr_in   gradients of x and of r_out; either may be NULL for zeros (dx is
 *               NULL without w_pre), not both
 *   dy, dr      [N, d] in dtype; dr may be dr_in, dy may be dx; one array each
 *   dw_post, dw_pre  fp32 [d], each NULL exactly where the weight is
 *   dgate       fp32 [d], or [N, d] in dtype with gate_rows, NULL without a gate
 *   workspace   at least ckl_add_norm_bwd_workspace(N, d, sums) bytes, sums = how
 *               many of dw_post, dw_pre and a gate [d]'s gradient there are;
 *               256-byte aligned, need not be cleared, not shared by calls that
 *               may overlap
 * Sums over rows are fp32 in a fixed order.  N = 0: their outputs are zeros. */
int ckl_add_norm_bwd(int dtype, const void* y, const void* r, const ckl_norm* how, int64_t N, int64_t d,
                     const float* stats, const void* dx, const void* dr_in, void* dy, void* dr, float* dw_post,
                     float* dw_pre, void* dgate, void* workspace, uint64_t workspace_bytes, hipStream_t stream);
int ckl_add_norm_bwd_workspace(int64_t N, int64_t d, int sums, uint64_t* bytes_out);

/* Chunk planner of the fused call (pure host computation, needs no GPU).  The
 * sequence is cut into chunks of C rows so that the loss's own device memory
 * stays bounded independently of N ("A New Trick...", section "Does this
 * matter for longer documents?": peak memory barely grows with input length).
 *   dtype         ckl_dtype of H and W
 *   budget_bytes  0 = CKL_WORKSPACE_BYTES or 6 GiB
 *   chunk_out, workspace_bytes_out  (may be NULL) the rows per chunk a call
 *                 with chunk = 0 uses, and the exact bytes it allocates for its
 *                 workspace: the largest multiple of 256 rows that fits (or N if
 *                 N < 256), evened out over the resulting chunk count, then
 *                 lowered by 256-row steps until it fits (the workspace is not
 *                 monotonic in the chunk: the dH split count depends on it)
 * Returns CKL_EBUDGET if not even 256 rows (or N) fit, CKL_EINVAL /
 * CKL_EUNSUPPORTED for shapes the calls reject. */
int ckl_plan(int64_t N, int64_t d, int64_t V, int64_t K, int dtype, uint64_t budget_bytes, int64_t* chunk_out,
             uint64_t* workspace_bytes_out);

/* The planner for one of the calls with a caller-given chunk: pass = ckl_pass
 * (the forward-only call needs no dH split-K slabs, so it can take longer
 * chunks); chunk > 0 checks min(chunk, N) rows against the budget
 * (CKL_EBUDGET if they do not fit), chunk = 0 plans as ckl_plan does. */
int ckl_plan_pass(int pass, int64_t N, int64_t d, int64_t V, int64_t K, int dtype, int64_t chunk,
                  uint64_t budget_bytes, int64_t* chunk_out, uint64_t* workspace_bytes_out);

/* Frees every cached workspace (after synchronising the device). */
void ckl_release_workspace(void);

/* Bytes currently held in cached workspaces (all devices and streams). */
uint64_t ckl_workspace_bytes_held(void);

/* Human-readable name of a status code. */
const char* ckl_strerror(int status);

/* Test entry: the row pass alone on caller-given fp32 logits Z [R, V]
 * (row stride V): log-normaliser, teacher softmax, gather, KL and the logit
 * gradient with weight `scale` for rows whose mask is 1 (or all rows if mask
 * is NULL).  Z is first turned into what the logits GEMM leaves in the
 * workspace (per 128-id slice: max m and exp(z - m) in the gradient's element
 * type), then the production row kernels run.  Outputs (device, caller-owned):
 *   zg_out          fp32 [R, K]  the logits at the teacher ids as the row pass read them
 *                                (copied from Z through the same id tables the
 *                                logits contraction fills: Z[r, id] bit for bit)
 *   scatter_ids_out int32 [R, K] the ids the top-K values were scattered to
 *   G_out           [R, V]       gradient, bf16 if g_bf16 else fp32
 *   kl_out, lse_out fp32 [R]     per-row KL and logsumexp (both 0 for masked rows)
 * Synchronises `stream` before returning. */
int ckl_debug_rows(const float* Z, const int32_t* idx, const float* tlogit, const uint8_t* mask, int64_t R,
                   int64_t V, int64_t K, float scale, int g_bf16, float* zg_out, int32_t* scatter_ids_out,
                   void* G_out, float* kl_out, float* lse_out, hipStream_t stream);

/* Measurement support.  While enabled, every kernel launch of a loss call
 * (ckl_fwd_bwd*, ckl_fwd, ckl_bwd, ckl_topk), and all launches of one call of the
 * other operators together, are bracketed by HIP events on the call's stream.
 * ckl_timing_query waits for the recorded events and returns the summed
 * milliseconds and launch count of one kernel kind: 0 logits GEMM, 1 row pass,
 * 2 dH GEMM, 3 dH split reduce, 4 dW GEMM, 5 other (of a loss call, and the
 * log-probabilities, the residual's norms and dropout), 6 top-K (ckl_topk),
 * 7 embedding, 8 sampling, 9 8-bit products and quantisers.  Not for concurrent use
 * from several threads. */
int ckl_timing_enable(int on);
int ckl_timing_query(int kind, double* total_ms, int64_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* CKL_H_ */
