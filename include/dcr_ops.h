/*
 * dcr_ops.h — the operators around a refit: NVFP4 quantisation of weights and
 * activations, the product of NVFP4 operands, routing to experts, scores of
 * tokens, the policy loss whose updates a refit carries, and the optimiser's
 * step that makes them.
 *
 * Conventions are those of dcr.h, with one difference: these calls are
 * stream-ordered and return without waiting for the GPU (as dcr_dense_refit
 * does), so they can be captured into a CUDA graph.  A bad argument is
 * refused with DCR_ERR_INVALID before anything is launched; sizes of zero are
 * valid and launch nothing (no scale is written, but dcr_policy_loss of no rows
 * still writes a loss of 0).  Device buffers belong to the caller; no call
 * keeps an address after it returns, so calls on several streams may overlap.
 * What a call writes may overlap nothing else that it is given, except where it
 * says that an output may be one of its inputs, which is then the same memory,
 * laid out alike.  From dcr_token_scores on other overlaps are refused, matrices
 * by their rows: columns of one buffer side by side are no overlap.
 *
 * NVFP4.  A matrix [rows, cols] is held as codes [rows, cols / 2] (e2m1, two
 * per byte, the even column in the low nibble), scales [rows, cols / 16]
 * (e4m3, one per 16 consecutive columns) and a 32-bit scale t, one for the
 * matrix or one per row.  These are the row-major bytes of 4- and 8-bit
 * tensors in dcr_tensor_desc, so trainer arenas are written and receiver
 * arenas read where they lie.  A code c in a block of scale s stands for
 * c * (s * t).  Quantisation, every step rounded to nearest even in 32 bits:
 *   t = amax * (1 / 2688), amax the largest finite |x| of the matrix or row
 *       (t = 1 if that is 0); 2688 = 6 * 448, the largest code times the
 *       largest scale;
 *   s = e4m3(min(a / (6 t), 448)), a the largest |x| of the block;
 *   r = min(1 / (s t), FLT_MAX), or 0 if s t = 0;
 *   code = e2m1(x r), saturating at +-6.
 * A block that holds a NaN gets a NaN scale (0x7F), so that it reads back as
 * NaN; infinities take the largest code.
 */
#ifndef DCR_OPS_H
#define DCR_OPS_H

#include "dcr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of inputs and outputs. */
enum { DCR_F32 = 0, DCR_BF16 = 1, DCR_F16 = 2, DCR_NONE = 3 };

/* Where the 32-bit scale comes from: GIVEN, scale[0] is read; TENSOR, it is
 * computed from all of x and written to scale[0] (x is read twice); ROW, one
 * per row is computed and written to scale[rows]. */
enum { DCR_SCALE_GIVEN = 0, DCR_SCALE_TENSOR = 1, DCR_SCALE_ROW = 2 };

/* One NVFP4 matrix (device pointers; codes 16-byte aligned). */
typedef struct {
    const void* codes;
    const void* scales;
    const float* scale;
    uint64_t scale_count;   /* entries of scale */
} dcr_nvfp4;

/* Quantise x [rows, cols] (dtype, rows row_stride elements apart, cols a
 * multiple of 16) to codes (16-byte aligned), scales and scale.  values
 * (nullable, [rows, cols] contiguous, 16-byte aligned, of values_dtype;
 * DCR_NONE without) receives what the codes stand for, rounded once to its
 * type: the weights that a quantisation-aware forward pass computes with.
 * The gradient of a quantisation-aware pass goes straight through.  A block's
 * largest value is kept to a sixteenth, the rounding of its scale, unless the
 * scale is GIVEN and too small or the block lies far below its matrix or row:
 * where its largest value is under amax / 28672 the scale is a subnormal e4m3
 * number, rounded down by as much as a third (largest values then saturate) or
 * to 0.  workspace (TENSOR only, device, at least DCR_QUANT_PARTIALS floats)
 * holds partial maxima during the call. */
#define DCR_QUANT_PARTIALS 1216u
int dcr_nvfp4_quantize(const void* x, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t row_stride,
                       uint32_t scale_mode, float* scale, void* codes, void* scales, void* values,
                       uint32_t values_dtype, void* workspace, void* stream);

/* y [m, n] (dtype, rows y_stride elements apart) = x w^T, x [m, k] and w
 * [n, k] both NVFP4, k a multiple of 32: the product of the two 32-bit scales
 * times a sum that is held in 32 bits, rounded once.  e4m3 scales are not
 * negative.  x->scale_count is 1 or m, w->scale_count 1 or the number of
 * experts.  The same call gives the same bits every time; which kernel and how
 * many parts of k a row's sum has goes by the sizes, so that a row alone and the
 * same row in a larger batch may differ by the rounding of 32-bit sums.
 * experts > 0: w is [experts * n, k], one matrix after another, and offsets
 * (device, experts + 1 entries, not decreasing) says which rows of x belong
 * to which: rows offsets[e] to offsets[e + 1] are multiplied by matrix e.
 * Rows that no expert has are left as they are.  experts <= DCR_MAX_EXPERTS;
 * experts = 0 and offsets = NULL for one matrix.
 * Test only: with DCR_TEST_STALL added to dtype no operand is ever loaded, so
 * that the kernel's waits run out (after about a second): it ends with y
 * incomplete, and dcr_ops_status reports DCR_ERR_TIMEOUT. */
#define DCR_MAX_EXPERTS 1024u
#define DCR_TEST_STALL 0x80000000u
int dcr_nvfp4_matmul(const dcr_nvfp4* x, const dcr_nvfp4* w, uint64_t m, uint64_t n, uint64_t k,
                     const int32_t* offsets, uint32_t experts, void* y, uint32_t dtype, uint64_t y_stride,
                     void* stream);

/* y = x w^T for activations x [m, k] (x_dtype, rows x_stride elements apart):
 * x is quantised with a scale per row, so that a row's codes and scales do not
 * depend on the rows beside it, then multiplied as in dcr_nvfp4_matmul.  workspace
 * (device, 16-byte aligned, DCR_LINEAR_WORKSPACE bytes) holds the quantised
 * activations during the call.  The size is a function's, in 64 bits whatever
 * the types of m and k. */
#define DCR_LINEAR_WORKSPACE(m, k) ((m) * ((k) / 2 + (k) / 16 + 4) + 4)
#ifdef __cplusplus
    constexpr uint64_t dcr_linear_workspace(uint64_t m, uint64_t k) { return DCR_LINEAR_WORKSPACE(m, k); }
#else
    static inline uint64_t dcr_linear_workspace(uint64_t m, uint64_t k) { return DCR_LINEAR_WORKSPACE(m, k); }
#endif
#undef DCR_LINEAR_WORKSPACE
#define DCR_LINEAR_WORKSPACE(m, k) dcr_linear_workspace(m, k)
int dcr_nvfp4_linear(const void* x, uint32_t x_dtype, uint64_t x_stride, const dcr_nvfp4* w, uint64_t m, uint64_t n,
                     uint64_t k, const int32_t* offsets, uint32_t experts, void* y, uint32_t dtype,
                     uint64_t y_stride, void* workspace, void* stream);

/* Clipped policy loss with a KL term, from logits [rows, vocab] (dtype, rows
 * row_stride elements apart), with the gradient by the logits.  Per row, with
 * token y, old log-probability o, reference q, advantage A and weight w:
 *   z = logits / temperature,  lp = z_y - log sum_j exp(z_j),
 *   u = exp(lp - o) A,  c = clip(exp(lp - o), 1 - clip_low, 1 + clip_high) A,
 *   l = -min(u, c) + kl_coef (exp(q - lp) - (q - lp) - 1),
 *   loss = sum_rows w l,  grad_j = d loss / d logits_j.
 * An exponential that overflows 32 bits at a finite argument counts as the
 * largest 32-bit number, so that an advantage of 0 times it is 0.
 * A row whose weight is 0 or whose token lies outside [0, vocab) is left out:
 * its logits are not read, its log-probability and loss are 0 and its
 * gradient is 0, whatever its logits hold.  ref_logp may be NULL if kl_coef
 * is 0.  grad (same dtype, rows grad_stride elements apart) may be NULL, and
 * may be logits itself.  row_loss [rows] receives w l, loss [1] their sum in
 * a fixed order. */
typedef struct {
    float temperature, clip_low, clip_high, kl_coef;
} dcr_policy_opts;
int dcr_policy_loss(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                    const int64_t* tokens, const float* old_logp, const float* ref_logp,
                    const float* advantages, const float* weights, const dcr_policy_opts* opts, float* loss,
                    float* row_loss, float* logp, void* grad, uint64_t grad_stride, void* stream);

/* lp of dcr_policy_loss alone (0 where the token lies outside [0, vocab)). */
int dcr_token_logprobs(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                       const int64_t* tokens, float temperature, float* logp, void* stream);

/* ---- scores of given tokens --------------------------------------------
 * Per row of logits x [rows, vocab] (dtype, rows row_stride elements apart),
 * with token y and z = x / temperature, M = max_j x_j:
 *   r = sum_j exp((x_j - M) / temperature) - 1   (one maximum left out),
 *   logp = (x_y - M) / temperature - log(1 + r),
 *   D = sum_j exp((x_j - M) / temperature) (M - x_j) / temperature / (1 + r),
 *   entropy = log(1 + r) + D,
 * and the `top` likeliest tokens, the lowest index first among equal ones,
 * with their log-probabilities: top_logp and top_tokens [rows, top], top at
 * most DCR_MAX_TOP and vocab.  A NaN stands behind every number there.  stats
 * [rows, 3] receives M, r and D, which dcr_token_scores_grad takes.  logp,
 * entropy, stats and top_logp are held in 32 bits.  A row whose token lies
 * outside [0, vocab) is left out: its logits are not read, its outputs are 0
 * and its alternatives' tokens -1.  logp, entropy and stats may each be NULL. */
#define DCR_MAX_TOP 64u
int dcr_token_scores(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                     const int64_t* tokens, float temperature, uint32_t top, float* logp, float* entropy,
                     float* top_logp, int64_t* top_tokens, float* stats, void* stream);

/* The gradient by the logits of a loss whose derivatives by logp and entropy
 * are grad_logp and grad_entropy [rows] (either may be NULL: 0):
 *   grad_j = (grad_logp (delta_jy - p_j)
 *             - grad_entropy p_j ((x_j - M) / temperature + D)) / temperature,
 * p_j = exp((x_j - M) / temperature) / (1 + r), the token's own factor 1 - p_y
 * from r where x_y = M.  Alternatives carry no gradient.  grad (same dtype,
 * rows grad_stride elements apart) may be logits itself.  The gradient of a
 * row whose token lies outside [0, vocab), or whose two derivatives are 0, is
 * 0 and its logits are not read. */
int dcr_token_scores_grad(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                          const int64_t* tokens, const float* stats, const float* grad_logp,
                          const float* grad_entropy, float temperature, void* grad, uint64_t grad_stride,
                          void* stream);

/* ---- routing to experts ------------------------------------------------
 * Per token, from the router's logits x [tokens, experts] (dtype, rows
 * row_stride elements apart): s = softmax(x) or sigmoid(x); the k experts of
 * largest s + bias (bias [experts], float, nullable), the lowest index first
 * among equal ones, in that order; with groups > 1 only from the group_top
 * groups (of experts / groups consecutive experts) whose group_by (1 or 2)
 * best sum highest.  Which experts are chosen is decided as with scores in 64
 * bits; without a bias, and with one group or group_by 1, by the logits
 * themselves.  Their weights are s without the bias, divided by the sum over
 * the chosen ones if renormalise is not 0, times scale.  An expert whose logit
 * or s + bias is -inf or NaN is never chosen; a token that mask (bytes,
 * nullable) has a 0 for chooses none.  Slots without an expert hold expert -1,
 * weight 0 and position -1.
 * experts, weights, positions [tokens, k]; offsets [experts + 1]: the rows of
 * expert e are offsets[e] to offsets[e + 1], as dcr_nvfp4_matmul takes them,
 * ordered by token; positions: the row of a slot; order [tokens * k]: the slot
 * (token * k + place) of a row, -1 behind the last.  workspace: device,
 * 16-byte aligned, DCR_ROUTE_WORKSPACE(experts) bytes.  tokens * k < 2^31. */
enum { DCR_SOFTMAX = 0, DCR_SIGMOID = 1 };
#define DCR_MAX_CHOSEN 32u
#define DCR_MAX_GROUPS 32u
#define DCR_ROUTE_PARTS 152u
#define DCR_ROUTE_WORKSPACE(experts) (16ull * DCR_ROUTE_PARTS * (((experts) + 3) / 4))
typedef struct {
    uint32_t scoring, k, groups, group_top, group_by, renormalise;
    float scale;
} dcr_route_opts;
int dcr_route(const void* logits, uint32_t dtype, uint64_t tokens, uint32_t experts, uint64_t row_stride,
              const float* bias, const uint8_t* mask, const dcr_route_opts* opts, int32_t* chosen, float* weights,
              int32_t* offsets, int32_t* order, int32_t* positions, void* workspace, void* stream);

/* The gradient by the logits of a loss whose derivative by the weights is
 * grad_weights [tokens, k]; the choice itself and the bias carry none.  grad
 * [tokens, experts] (dtype, rows grad_stride elements apart) may be logits
 * itself; opts: scoring, k, renormalise and scale are used. */
int dcr_route_grad(const void* logits, uint32_t dtype, uint64_t tokens, uint32_t experts, uint64_t row_stride,
                   const int32_t* chosen, const float* grad_weights, const dcr_route_opts* opts, void* grad,
                   uint64_t grad_stride, void* stream);

/* Rows into the experts' order: out[positions[t, j]] = x[t], times weights[t,
 * j] if weights is not NULL, rounded once.  x [tokens, cols] (x_dtype, rows
 * x_stride elements apart), out (dtype, rows out_stride apart) of `rows` rows;
 * positions [tokens, k] as from dcr_route; one that lies outside [0, rows) is
 * passed over, and rows of out that none names are left as they are. */
int dcr_experts_gather(const void* x, uint32_t x_dtype, uint64_t tokens, uint64_t cols, uint64_t x_stride,
                       const int32_t* positions, uint32_t k, const float* weights, void* out, uint32_t dtype,
                       uint64_t rows, uint64_t out_stride, void* stream);

/* The rows back: out[t] = sum_j weights[t, j] y[positions[t, j]] (weights
 * NULL: 1), summed in 32 bits in the order of j and rounded once; a token
 * without a row gets 0, whatever the other rows hold.  y: `rows` rows.  With
 * weights NULL it is the gradient of dcr_experts_gather by x. */
int dcr_experts_combine(const void* y, uint32_t y_dtype, uint64_t rows, uint64_t cols, uint64_t y_stride,
                        const int32_t* positions, const float* weights, uint64_t tokens, uint32_t k, void* out,
                        uint32_t dtype, uint64_t out_stride, void* stream);

/* Gradients of dcr_experts_combine from that of its output, grad [tokens,
 * cols] (dtype): grad_y[positions[t, j]] = weights[t, j] grad[t] (y_dtype,
 * nullable; rows that no slot has are left as they are), and grad_weights[t,
 * j] (nullable) is the dot product of y[positions[t, j]] and grad[t], 0 for a
 * slot without a row.  weights NULL: 1.  grad_y may be y itself, in the same
 * place, and grad_weights weights. */
int dcr_experts_combine_grad(const void* y, uint32_t y_dtype, uint64_t rows, uint64_t cols, uint64_t y_stride,
                             const int32_t* positions, const float* weights, uint64_t tokens, uint32_t k,
                             const void* grad, uint32_t dtype, uint64_t grad_stride, void* grad_y,
                             uint64_t grad_y_stride, float* grad_weights, void* stream);

/* ---- the trainer's step ------------------------------------------------
 * norm [1] = the square root of the sum of the squares of every gradient:
 * `count` tensors of n contiguous values of dtype.  Up to 65 squares are
 * added up in 32 bits (scaled by a power of two where these would not hold
 * them) and the sums of these in 64, all in a fixed order; a norm beyond the
 * largest float is infinite.  workspace: device, 8-byte aligned,
 * DCR_NORM_WORKSPACE bytes. */
#define DCR_NORM_WORKSPACE 9728u
typedef struct {
    const void* values;
    uint64_t n;
} dcr_grad;
int dcr_grad_norm(const dcr_grad* grads, uint32_t count, uint32_t dtype, void* workspace, float* norm, void* stream);

/* One AdamW step over `count` tensors of n contiguous values each, in place:
 *   g = grad * grad_scale (times max_norm / N if N = |grad_scale| norm[0] > max_norm > 0),
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   w = w (1 - lr weight_decay) - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps).
 * The factors of lr, betas and step are formed in 64 bits; every operation on
 * the values is rounded to 32 bits by itself, in that order, w to its type at
 * the end and the copy (copy_dtype, DCR_NONE without), from the same 32 bits,
 * to its own: a master in 32 bits and 16-bit weights in a refit's arena are
 * written together.  16-bit weights without a master are rounded to nearest,
 * and so lose updates below half of their last bit.
 * state_bits 32: m and v are floats.  state_bits 8: m and sqrt(v) are held as
 * e4m3 values (m, v: n bytes) times a 32-bit scale per 256 consecutive values
 * of a tensor (m_scale, v_scale: ceil(n / 256) floats), the scale being the
 * block's largest magnitude times 1 / 448.  A value between two of e4m3 is
 * rounded up with the probability of its distance from the lower one, so that
 * moments keep moving on average although a step changes them by less than
 * half an e4m3 step; sqrt(v) above 0 is never rounded to 0.  The random bits
 * are a hash of seed, step and the value's number in the call: the same call
 * gives the same bits.  A block with an infinite or NaN moment reads back as
 * NaN.  norm (device, nullable): if N is not finite the step is left out
 * whole: nothing is written.  device_step, device_lr (device, nullable) stand
 * in step's and lr's place, for captured graphs (their factors are formed in
 * 32 bits); the step is the number of
 * this update, from 1, and is not changed.  Tensors that are written may not
 * overlap any other, nor norm, device_step or device_lr. */
typedef struct {
    void* w;
    const void* grad;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    void* copy;
    uint64_t n;
} dcr_adamw_tensor;
typedef struct {
    double lr, beta1, beta2, eps, weight_decay, grad_scale, max_norm;
    uint64_t step;
    const float* norm;
    const int64_t* device_step;
    const float* device_lr;
    uint32_t seed, state_bits;
} dcr_adamw_opts;
#define DCR_ADAMW_BLOCK 256u
int dcr_adamw(const dcr_adamw_tensor* tensors, uint32_t count, uint32_t w_dtype, uint32_t grad_dtype,
              uint32_t copy_dtype, const dcr_adamw_opts* opts, void* stream);

/* Waits for `stream` and reports whether any operator on the current device
 * gave up a wait since the last report: every wait inside a kernel is
 * bounded (about a second), after which the kernel ends with its output
 * incomplete.  DCR_OK, DCR_ERR_TIMEOUT or DCR_ERR_CUDA. */
int dcr_ops_status(void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DCR_OPS_H */
