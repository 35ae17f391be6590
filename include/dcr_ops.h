/*
 * dcr_ops.h — the operators around a refit: NVFP4 quantisation of weights and
 * activations, the product of NVFP4 operands, and the policy loss whose
 * updates a refit carries.
 *
 * Conventions are those of dcr.h, with one difference: these calls are
 * stream-ordered and return without waiting for the GPU (as dcr_dense_refit
 * does), so they can be captured into a CUDA graph.  A bad argument is
 * refused with DCR_ERR_INVALID before anything is launched; sizes of zero are
 * valid and launch nothing (no scale is written, but dcr_policy_loss of no rows
 * still writes a loss of 0).  Device buffers belong to the caller; no call
 * keeps an address after it returns, so calls on several streams may overlap.
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

/* Waits for `stream` and reports whether any operator on the current device
 * gave up a wait since the last report: every wait inside a kernel is
 * bounded (about a second), after which the kernel ends with its output
 * incomplete.  DCR_OK, DCR_ERR_TIMEOUT or DCR_ERR_CUDA. */
int dcr_ops_status(void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DCR_OPS_H */
