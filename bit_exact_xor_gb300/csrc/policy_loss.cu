// Clipped policy loss with a KL term, its gradient by the logits, and the
// log-probabilities of tokens (include/dcr_ops.h).
#include "ops_internal.h"

namespace dcr {
namespace {

struct LossArgs {
    const void* logits;
    void* grad;
    uint64_t rows, vocab, row_stride, grad_stride;
    const int64_t* tokens;
    const float* old_logp;      // null: log-probabilities alone
    const float* ref_logp;
    const float* advantages;
    const float* weights;
    float* row_loss;
    float* logp;
    float inv_temp, lo, hi, kl;
};

// The running maximum and sum of exponentials of two stretches of a row,
// joined.  A stretch without a finite value has maximum -inf and sum 0.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2)
{
    float t = fmaxf(m, m2);
    float a = m == t ? 1.0f : __expf(m - t), b = m2 == t ? 1.0f : __expf(m2 - t);
    s = s * a + s2 * b;
    m = t;
}

// Loss of a row and its derivative by the log-probability.
__device__ __forceinline__ void row_loss(const LossArgs& A, uint64_t row, float lp, float& loss, float& slope)
{
    const float adv = A.advantages[row], ratio = expf(lp - A.old_logp[row]);
    const float u = ratio * adv, c = fminf(fmaxf(ratio, A.lo), A.hi) * adv;
    const bool clipped = c < u;
    loss = clipped ? -c : -u;
    slope = clipped ? 0.0f : -u;
    if (A.kl != 0.0f) {
        const float k = A.ref_logp[row] - lp, e = expf(k);
        loss += A.kl * (e - k - 1.0f);
        slope += A.kl * (1.0f - e);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) loss_kernel(LossArgs A)
{
    __shared__ float pm[8], ps[8];
    const uint64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(A.logits) + row * A.row_stride;
    T* g = A.grad ? static_cast<T*>(A.grad) + row * A.grad_stride : nullptr;
    const int64_t y = A.tokens[row];
    const float w = A.weights ? A.weights[row] : 1.0f;
    if (w == 0.0f || y < 0 || uint64_t(y) >= A.vocab) {
        if (threadIdx.x == 0) {
            A.logp[row] = 0.0f;
            if (A.row_loss) A.row_loss[row] = 0.0f;
        }
        if (g)
            for (uint64_t i = threadIdx.x; i < A.vocab; i += 256) g[i] = from_f32<T>(0.0f);
        return;
    }
    float m = -INFINITY, s = 0.0f;
    for (uint64_t i = threadIdx.x; i < A.vocab; i += 256) join(m, s, to_f32(x[i]) * A.inv_temp, 1.0f);
    for (int o = 16; o; o >>= 1) join(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
    if (threadIdx.x % 32 == 0) pm[threadIdx.x / 32] = m, ps[threadIdx.x / 32] = s;
    __syncthreads();
    m = pm[0], s = ps[0];
    for (int i = 1; i < 8; ++i) join(m, s, pm[i], ps[i]);
    const float lse = m + logf(s);
    const float lp = to_f32(x[y]) * A.inv_temp - lse;
    if (threadIdx.x == 0) A.logp[row] = lp;
    if (!A.old_logp) return;
    float loss, slope;
    row_loss(A, row, lp, loss, slope);
    if (threadIdx.x == 0) A.row_loss[row] = w * loss;
    if (!g) return;
    const float c = w * slope * A.inv_temp;
    __syncthreads();   // grad may be logits: x[y] has been read by all
    for (uint64_t i = threadIdx.x; i < A.vocab; i += 256) {
        float p = __expf(to_f32(x[i]) * A.inv_temp - lse);
        g[i] = from_f32<T>(c * ((int64_t(i) == y ? 1.0f : 0.0f) - p));
    }
}

// The rows' losses summed in a fixed order: thread i takes rows i, i + 1024,
// ..., then a tree over the threads.
__global__ void __launch_bounds__(1024) sum_kernel(const float* v, uint64_t n, float* out)
{
    __shared__ double part[32];
    double s = 0.0;
    for (uint64_t i = threadIdx.x; i < n; i += 1024) s += v[i];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = part[threadIdx.x];
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (threadIdx.x == 0) *out = float(s);
    }
}

int launch(const LossArgs& A, uint32_t dtype, float* loss, cudaStream_t s)
{
    if (A.rows == 0 && !loss) return DCR_OK;
    if (A.rows) with_dtype(dtype, [&](auto t) { loss_kernel<decltype(t)><<<unsigned(A.rows), 256, 0, s>>>(A); });
    if (loss) sum_kernel<<<1, 1024, 0, s>>>(A.row_loss, A.rows, loss);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "policy loss launch");
}

int check(const char* what, const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
          const int64_t* tokens, float temperature, const float* logp)
{
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "%s: unknown dtype %u", what, dtype);
    if (!(temperature > 0.0f) || temperature > 3.0e38f)
        return set_error(DCR_ERR_INVALID, "%s: temperature must be positive and finite", what);
    if (vocab == 0 || vocab >= 1ull << 31 || rows >= 1ull << 31 || row_stride >= 1ull << 40)
        return set_error(DCR_ERR_INVALID, "%s: vocab must be at least 1 and sizes below 2^31", what);
    if (row_stride < vocab) return set_error(DCR_ERR_INVALID, "%s: row_stride below vocab", what);
    if (rows && (!logits || !tokens || !logp)) return set_error(DCR_ERR_INVALID, "%s: NULL argument", what);
    if (uintptr_t(logits) % dtype_size(dtype) || uintptr_t(tokens) % 8 || uintptr_t(logp) % 4)
        return set_error(DCR_ERR_INVALID, "%s: misaligned buffer", what);
    return DCR_OK;
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_policy_loss(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                               const int64_t* tokens, const float* old_logp, const float* ref_logp,
                               const float* advantages, const float* weights, const dcr_policy_opts* opts, float* loss,
                               float* row_loss, float* logp, void* grad, uint64_t grad_stride, void* stream)
{
    if (!opts || !loss) return set_error(DCR_ERR_INVALID, "dcr_policy_loss: NULL argument");
    if (int rc = dcr::check("dcr_policy_loss", logits, dtype, rows, vocab, row_stride, tokens, opts->temperature, logp)) return rc;
    if (!(opts->clip_low >= 0.0f) || !(opts->clip_high >= 0.0f) || !(opts->kl_coef >= 0.0f))
        return set_error(DCR_ERR_INVALID, "dcr_policy_loss: clip_low, clip_high and kl_coef must not be negative");
    if (rows && (!old_logp || !advantages || !weights || !row_loss))
        return set_error(DCR_ERR_INVALID, "dcr_policy_loss: NULL argument");
    if (rows && opts->kl_coef != 0.0f && !ref_logp)
        return set_error(DCR_ERR_INVALID, "dcr_policy_loss: kl_coef needs ref_logp");
    if (grad && (grad_stride < vocab || grad_stride >= 1ull << 40))
        return set_error(DCR_ERR_INVALID, "dcr_policy_loss: bad grad_stride");
    if (grad == logits && grad && grad_stride != row_stride)
        return set_error(DCR_ERR_INVALID, "dcr_policy_loss: grad in place of logits needs the same stride");
    if (uintptr_t(grad) % dtype_size(dtype) || uintptr_t(old_logp) % 4 || uintptr_t(ref_logp) % 4 ||
        uintptr_t(advantages) % 4 || uintptr_t(weights) % 4 || uintptr_t(loss) % 4 || uintptr_t(row_loss) % 4)
        return set_error(DCR_ERR_INVALID, "dcr_policy_loss: misaligned buffer");
    LossArgs A{logits, grad, rows, vocab, row_stride, grad_stride, tokens, old_logp, ref_logp, advantages, weights,
               row_loss, logp, 1.0f / opts->temperature, 1.0f - opts->clip_low, 1.0f + opts->clip_high, opts->kl_coef};
    return launch(A, dtype, loss, static_cast<cudaStream_t>(stream));
}

extern "C" int dcr_token_logprobs(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                                  const int64_t* tokens, float temperature, float* logp, void* stream)
{
    if (int rc = dcr::check("dcr_token_logprobs", logits, dtype, rows, vocab, row_stride, tokens, temperature, logp)) return rc;
    LossArgs A{};
    A.logits = logits, A.rows = rows, A.vocab = vocab, A.row_stride = row_stride;
    A.tokens = tokens, A.logp = logp, A.inv_temp = 1.0f / temperature;
    return launch(A, dtype, nullptr, static_cast<cudaStream_t>(stream));
}
