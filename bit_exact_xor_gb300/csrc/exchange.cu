// Rows between the tokens' order and the experts' order, and the gradients of
// both ways (include/dcr_ops.h).
//
// A team of threads takes a token, 8 columns a thread at a time: a token's row
// is read once and written to its k rows, or its k rows are read and summed in
// registers.  Everything is bound by these rows' bytes: 65520 rows of 6144
// values, an eighth of them without a token, gathered in 120 us (bf16, 6.6
// TB/s), summed in 216 (f32, 7.0 TB/s) or about 140 (bf16), the gradients of the
// sum in 450 (f32, 6.5 TB/s).
#include <algorithm>

#include "ops_internal.h"

namespace dcr {
namespace {

struct ExchangeArgs {
    const void* tokens_side;    // x of a gather, the output's gradient of a combine
    const void* rows_side;      // y of a combine
    void* out;                  // rows of a gather, sums of a combine, y's gradient
    const int32_t* positions;
    const float* weights;
    float* grad_weights;
    uint64_t tokens, cols, rows;
    uint64_t token_stride, row_stride, out_stride;
    uint32_t k;
};

constexpr int kThreads = 256;

// 8 values of a thread: consecutive ones in 16-byte words where all is laid
// out so (VEC), else every `team`th, the first n of them, so that neighbouring
// threads still read neighbouring values.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, uint32_t team, uint32_t n, float (&v)[8])
{
    if (VEC) {
        uint4 q[sizeof(T) / 2];
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
        const T* t = reinterpret_cast<const T*>(q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = uint32_t(i) < n ? to_f32(p[i * team]) : 0.0f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, uint32_t team, uint32_t n, const float (&v)[8])
{
    if (VEC) {
        uint4 q[sizeof(T) / 2];
        T* t = reinterpret_cast<T*>(q);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(v[i]);
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = q[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (uint32_t(i) < n) p[i * team] = from_f32<T>(v[i]);
    }
}

// The token and the columns of a thread: blockIdx.x counts pieces of `piece`
// columns within groups of tokens, one for each team.
template <bool VEC>
struct Place {
    uint64_t token, begin, end;
    uint32_t team;
    __device__ __forceinline__ Place(const ExchangeArgs& A, uint32_t team_, uint32_t pieces, uint64_t piece) : team(team_)
    {
        token = uint64_t(blockIdx.x / pieces) * (kThreads / team) + threadIdx.x / team;
        begin = uint64_t(blockIdx.x % pieces) * piece + threadIdx.x % team * (VEC ? 8 : 1);
        end = min(uint64_t(blockIdx.x % pieces + 1) * piece, A.cols);
    }
    // how many of the values from column c on exist
    __device__ __forceinline__ uint32_t count(uint64_t c) const { return VEC ? 8 : uint32_t(min((end - c + team - 1) / team, uint64_t(8))); }
};

template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(kThreads) gather_kernel(const ExchangeArgs A, uint32_t team, uint32_t pieces, uint32_t piece)
{
    const Place<VEC> P(A, team, pieces, piece);
    if (P.token >= A.tokens) return;
    const int32_t* pos = A.positions + P.token * A.k;
    const float* w = A.weights ? A.weights + P.token * A.k : nullptr;
    const TI* x = static_cast<const TI*>(A.tokens_side) + P.token * A.token_stride;
    for (uint64_t c = P.begin; c < P.end; c += team * 8) {
        const uint32_t n = P.count(c);
        float v[8];
        load8<TI, VEC>(x + c, team, n, v);
        for (uint32_t j = 0; j < A.k; ++j) {
            const uint64_t row = uint64_t(int64_t(pos[j]));
            if (row >= A.rows) continue;
            TO* out = static_cast<TO*>(A.out) + row * A.out_stride + c;
            if (w) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = v[i] * w[j];
                store8<TO, VEC>(out, team, n, u);
            } else {
                store8<TO, VEC>(out, team, n, v);
            }
        }
    }
}

// As many threads as an SM holds: rows at unrelated places want many loads under way (65520 rows of bf16 values: 156 us with
// 1536 threads an SM; 8 rows on their way a thread and fewer threads: 203; 32 bytes of a row a thread: 170).  That is 32
// registers, and spills: 12 to 36 bytes a thread in whole words, 100 of loads for f32, up to 432 where a row is no whole words.
// With and without that bound: 6144 columns bf16 155 and 180 us, f32 254 and 250; 2049 columns bf16 112 and 208, f32 111 and 183.
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(kThreads, 8) combine_kernel(const ExchangeArgs A, uint32_t team, uint32_t pieces, uint32_t piece)
{
    const Place<VEC> P(A, team, pieces, piece);
    if (P.token >= A.tokens) return;
    const int32_t* pos = A.positions + P.token * A.k;
    const float* w = A.weights ? A.weights + P.token * A.k : nullptr;
    TO* out = static_cast<TO*>(A.out) + P.token * A.out_stride;
    for (uint64_t c = P.begin; c < P.end; c += team * 8) {
        const uint32_t n = P.count(c);
        float s[8] = {};
#pragma unroll 4
        for (uint32_t j = 0; j < A.k; ++j) {
            const uint64_t row = uint64_t(int64_t(pos[j]));
            if (row >= A.rows) continue;
            float v[8];
            load8<TI, VEC>(static_cast<const TI*>(A.rows_side) + row * A.row_stride + c, team, n, v);
            const float f = w ? w[j] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = fmaf(f, v[i], s[i]);
        }
        store8<TO, VEC>(out + c, team, n, s);
    }
}

constexpr int kAtOnce = 4;     // rows whose products with the gradient are summed at once
constexpr uint64_t kFullWarps = 152 * 16;      // of combine_grad_kernel, which fill the SMs

// TY: type of y and its gradient, TG: of the output's gradient.
template <typename TY, typename TG, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const ExchangeArgs A, uint32_t team)
{
    __shared__ float part[kThreads / 32][kAtOnce];
    const Place<VEC> P(A, team, 1, A.cols);
    const bool on = P.token < A.tokens;
    const int32_t* pos = A.positions + P.token * A.k;
    const float* w = A.weights ? A.weights + P.token * A.k : nullptr;
    const TG* g = static_cast<const TG*>(A.tokens_side) + P.token * A.token_stride;
    for (uint32_t j = 0; j < A.k; j += kAtOnce) {
        uint64_t row[kAtOnce];
        float f[kAtOnce], dot[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            row[i] = on && j + i < A.k ? uint64_t(int64_t(pos[j + i])) : ~0ull;
            f[i] = row[i] < A.rows && w ? w[j + i] : 1.0f;
            dot[i] = 0.0f;
        }
        for (uint64_t c = P.begin; on && c < A.cols; c += team * 8) {
            const uint32_t n = P.count(c);
            float v[8], y[kAtOnce][8];
            load8<TG, VEC>(g + c, team, n, v);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (A.grad_weights && row[i] < A.rows) load8<TY, VEC>(static_cast<const TY*>(A.rows_side) + row[i] * A.row_stride + c, team, n, y[i]);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (row[i] >= A.rows) continue;
                if (A.grad_weights) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[i] = fmaf(v[e], y[i][e], dot[i]);
                }
                if (A.out) {
                    float u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = v[e] * f[i];
                    store8<TY, VEC>(static_cast<TY*>(A.out) + row[i] * A.out_stride + c, team, n, u);
                }
            }
        }
        if (!A.grad_weights) continue;
        const uint32_t width = min(team, 32u);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            for (uint32_t o = width / 2; o; o >>= 1) dot[i] += __shfl_xor_sync(~0u, dot[i], o);
        if (team > 32) {
            // the block's warps that share a token
            __syncthreads();
            if (threadIdx.x % 32 == 0) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) part[threadIdx.x / 32][i] = dot[i];
            }
            __syncthreads();
            const uint32_t first = threadIdx.x / team * (team / 32);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                dot[i] = 0.0f;
                for (uint32_t q = 0; q < team / 32; ++q) dot[i] += part[first + q][i];
            }
        }
        if (on && threadIdx.x % team == 0) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (j + i < A.k) A.grad_weights[P.token * A.k + j + i] = row[i] < A.rows ? dot[i] : 0.0f;
        }
    }
}

// Threads of a token: as many as have 8 columns, up to a block.
uint32_t team_of(uint64_t cols)
{
    uint32_t t = 1;
    while (t < kThreads && t * 8ull < cols) t *= 2;
    return t;
}

bool aligned(const void* p, uint64_t stride, uint32_t size) { return uintptr_t(p) % 16 == 0 && stride * size % 16 == 0; }

// A kernel over (tokens x pieces of columns): a piece is one step of a team.
template <typename K>
int launch_pieces(K kernel, const ExchangeArgs& A, const char* what, cudaStream_t s)
{
    const uint32_t team = team_of(A.cols);
    const uint64_t groups = (A.tokens + kThreads / team - 1) / (kThreads / team);
    uint64_t pieces = (A.cols + team * 8 - 1) / (team * 8);
    pieces = std::max<uint64_t>(1, std::min<uint64_t>(pieces, ((1ull << 31) - 1) / groups));
    const uint64_t steps = (A.cols + team * 8 * pieces - 1) / (team * 8 * pieces);
    const LaunchAttrs at(groups * pieces, kThreads, 0, 1, false, s);
    const cudaError_t e = cudaLaunchKernelEx(&at.cfg, kernel, A, team, uint32_t(pieces), uint32_t(steps * team * 8));
    return e == cudaSuccess ? DCR_OK : cuda_error(e, what);
}

int check(const char* what, uint32_t a, uint32_t b, uint64_t tokens, uint64_t cols, uint64_t rows, uint32_t k, const int32_t* positions, const float* weights)
{
    if (a > DCR_F16 || b > DCR_F16) return set_error(DCR_ERR_INVALID, "%s: unknown dtype", what);
    if (k == 0 || k > DCR_MAX_CHOSEN) return set_error(DCR_ERR_INVALID, "%s: k must be 1 to %u", what, DCR_MAX_CHOSEN);
    if (tokens >= 1ull << 31 || tokens * k >= 1ull << 31 || rows >= 1ull << 31 || cols >= 1ull << 31)
        return set_error(DCR_ERR_INVALID, "%s: tokens * k, rows and cols must be below 2^31", what);
    if (tokens && !positions) return set_error(DCR_ERR_INVALID, "%s: NULL argument", what);
    if (uintptr_t(positions) % 4 || uintptr_t(weights) % 4) return set_error(DCR_ERR_INVALID, "%s: misaligned buffer", what);
    return DCR_OK;
}

int check_matrix(const char* what, const char* name, const void* p, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t stride)
{
    if (stride < cols || stride >= 1ull << 40) return set_error(DCR_ERR_INVALID, "%s: bad stride of %s", what, name);
    if (rows && cols && !p) return set_error(DCR_ERR_INVALID, "%s: %s is NULL", what, name);
    if (uintptr_t(p) % dtype_size(dtype)) return set_error(DCR_ERR_INVALID, "%s: %s is misaligned", what, name);
    return DCR_OK;
}

// Calls f with values of both types and whether all is laid out in 16-byte words.
template <typename F>
int with_types(uint32_t a, uint32_t b, bool vec, F f)
{
    return with_dtype(a, [&](auto x) {
        return with_dtype(b, [&](auto y) { return vec ? f(x, y, std::true_type()) : f(x, y, std::false_type()); });
    });
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_experts_gather(const void* x, uint32_t x_dtype, uint64_t tokens, uint64_t cols, uint64_t x_stride,
                                  const int32_t* positions, uint32_t k, const float* weights, void* out, uint32_t dtype, uint64_t rows,
                                  uint64_t out_stride, void* stream)
{
    static const char what[] = "dcr_experts_gather";
    if (int rc = dcr::check(what, x_dtype, dtype, tokens, cols, rows, k, positions, weights)) return rc;
    if (int rc = check_matrix(what, "x", x, x_dtype, tokens, cols, x_stride)) return rc;
    if (int rc = check_matrix(what, "out", out, dtype, rows, cols, out_stride)) return rc;
    if (tokens == 0 || cols == 0 || rows == 0) return DCR_OK;
    if (int rc = check_overlap(what, {{"out", out, dtype_size(dtype), rows, cols, out_stride}},
                               {{"x", x, dtype_size(x_dtype), tokens, cols, x_stride}, {"positions", positions, tokens * k * 4}, {"weights", weights, tokens * k * 4}}))
        return rc;
    ExchangeArgs A{};
    A.tokens_side = x, A.out = out, A.positions = positions, A.weights = weights;
    A.tokens = tokens, A.cols = cols, A.rows = rows, A.token_stride = x_stride, A.out_stride = out_stride, A.k = k;
    const bool vec = cols % 8 == 0 && aligned(x, x_stride, dtype_size(x_dtype)) && aligned(out, out_stride, dtype_size(dtype));
    return with_types(x_dtype, dtype, vec, [&](auto a, auto b, auto v) {
        return launch_pieces(gather_kernel<decltype(a), decltype(b), decltype(v)::value>, A, "experts gather launch", static_cast<cudaStream_t>(stream));
    });
}

extern "C" int dcr_experts_combine(const void* y, uint32_t y_dtype, uint64_t rows, uint64_t cols, uint64_t y_stride, const int32_t* positions,
                                   const float* weights, uint64_t tokens, uint32_t k, void* out, uint32_t dtype, uint64_t out_stride,
                                   void* stream)
{
    static const char what[] = "dcr_experts_combine";
    if (int rc = dcr::check(what, y_dtype, dtype, tokens, cols, rows, k, positions, weights)) return rc;
    if (int rc = check_matrix(what, "y", y, y_dtype, rows, cols, y_stride)) return rc;
    if (int rc = check_matrix(what, "out", out, dtype, tokens, cols, out_stride)) return rc;
    if (tokens == 0 || cols == 0) return DCR_OK;
    if (int rc = check_overlap(what, {{"out", out, dtype_size(dtype), tokens, cols, out_stride}},
                               {{"y", y, dtype_size(y_dtype), rows, cols, y_stride}, {"positions", positions, tokens * k * 4}, {"weights", weights, tokens * k * 4}}))
        return rc;
    ExchangeArgs A{};
    A.rows_side = y, A.out = out, A.positions = positions, A.weights = weights;
    A.tokens = tokens, A.cols = cols, A.rows = rows, A.row_stride = y_stride, A.out_stride = out_stride, A.k = k;
    const bool vec = cols % 8 == 0 && aligned(y, y_stride, dtype_size(y_dtype)) && aligned(out, out_stride, dtype_size(dtype));
    return with_types(y_dtype, dtype, vec, [&](auto a, auto b, auto v) {
        return launch_pieces(combine_kernel<decltype(a), decltype(b), decltype(v)::value>, A, "experts combine launch", static_cast<cudaStream_t>(stream));
    });
}

extern "C" int dcr_experts_combine_grad(const void* y, uint32_t y_dtype, uint64_t rows, uint64_t cols, uint64_t y_stride,
                                        const int32_t* positions, const float* weights, uint64_t tokens, uint32_t k, const void* grad,
                                        uint32_t dtype, uint64_t grad_stride, void* grad_y, uint64_t grad_y_stride, float* grad_weights,
                                        void* stream)
{
    static const char what[] = "dcr_experts_combine_grad";
    if (int rc = dcr::check(what, y_dtype, dtype, tokens, cols, rows, k, positions, weights)) return rc;
    if (int rc = check_matrix(what, "y", grad_weights ? y : nullptr, y_dtype, grad_weights ? rows : 0, cols, grad_weights ? y_stride : cols)) return rc;
    if (int rc = check_matrix(what, "grad", grad, dtype, tokens, cols, grad_stride)) return rc;
    if (int rc = check_matrix(what, "grad_y", grad_y, y_dtype, 0, cols, grad_y ? grad_y_stride : cols)) return rc;
    if (uintptr_t(grad_weights) % 4) return set_error(DCR_ERR_INVALID, "%s: misaligned buffer", what);
    if (tokens == 0 || (!grad_y && !grad_weights)) return DCR_OK;
    // each value of y, and each weight, is read by the threads that write its gradient, and before that
    const Memory in_y = {"y", grad_weights ? y : nullptr, dtype_size(y_dtype), rows, cols, y_stride}, in_w = {"weights", weights, tokens * k * 4},
                 none, out_y = {"grad_y", grad_y, dtype_size(y_dtype), rows, cols, grad_y_stride}, out_w = {"grad_weights", grad_weights, tokens * k * 4};
    const Memory in_grad = {"grad", grad, dtype_size(dtype), tokens, cols, grad_stride}, in_pos = {"positions", positions, tokens * k * 4};
    if (int rc = check_overlap(what, {out_y, out_w}, {in_grad, in_pos})) return rc;
    if (int rc = check_overlap(what, {out_y}, {grad_y == y && grad_y_stride == y_stride ? none : in_y, in_w})) return rc;
    if (int rc = check_overlap(what, {out_w}, {grad_weights == weights ? none : in_w, in_y})) return rc;
    ExchangeArgs A{};
    A.tokens_side = grad, A.rows_side = y, A.out = grad_y, A.positions = positions, A.weights = weights, A.grad_weights = grad_weights;
    A.tokens = tokens, A.cols = cols, A.rows = rows, A.token_stride = grad_stride, A.row_stride = y_stride, A.out_stride = grad_y_stride, A.k = k;
    const uint32_t ys = dtype_size(y_dtype);
    const bool vec = cols % 8 == 0 && aligned(grad, grad_stride, dtype_size(dtype)) && (!grad_weights || aligned(y, y_stride, ys)) &&
                     (!grad_y || aligned(grad_y, grad_y_stride, ys));
    // A warp a token needs no barriers (2432 tokens of 8 rows of 1024 bf16 values: 27 -> 17 us); a block shares one where
    // tokens are few, or rows so long that their pieces are better read at once (8190 of 6144 f32 values: 469 -> 450).
    const bool warps = tokens >= kFullWarps && cols * ys <= 16384;
    const uint32_t team = std::min(team_of(cols), warps ? 32u : uint32_t(kThreads));
    return with_types(y_dtype, dtype, vec, [&](auto a, auto b, auto v) {
        const LaunchAttrs at((tokens + kThreads / team - 1) / (kThreads / team), kThreads, 0, 1, false, static_cast<cudaStream_t>(stream));
        const cudaError_t e = cudaLaunchKernelEx(&at.cfg, combine_grad_kernel<decltype(a), decltype(b), decltype(v)::value>, A, team);
        return e == cudaSuccess ? DCR_OK : cuda_error(e, "experts combine gradient launch");
    });
}
