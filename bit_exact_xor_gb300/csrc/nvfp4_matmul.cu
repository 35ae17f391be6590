// Product of two NVFP4 operands, dense or per expert (include/dcr_ops.h).
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "ops_internal.h"

namespace dcr {
namespace {

struct MatmulArgs {
    dcr_nvfp4 x, w;
    uint32_t m, n, k, experts;
    const int32_t* offsets;
    void* y;
    uint64_t y_stride;
};

__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    uint32_t h = ((code & 7u) << 9) | ((code & 8u) << 12);
    return __half2float(__ushort_as_half((unsigned short)h)) * 16384.0f;
}

__device__ __forceinline__ float value_at(const dcr_nvfp4& a, uint64_t row, uint32_t k, uint32_t i)
{
    uint32_t c = static_cast<const uint8_t*>(a.codes)[(row * k + i) / 2] >> (4 * (i % 2));
    __nv_fp8_e4m3 s;
    s.__x = static_cast<const uint8_t*>(a.scales)[row * (k / 16) + i / 16];
    return e2m1_value(c & 15u) * float(s);
}

// A 32x32 tile of y a block, 4 values a thread, operands spread to 32 bits in
// shared memory.
template <typename T>
__global__ void __launch_bounds__(256) matmul_kernel(MatmulArgs A)
{
    __shared__ float xs[32][33], ws[32][33];
    const uint32_t e = blockIdx.z;
    int64_t lo = 0, hi = A.m;
    if (A.offsets) {
        lo = min(max(int64_t(A.offsets[e]), int64_t(0)), int64_t(A.m));
        hi = min(max(int64_t(A.offsets[e + 1]), int64_t(0)), int64_t(A.m));
    }
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const uint32_t n0 = blockIdx.x * 32;
    for (int64_t m0 = lo + 32ll * blockIdx.y; m0 < hi; m0 += 32ll * gridDim.y) {
        float acc[4] = {};
        for (uint32_t k0 = 0; k0 < A.k; k0 += 32) {
            for (int i = ty; i < 32; i += 8) {
                xs[i][tx] = m0 + i < hi ? value_at(A.x, m0 + i, A.k, k0 + tx) : 0.0f;
                ws[i][tx] = n0 + i < A.n ? value_at(A.w, uint64_t(e) * A.n + n0 + i, A.k, k0 + tx) : 0.0f;
            }
            __syncthreads();
            for (int q = 0; q < 32; ++q)
                for (int i = 0; i < 4; ++i) acc[i] += xs[ty + 8 * i][q] * ws[tx][q];
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i) {
            int64_t r = m0 + ty + 8 * i;
            if (r < hi && n0 + tx < A.n)
                static_cast<T*>(A.y)[r * A.y_stride + n0 + tx] = from_f32<T>(
                    acc[i] * (A.x.scale[A.x.scale_count > 1 ? r : 0] * A.w.scale[A.w.scale_count > 1 ? e : 0]));
        }
    }
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_nvfp4_matmul(const dcr_nvfp4* x, const dcr_nvfp4* w, uint64_t m, uint64_t n, uint64_t k,
                                const int32_t* offsets, uint32_t experts, void* y, uint32_t dtype, uint64_t y_stride,
                                void* stream)
{
    if (!x || !w) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: NULL argument");
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: unknown dtype %u", dtype);
    if (k == 0 || k % 32) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: k must be a positive multiple of 32");
    if (experts > DCR_MAX_EXPERTS) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: more than %u experts", DCR_MAX_EXPERTS);
    if ((experts > 0) != (offsets != nullptr))
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: experts and offsets do not go together");
    const uint64_t wrows = n * (experts ? experts : 1);
    if (m >= 1ull << 31 || n >= 1ull << 31 || k >= 1ull << 31 || wrows >= 1ull << 31 || y_stride >= 1ull << 40)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: matrix too large");
    if (y_stride < n) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: y_stride below n");
    if (x->scale_count != 1 && x->scale_count != m)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: x needs one scale or one per row");
    if (w->scale_count != 1 && (experts == 0 || w->scale_count != experts))
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: w needs one scale or one per expert");
    if (m == 0 || n == 0) return DCR_OK;
    if (!x->codes || !x->scales || !x->scale || !w->codes || !w->scales || !w->scale || !y)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: NULL argument");
    if (uintptr_t(x->codes) % 16 || uintptr_t(w->codes) % 16 || uintptr_t(y) % dtype_size(dtype) ||
        uintptr_t(x->scale) % 4 || uintptr_t(w->scale) % 4 || uintptr_t(offsets) % 4)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: misaligned buffer");
    MatmulArgs A{*x, *w, uint32_t(m), uint32_t(n), uint32_t(k), experts, offsets, y, y_stride};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    dim3 grid(unsigned((n + 31) / 32), unsigned(m < 32 * 512 ? (m + 31) / 32 : 512), experts ? experts : 1);
    with_dtype(dtype, [&](auto t) { matmul_kernel<decltype(t)><<<grid, 256, 0, s>>>(A); });
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "NVFP4 product launch");
}
