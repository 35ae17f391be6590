// NVFP4 quantisation: e2m1 codes, an e4m3 scale per 16 values and a 32-bit
// scale per matrix or row (the formulas stand in include/dcr_ops.h).
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "ops_internal.h"

namespace dcr {
namespace {

constexpr float kInvMax = 1.0f / 2688.0f;   // 1 / (largest code * largest scale)
constexpr float kFltMax = 3.402823466e38f;

struct QuantArgs {
    const void* x;
    float* scale;
    uint8_t* codes;
    uint8_t* scales;
    void* values;
    uint64_t rows, cols, row_stride;
};

__device__ __forceinline__ float finite_abs(float v)
{
    float a = fabsf(v);
    return a <= kFltMax ? a : 0.0f;   // infinities and NaN count as 0
}

// t of a matrix or row from its largest finite |x|; amax * kInvMax rounds to
// a t that grows with amax, so a maximum may be taken over either.
__device__ __forceinline__ float scale_or_one(float t) { return t > 0.0f ? t : 1.0f; }

// Two fp32 values to two e2m1 codes in a byte, `lo` in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{ .reg .b8 b; cvt.rn.satfinite.e2m1x2.f32 b, %1, %2; cvt.u32.u8 %0, b; }" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One block of 16: its scale byte, 8 bytes of codes, and s * t.
__device__ __forceinline__ void quantize_block(const float (&v)[16], float t, uint32_t& scale, uint2& codes, float& st)
{
    float a = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        a = fmaxf(a, fabsf(v[i]));
        nan |= v[i] != v[i];
    }
    float u = fminf(__fdiv_rn(a, __fmul_rn(6.0f, t)), 448.0f);
    __nv_fp8_e4m3 s8(u);
    scale = nan ? 0x7Fu : uint32_t(s8.__x);
    float s = float(s8);
    st = __fmul_rn(s, t);
    float r = st > 0.0f ? fminf(__frcp_rn(st), kFltMax) : 0.0f;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i / 4] |= e2m1x2(__fmul_rn(v[2 * i], r), __fmul_rn(v[2 * i + 1], r)) << (8 * (i % 4));
    codes = make_uint2(c[0], c[1]);
    if (nan) st = __int_as_float(0x7FFFFFFF);
}

// The value of an e2m1 code: its 2-bit exponent and 1-bit mantissa sit at the
// top of a half's exponent and mantissa once moved there; the bias differs by
// 14, so a product with 2^14 corrects it (subnormal codes come out right too).
__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    uint32_t h = ((code & 7u) << 9) | ((code & 8u) << 12);
    return __half2float(__ushort_as_half((unsigned short)h)) * 16384.0f;
}

template <typename T>
__global__ void amax_kernel(const T* x, uint64_t rows, uint64_t cols, uint64_t row_stride, int* scale)
{
    float a = 0.0f;
    uint64_t n = rows * cols;
    for (uint64_t i = uint64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += uint64_t(gridDim.x) * blockDim.x)
        a = fmaxf(a, finite_abs(to_f32(x[(i / cols) * row_stride + i % cols])));
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
    // non-negative floats order as their bits do: the maximum does not depend on the order of the atomics
    if (threadIdx.x % 32 == 0 && a > 0.0f) atomicMax(scale, __float_as_int(__fmul_rn(a, kInvMax)));
}

template <typename T, typename V, int MODE>
__global__ void quantize_kernel(QuantArgs A)
{
    const uint32_t bpr = uint32_t(A.cols / 16);
    for (uint64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(A.x) + row * A.row_stride;
        float t;
        if (MODE == DCR_SCALE_ROW) {
            __shared__ float part[32];
            float a = 0.0f;
            for (uint64_t i = threadIdx.x; i < A.cols; i += blockDim.x) a = fmaxf(a, finite_abs(to_f32(x[i])));
            for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
            if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = a;
            __syncthreads();
            for (uint32_t i = 0; i < blockDim.x / 32; ++i) a = fmaxf(a, part[i]);
            __syncthreads();
            t = scale_or_one(__fmul_rn(a, kInvMax));
            if (threadIdx.x == 0) A.scale[row] = t;
        } else {
            t = *(volatile const float*)A.scale;
            if (MODE == DCR_SCALE_TENSOR) {
                // 0 (nothing above 0) stands for 1; a block that reads the 1 already written agrees
                if (t == 0.0f && row == 0 && threadIdx.x == 0) *(volatile float*)A.scale = 1.0f;
                t = scale_or_one(t);
            }
        }
        for (uint32_t b = threadIdx.x; b < bpr; b += blockDim.x) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = to_f32(x[16ull * b + i]);
            uint32_t s;
            uint2 c;
            float st;
            quantize_block(v, t, s, c, st);
            uint64_t at = row * bpr + b;
            reinterpret_cast<uint2*>(A.codes)[at] = c;
            A.scales[at] = uint8_t(s);
            if (A.values) {
                V* out = static_cast<V*>(A.values) + 16 * at;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    out[i] = from_f32<V>(__fmul_rn(e2m1_value(((i < 8 ? c.x : c.y) >> (4 * (i % 8))) & 15u), st));
            }
        }
    }
}

template <typename T>
int quantize(const QuantArgs& A, uint32_t mode, uint32_t values_dtype, cudaStream_t s)
{
    if (mode == DCR_SCALE_TENSOR) {
        cudaError_t e = cudaMemsetAsync(A.scale, 0, 4, s);
        if (e != cudaSuccess) return cuda_error(e, "clearing the scale");
        uint64_t want = (A.rows * A.cols + 1023) / 1024;
        amax_kernel<T><<<unsigned(want < 2432 ? want : 2432), 256, 0, s>>>(static_cast<const T*>(A.x), A.rows, A.cols,
                                                                            A.row_stride, reinterpret_cast<int*>(A.scale));
    }
    unsigned grid = unsigned(A.rows < 65536 ? A.rows : 65536);
    with_dtype(values_dtype, [&](auto v) {
        using V = decltype(v);
        if (mode == DCR_SCALE_ROW) quantize_kernel<T, V, DCR_SCALE_ROW><<<grid, 128, 0, s>>>(A);
        else if (mode == DCR_SCALE_TENSOR) quantize_kernel<T, V, DCR_SCALE_TENSOR><<<grid, 128, 0, s>>>(A);
        else quantize_kernel<T, V, DCR_SCALE_GIVEN><<<grid, 128, 0, s>>>(A);
    });
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "NVFP4 quantise launch");
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_nvfp4_quantize(const void* x, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t row_stride,
                                  uint32_t scale_mode, float* scale, void* codes, void* scales, void* values,
                                  uint32_t values_dtype, void* stream)
{
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: unknown dtype %u", dtype);
    if (scale_mode > DCR_SCALE_ROW) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: unknown scale mode %u", scale_mode);
    if (cols % 16) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: cols must be a multiple of 16");
    if (rows >= 1ull << 32 || cols >= 1ull << 32 || row_stride >= 1ull << 40)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: matrix too large");
    if (row_stride < cols) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: row_stride below cols");
    if (rows == 0 || cols == 0) return DCR_OK;
    if ((values != nullptr) != (values_dtype <= DCR_F16))
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: values and values_dtype do not go together");
    if (!x || !scale || !codes || !scales) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: NULL argument");
    if (uintptr_t(codes) % 16 || uintptr_t(values) % 16 || uintptr_t(scale) % 4 || uintptr_t(x) % dtype_size(dtype))
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: misaligned buffer");
    QuantArgs A{x, scale, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), values, rows, cols, row_stride};
    return with_dtype(dtype, [&](auto t) {
        return quantize<decltype(t)>(A, scale_mode, values_dtype, static_cast<cudaStream_t>(stream));
    });
}
