// Internal definitions shared by the operators of include/dcr_ops.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/dcr_ops.h"

namespace dcr {

int set_error(int code, const char* fmt, ...);
int cuda_error(cudaError_t e, const char* what);

inline uint32_t dtype_size(uint32_t d) { return d == DCR_F32 ? 4 : 2; }

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// Calls f with a value of the element type that `dtype` names.
template <typename F>
auto with_dtype(uint32_t dtype, F f)
{
    if (dtype == DCR_BF16) return f(__nv_bfloat16());
    if (dtype == DCR_F16) return f(__half());
    return f(float());
}

}  // namespace dcr
