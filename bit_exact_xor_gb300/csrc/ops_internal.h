// Internal definitions shared by the operators of include/dcr_ops.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/dcr_ops.h"
#include "overlap.h"

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

// Programmatic dependent launch: a kernel of one call that follows another of
// the same call is launched while that one still runs (launch_dependents),
// and waits for its end and its writes (grid_wait) before it reads them.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Attributes of a launch: blocks of a cluster, and whether it may begin
// before the kernel ahead of it in the stream has ended.
struct LaunchAttrs {
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = {};
    LaunchAttrs(uint64_t grid, unsigned threads, size_t smem, unsigned cluster, bool dependent, cudaStream_t s)
    {
        cfg.gridDim = dim3(unsigned(grid));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = at;
        if (cluster > 1) {
            at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            at[cfg.numAttrs].val.clusterDim.x = cluster;
            at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
            ++cfg.numAttrs;
        }
        if (dependent) {
            at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
            ++cfg.numAttrs;
        }
    }
};

// Launches of the operators' kernels with checked arguments (dcr_nvfp4_linear
// is the two of them).
int quantize_launch(const void* x, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t row_stride, uint32_t scale_mode,
                    float* scale, void* codes, void* scales, void* values, uint32_t values_dtype, void* workspace,
                    cudaStream_t s);
int matmul_launch(const dcr_nvfp4& x, const dcr_nvfp4& w, uint64_t m, uint64_t n, uint64_t k, const int32_t* offsets,
                  uint32_t experts, void* y, uint32_t dtype, uint64_t y_stride, bool dependent, cudaStream_t s);

// Calls f with a value of the element type that `dtype` names.
template <typename F>
auto with_dtype(uint32_t dtype, F f)
{
    if (dtype == DCR_BF16) return f(__nv_bfloat16());
    if (dtype == DCR_F16) return f(__half());
    return f(float());
}

}  // namespace dcr
