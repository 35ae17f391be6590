// NVFP4 quantisation: e2m1 codes, an e4m3 scale per 16 values and a 32-bit
// scale per matrix or row (the formulas stand in include/dcr_ops.h).
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "ops_internal.h"

namespace dcr {
namespace {

constexpr float kInvMax = 1.0f / 2688.0f;   // 1 / (largest code * largest scale)
constexpr float kFltMax = 3.402823466e38f;

struct QuantArgs {
    const void* x;
    float* scale;
    const float* partial;   // TENSOR: per block of amax_kernel, the largest t
    uint8_t* codes;
    uint8_t* scales;
    void* values;
    uint64_t rows, row_stride;
    uint64_t blocks;        // of 16 values, in the matrix
    uint32_t bpr;           // in a row
    uint32_t n_partial;
};

// t of a matrix or row from its largest finite |x|: amax * kInvMax grows with
// amax also after rounding, so the maximum may be taken over either.
__device__ __forceinline__ float scale_or_one(float t) { return t > 0.0f ? t : 1.0f; }

// Two fp32 values to two e2m1 codes in a byte, `lo` in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{ .reg .b8 b; cvt.rn.satfinite.e2m1x2.f32 b, %1, %2; cvt.u32.u8 %0, b; }" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The raw words of one block of 16 values, in memory order.
template <typename T>
struct Raw {
    static constexpr int kWords = sizeof(T) * 4;
    uint32_t w[kWords];
};

__device__ __forceinline__ void unpack(const Raw<float>& r, float (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = __uint_as_float(r.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw<__half>& r, float (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// One block from memory.  VEC: every row starts on a 16-byte boundary.
// Otherwise the 16-byte words around the block are read and shifted into
// place where they lie inside the matrix (from `lo` to `hi`), and single
// values at its two ends.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load_block(const T* p, const uint8_t* lo, const uint8_t* hi)
{
    constexpr int W = Raw<T>::kWords;
    Raw<T> r;
    if (VEC) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
            r.w[4 * i] = q.x, r.w[4 * i + 1] = q.y, r.w[4 * i + 2] = q.z, r.w[4 * i + 3] = q.w;
        }
        return r;
    }
    const uint32_t off = uintptr_t(p) & 15;
    const uint8_t* a = reinterpret_cast<const uint8_t*>(p) - off;
    if (a >= lo && a + 4 * W + 16 <= hi) {
        uint32_t w[W + 4];
#pragma unroll
        for (int i = 0; i < W / 4 + 1; ++i) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(a) + i);
            w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
#pragma unroll
        for (int i = 0; i < W + 2; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < W + 1; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (off & 3));
        return r;
    }
    if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = uint32_t(h[2 * i]) | uint32_t(h[2 * i + 1]) << 16;
    }
    return r;
}

// The largest finite |x| of a block (infinities and NaN count as 0): the
// bits of |x| order as the values do.
template <typename T>
__device__ __forceinline__ float finite_amax(const Raw<T>& r)
{
    float v[16];
    unpack(r, v);
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]));   // a NaN is passed over
    if (a > kFltMax) {
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(v[i]) <= kFltMax ? fabsf(v[i]) : 0.0f);
    }
    return a;
}

__device__ __forceinline__ float warp_max(float a)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
    return a;
}

template <int THREADS>
__device__ __forceinline__ float block_max(float a)
{
    __shared__ float part[THREADS / 32];
    a = warp_max(a);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) a = fmaxf(a, part[i]);
    return a;
}

// One block of 16 quantised and written: its scale byte, 8 bytes of codes
// and, with values, what they stand for.
template <typename T, typename V, bool VALUES>
__device__ __forceinline__ void quantize_block(const QuantArgs& A, uint64_t b, const Raw<T>& raw, float t)
{
    float v[16];
    unpack(raw, v);
    float a = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        a = fmaxf(a, fabsf(v[i]));
        nan |= v[i] != v[i];
    }
    const float u = fminf(__fdiv_rn(a, __fmul_rn(6.0f, t)), 448.0f);
    const __nv_fp8_e4m3 s8(u);
    float st = __fmul_rn(float(s8), t);
    const float r = st > 0.0f ? fminf(__frcp_rn(st), kFltMax) : 0.0f;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i / 4] |= e2m1x2(__fmul_rn(v[2 * i], r), __fmul_rn(v[2 * i + 1], r)) << (8 * (i % 4));
    reinterpret_cast<uint2*>(A.codes)[b] = make_uint2(c[0], c[1]);
    A.scales[b] = nan ? 0x7F : uint8_t(s8.__x);
    if (!VALUES) return;
    if (nan) st = __int_as_float(0x7FFFFFFF);
    alignas(16) V o[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // the magnitudes' upper 16 bits as 32-bit floats, looked up bytewise: four codes a lookup
        const uint32_t m = c[h] & 0x77777777u;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t sel = m >> (16 * q), cc = c[h] >> (16 * q);
            const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel), lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
            const uint32_t w0 = __byte_perm(lo, hi, 0x5140) | ((cc << 12) & 0x8000u) | ((cc << 24) & 0x80000000u);
            const uint32_t w1 = __byte_perm(lo, hi, 0x7362) | ((cc << 4) & 0x8000u) | ((cc << 16) & 0x80000000u);
            const int i = 8 * h + 4 * q;
            o[i] = from_f32<V>(__fmul_rn(__uint_as_float(w0 << 16), st));
            o[i + 1] = from_f32<V>(__fmul_rn(__uint_as_float(w0 & 0xFFFF0000u), st));
            o[i + 2] = from_f32<V>(__fmul_rn(__uint_as_float(w1 << 16), st));
            o[i + 3] = from_f32<V>(__fmul_rn(__uint_as_float(w1 & 0xFFFF0000u), st));
        }
    }
    uint4* out = reinterpret_cast<uint4*>(static_cast<V*>(A.values) + 16 * b);
#pragma unroll
    for (int i = 0; i < int(sizeof(o) / 16); ++i) out[i] = reinterpret_cast<const uint4*>(o)[i];
}

// Where block b lies.  FLAT: the rows follow each other without a gap.
template <typename T, bool FLAT>
__device__ __forceinline__ const T* block_at(const QuantArgs& A, uint64_t b)
{
    const T* x = static_cast<const T*>(A.x);
    if (FLAT) return x + 16 * b;
    uint64_t row;
    uint32_t in;
    if (A.blocks >> 32) {
        row = b / A.bpr;
        in = uint32_t(b - row * A.bpr);
    } else {
        const uint32_t r = uint32_t(b) / A.bpr;
        row = r;
        in = uint32_t(b) - r * A.bpr;
    }
    return x + row * A.row_stride + 16ull * in;
}

template <typename T>
__device__ __forceinline__ const uint8_t* matrix_end(const QuantArgs& A)
{
    return reinterpret_cast<const uint8_t*>(static_cast<const T*>(A.x) + (A.rows - 1) * A.row_stride + 16ull * A.bpr);
}

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // blocks of 16 a thread has in flight

// Bound by reading x once: 131072 x 6144 bf16 in 226 us (7.1 TB/s).  Each
// block leaves its largest t; there are no atomics and nothing has to be
// cleared before.
template <typename T, bool VEC, bool FLAT>
__global__ void __launch_bounds__(kThreads) amax_kernel(QuantArgs A, float* partial)
{
    const uint8_t *lo = static_cast<const uint8_t*>(A.x), *hi = matrix_end<T>(A);
    launch_dependents();
    float a = 0.0f;
    const uint64_t step = uint64_t(gridDim.x) * kThreads;
    for (uint64_t b = uint64_t(blockIdx.x) * kThreads + threadIdx.x; b < A.blocks; b += kUnroll * step) {
        Raw<T> r[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (b + i * step < A.blocks) r[i] = load_block<T, VEC>(block_at<T, FLAT>(A, b + i * step), lo, hi);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (b + i * step < A.blocks) a = fmaxf(a, finite_amax(r[i]));
    }
    a = block_max<kThreads>(a);
    if (threadIdx.x == 0) partial[blockIdx.x] = __fmul_rn(a, kInvMax);
}

// GIVEN and TENSOR: bound by reading x and writing the outputs: 131072 x 6144
// bf16 with bf16 values in 567 us (6.5 TB/s); both passes 809 us, against 541
// for the bytes read and written once and 778 with the second read.  Four
// blocks of 16 a thread are in flight.  TENSOR runs
// through the matrix from its end, where amax_kernel has just left off, so
// that what the L2 still holds is read from there.
template <typename T, typename V, int MODE, bool VALUES, bool VEC, bool FLAT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(QuantArgs A)
{
    const uint8_t *lo = static_cast<const uint8_t*>(A.x), *hi = matrix_end<T>(A);
    float t;
    if (MODE == DCR_SCALE_TENSOR) {
        grid_wait();
        t = 0.0f;
        for (uint32_t i = threadIdx.x; i < A.n_partial; i += kThreads) t = fmaxf(t, A.partial[i]);
        t = scale_or_one(block_max<kThreads>(t));
        if (blockIdx.x == 0 && threadIdx.x == 0) *A.scale = t;
    } else {
        t = *A.scale;
    }
    const uint64_t step = uint64_t(gridDim.x) * kThreads;
    for (uint64_t b = uint64_t(blockIdx.x) * kThreads + threadIdx.x; b < A.blocks; b += kUnroll * step) {
        Raw<T> r[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const uint64_t at = b + i * step;
            if (at < A.blocks)
                r[i] = load_block<T, VEC>(block_at<T, FLAT>(A, MODE == DCR_SCALE_TENSOR ? A.blocks - 1 - at : at), lo, hi);
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const uint64_t at = b + i * step;
            if (at < A.blocks) quantize_block<T, V, VALUES>(A, MODE == DCR_SCALE_TENSOR ? A.blocks - 1 - at : at, r[i], t);
        }
    }
}

constexpr int kRowBlocks = 4;   // blocks of 16 a thread keeps in registers

// ROW, bound by reading x and writing the outputs (4096 x 14336 bf16: 31 us,
// 4.8 TB/s; small calls by the latency of one row, 333 x 6144: 5.3 us): TPR threads a row (a warp, or the whole block), which keep the row in
// registers between its maximum and its codes; what a longer row has beyond
// that is read again.
template <typename T, typename V, int TPR, bool VALUES, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(QuantArgs A)
{
    const uint8_t *lo = static_cast<const uint8_t*>(A.x), *hi = matrix_end<T>(A);
    const uint32_t lane = threadIdx.x % TPR;
    launch_dependents();
    for (uint64_t row = uint64_t(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR; row < A.rows;
         row += uint64_t(gridDim.x) * (kThreads / TPR)) {
        const T* x = static_cast<const T*>(A.x) + row * A.row_stride;
        Raw<T> r[kRowBlocks];
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i)
            if (lane + i * TPR < A.bpr) r[i] = load_block<T, VEC>(x + 16ull * (lane + i * TPR), lo, hi);
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i)
            if (lane + i * TPR < A.bpr) a = fmaxf(a, finite_amax(r[i]));
        for (uint32_t b = lane + kRowBlocks * TPR; b < A.bpr; b += TPR)
            a = fmaxf(a, finite_amax(load_block<T, VEC>(x + 16ull * b, lo, hi)));
        if (TPR == 32) a = warp_max(a);
        else a = block_max<kThreads>(a);
        const float t = scale_or_one(__fmul_rn(a, kInvMax));
        if (lane == 0) A.scale[row] = t;
        const uint64_t at = row * A.bpr;
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i)
            if (lane + i * TPR < A.bpr) quantize_block<T, V, VALUES>(A, at + lane + i * TPR, r[i], t);
        for (uint32_t b = lane + kRowBlocks * TPR; b < A.bpr; b += TPR)
            quantize_block<T, V, VALUES>(A, at + b, load_block<T, VEC>(x + 16ull * b, lo, hi), t);
        if (TPR != 32) __syncthreads();   // block_max's words are used again
    }
}

template <typename F>
auto with_bool(bool v, F f)
{
    return v ? f(std::true_type()) : f(std::false_type());
}

// By the launch's own status: the thread's last error may be another call's.
template <typename K, typename... X>
cudaError_t go(K kernel, unsigned grid, bool dependent, cudaStream_t s, const X&... args)
{
    const LaunchAttrs at(grid, kThreads, 0, 1, dependent, s);
    return cudaLaunchKernelEx(&at.cfg, kernel, args...);
}

template <typename T, typename V, bool VALUES>
cudaError_t launch(const QuantArgs& A, uint32_t mode, float* partial, cudaStream_t s)
{
    const bool vec = uintptr_t(A.x) % 16 == 0 && A.row_stride * sizeof(T) % 16 == 0;
    const bool flat = A.row_stride == 16ull * A.bpr || A.rows == 1;
    if (mode == DCR_SCALE_ROW) {
        const uint64_t per = A.bpr <= 32 * kRowBlocks ? kThreads / 32 : 1, want = (A.rows + per - 1) / per;
        const unsigned grid = unsigned(want < 1u << 20 ? want : 1u << 20);
        return with_bool(vec, [&](auto ve) {
            if (per == 1) return go(quantize_rows_kernel<T, V, kThreads, VALUES, ve.value>, grid, false, s, A);
            return go(quantize_rows_kernel<T, V, 32, VALUES, ve.value>, grid, false, s, A);
        });
    }
    const uint64_t want = (A.blocks + kThreads - 1) / kThreads;
    const unsigned grid = unsigned(want < DCR_QUANT_PARTIALS ? want : DCR_QUANT_PARTIALS);
    return with_bool(vec, [&](auto ve) {
        return with_bool(flat, [&](auto fl) {
            if (mode != DCR_SCALE_TENSOR)
                return go(quantize_kernel<T, V, DCR_SCALE_GIVEN, VALUES, ve.value, fl.value>, grid, false, s, A);
            QuantArgs B = A;
            B.partial = partial;
            B.n_partial = grid;
            const cudaError_t e = go(amax_kernel<T, ve.value, fl.value>, grid, false, s, A, partial);
            if (e != cudaSuccess) return e;
            return go(quantize_kernel<T, V, DCR_SCALE_TENSOR, VALUES, ve.value, fl.value>, grid, true, s, B);
        });
    });
}

}  // namespace

int quantize_launch(const void* x, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t row_stride, uint32_t scale_mode,
                    float* scale, void* codes, void* scales, void* values, uint32_t values_dtype, void* workspace,
                    cudaStream_t s)
{
    QuantArgs A{x, scale, nullptr, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), values, rows, row_stride,
                rows * (cols / 16), uint32_t(cols / 16), 0};
    float* partial = static_cast<float*>(workspace);
    const cudaError_t e = with_dtype(dtype, [&](auto t) {
        if (!values) return launch<decltype(t), float, false>(A, scale_mode, partial, s);
        return with_dtype(values_dtype, [&](auto v) { return launch<decltype(t), decltype(v), true>(A, scale_mode, partial, s); });
    });
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "NVFP4 quantise launch");
}

}  // namespace dcr

using namespace dcr;

extern "C" int dcr_nvfp4_quantize(const void* x, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t row_stride,
                                  uint32_t scale_mode, float* scale, void* codes, void* scales, void* values,
                                  uint32_t values_dtype, void* workspace, void* stream)
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
    if (!x || !scale || !codes || !scales || (scale_mode == DCR_SCALE_TENSOR && !workspace))
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: NULL argument");
    if (uintptr_t(codes) % 16 || uintptr_t(values) % 16 || uintptr_t(scale) % 4 || uintptr_t(workspace) % 4 || uintptr_t(x) % dtype_size(dtype))
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_quantize: misaligned buffer");
    return quantize_launch(x, dtype, rows, cols, row_stride, scale_mode, scale, codes, scales, values, values_dtype,
                           workspace, static_cast<cudaStream_t>(stream));
}
