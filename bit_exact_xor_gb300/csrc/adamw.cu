// The trainer's step: the norm of all gradients, and AdamW over many tensors
// at once with moments in 32 or 8 bits (include/dcr_ops.h).
//
// The tensors' addresses travel as a kernel parameter (up to 424 of them a
// launch), so that a call copies nothing to the device and can be captured.  A
// block takes a chunk of one tensor, a warp 256 consecutive values of it at a
// time: the block of values that shares a scale of an 8-bit moment, 8 a lane.
// The loads of a warp's next values come before the arithmetic on these.
//
// Moments in 32 bits are bound by DRAM: 235 million values in 195 tensors (16-bit
// gradients and copies) in 958 us, 6.9 TB/s of what it moves.  Their norm takes
// 79 (6.0 TB/s): a block has no loads under way between two chunks.  Moments in 8
// bits are bound by instruction issue, 82 instructions a value, of which a
// correctly rounded root and quotient are a third: 185 million values in 574 us,
// 5.1 TB/s (685 without the loads ahead).
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <vector>

#include "ops_internal.h"

namespace dcr {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kBlock = DCR_ADAMW_BLOCK;     // values a warp takes at a time
constexpr uint32_t kRound = kThreads / 32 * kBlock;

// A table of tensors as a kernel's parameter: a call with few of them does not carry the space of many.
constexpr int kFew = 48, kMany = 424;

struct Entry {
    dcr_adamw_tensor t;
    uint64_t first;       // the call's values before this tensor
};
template <int N>
struct Table {
    Entry e[N];
    uint32_t chunk[N + 1];   // the launch's chunks before each tensor
    uint32_t count;
};

struct AdamwArgs {
    float beta1, beta2, rest1, rest2, eps, decay, step_size, inv_root;   // rest: 1 - beta; inv_root: 1 / sqrt(1 - beta2^step)
    float grad_scale, max_norm, lr, weight_decay, log1, log2;
    const float* norm;
    const int64_t* step_at;
    const float* lr_at;
    uint64_t step;
    uint32_t per;         // values a chunk
    uint32_t seed;
    uint32_t w_half, g_half;   // 16-bit weights and gradients are f16
    uint32_t copy_dtype;
};

// 32 bits that depend on every bit of x: the output function of a permuted
// congruential generator (O'Neill 2014) behind one step of it.
__device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x = x * 747796405u + 2891336453u;
    x = ((x >> ((x >> 28) + 4)) ^ x) * 277803737u;
    return (x >> 22) ^ x;
}

// 8 values of a lane, as they lie in memory.
template <int BYTES>
struct Raw8 {
    uint32_t w[2 * BYTES];
};

__device__ __forceinline__ void load(Raw8<4>& r, const void* p)
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p));
}
__device__ __forceinline__ void load(Raw8<2>& r, const void* p)
{
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "l"(p));
}
__device__ __forceinline__ void load(Raw8<1>& r, const void* p)
{
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p));
}
__device__ __forceinline__ void store(const Raw8<4>& r, void* p)
{
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]),
                 "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7]), "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store(const Raw8<2>& r, void* p)
{
    asm volatile("st.global.v4.b32 [%4], {%0, %1, %2, %3};" ::"r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "l"(p) : "memory");
}
__device__ __forceinline__ void store(const Raw8<1>& r, void* p)
{
    asm volatile("st.global.v2.b32 [%2], {%0, %1};" ::"r"(r.w[0]), "r"(r.w[1]), "l"(p) : "memory");
}

// The lane's 8 values of the 256 from `at`: 8 consecutive ones where every
// pointer is aligned and all 256 there, else every 32nd, those below n.
template <bool VEC, int BYTES>
__device__ __forceinline__ void read8(Raw8<BYTES>& r, const void* base, uint64_t at, uint64_t n)
{
    const uint32_t lane = threadIdx.x % 32;
    if constexpr (VEC) {
        load(r, static_cast<const uint8_t*>(base) + (at + lane * 8) * BYTES);
    } else {
#pragma unroll
        for (int i = 0; i < 2 * BYTES; ++i) r.w[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t i = at + lane + 32 * j;
            if (i < n) {
                if (BYTES == 4) r.w[j % (2 * BYTES)] = static_cast<const uint32_t*>(base)[i];
                if (BYTES == 2) r.w[j * BYTES / 4] |= uint32_t(static_cast<const uint16_t*>(base)[i]) << (16 * (j % 2));
                if (BYTES == 1) r.w[j * BYTES / 4] |= uint32_t(static_cast<const uint8_t*>(base)[i]) << (8 * (j % 4));
            }
        }
    }
}
template <bool VEC, int BYTES>
__device__ __forceinline__ void write8(const Raw8<BYTES>& r, void* base, uint64_t at, uint64_t n)
{
    const uint32_t lane = threadIdx.x % 32;
    if constexpr (VEC) {
        store(r, static_cast<uint8_t*>(base) + (at + lane * 8) * BYTES);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t i = at + lane + 32 * j;
            if (i < n) {
                if (BYTES == 4) static_cast<uint32_t*>(base)[i] = r.w[j % (2 * BYTES)];
                if (BYTES == 2) static_cast<uint16_t*>(base)[i] = uint16_t(r.w[j * BYTES / 4] >> (16 * (j % 2)));
                if (BYTES == 1) static_cast<uint8_t*>(base)[i] = uint8_t(r.w[j * BYTES / 4] >> (8 * (j % 4)));
            }
        }
    }
}

__device__ __forceinline__ void values(const Raw8<4>& r, float2 (&v)[4], bool)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
}
__device__ __forceinline__ void values(const Raw8<2>& r, float2 (&v)[4], bool half)
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = half ? __half22float2(*reinterpret_cast<const __half2*>(&r.w[j]))
                    : make_float2(__uint_as_float(r.w[j] << 16), __uint_as_float(r.w[j] & 0xFFFF0000u));
}
// e4m3 codes
__device__ __forceinline__ void values(const Raw8<1>& r, float2 (&v)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(r.w[j / 2] >> (16 * (j % 2))), __NV_E4M3);
        v[j] = __half22float2(__half2(h));
    }
}
__device__ __forceinline__ Raw8<4> packed(const float2 (&v)[4], Raw8<4>, bool)
{
    Raw8<4> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[2 * j] = __float_as_uint(v[j].x), r.w[2 * j + 1] = __float_as_uint(v[j].y);
    return r;
}
__device__ __forceinline__ Raw8<2> packed(const float2 (&v)[4], Raw8<2>, bool half)
{
    Raw8<2> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (half) {
            const __half2 h = __float22half2_rn(v[j]);
            r.w[j] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 b = __float22bfloat162_rn(v[j]);
            r.w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
    return r;
}

// Two products in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t r;
    asm("{ .reg .b64 x, y; mov.b64 x, {%1, %2}; mov.b64 y, {%3, %4}; mul.rn.f32x2 %0, x, y; }" : "=l"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
    return f;
}
// Not in one instruction: that would be merged with the product into a
// multiply-add, which rounds once.
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The largest magnitude of three, NaN if one is.
__device__ __forceinline__ float largest(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// The scale of a block of 256 values from the lanes' own, and 1 / it.
struct Scale {
    float s, inv;
    __device__ __forceinline__ explicit Scale(const float2 (&x)[4])
    {
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = largest(a, x[j].x, x[j].y);
        // magnitudes order as their bits do, NaN above all
        s = __fmul_rn(__uint_as_float(__reduce_max_sync(~0u, __float_as_uint(a) & 0x7FFFFFFFu)), 1.0f / 448.0f);
        if (!(s <= FLT_MAX)) s = NAN;
        inv = s > 0.0f ? fminf(__frcp_rn(s), FLT_MAX) : 0.0f;
    }
};

// |x| inv as e4m3 codes, in the last byte: a value of e4m3 is one of 32 bits
// whose exponent is 120 larger, cut to 3 bits of mantissa; 16 random bits, a
// half below their last one, are added to what is cut off.  That is at most
// 2^20 - 8 units of the last place of 448, so that a largest value less than 8
// above 448 keeps 448's code and does not become a NaN's.  It is within three
// where the scale is a normal number.  A subnormal one (largest values of 1.3e-36
// to 5.3e-36) is itself off by up to 2^-22 of it, 3.5 units instead of 0.9, which
// makes six; below, 1 / scale is cut to the largest number, and values are
// smaller.  (A block that is not finite has a NaN for its scale, and any codes.)
__device__ __forceinline__ uint2 encode2(float2 x, float inv, uint32_t random0, uint32_t random1)
{
    const float2 y = mul2(mul2(make_float2(fabsf(x.x), fabsf(x.y)), both(inv)), both(0x1p-120f));
    return make_uint2((__float_as_uint(y.x) + random0 * 16) * 16 + 128, (__float_as_uint(y.y) + random1 * 16) * 16 + 128);
}

// What a whole launch shares.
struct Common {
    float coef, decay, step_size, inv_root;
    uint32_t key;
    bool skip;
    __device__ __forceinline__ explicit Common(const AdamwArgs& A)
    {
        coef = A.grad_scale;
        skip = false;
        if (A.norm) {
            const float n = *A.norm * fabsf(A.grad_scale);
            skip = !(n <= FLT_MAX);
            if (A.max_norm > 0.0f && n > A.max_norm) coef = __fmul_rn(A.grad_scale, __fdiv_rn(A.max_norm, n));
        }
        const float lr = A.lr_at ? *A.lr_at : A.lr;
        uint64_t step = A.step;
        decay = A.decay, step_size = A.step_size, inv_root = A.inv_root;
        if (A.step_at || A.lr_at) {
            if (A.step_at) step = uint64_t(max(*A.step_at, int64_t(1)));
            // 1 - beta^step as -(exp(step log beta) - 1), which keeps its digits where it is small
            const float t = float(step);
            decay = __fsub_rn(1.0f, __fmul_rn(lr, A.weight_decay));
            step_size = __fdiv_rn(lr, -expm1f(t * A.log1));
            inv_root = __frsqrt_rn(-expm1f(t * A.log2));
        }
        key = mix(mix(A.seed) + uint32_t(step));
    }
};

// What a lane reads of 256 values before it can begin; the weights come in
// meanwhile.
template <int GB, int BITS>
struct Loaded {
    Raw8<GB> g;
    Raw8<BITS / 8> m, v;
    float ms, vs;
    template <bool VEC>
    __device__ __forceinline__ void read(const Entry& E, uint64_t at)
    {
        read8<VEC>(g, E.t.grad, at, E.t.n);
        read8<VEC>(m, E.t.m, at, E.t.n);
        read8<VEC>(v, E.t.v, at, E.t.n);
        if (BITS == 8) ms = E.t.m_scale[at / kBlock], vs = E.t.v_scale[at / kBlock];
    }
};

template <int WB, int GB, int BITS, bool VEC>
__device__ __forceinline__ void update(const Entry& E, const AdamwArgs& A, const Common& C, uint64_t at, const Loaded<GB, BITS>& L)
{
    const uint64_t n = E.t.n;
    const uint32_t lane = threadIdx.x % 32;
    Raw8<WB> rw;
    read8<VEC>(rw, E.t.w, at, n);
    const Raw8<GB>& rg = L.g;
    const Raw8<BITS / 8>&rm = L.m, &rv = L.v;
    const float ms = L.ms, vs = L.vs;
    float2 w[4], g[4], m[4], v[4], root[4];
    values(rg, g, A.g_half);
    if constexpr (BITS == 8) {
        values(rm, m);
        values(rv, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = mul2(m[j], both(ms));
            v[j] = mul2(v[j], both(vs));
            v[j] = mul2(v[j], v[j]);
        }
    } else {
        values(rm, m, false);
        values(rv, v, false);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        g[j] = mul2(g[j], both(C.coef));
        m[j] = add2(mul2(m[j], both(A.beta1)), mul2(g[j], both(A.rest1)));
        v[j] = add2(mul2(v[j], both(A.beta2)), mul2(mul2(g[j], g[j]), both(A.rest2)));
        root[j] = make_float2(__fsqrt_rn(v[j].x), __fsqrt_rn(v[j].y));
        const float2 below = add2(mul2(root[j], both(C.inv_root)), both(A.eps));
        g[j] = make_float2(__fdiv_rn(m[j].x, below.x), __fdiv_rn(m[j].y, below.y));
    }
    values(rw, w, A.w_half);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = add2(mul2(w[j], both(C.decay)), mul2(g[j], both(-C.step_size)));
    write8<VEC>(packed(w, rw, A.w_half), E.t.w, at, n);
    if (A.copy_dtype == DCR_F32) write8<VEC>(packed(w, Raw8<4>(), false), E.t.copy, at, n);
    else if (A.copy_dtype != DCR_NONE) write8<VEC>(packed(w, Raw8<2>(), A.copy_dtype == DCR_F16), E.t.copy, at, n);
    if constexpr (BITS == 32) {
        write8<VEC>(packed(m, rm, false), E.t.m, at, n);
        write8<VEC>(packed(v, rv, false), E.t.v, at, n);
    } else {
        if (!VEC) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (at + lane + 64 * j >= n) m[j].x = root[j].x = 0.0f;
                if (at + lane + 64 * j + 32 >= n) m[j].y = root[j].y = 0.0f;
            }
        }
        const Scale sm(m), sv(root);
        // a random number for each value's number in the call, whose upper half is nearly always the same for all 256
        const uint64_t first = E.first + at;
        const uint32_t low = uint32_t(first), key = mix(C.key + uint32_t(first >> 32));
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = mix((low + (VEC ? lane * 8 + j : lane + 32 * j)) ^ key);
        if (low > 0xFFFFFFFFu - kBlock) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint64_t i = first + (VEC ? lane * 8 + j : lane + 32 * j);
                h[j] = mix(uint32_t(i) ^ mix(C.key + uint32_t(i >> 32)));
            }
        }
        Raw8<1> cm, cv;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t a[4], b[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 x = m[2 * i + j], y = root[2 * i + j];
                const uint32_t h0 = h[4 * i + 2 * j], h1 = h[4 * i + 2 * j + 1];
                const uint2 p = encode2(x, sm.inv, h0 & 0xFFFFu, h1 & 0xFFFFu);
                uint2 q = encode2(y, sv.inv, h0 >> 16, h1 >> 16);
                if (y.x != 0.0f) q.x = max(q.x, 1u << 24);
                if (y.y != 0.0f) q.y = max(q.y, 1u << 24);
                // the first moment's sign beside its code
                a[2 * j] = (p.x & 0x7FFFFFFFu) | (__float_as_uint(x.x) & 0x80000000u);
                a[2 * j + 1] = (p.y & 0x7FFFFFFFu) | (__float_as_uint(x.y) & 0x80000000u);
                b[2 * j] = q.x, b[2 * j + 1] = q.y;
            }
            cm.w[i] = __byte_perm(__byte_perm(a[0], a[1], 0x0073), __byte_perm(a[2], a[3], 0x0073), 0x5410);
            cv.w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0073), __byte_perm(b[2], b[3], 0x0073), 0x5410);
        }
        write8<VEC>(cm, E.t.m, at, n);
        write8<VEC>(cv, E.t.v, at, n);
        if (lane == 0) E.t.m_scale[at / kBlock] = sm.s, E.t.v_scale[at / kBlock] = sv.s;
    }
}

// The tensor that chunk c of a table lies in.
template <typename TABLE>
__device__ __forceinline__ uint32_t tensor_of(const TABLE& T, uint32_t c)
{
    uint32_t lo = 0, hi = T.count;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (T.chunk[mid] <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

// 8 bits: 64 registers, for four blocks an SM (80 and three: 596 us; the weights
// loaded ahead, too, which spills: 589; two rounds unrolled, without moves
// between them: 671).
template <int WB, int GB, int BITS, int N>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 4 : 2) adamw_kernel(const __grid_constant__ Table<N> T, const AdamwArgs A)
{
    const Common C(A);
    if (C.skip) return;
    const uint32_t k = tensor_of(T, blockIdx.x);
    const Entry E = T.e[k];
    const uint64_t begin = uint64_t(blockIdx.x - T.chunk[k]) * A.per, end = min(begin + A.per, E.t.n);
    // 8 consecutive values of each kind as one access
    const uintptr_t odd = (uintptr_t(E.t.w) & (8 * WB - 1)) | (uintptr_t(E.t.grad) & (8 * GB - 1)) | ((uintptr_t(E.t.m) | uintptr_t(E.t.v)) & (BITS - 1)) |
                          (uintptr_t(E.t.copy) & (A.copy_dtype == DCR_F32 ? 31 : 15));
    uint64_t at = begin + threadIdx.x / 32 * kBlock;
    const uint64_t whole = odd == 0 ? min(end, E.t.n / kBlock * kBlock) : begin;
    if (at < whole) {
        // the next values are on their way while these are computed
        Loaded<GB, BITS> now, next;
        next.template read<true>(E, at);
        for (; at < whole; at += kRound) {
            now = next;
            if (at + kRound < whole) next.template read<true>(E, at + kRound);
            update<WB, GB, BITS, true>(E, A, C, at, now);
        }
    }
    for (; at < end; at += kRound) {
        Loaded<GB, BITS> now;
        now.template read<false>(E, at);
        update<WB, GB, BITS, false>(E, A, C, at, now);
    }
}

// ---- the norm -------------------------------------------------------------------------------------------------------

constexpr int kNormFew = 160, kNormMany = 1280;
constexpr uint32_t kNormPer = 16384;   // values a chunk

template <int N>
struct NormTable {
    dcr_grad e[N];
    uint32_t chunk[N + 1];
    uint32_t count;
};

// The values of a chunk that a thread takes: 16-byte words from lo on, and at
// most one value (of index `single`) before or behind them.
template <typename T>
struct Share {
    static constexpr int V = 16 / sizeof(T);
    const T* p;
    uint64_t lo, single;
    uint32_t words;
    bool one;
    __device__ __forceinline__ Share(const T* p_, uint64_t begin, uint64_t end) : p(p_)
    {
        lo = min(begin + (16 - (uintptr_t(p + begin) & 15)) % 16 / sizeof(T), end);
        words = uint32_t((end - lo) / V);
        single = threadIdx.x < V ? begin + threadIdx.x : lo + words * V + (threadIdx.x - V);
        one = threadIdx.x < V ? single < lo : threadIdx.x < 2 * V && single < end;
    }
    __device__ __forceinline__ const uint4* word(uint32_t i) const { return reinterpret_cast<const uint4*>(p + lo) + i; }
};

// A thread's squares of its values times `scale`.
template <typename T>
__device__ __noinline__ float scaled_squares(const T* p, uint64_t begin, uint64_t end, float scale)
{
    const Share<T> S(p, begin, end);
    float q = 0.0f;
    for (uint32_t i = threadIdx.x; i < S.words; i += kThreads) {
        const uint4 x = *S.word(i);
        const T* t = reinterpret_cast<const T*>(&x);
#pragma unroll
        for (int j = 0; j < S.V; ++j) q = fmaf(to_f32(t[j]) * scale, to_f32(t[j]) * scale, q);
    }
    const float v = S.one ? to_f32(p[S.single]) * scale : 0.0f;
    return fmaf(v, v, q);
}

// Partial sums of squares: each block takes every gridDim-th chunk, whose
// squares a thread adds up in 32 bits (65 at most) and over chunks in 64.  A
// thread whose sum overflows takes its values again times 2^-70 (squares up to
// 2^116), and one whose sum is so small, although values are not 0, that it may
// lack squares below the smallest normal number, times 2^100 (of values below
// 2^-50; the smallest number's square is 2^-98).
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 8) squares_kernel(const __grid_constant__ NormTable<N> A, double* part, bool more)
{
    __shared__ double sums[kThreads / 32];
    double s = 0.0;
    for (uint32_t c = blockIdx.x; c < A.chunk[A.count]; c += gridDim.x) {
        const uint32_t k = tensor_of(A, c);
        const uint64_t begin = uint64_t(c - A.chunk[k]) * kNormPer, end = min(begin + kNormPer, A.e[k].n);
        const T* p = static_cast<const T*>(A.e[k].values);
        const Share<T> S(p, begin, end);
        float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t any = 0;
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < S.words; i += kThreads) {
            const uint4 x = *S.word(i);
            const T* t = reinterpret_cast<const T*>(&x);
#pragma unroll
            for (int j = 0; j < S.V; ++j) q[j % 4] = fmaf(to_f32(t[j]), to_f32(t[j]), q[j % 4]);
            any |= x.x | x.y | x.z | x.w;
        }
        if (S.one) {
            const float v = to_f32(p[S.single]);
            q[0] = fmaf(v, v, q[0]);
            any |= __float_as_uint(v);
        }
        double sum = double(q[0] + q[1]) + double(q[2] + q[3]);
        if (!(sum <= FLT_MAX)) sum = double(scaled_squares(p, begin, end, 0x1p-70f)) * 0x1p140;
        else if (any != 0 && sum < 0x1p-100) sum = double(scaled_squares(p, begin, end, 0x1p100f)) * 0x1p-200;
        s += sum;
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 32; ++i) s += sums[i];
        part[blockIdx.x] = more ? part[blockIdx.x] + s : s;
    }
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, uint32_t n, float* norm)
{
    __shared__ double sums[kThreads / 32];
    grid_wait();
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) s += part[i];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 32; ++i) s += sums[i];
        *norm = float(sqrt(s));
    }
}

constexpr uint32_t kNormBlocks = DCR_NORM_WORKSPACE / sizeof(double);   // 8 a SM

template <typename T, int N>
int squares_launch(const dcr_grad* grads, uint32_t count, double* part, uint32_t grid, bool more, cudaStream_t s)
{
    NormTable<N> A;
    A.count = count;
    uint32_t chunks = 0;
    for (uint32_t i = 0; i < count; ++i) {
        A.e[i] = grads[i];
        A.chunk[i] = chunks;
        chunks += uint32_t((grads[i].n + kNormPer - 1) / kNormPer);
    }
    A.chunk[count] = chunks;
    const LaunchAttrs at(grid, kThreads, 0, 1, false, s);
    const cudaError_t e = cudaLaunchKernelEx(&at.cfg, squares_kernel<T, N>, A, part, more);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "gradient norm launch");
}

template <int WB, int GB, int BITS, int N>
int adamw_launch(const dcr_adamw_tensor* t, uint32_t count, uint64_t first, const AdamwArgs& A, cudaStream_t s)
{
    Table<N> T;
    T.count = count;
    uint32_t chunks = 0;
    for (uint32_t i = 0; i < count; ++i) {
        T.e[i] = Entry{t[i], first};
        T.chunk[i] = chunks;
        chunks += uint32_t((t[i].n + A.per - 1) / A.per);
        first += t[i].n;
    }
    T.chunk[count] = chunks;
    const LaunchAttrs at(chunks, kThreads, 0, 1, false, s);
    const cudaError_t e = cudaLaunchKernelEx(&at.cfg, adamw_kernel<WB, GB, BITS, N>, T, A);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "AdamW launch");
}

template <int WB, int GB, int BITS>
int adamw_all(const std::vector<dcr_adamw_tensor>& t, AdamwArgs A, cudaStream_t s)
{
    uint64_t total = 0;
    for (const auto& x : t) total += x.n;
    // chunks of 16 rounds where there are enough to fill the SMs several times over, smaller ones otherwise
    A.per = kRound;
    while (A.per < 16 * kRound && total / (2 * A.per) >= 16 * 152) A.per *= 2;
    uint64_t first = 0;
    for (size_t i = 0; i < t.size(); i += kMany) {
        const uint32_t n = uint32_t(std::min<size_t>(kMany, t.size() - i));
        const int rc = n <= kFew ? adamw_launch<WB, GB, BITS, kFew>(&t[i], n, first, A, s) : adamw_launch<WB, GB, BITS, kMany>(&t[i], n, first, A, s);
        if (rc != DCR_OK) return rc;
        for (uint32_t j = 0; j < n; ++j) first += t[i + j].n;
    }
    return DCR_OK;
}

// Memory of a call: what is written may not overlap anything else.
struct Range {
    uintptr_t lo, hi;
    bool out;
    bool operator<(const Range& o) const { return lo < o.lo; }
};

// kinds: the ranges of all weights, of all gradients and so on, each of which
// a program mostly has in the order of their addresses.
constexpr size_t kKinds = 8;
bool overlapping(std::vector<Range> (&kinds)[kKinds])
{
    for (auto& k : kinds)
        if (!std::is_sorted(k.begin(), k.end())) std::sort(k.begin(), k.end());
    for (size_t step = 1; step < kKinds; step *= 2)
        for (size_t i = 0; i + step < kKinds; i += 2 * step) {
            std::vector<Range> both(kinds[i].size() + kinds[i + step].size());
            std::merge(kinds[i].begin(), kinds[i].end(), kinds[i + step].begin(), kinds[i + step].end(), both.begin());
            kinds[i].swap(both);
        }
    uintptr_t read = 0, written = 0;
    for (const Range& x : kinds[0]) {
        if (x.lo < written || (x.out && x.lo < read)) return true;
        uintptr_t& end = x.out ? written : read;
        end = std::max(end, x.hi);
    }
    return false;
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_grad_norm(const dcr_grad* grads, uint32_t count, uint32_t dtype, void* workspace, float* norm, void* stream)
{
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "dcr_grad_norm: unknown dtype %u", dtype);
    if (!norm || !workspace || (count && !grads)) return set_error(DCR_ERR_INVALID, "dcr_grad_norm: NULL argument");
    if (uintptr_t(norm) % 4 || uintptr_t(workspace) % 8) return set_error(DCR_ERR_INVALID, "dcr_grad_norm: misaligned buffer");
    try {
        std::vector<dcr_grad> t;
        t.reserve(count);
        uint64_t chunks = 0;
        for (uint32_t i = 0; i < count; ++i) {
            if (grads[i].n == 0) continue;
            if (!grads[i].values) return set_error(DCR_ERR_INVALID, "dcr_grad_norm: tensor %u is NULL", i);
            if (uintptr_t(grads[i].values) % dtype_size(dtype)) return set_error(DCR_ERR_INVALID, "dcr_grad_norm: tensor %u is misaligned", i);
            if (grads[i].n >= 1ull << 40) return set_error(DCR_ERR_INVALID, "dcr_grad_norm: tensor %u is too large", i);
            chunks += (grads[i].n + kNormPer - 1) / kNormPer;
            t.push_back(grads[i]);
        }
        if (chunks >= 1ull << 31) return set_error(DCR_ERR_INVALID, "dcr_grad_norm: too large");
        const Memory out = {"norm", norm, 4}, work = {"workspace", workspace, DCR_NORM_WORKSPACE};
        if (int rc = check_overlap("dcr_grad_norm", {out, work}, {})) return rc;
        for (const dcr_grad& g : t)
            if (int rc = check_overlap("dcr_grad_norm", {out, work}, {{"a gradient", g.values, g.n * dtype_size(dtype)}})) return rc;
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        double* part = static_cast<double*>(workspace);
        const uint32_t grid = uint32_t(std::min<uint64_t>(std::max<uint64_t>(chunks, 1), kNormBlocks));
        size_t i = 0;
        do {
            const uint32_t n = uint32_t(std::min<size_t>(kNormMany, t.size() - i));
            const int rc = with_dtype(dtype, [&](auto x) {
                using T = decltype(x);
                return n <= kNormFew ? squares_launch<T, kNormFew>(t.data() + i, n, part, grid, i != 0, s)
                                     : squares_launch<T, kNormMany>(t.data() + i, n, part, grid, i != 0, s);
            });
            if (rc != DCR_OK) return rc;
            i += n;
        } while (i < t.size());
        const LaunchAttrs at(1, kThreads, 0, 1, true, s);
        const cudaError_t e = cudaLaunchKernelEx(&at.cfg, norm_kernel, static_cast<const double*>(part), grid, norm);
        return e == cudaSuccess ? DCR_OK : cuda_error(e, "gradient norm launch");
    } catch (const std::exception&) {
        return set_error(DCR_ERR_NOMEM, "dcr_grad_norm: out of host memory");
    }
}

extern "C" int dcr_adamw(const dcr_adamw_tensor* tensors, uint32_t count, uint32_t w_dtype, uint32_t grad_dtype, uint32_t copy_dtype,
                         const dcr_adamw_opts* opts, void* stream)
{
    if (!opts || (count && !tensors)) return set_error(DCR_ERR_INVALID, "dcr_adamw: NULL argument");
    if (w_dtype > DCR_F16 || grad_dtype > DCR_F16 || copy_dtype > DCR_NONE) return set_error(DCR_ERR_INVALID, "dcr_adamw: unknown dtype");
    const dcr_adamw_opts& o = *opts;
    if (o.state_bits != 32 && o.state_bits != 8) return set_error(DCR_ERR_INVALID, "dcr_adamw: state_bits must be 32 or 8");
    if (!(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0)) return set_error(DCR_ERR_INVALID, "dcr_adamw: betas must lie in [0, 1)");
    auto finite = [](double v) { return std::isfinite(float(v)); };    // in the 32 bits that the kernel computes in
    if (!finite(o.lr) || o.lr < 0.0 || !finite(o.weight_decay) || o.weight_decay < 0.0 || !finite(o.eps) || o.eps < 0.0)
        return set_error(DCR_ERR_INVALID, "dcr_adamw: lr, weight_decay and eps must be finite and not negative");
    if (!finite(o.grad_scale)) return set_error(DCR_ERR_INVALID, "dcr_adamw: grad_scale must be finite");
    if (!finite(o.max_norm) || o.max_norm < 0.0 || (o.max_norm > 0.0 && !o.norm))
        return set_error(DCR_ERR_INVALID, "dcr_adamw: max_norm must be finite, not negative, and needs a norm");
    if (o.step == 0 && !o.device_step) return set_error(DCR_ERR_INVALID, "dcr_adamw: step counts from 1");
    if (uintptr_t(o.norm) % 4 || uintptr_t(o.device_lr) % 4 || uintptr_t(o.device_step) % 8)
        return set_error(DCR_ERR_INVALID, "dcr_adamw: misaligned buffer");
    try {
        std::vector<dcr_adamw_tensor> t;
        std::vector<Range> used[kKinds];
        t.reserve(count);
        for (auto& u : used) u.reserve(count);
        auto use = [&](int kind, const void* p, uint64_t bytes, bool out) { used[kind].push_back(Range{uintptr_t(p), uintptr_t(p) + bytes, out}); };
        // every block reads these, while others write
        if (o.norm) use(7, o.norm, 4, false);
        if (o.device_step) use(7, o.device_step, 8, false);
        if (o.device_lr) use(7, o.device_lr, 4, false);
        uint64_t chunks = 0;
        for (uint32_t i = 0; i < count; ++i) {
            dcr_adamw_tensor x = tensors[i];
            if (x.n == 0) continue;
            if (copy_dtype == DCR_NONE) x.copy = nullptr;
            if (!x.w || !x.grad || !x.m || !x.v || (copy_dtype != DCR_NONE && !x.copy) || (o.state_bits == 8 && (!x.m_scale || !x.v_scale)))
                return set_error(DCR_ERR_INVALID, "dcr_adamw: tensor %u has a NULL pointer", i);
            if (x.n >= 1ull << 40) return set_error(DCR_ERR_INVALID, "dcr_adamw: tensor %u is too large", i);
            const uint32_t sb = o.state_bits / 8, cb = copy_dtype == DCR_NONE ? 1 : dtype_size(copy_dtype);
            if (uintptr_t(x.w) % dtype_size(w_dtype) || uintptr_t(x.grad) % dtype_size(grad_dtype) || uintptr_t(x.copy) % cb ||
                uintptr_t(x.m) % sb || uintptr_t(x.v) % sb || (sb == 1 && (uintptr_t(x.m_scale) % 4 || uintptr_t(x.v_scale) % 4)))
                return set_error(DCR_ERR_INVALID, "dcr_adamw: tensor %u is misaligned", i);
            use(0, x.w, x.n * dtype_size(w_dtype), true);
            use(1, x.grad, x.n * dtype_size(grad_dtype), false);
            use(2, x.m, x.n * sb, true);
            use(3, x.v, x.n * sb, true);
            if (copy_dtype != DCR_NONE) use(4, x.copy, x.n * cb, true);
            if (sb == 1) {
                const uint64_t blocks = (x.n + kBlock - 1) / kBlock;
                use(5, x.m_scale, blocks * 4, true);
                use(6, x.v_scale, blocks * 4, true);
            }
            chunks += (x.n + kRound - 1) / kRound;
            t.push_back(x);
        }
        if (chunks >= 1ull << 31) return set_error(DCR_ERR_INVALID, "dcr_adamw: too large");
        if (overlapping(used)) return set_error(DCR_ERR_INVALID, "dcr_adamw: tensors overlap");
        if (t.empty()) return DCR_OK;
        AdamwArgs A{};
        const double c1 = 1.0 - std::pow(o.beta1, double(o.step)), c2 = 1.0 - std::pow(o.beta2, double(o.step));
        A.beta1 = float(o.beta1), A.beta2 = float(o.beta2), A.rest1 = float(1.0 - o.beta1), A.rest2 = float(1.0 - o.beta2);
        A.eps = float(o.eps), A.decay = float(1.0 - o.lr * o.weight_decay), A.step_size = float(o.lr / c1), A.inv_root = float(1.0 / std::sqrt(c2));
        A.grad_scale = float(o.grad_scale), A.max_norm = float(o.max_norm), A.lr = float(o.lr), A.weight_decay = float(o.weight_decay);
        A.log1 = float(std::log(o.beta1)), A.log2 = float(std::log(o.beta2));
        A.norm = o.norm, A.step_at = o.device_step, A.lr_at = o.device_lr, A.step = o.step, A.seed = o.seed;
        A.w_half = w_dtype == DCR_F16, A.g_half = grad_dtype == DCR_F16, A.copy_dtype = copy_dtype;
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        auto bits = [&](auto wb, auto gb) {
            return o.state_bits == 32 ? adamw_all<decltype(wb)::value, decltype(gb)::value, 32>(t, A, s)
                                      : adamw_all<decltype(wb)::value, decltype(gb)::value, 8>(t, A, s);
        };
        using Two = std::integral_constant<int, 2>;
        using Four = std::integral_constant<int, 4>;
        if (w_dtype == DCR_F32) return grad_dtype == DCR_F32 ? bits(Four(), Four()) : bits(Four(), Two());
        return grad_dtype == DCR_F32 ? bits(Two(), Four()) : bits(Two(), Two());
    } catch (const std::exception&) {
        return set_error(DCR_ERR_NOMEM, "dcr_adamw: out of host memory");
    }
}
