// Rows of logits as the kernels of policy_loss.cu and token_scores.cu read
// them: 16-byte words whose first and last may be cut, and exponentials of
// differences from a maximum.
#pragma once

#include <cmath>
#include <type_traits>

#include "ops_internal.h"

namespace dcr {
namespace {

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The 16 bytes of a word as its values.
template <typename T>
struct Word;
template <>
struct Word<float> {
    static constexpr int kN = 4;
    static constexpr uint32_t kLow = 0xFF800000u;   // -inf
    static __device__ __forceinline__ void values(const uint4& q, float (&v)[4])
    {
        v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4])
    {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Word<__nv_bfloat16> {
    static constexpr int kN = 8;
    static constexpr uint32_t kLow = 0xFF80FF80u;
    static __device__ __forceinline__ void values(const uint4& q, float (&v)[8])
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Word<__half> {
    static constexpr int kN = 8;
    static constexpr uint32_t kLow = 0xFC00FC00u;
    static __device__ __forceinline__ void values(const uint4& q, float (&v)[8])
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// A word with -inf in the place of its value j.
template <typename T>
__device__ __forceinline__ uint4 without(const uint4& q, uint32_t j)
{
    constexpr uint32_t kPer = 4 / sizeof(T);
    const uint32_t at = j / kPer, mask = kPer == 1 ? ~0u : 0xFFFFu << (16 * (j % kPer)), low = Word<T>::kLow & mask;
    return make_uint4(at == 0 ? (q.x & ~mask) | low : q.x, at == 1 ? (q.y & ~mask) | low : q.y,
                      at == 2 ? (q.z & ~mask) | low : q.z, at == 3 ? (q.w & ~mask) | low : q.w);
}

// Largest value of a word (a NaN is passed over), two at a time where two
// share a register.
__device__ __forceinline__ float word_max(const uint4& q, float)
{
    return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
}
template <typename T>
__device__ __forceinline__ float word_max(const uint4& q, T)
{
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2* h = reinterpret_cast<const T2*>(&q);
    const T2 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(to_f32(a.x), to_f32(a.y));
}

// exp((x - m) / T) = 2^(x sc - m sc), sc = log2(e) / T: one multiply-add with
// the rounded product msc = m sc, whose rounding error is the same factor on
// every term (the row's sum is corrected for it once).  That holds while the
// factor 2^excess is near 1: it is half a unit of msc's last place at most,
// 2^-5 below |msc| = 2^20.  Beyond (a row far from 0, a temperature near 0)
// the difference comes first.  The row's sum takes a second multiply-add with
// the rest of sc: over a large vocabulary most of it comes from terms far
// below the maximum, where sc's rounding shifts every one the same way (a
// row's log-probability by up to 1e-6).  There sc is rounded down, so that the
// rest is positive and -inf stays -inf.
struct Exponent {
    float sc, lo, m, msc;
    bool plain;
    __device__ __forceinline__ Exponent(float m_, float sc_, float lo_)
        : sc(sc_), lo(lo_), m(m_), msc(m_ * sc_), plain(fabsf(m_ * sc_) < 1048576.0f)
    {
    }
    template <bool PLAIN>
    __device__ __forceinline__ float term(float x) const
    {
        return exp2_fast(PLAIN ? fmaf(x, lo, fmaf(x, sc, -msc)) : fmaf(x - m, lo, (x - m) * sc));
    }
    __device__ __forceinline__ float term_excess() const { return plain ? fmaf(m, lo, fmaf(m, sc, -msc)) : 0.0f; }
    template <bool PLAIN>
    __device__ __forceinline__ float of(float x) const
    {
        return exp2_fast(PLAIN ? fmaf(x, sc, -msc) : (x - m) * sc);
    }
    // log2 of the factor that all terms carry
    __device__ __forceinline__ float excess() const { return plain ? fmaf(m, sc, -msc) : 0.0f; }
};

template <typename T, bool PLAIN>
__device__ __forceinline__ float word_sum(const uint4& q, const Exponent& e)
{
    float v[Word<T>::kN], s[2] = {0.0f, 0.0f};
    Word<T>::values(q, v);
#pragma unroll
    for (int i = 0; i < Word<T>::kN; ++i) s[i & 1] += e.term<PLAIN>(v[i]);
    return s[0] + s[1];
}

template <typename T>
__device__ __forceinline__ bool word_nan(const uint4& q)
{
    float v[Word<T>::kN];
    Word<T>::values(q, v);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < Word<T>::kN; ++i) nan |= v[i] != v[i];
    return nan;
}

// A row as 16-byte words, the first of which may begin before it and the last
// end behind it: `skip` values of the first word belong to what lies before.
template <typename T>
struct Row {
    T* base;          // on a 16-byte boundary, at or below the row's start
    uint32_t skip, vocab, words, lo, hi;   // whole words: lo to hi
    __device__ __forceinline__ Row(const T* p, uint32_t v)
    {
        skip = uint32_t((uintptr_t(p) & 15) / sizeof(T));
        base = const_cast<T*>(p) - skip;
        vocab = v;
        words = (skip + v + Word<T>::kN - 1) / Word<T>::kN;
        lo = skip ? 1 : 0;
        hi = (skip + v) / Word<T>::kN;
    }
    __device__ __forceinline__ bool whole(uint32_t g) const { return g >= lo && g < hi; }
    __device__ __forceinline__ bool cut(uint32_t g) const { return g < words && !whole(g); }
    // word g, with -inf where it is not the row: whole words by a predicated load that nothing waits for before its
    // use, the (at most two) others value by value
    __device__ __forceinline__ uint4 load_whole(uint32_t g) const
    {
        uint4 q;
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %5, 0; mov.u32 %0, %6; mov.u32 %1, %6; mov.u32 %2, %6; mov.u32 %3, %6;\n"
            "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4]; }"
            : "=&r"(q.x), "=&r"(q.y), "=&r"(q.z), "=&r"(q.w)
            : "l"(base + uint64_t(g) * Word<T>::kN), "r"(uint32_t(whole(g))), "n"(Word<T>::kLow));
        return q;
    }
    __device__ __noinline__ uint4 load_cut(uint32_t g) const
    {
        union { uint4 q; T t[Word<T>::kN]; } u;
        u.q = make_uint4(Word<T>::kLow, Word<T>::kLow, Word<T>::kLow, Word<T>::kLow);
        for (int i = 0; i < Word<T>::kN; ++i) {
            const uint32_t at = g * Word<T>::kN + i;
            if (at >= skip && at - skip < vocab) u.t[i] = base[at];
        }
        return u.q;
    }
    __device__ __forceinline__ uint4 load(uint32_t g) const { return cut(g) ? load_cut(g) : load_whole(g); }
};

// Sum of exp((x - m) / T) over words whose largest value is m.
template <typename T, int NV>
__device__ __forceinline__ float words_sum(const uint4 (&q)[NV], float m, float sc, float lo)
{
    float s = 0.0f;
    if (fabsf(m) == INFINITY || m != m) {
        // nothing above -inf: nothing to add; +inf: exp(inf - inf) is not a number, although the sum is not one only if
        // a value is not
        bool nan = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) nan |= word_nan<T>(q[i]);
        return nan ? NAN : 0.0f;
    }
    const Exponent e(m, sc, lo);
    if (e.plain) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s += word_sum<T, true>(q[i], e);
        return s * exp2f(-e.term_excess());
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) s += word_sum<T, false>(q[i], e);
    return s;
}

// The values of word k of a row that begins `skip` values into its first
// word, one by one.
template <typename T>
__device__ __noinline__ void store_values(T* row, uint32_t skip, uint32_t vocab, uint32_t k, uint4 w)
{
    union { uint4 q; T t[Word<T>::kN]; } u;
    u.q = w;
    for (int j = 0; j < Word<T>::kN; ++j) {
        const uint32_t at = k * Word<T>::kN + j;
        if (at >= skip && at - skip < vocab) row[at - skip] = u.t[j];
    }
}

}  // namespace
}  // namespace dcr
