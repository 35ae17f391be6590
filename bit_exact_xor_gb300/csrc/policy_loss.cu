// Clipped policy loss with a KL term, its gradient by the logits, and the
// log-probabilities of tokens (include/dcr_ops.h).
//
// A row is read once: each thread keeps its share of it in registers, as
// 16-byte words, between the statistics (maximum m, then the sum s of
// exp((x - m) / T) against the block's maximum) and the gradient.  Long rows
// are shared by the blocks of a cluster, which exchange (m, s) through
// distributed shared memory once.  What does not fit on the chip that way is
// read again.
//
// Bound by its traffic in long batches: 4096 rows of 128256 bf16 values in 375
// us, 4.9 TB/s of what it moves (a quarter of the rows is left out: read 0.79
// GB, written 1.05 GB), of which keeping the token's term apart is about 9;
// by the chain of loads, two block-wide steps, two cluster-wide ones and
// stores in short ones (1021 rows of 32771 values: 43 us, five rounds of
// blocks).
#include <cfloat>
#include <cmath>
#include <type_traits>

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
    float sc;                   // log2(e) / temperature, rounded to nearest
    float sc_dn, sc_lo;         // the same rounded down, and the (positive) rest
};

constexpr int kMaxCluster = 8;

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

// exp(v), the largest number where that overflows although v is finite: what
// is multiplied by 0 then (an advantage, a probability) is 0 as in exact
// arithmetic, and not NaN.
__device__ __forceinline__ float exp_finite(float v)
{
    const float e = expf(v);
    return v < INFINITY ? fminf(e, FLT_MAX) : e;
}

// Loss of a row and its derivative by the log-probability.
__device__ __forceinline__ void row_loss(const LossArgs& A, float adv, float old, float ref, float lp, float& loss, float& slope)
{
    const float ratio = exp_finite(lp - old);
    const float u = ratio * adv, c = fminf(fmaxf(ratio, A.lo), A.hi) * adv;
    const bool clipped = c < u;
    loss = clipped ? -c : -u;
    slope = clipped ? 0.0f : -u;
    if (A.kl != 0.0f) {
        const float k = ref - lp, e = exp_finite(k);
        loss += A.kl * (e - k - 1.0f);
        slope += A.kl * (1.0f - e);
    }
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

// Blocks on an SM: what bounds the kernel is how many words are in flight, so
// registers are held to what that takes (4096 rows of 128256 bf16 values,
// 8 words a thread, before sums and the token's term took their present form:
// 495 us with two blocks of 256 threads, 405 with three, 347 with four).
constexpr int resident_blocks(int th, int nv) { return (nv >= 6 ? 1024 : nv >= 4 ? 1536 : 2048) / th; }

// TH threads a block, NV words a thread kept, `cluster` blocks a row.
template <typename T, int TH, int NV>
__global__ void __launch_bounds__(TH, resident_blocks(TH, NV)) loss_kernel(LossArgs A, uint32_t cluster)
{
    constexpr int N = Word<T>::kN;
    __shared__ float part[TH / 16];
    __shared__ float2 all[kMaxCluster];
    launch_dependents();
    const uint32_t rank = cluster > 1 ? blockIdx.x % cluster : 0;
    const uint64_t row = blockIdx.x / cluster;
    const uint32_t vocab = uint32_t(A.vocab);
    const T* x = static_cast<const T*>(A.logits) + row * A.row_stride;
    T* g = A.grad ? static_cast<T*>(A.grad) + row * A.grad_stride : nullptr;
    const uint32_t step = cluster * TH, first = rank * TH + threadIdx.x;   // this thread's words: first + i * step

    const int64_t token = A.tokens[row];
    const float w = A.weights ? A.weights[row] : 1.0f;
    // asked for now, so that they are there when the statistics are
    const float adv = A.old_logp ? A.advantages[row] : 0.0f, old = A.old_logp ? A.old_logp[row] : 0.0f;
    const float ref = A.ref_logp ? A.ref_logp[row] : 0.0f;
    const bool on = w != 0.0f && token >= 0 && token < int64_t(vocab);
    const uint32_t y = uint32_t(token);
    const float sc = A.sc;
    // m: the row's maximum; others: the sum of exp((x_j - m) / T) without the token's own term, which is ey.  Formed
    // from others, 1 - p = others / (others + ey) and log p keep their accuracy where the token is nearly certain: a sum
    // over all values has rounded away what is left beside 1 there.
    float m = -INFINITY, others = 0.0f, ey = 0.0f;
    uint4 q[NV];
    float xy = 0.0f;
    const Row<T> in(x, vocab);
    // where the token's value is: its word, the place in it, whether this thread has it
    const uint32_t yword = (in.skip + y) / N, yat = (in.skip + y) % N;
    const bool mine = yword % step == first;
    if (on) {
        // another block's shared memory may be written once that block is known to run: all say so here, and wait for it
        // while their loads are under way (a row is on in all blocks of its cluster or in none)
        if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
#pragma unroll
        for (int i = 0; i < NV; ++i) q[i] = in.load_whole(first + i * step);
        xy = to_f32(x[y]);
        if (cluster > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in.cut(first + i * step)) q[i] = in.load_cut(first + i * step);
#pragma unroll
        for (int i = 0; i < NV; ++i) m = fmaxf(m, word_max(q[i], T()));
        for (uint32_t k = first + NV * step; k < in.words; k += step) m = fmaxf(m, word_max(in.load(k), T()));
        if (mine) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (first + i * step == yword) q[i] = without<T>(q[i], yat);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TH / 32; ++i) m = fmaxf(m, part[i]);
        float s = words_sum<T, NV>(q, m, A.sc_dn, A.sc_lo);
        for (uint32_t k = first + NV * step; k < in.words; k += step) {
            const uint4 word = in.load(k), e[1] = {k == yword ? without<T>(word, yat) : word};
            s += words_sum<T, 1>(e, m, A.sc_dn, A.sc_lo);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (threadIdx.x % 32 == 0) part[TH / 32 + threadIdx.x / 32] = s;
        __syncthreads();   // also: grad may be logits, and everybody has read x[y]
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < TH / 32; ++i) s += part[TH / 32 + i];
        if (cluster > 1) {
            if (threadIdx.x < cluster) {
                const uint32_t at = uint32_t(__cvta_generic_to_shared(&all[rank]));
                asm volatile(
                    "{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, %1; st.shared::cluster.v2.f32 [a], {%2, %3}; }" ::"r"(at),
                    "r"(threadIdx.x), "f"(m), "f"(s)
                    : "memory");
            }
            asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
            for (uint32_t i = 0; i < cluster; ++i) m = fmaxf(m, all[i].x);
            s = 0.0f;
            // maxima that are equal (infinite ones among them) need no factor
            for (uint32_t i = 0; i < cluster; ++i) s += all[i].x == m ? all[i].y : all[i].y * exp2_fast((all[i].x - m) * sc);
        }
        if (m == INFINITY && s == s) s = 1.0f;
        others = s;
        // not a number where the token's value is infinite and the maximum
        ey = xy != m ? exp2_fast((xy - m) * sc) : fabsf(m) == INFINITY ? NAN : 1.0f;
    }
    const float s = others + ey;

    float c = 0.0f;
    if (on) {
        // log s with what the sum's rounding left out, which is most of it beside ey = 1
        const float lp = (xy - m) * A.inv_temp - logf(s) - __fdividef(others - (s - ey), s);
        float loss = 0.0f, slope = 0.0f;
        if (A.old_logp) row_loss(A, adv, old, ref, lp, loss, slope);
        if (rank == 0 && threadIdx.x == 0) {
            A.logp[row] = lp;
            if (A.row_loss) A.row_loss[row] = w * loss;
        }
        c = w * slope * A.inv_temp;
    } else if (rank == 0 && threadIdx.x == 0) {
        A.logp[row] = 0.0f;
        if (A.row_loss) A.row_loss[row] = 0.0f;
    }
    if (!g) return;

    // grad_j = -c exp((x_j - m) / T) / s, and c others / s for the token.  The words go out as they came in where the
    // gradient's row lies on the same offset from a 16-byte boundary.
    const Exponent e(m, sc, 0.0f);
    const float d = on ? -c / s * exp2f(-e.excess()) : 0.0f;
    const Row<T> out(g, vocab);
    const bool same = out.skip == in.skip;
    auto put = [&](uint32_t k, const uint4& q, auto plain) {
        float v[N];
        Word<T>::values(q, v);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = d * e.of<decltype(plain)::value>(v[j]);
        const uint4 w = Word<T>::pack(v);
        if (same && in.whole(k)) *reinterpret_cast<uint4*>(out.base + uint64_t(k) * N) = w;
        else if (k < in.words) store_values<T>(g, in.skip, vocab, k, w);
    };
    auto put_all = [&](auto plain) {
#pragma unroll
        for (int i = 0; i < NV; ++i) put(first + i * step, q[i], plain);
        for (uint32_t k = first + NV * step; k < in.words; k += step) put(k, in.load(k), plain);
    };
    if (!on) {
        for (uint32_t k = rank * TH + threadIdx.x; k < out.words; k += step) {
            if (out.whole(k)) *reinterpret_cast<uint4*>(out.base + uint64_t(k) * N) = make_uint4(0, 0, 0, 0);
            else store_values<T>(g, out.skip, vocab, k, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    if (e.plain) put_all(std::true_type());
    else put_all(std::false_type());
    // the token's own value, by the thread that wrote its word
    if (mine) g[y] = from_f32<T>(c * (others / s));
}

// The rows' losses summed in a fixed order: thread i takes rows i, i + 1024,
// ..., then a tree over the threads.
__global__ void __launch_bounds__(1024) sum_kernel(const float* v, uint64_t n, float* out)
{
    __shared__ double part[32];
    grid_wait();
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

template <typename T, int TH, int NV>
int launch_rows(const LossArgs& A, uint32_t cluster, cudaStream_t s)
{
    const LaunchAttrs at(A.rows * cluster, TH, 0, cluster, false, s);
    const cudaError_t e = cudaLaunchKernelEx(&at.cfg, loss_kernel<T, TH, NV>, A, cluster);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "policy loss launch");
}

// As few blocks of 256 threads as hold the row with up to 8 words a thread,
// then as few words as that takes; for short rows blocks of 128.  (2048 rows
// of 50000 f16 values: 89 us as 4 blocks x 8 words, 112 as 7 x 4, although
// that keeps less.)
template <typename T>
int launch_rows(const LossArgs& A, cudaStream_t s)
{
    const bool aligned = uintptr_t(A.logits) % 16 == 0 && A.row_stride * sizeof(T) % 16 == 0;
    const uint64_t words = (A.vocab * sizeof(T) + 15) / 16 + (aligned ? 0 : 1);
    if (words <= 128) return launch_rows<T, 128, 1>(A, 1, s);
    if (words <= 256) return launch_rows<T, 128, 2>(A, 1, s);
    if (words <= 512) return launch_rows<T, 128, 4>(A, 1, s);
    // a row that eight such blocks do not hold: blocks of 512 (512 rows of 300000 f32 values: 356 -> 282 us; on rows
    // that the smaller blocks hold they are no faster: 347 -> 365 us at 128256 bf16 values then)
    if (words > 2048 * kMaxCluster)
        return launch_rows<T, 512, 8>(A, words > 4096 * kMaxCluster ? kMaxCluster : uint32_t((words + 4095) / 4096), s);
    const uint32_t cluster = uint32_t((words + 2047) / 2048);
    const uint64_t nv = (words + 256 * cluster - 1) / (256 * cluster);
    if (nv <= 4) return launch_rows<T, 256, 4>(A, cluster, s);
    if (nv <= 6) return launch_rows<T, 256, 6>(A, cluster, s);
    return launch_rows<T, 256, 8>(A, cluster, s);
}

int launch(LossArgs A, uint32_t dtype, float temperature, float* loss, cudaStream_t s)
{
    // 1 / T and log2(e) / T stay finite for the smallest T, too (0 times them is 0); the rest of the second is positive and
    // no larger than its rounding, and adds nothing even to the largest logits where there is none
    const double most = FLT_MAX, sc = std::fmin(1.4426950408889634 / temperature, most);
    A.inv_temp = float(std::fmin(1.0 / temperature, most));
    A.sc = float(sc);
    A.sc_dn = A.sc > sc ? std::nextafterf(A.sc, 0.0f) : A.sc;
    A.sc_lo = std::fmax(float(sc - A.sc_dn), FLT_TRUE_MIN);
    if (A.rows == 0 && !loss) return DCR_OK;
    if (A.rows) {
        const int rc = with_dtype(dtype, [&](auto t) { return launch_rows<decltype(t)>(A, s); });
        if (rc != DCR_OK) return rc;
    }
    if (!loss) return DCR_OK;
    const LaunchAttrs at(1, 1024, 0, 1, A.rows != 0, s);
    const cudaError_t e = cudaLaunchKernelEx(&at.cfg, sum_kernel, static_cast<const float*>(A.row_loss), A.rows, loss);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "policy loss launch");
}

int check(const char* what, const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
          const int64_t* tokens, float temperature, const float* logp)
{
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "%s: unknown dtype %u", what, dtype);
    if (!(temperature > 0.0f) || temperature > 3.0e38f)
        return set_error(DCR_ERR_INVALID, "%s: temperature must be positive and finite", what);
    if (vocab == 0 || vocab >= 1ull << 31 || rows >= 1ull << 28 || row_stride >= 1ull << 40)
        return set_error(DCR_ERR_INVALID, "%s: vocab must be at least 1 and below 2^31, rows below 2^28", what);
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
               row_loss, logp, 0.0f, 1.0f - opts->clip_low, 1.0f + opts->clip_high, opts->kl_coef};
    return launch(A, dtype, opts->temperature, loss, static_cast<cudaStream_t>(stream));
}

extern "C" int dcr_token_logprobs(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                                  const int64_t* tokens, float temperature, float* logp, void* stream)
{
    if (int rc = dcr::check("dcr_token_logprobs", logits, dtype, rows, vocab, row_stride, tokens, temperature, logp)) return rc;
    LossArgs A{};
    A.logits = logits, A.rows = rows, A.vocab = vocab, A.row_stride = row_stride;
    A.tokens = tokens, A.logp = logp;
    return launch(A, dtype, temperature, nullptr, static_cast<cudaStream_t>(stream));
}
