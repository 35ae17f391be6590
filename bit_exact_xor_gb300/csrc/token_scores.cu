// Scores of given tokens: log-probability, entropy and likeliest alternatives
// of each row of logits, and the gradient of the first two
// (include/dcr_ops.h).
//
// One pass: each thread reads its words of the row in chunks of 6 and keeps a
// running maximum m, the sum of exp((x - m) / T) and the sum of that times the
// exponent; maxima and sums meet once, at the end.  The chunk that holds a
// thread's maximum is summed apart, so that the threads whose maximum is the
// row's can read that chunk again and leave the maximum itself out: the sum
// of the others keeps the digits that are lost beside a 1, and with them the
// log-probability and the entropy of nearly certain rows.
//
// Alternatives: the pass also leaves the maximum of each chunk.  From the
// threads' maxima comes a bound that at least `top` values reach; the few
// chunks that reach it are read again, and their values of that size sorted.
// Where those are too many (equal ones above all: masked rows), the values
// above the bound are taken, and the first of the equal ones in the order of
// their indexes, then of NaN; where that does not fit either, the largest is
// searched `top` times.
//
// Long batches are bound by instruction issue, 8 to 9 a value, and by the steps
// at a row's end: 4096 rows of 128256 bf16 values in 173 us (6.1 TB/s), with
// 20 alternatives in 213; 4096 of 32768 f32 values in 84 (6.4 TB/s) and their
// gradient in 168 (6.4 TB/s).  Few rows are bound by latency: 8 rows of 128256
// in 7.8 us, with 20 alternatives in 12.0.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "logits.cuh"

namespace dcr {
namespace {

struct ScoreArgs {
    const void* logits;
    uint64_t rows, vocab, row_stride;
    const int64_t* tokens;
    float* logp;
    float* entropy;
    float* top_logp;
    int64_t* top_tokens;
    float* stats;
    uint32_t top;
    float inv_temp;
    float sc;             // log2(e) / temperature, rounded to nearest
    float sc_dn, sc_lo;   // the same rounded down, and the (positive) rest
};

constexpr int kWords = 6;          // words of a chunk
constexpr uint32_t kBuckets = 16;  // chunk maxima that a thread keeps
constexpr uint32_t kList = 512;    // values that are sorted
constexpr int kMaxBlocks = 8;      // of a cluster
constexpr float kLn2 = 0.69314718055994531f;

// The larger one, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum of exp((x - m) / T) =: e over words, and of e log2(e).
struct Sums {
    float s, t;
};

// Two multiply-adds, or sums, in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 z, x, y, z; mov.b64 {%0, %1}, z; }"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The sums of a chunk without -inf and not far from 0; its words are `step`
// apart, and those from `left` on lie behind the row.
template <typename T>
__device__ __forceinline__ Sums plain_sums(const uint4 (&q)[kWords], const Exponent& e, uint32_t left, uint32_t step)
{
    float2 s = both(0.0f), t = both(0.0f);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if (i * step >= left) break;
        float v[Word<T>::kN];
        Word<T>::values(q[i], v);
#pragma unroll
        for (int j = 0; j < Word<T>::kN; j += 2) {
            const float2 x = make_float2(v[j], v[j + 1]), d = fma2(x, both(e.lo), fma2(x, both(e.sc), both(-e.msc)));
            const float2 p = make_float2(exp2_fast(d.x), exp2_fast(d.y));
            s = add2(s, p);
            t = fma2(p, d, t);
        }
    }
    return {s.x + s.y, t.x + t.y};
}

// A word whose values below lowest() are that, -inf among them; NaN stays.
template <typename T>
__device__ __forceinline__ float lowest()
{
    return std::is_same<T, __half>::value ? -65504.0f : -1e30f;
}
__device__ __forceinline__ uint4 not_below(const uint4& q, float)
{
    return make_uint4(__float_as_uint(max_nan(__uint_as_float(q.x), -1e30f)), __float_as_uint(max_nan(__uint_as_float(q.y), -1e30f)),
                      __float_as_uint(max_nan(__uint_as_float(q.z), -1e30f)), __float_as_uint(max_nan(__uint_as_float(q.w), -1e30f)));
}
template <typename T>
__device__ __forceinline__ uint4 not_below(const uint4& q, T)
{
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T l = from_f32<T>(lowest<T>());
    T2 low;
    low.x = l, low.y = l;
    union { uint4 w; T2 t[4]; } u;
    u.w = q;
#pragma unroll
    for (int i = 0; i < 4; ++i) u.t[i] = __hmax2_nan(u.t[i], low);
    return u.w;
}

// The same, where a value may be -inf, or left out as if it were, one by one.
template <bool PLAIN, int N>
__device__ __forceinline__ void add_values(Sums& a, const float (&v)[N], const Exponent& e)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x = PLAIN ? fmaf(v[i], e.lo, fmaf(v[i], e.sc, -e.msc)) : fmaf(v[i] - e.m, e.lo, (v[i] - e.m) * e.sc);
        // -200: exp of it is 0, and so is its product with it, which with -inf would not be a number
        const float d = max_nan(x, -200.0f), p = exp2_fast(d);
        a.s += p;
        a.t = fmaf(p, d, a.t);
    }
}

// What every exponent has too much is taken out of the sums.
__device__ __forceinline__ void correct(Sums& a, const Exponent& e)
{
    const float x = e.term_excess(), f = exp2f(-x);
    a.t = fmaf(-x, a.s, a.t) * f;
    a.s *= f;
}

// The same over the values below m, and how many are equal to it (m is finite or +inf).
template <typename T, int NV>
__device__ __forceinline__ Sums chunk_sums_below(const uint4 (&q)[NV], float m, const ScoreArgs& A, float& count)
{
    const Exponent e(m, A.sc_dn, A.sc_lo);
    Sums a = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float v[Word<T>::kN];
        Word<T>::values(q[i], v);
#pragma unroll
        for (int j = 0; j < Word<T>::kN; ++j) {
            if (v[j] == m) count += 1.0f;
            v[j] = v[j] == m ? -INFINITY : v[j];
        }
        if (e.plain) add_values<true>(a, v, e);
        else add_values<false>(a, v, e);
    }
    correct(a, e);
    return a;
}

// A maximum, the values that are equal to it, and the sums over the others.
struct Part {
    float m, count, s, t;
    // b's share from its own maximum to this one's, which is no smaller
    __device__ __forceinline__ void add(const Part& b, float sc)
    {
        if (b.m == m) {
            count += b.count, s += b.s, t += b.t;
        } else if (b.m == -INFINITY) {
            s += b.s, t += b.t;      // nothing, or NaN
        } else {
            const float d = (b.m - m) * sc, f = exp2_fast(d), all = b.s + b.count;
            s = fmaf(f, all, s);
            if (f != 0.0f) t = fmaf(f, fmaf(d, all, b.t), t);
        }
    }
};

// Order of values, and of (value, index) with the lower index above.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);    // -0 is 0
    return x != x ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o)
{
    return o == 0 ? NAN : __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) { return uint64_t(order_of(x)) << 32 | uint32_t(~index); }

__device__ __forceinline__ uint4 load_word(const void* p)
{
    uint4 q;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p));
    return q;
}

// This block's words of a row.
template <typename T>
struct Share {
    Row<T> in;
    uint32_t first, step;   // of this thread
    uint32_t chunks;        // of the block
    __device__ __forceinline__ Share(const T* x, uint32_t vocab, uint32_t rank, uint32_t blocks)
        : in(x, vocab), first(rank * blockDim.x + threadIdx.x), step(blocks * blockDim.x), chunks((in.words + kWords * step - 1) / (kWords * step))
    {
    }
    __device__ __forceinline__ void load(uint32_t c, uint4 (&q)[kWords]) const
    {
        const uint32_t k = first + c * kWords * step, block = k - threadIdx.x;
        if (block >= in.lo && block + (kWords - 1) * step + blockDim.x <= in.hi) {   // nothing of the block's chunk is cut
            const T* p = in.base + uint64_t(k) * Word<T>::kN;
#pragma unroll
            for (int i = 0; i < kWords; ++i) q[i] = load_word(p + uint64_t(i * step) * Word<T>::kN);
            return;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) q[i] = in.load_whole(k + i * step);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (in.cut(k + i * step)) q[i] = in.load_cut(k + i * step);
    }
    // f(value, index) for the values of word k
    template <typename F>
    __device__ __forceinline__ void each(const uint4& q, uint32_t k, F f) const
    {
        float v[Word<T>::kN];
        Word<T>::values(q, v);
#pragma unroll
        for (int j = 0; j < Word<T>::kN; ++j) {
            const uint32_t at = k * Word<T>::kN + j - in.skip;
            if (k < in.words && at < in.vocab) f(v[j], at);      // before the row: at is huge
        }
    }
    template <typename F>
    __device__ __forceinline__ void each_of_chunk(uint32_t c, F f) const
    {
        uint4 q[kWords];
        load(c, q);
#pragma unroll
        for (int i = 0; i < kWords; ++i) each(q[i], first + (c * kWords + i) * step, f);
    }
};

// The sums over a chunk whose largest value is no larger than m, in rows that
// hold -inf, NaN or an infinite m, or lie far from 0.  Apart, with the chunk
// read again, so that the common case has its registers (2048 rows of 128256
// bf16 values: 90 us, 97 with every seventh value -inf, 242 far from 0).
template <typename T>
__device__ __noinline__ Sums rare_sums(const T* x, uint32_t vocab, uint32_t rank, uint32_t blocks, uint32_t c, float m, float sc, float lo)
{
    const Share<T> S(x, vocab, rank, blocks);
    Sums a = {0.0f, 0.0f};
    const Exponent e(m, sc, lo);
    bool nan = false;
    for (int i = 0; i < kWords; ++i) {
        const uint4 q = S.in.load(S.first + (c * kWords + i) * S.step);
        float v[Word<T>::kN];
        Word<T>::values(q, v);
        nan |= word_nan<T>(q);
        if (e.plain) add_values<true>(a, v, e);
        else add_values<false>(a, v, e);
    }
    if (fabsf(m) == INFINITY) {
        a.s = a.t = nan ? NAN : 0.0f;
        return a;
    }
    correct(a, e);
    return a;
}

template <int TH>
struct TopMemory {
    float chunk_max[kBuckets][TH];
    uint64_t list[kList];
    uint16_t bucket[kBuckets * TH];   // those that hold a value of the list: index in chunk_max
    uint64_t best[DCR_MAX_TOP];    // this block's, the largest first; 0: none
    uint64_t part[TH / 32];
    uint32_t bound[TH / 32];
    uint32_t count, buckets, scan[TH / 32];
    uint64_t lists[kMaxBlocks * DCR_MAX_TOP];   // in the cluster's first block: all blocks' best
};

// The n largest of list[0..count) to best.
template <int TH>
__device__ __forceinline__ void sort_list(TopMemory<TH>& M, uint32_t count, uint32_t n)
{
    for (uint32_t i = threadIdx.x; i < count; i += TH) {
        const uint64_t mine = M.list[i];
        uint32_t above = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < count; ++j) above += M.list[j] > mine;
        if (above < n && mine != 0) M.best[above] = mine;
    }
}

// The same of `lists` sorted lists of n, one after another: in each other
// list it is searched how many are larger.
template <int TH>
__device__ __forceinline__ void merge_lists(TopMemory<TH>& M, uint32_t lists, uint32_t n)
{
    for (uint32_t i = threadIdx.x; i < lists * n; i += TH) {
        const uint64_t mine = M.lists[i];
        uint32_t above = i % n;
        for (uint32_t l = 0; l < lists; ++l) {
            if (l == i / n) continue;
            uint32_t lo = 0, hi = n;        // the first that is not larger
            while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if (M.lists[l * n + mid] > mine) lo = mid + 1;
                else hi = mid;
            }
            above += lo;
        }
        if (above < n && mine != 0) M.best[above] = mine;
    }
}

// Before a barrier: a warp's part of the bound, which at least ceil(n / W) of
// its lanes' maxima reach.
template <int TH>
__device__ __forceinline__ void start_top(TopMemory<TH>& M, float mine, uint32_t n)
{
    const uint32_t lane = threadIdx.x % 32;
    uint32_t left = order_of(mine), most = 0;
    for (uint32_t i = 0; i < (n + TH / 32 - 1) / (TH / 32); ++i) {
        most = __reduce_max_sync(~0u, left);
        const uint32_t who = __ballot_sync(~0u, left == most);
        if (lane == __ffs(who) - 1) left = 0;
    }
    if (lane == 0) M.bound[threadIdx.x / 32] = most;
    if (threadIdx.x == 0) M.count = M.buckets = 0;
    if (threadIdx.x < n) M.best[threadIdx.x] = 0;
}

template <int TH>
__device__ __forceinline__ uint32_t bound_of(const TopMemory<TH>& M)
{
    uint32_t bound = M.bound[0];
#pragma unroll
    for (uint32_t i = 1; i < TH / 32; ++i) bound = min(bound, M.bound[i]);
    return bound;
}

// The buckets that hold a value of at least this order, so that their words
// can be shared out among all threads.
template <typename T, int TH>
__device__ __forceinline__ void list_buckets(TopMemory<TH>& M, const Share<T>& S, uint32_t least)
{
    for (uint32_t b = 0; b < min(S.chunks, kBuckets); ++b)
        if (order_of(M.chunk_max[b][threadIdx.x]) >= least) M.bucket[atomicAdd(&M.buckets, 1u)] = uint16_t(b * TH + threadIdx.x);
}

// The values of at least this order of the buckets listed, to the list; where
// a value stands there does not matter.
template <typename T, int TH>
__device__ __forceinline__ void list_values(TopMemory<TH>& M, const Share<T>& S, uint32_t least)
{
    const uint32_t words = M.buckets * kWords;
    for (uint32_t i = threadIdx.x; i < words; i += TH) {
        const uint32_t from = M.bucket[i / kWords];
        for (uint32_t c = from / TH; c < S.chunks; c += kBuckets) {
            const uint32_t k = S.first - threadIdx.x + from % TH + (c * kWords + i % kWords) * S.step;
            S.each(S.in.load(k), k, [&](float v, uint32_t at) {
                if (order_of(v) >= least) {
                    const uint32_t p = atomicAdd(&M.count, 1u);
                    if (p < kList) M.list[p] = key_of(v, at);
                }
            });
        }
    }
}

// The n largest of the block's share to best, sorted, where the list does not
// hold all that reach the bound, or fewer than n do.
template <typename T, int TH>
__device__ __noinline__ void search_top(TopMemory<TH>& M, const T* x, uint32_t vocab, uint32_t rank, uint32_t blocks, uint32_t count, uint32_t n)
{
    constexpr uint32_t W = TH / 32;
    const Share<T> S(x, vocab, rank, blocks);
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, bound = bound_of(M);
    __syncthreads();
    if (count > kList) {
        // more than the list holds: those above the bound, then the first that are equal to it, then the first NaN
        if (threadIdx.x == 0) M.count = M.buckets = 0;
        __syncthreads();
        list_buckets(M, S, bound + 1);
        __syncthreads();
        const bool fits = M.buckets <= kList - DCR_MAX_TOP;
        if (fits) list_values(M, S, bound + 1);
        __syncthreads();
        count = M.count;
        if (fits && count <= kList - DCR_MAX_TOP) {
            uint32_t need = count < n ? n - count : 0, at = count;
            // a bound of -inf is also that of threads that met no number: what is missing then is NaN, of order 0
            for (uint32_t pass = 0, order = bound; pass < 2; ++pass, order = 0) {
                for (uint32_t k = S.first; need && k - threadIdx.x < S.in.words; k += S.step) {
                    // all threads go through words of one stride at a time, in the order of the indexes
                    const uint4 q = S.in.load(k);
                    uint32_t equal = 0;
                    S.each(q, k, [&](float v, uint32_t) { equal += order_of(v) == order; });
                    uint32_t before = equal;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t u = __shfl_up_sync(~0u, before, o);
                        if (lane >= uint32_t(o)) before += u;
                    }
                    __syncthreads();
                    if (lane == 31) M.scan[warp] = before;
                    __syncthreads();
                    before -= equal;
                    uint32_t all = 0;
                    for (uint32_t i = 0; i < W; ++i) {
                        if (i < warp) before += M.scan[i];
                        all += M.scan[i];
                    }
                    S.each(q, k, [&](float v, uint32_t i) {
                        if (order_of(v) == order && before++ < need) M.list[at + before - 1] = key_of(v, i);
                    });
                    const uint32_t taken = min(all, need);
                    at += taken, need -= taken;
                }
            }
            __syncthreads();
            sort_list(M, at, n);
            __syncthreads();
            return;
        }
    }
    // the largest, n times
    uint64_t last = ~0ull;
    for (uint32_t i = 0; i < n; ++i) {
        uint64_t best = 0;
        for (uint32_t c = 0; c < S.chunks; ++c)
            S.each_of_chunk(c, [&](float v, uint32_t at) {
                const uint64_t key = key_of(v, at);
                if (key < last && key > best) best = key;
            });
#pragma unroll
        for (int o = 16; o; o >>= 1) best = max(best, uint64_t(__shfl_xor_sync(~0u, static_cast<unsigned long long>(best), o)));
        __syncthreads();
        if (lane == 0) M.part[warp] = best;
        __syncthreads();
        for (uint32_t w = 0; w < W; ++w) best = max(best, M.part[w]);
        if (threadIdx.x == 0) M.best[i] = best;
        if (best == 0) break;
        last = best;
    }
    __syncthreads();
}

// A word, or four, into the shared memory of the cluster's first block.
__device__ __forceinline__ void to_first(const void* p, uint64_t v)
{
    asm volatile("{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, 0; st.shared::cluster.u64 [a], %1; }" ::"r"(uint32_t(__cvta_generic_to_shared(p))), "l"(v)
                 : "memory");
}
__device__ __forceinline__ void to_first(const void* p, const Part& v)
{
    asm volatile("{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, 0; st.shared::cluster.v4.f32 [a], {%1, %2, %3, %4}; }" ::"r"(
                     uint32_t(__cvta_generic_to_shared(p))),
                 "f"(v.m), "f"(v.count), "f"(v.s), "f"(v.t)
                 : "memory");
}

// 64 registers a thread: 80 leave a quarter of the threads out (4096 rows of
// 128256 values, 20 alternatives: 251 us), and chunks of 8 words do not fit (349).
template <typename T, int TH, bool TOP>
__global__ void __launch_bounds__(TH, 1024 / TH) scores_kernel(ScoreArgs A, uint32_t cluster)
{
    constexpr uint32_t W = TH / 32;
    __shared__ float warp_max_of[W];
    __shared__ float4 parts[W], blocks[kMaxBlocks];
    __shared__ TopMemory<TOP ? TH : 32> top_memory;
    const uint32_t rank = cluster > 1 ? blockIdx.x % cluster : 0, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint64_t row = blockIdx.x / cluster;
    const uint32_t vocab = uint32_t(A.vocab);
    const T* x = static_cast<const T*>(A.logits) + row * A.row_stride;
    const int64_t token = A.tokens[row];
    if (token < 0 || token >= int64_t(vocab)) {     // in all blocks of the row's cluster or in none
        if (rank == 0) {
            if (threadIdx.x == 0) {
                if (A.logp) A.logp[row] = 0.0f;
                if (A.entropy) A.entropy[row] = 0.0f;
                if (A.stats) A.stats[row * 3] = A.stats[row * 3 + 1] = A.stats[row * 3 + 2] = 0.0f;
            }
            for (uint32_t i = threadIdx.x; i < A.top; i += TH) A.top_logp[row * A.top + i] = 0.0f, A.top_tokens[row * A.top + i] = -1;
        }
        return;
    }
    // another block's shared memory may be written once that block is known to run: all say so here, and wait for it at the
    // end of their work
    if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    const Share<T> S(x, vocab, rank, cluster);
    // top: the sums over the chunk that the maximum m comes from (`at`); rest: those over the others
    float m = -INFINITY;
    Sums rest = {0.0f, 0.0f}, top = {0.0f, 0.0f};
    uint32_t at = 0;
    bool masked = false;
    for (uint32_t c = 0; c < S.chunks; ++c) {
        uint4 q[kWords];
        S.load(c, q);
        float cm = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWords; ++i) cm = fmaxf(cm, word_max(q[i], T()));
        if constexpr (TOP) {
            float& b = top_memory.chunk_max[c % kBuckets][threadIdx.x];
            b = c < kBuckets ? cm : fmaxf(b, cm);
        }
        const uint32_t k = S.first + c * kWords * S.step, left = k < S.in.words ? S.in.words - k : 0;
        if (left == 0) break;       // behind the row
        const bool higher = cm > m;
        if (higher) {
            rest.s += top.s, rest.t += top.t;
            if (m != -INFINITY) {       // otherwise nothing, or NaN
                const float d = (m - cm) * A.sc, f = exp2_fast(d);
                rest.t = f != 0.0f ? f * fmaf(d, rest.s, rest.t) : 0.0f * rest.s;
                rest.s *= f;
            }
            top = {0.0f, 0.0f}, m = cm, at = c;
        }
        if (m == -INFINITY) {
            // nothing so far, unless a value is none
            bool nan = false;
#pragma unroll
            for (int i = 0; i < kWords; ++i) nan |= word_nan<T>(q[i]);
            if (nan) rest.s = rest.t = NAN;
            continue;
        }
        if (masked) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) q[i] = not_below(q[i], T());
        }
        const Exponent e(m, A.sc_dn, A.sc_lo);
        Sums a = plain_sums<T>(q, e, left, S.step);
        if (!(fabsf(a.t) < INFINITY) || !e.plain) {
            // not a number where a value is -inf or none itself.  A row that holds one -inf holds more: from now on they are
            // finite values so far below the maximum (which only grows) that their part is 0
            a = rare_sums<T>(x, vocab, rank, cluster, c, m, A.sc_dn, A.sc_lo);
            masked = e.plain && (m - lowest<T>()) * A.sc > 200.0f;
        }
        else correct(a, e);
        if (higher) top = a;
        else rest.s += a.s, rest.t += a.t;
    }
    const float xy = to_f32(x[token]);      // there by the time that the sums are
    // the row's maximum in this block, and which threads have it
    float bm = value_of(__reduce_max_sync(~0u, order_of(m)));
    if (lane == 0) warp_max_of[warp] = bm;
    if constexpr (TOP) start_top(top_memory, m, A.top);
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < W; ++i) bm = fmaxf(bm, warp_max_of[i]);
    uint32_t bound = 0;
    if constexpr (TOP) {
        bound = bound_of(top_memory);
        list_buckets(top_memory, S, bound);
    }
    Part p = {m, 0.0f, rest.s + top.s, rest.t + top.t}, all = {bm, 0.0f, 0.0f, 0.0f};
    if (m == bm && m != -INFINITY) {
        // the chunk of the maximum again, without what is equal to it
        uint4 q[kWords];
        S.load(at, q);
        top = chunk_sums_below<T, kWords>(q, m, A, p.count);
        p.s = rest.s + top.s, p.t = rest.t + top.t;
    }
    all.add(p, A.sc);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        all.count += __shfl_xor_sync(~0u, all.count, o);
        all.s += __shfl_xor_sync(~0u, all.s, o);
        all.t += __shfl_xor_sync(~0u, all.t, o);
    }
    if (lane == 0) parts[warp] = make_float4(bm, all.count, all.s, all.t);
    __syncthreads();
    if constexpr (TOP) {
        // each bucket listed holds a value at least: more than the list has room for need not be collected
        const bool fits = top_memory.buckets <= kList;
        if (fits) list_values(top_memory, S, bound);
        __syncthreads();
        const uint32_t count = fits ? top_memory.count : kList + 1;
        if (count >= A.top && count <= kList) {
            sort_list(top_memory, count, A.top);
            __syncthreads();
        } else {
            search_top<T, TH>(top_memory, x, vocab, rank, cluster, count, A.top);
        }
    }
    all = {bm, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t i = 0; i < W; ++i) all.count += parts[i].y, all.s += parts[i].z, all.t += parts[i].w;
    if (cluster > 1) {
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        if (threadIdx.x == 0) to_first(&blocks[rank], all);
        if constexpr (TOP) {
            if (threadIdx.x < A.top) to_first(&top_memory.lists[rank * A.top + threadIdx.x], top_memory.best[threadIdx.x]);
        }
        asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
        if (rank == 0) {
            for (uint32_t i = 0; i < cluster; ++i) bm = fmaxf(bm, blocks[i].x);
            all = {bm, 0.0f, 0.0f, 0.0f};
            for (uint32_t i = 0; i < cluster; ++i) all.add({blocks[i].x, blocks[i].y, blocks[i].z, blocks[i].w}, A.sc);
            if constexpr (TOP) {
                merge_lists(top_memory, cluster, A.top);     // all have read best
                __syncthreads();
            }
        }
    }
    if (rank != 0) return;
    const float r = bm == INFINITY && all.s == all.s ? 0.0f : all.s + (all.count - 1.0f);
    const float lr = log1pf(r);
    const float d = fabsf(bm) == INFINITY ? NAN : -kLn2 * all.t / (1.0f + r);
    if (threadIdx.x == 0) {
        if (A.logp) A.logp[row] = (xy - bm) * A.inv_temp - lr;
        if (A.entropy) A.entropy[row] = lr + d;
        if (A.stats) A.stats[row * 3] = bm, A.stats[row * 3 + 1] = r, A.stats[row * 3 + 2] = d;
    }
    if constexpr (TOP) {
        for (uint32_t i = threadIdx.x; i < A.top; i += TH) {
            const uint64_t key = top_memory.best[i];
            A.top_logp[row * A.top + i] = (value_of(uint32_t(key >> 32)) - bm) * A.inv_temp - lr;
            A.top_tokens[row * A.top + i] = int64_t(uint32_t(~uint32_t(key)));
        }
    }
}

struct GradArgs {
    const void* logits;
    void* grad;
    uint64_t rows, vocab, row_stride, grad_stride;
    const int64_t* tokens;
    const float* stats;
    const float* grad_logp;
    const float* grad_entropy;
    float inv_temp, sc;
};

// `parts` blocks a row, each of which takes every parts-th piece of TH * NV
// words of it.
template <typename T, int TH, int NV>
__global__ void __launch_bounds__(TH) grad_kernel(GradArgs A, uint32_t parts)
{
    constexpr int N = Word<T>::kN;
    const uint64_t row = blockIdx.x / parts;
    const uint32_t vocab = uint32_t(A.vocab);
    const T* x = static_cast<const T*>(A.logits) + row * A.row_stride;
    T* g = static_cast<T*>(A.grad) + row * A.grad_stride;
    const int64_t token = A.tokens[row];
    const float ga = A.grad_logp ? A.grad_logp[row] : 0.0f, gb = A.grad_entropy ? A.grad_entropy[row] : 0.0f;
    const Row<T> in(x, vocab), out(g, vocab);
    if (token < 0 || token >= int64_t(vocab) || (ga == 0.0f && gb == 0.0f)) {
        for (uint32_t k = blockIdx.x % parts * TH + threadIdx.x; k < out.words; k += parts * TH) {
            if (out.whole(k)) *reinterpret_cast<uint4*>(out.base + uint64_t(k) * N) = make_uint4(0, 0, 0, 0);
            else store_values<T>(g, out.skip, vocab, k, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const float m = A.stats[row * 3], r = A.stats[row * 3 + 1], mean = A.stats[row * 3 + 2];
    // grad_j = e (a + b d) with d = log2 e, e = exp((x_j - m) / T), both with what their exponent has too much
    const Exponent e(m, A.sc, 0.0f);
    const float f = A.inv_temp / (1.0f + r), over = e.excess(), back = exp2f(-over);
    const float b = -gb * kLn2 * f * back, a = -(ga + (gb == 0.0f ? 0.0f : gb * mean)) * f * back - b * over;
    const bool same = out.skip == in.skip;
    const uint32_t yword = (in.skip + uint32_t(token)) / N, yat = (in.skip + uint32_t(token)) % N;
    for (uint32_t first = (blockIdx.x % parts) * (TH * NV) + threadIdx.x; first < in.words; first += parts * (TH * NV)) {
        uint4 q[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) q[i] = in.load_whole(first + i * TH);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in.cut(first + i * TH)) q[i] = in.load_cut(first + i * TH);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t k = first + i * TH;
            float v[N], w[N];
            Word<T>::values(q[i], v);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float d = max_nan(e.plain ? fmaf(v[j], e.sc, -e.msc) : (v[j] - m) * e.sc, -200.0f);
                w[j] = exp2_fast(d) * fmaf(b, d, a);
            }
            if (k == yword) {
                // the token's own value: 1 - p from the sum of the others where it is the largest
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j == int(yat)) w[j] = fmaf(ga * A.inv_temp, v[j] == m ? r / (1.0f + r) : 1.0f, v[j] == m ? -gb * mean * f : w[j]);
            }
            const uint4 z = Word<T>::pack(w);
            if (same && in.whole(k)) *reinterpret_cast<uint4*>(out.base + uint64_t(k) * N) = z;
            else if (k < in.words) store_values<T>(g, in.skip, vocab, k, z);
        }
    }
}

// 1 / T and log2(e) / T, which stay finite for the smallest T, too (0 times
// them is 0).
void scales_of(float temperature, float& inv, float& sc, float* dn, float* lo)
{
    const double most = FLT_MAX, s = std::fmin(1.4426950408889634 / temperature, most);
    inv = float(std::fmin(1.0 / temperature, most));
    sc = float(s);
    if (dn) {
        *dn = sc > s ? std::nextafterf(sc, 0.0f) : sc;
        *lo = std::fmax(float(s - *dn), FLT_TRUE_MIN);
    }
}

template <typename T, int TH>
int scores_launch(const ScoreArgs& A, uint32_t cluster, cudaStream_t s)
{
    const LaunchAttrs at(A.rows * cluster, TH, 0, cluster, false, s);
    const cudaError_t e = A.top ? cudaLaunchKernelEx(&at.cfg, scores_kernel<T, TH, true>, A, cluster)
                                : cudaLaunchKernelEx(&at.cfg, scores_kernel<T, TH, false>, A, cluster);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "token scores launch");
}

// Blocks of 128 or 256 threads, and one to eight of them for a row, whichever
// the model of a launch finds fastest: a block's chunks, each the time of
// DRAM's for what the SMs then have in flight (16 MB when full, 1024 threads an
// SM) or a load's latency, for as many blocks as come one after another on a
// slot; and in each round the steps at a row's end, which take longer where
// blocks have to meet.  (4096 rows of 128256 bf16 values, 20 alternatives: 208 us
// with 128 threads and 214 with 256, before rows with -inf were kept out of the
// slow sums, which took the first to 213; 1021 of 32771 f32 values: 35 and 41; 8
// rows of 128256 in clusters of eight: 15.4 and 12.0.)  A row of one chunk takes a
// warp, as long as its 32 maxima give a bound (2154 rows of 60, 5
// alternatives: 27 -> 15 us).
template <typename T>
int scores_launch(const ScoreArgs& A, cudaStream_t s)
{
    const uint64_t words = (A.vocab * sizeof(T) + 15) / 16 + 1;
    if (words <= 32 * kWords && A.top <= 32) return scores_launch<T, 32>(A, 1, s);
    uint32_t threads = 128, cluster = 1;
    double best = 1e300;
    for (uint32_t th = 128; th <= 256; th *= 2)
        for (uint32_t c = 1; c <= uint32_t(kMaxBlocks) && (c == 1 || (words >= uint64_t(c) * th && A.rows < 1u << 20)); c *= 2) {
            const double turns = double(A.rows) * c * th / (152.0 * 1024), chunks = std::ceil(double(words) / (c * th * kWords));
            const double us = chunks * std::max(1.0, 0.39 * kWords * std::min(1.0, turns)) * std::max(1.0, turns) + std::ceil(turns) * (c > 1 ? 6.0 : 4.0);
            if (us < best) best = us, threads = th, cluster = c;
        }
    return threads == 128 ? scores_launch<T, 128>(A, cluster, s) : scores_launch<T, 256>(A, cluster, s);
}

template <typename T, int TH, int NV>
int grad_launch(const GradArgs& A, uint64_t words, cudaStream_t s)
{
    const uint64_t parts = std::max<uint64_t>(1, std::min<uint64_t>((words + TH * NV - 1) / (TH * NV), ((1ull << 31) - 1) / A.rows));
    const LaunchAttrs at(A.rows * parts, TH, 0, 1, false, s);
    const cudaError_t e = cudaLaunchKernelEx(&at.cfg, grad_kernel<T, TH, NV>, A, uint32_t(parts));
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "token scores gradient launch");
}

int check(const char* what, const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride, const int64_t* tokens,
          float temperature)
{
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "%s: unknown dtype %u", what, dtype);
    if (!(temperature > 0.0f) || temperature > 3.0e38f) return set_error(DCR_ERR_INVALID, "%s: temperature must be positive and finite", what);
    if (vocab == 0 || vocab >= 1ull << 31 || rows >= 1ull << 28 || row_stride >= 1ull << 40)
        return set_error(DCR_ERR_INVALID, "%s: vocab must be at least 1 and below 2^31, rows below 2^28", what);
    if (row_stride < vocab) return set_error(DCR_ERR_INVALID, "%s: row_stride below vocab", what);
    if (rows && (!logits || !tokens)) return set_error(DCR_ERR_INVALID, "%s: NULL argument", what);
    if (uintptr_t(logits) % dtype_size(dtype) || uintptr_t(tokens) % 8) return set_error(DCR_ERR_INVALID, "%s: misaligned buffer", what);
    return DCR_OK;
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_token_scores(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride, const int64_t* tokens,
                                float temperature, uint32_t top, float* logp, float* entropy, float* top_logp, int64_t* top_tokens,
                                float* stats, void* stream)
{
    if (int rc = dcr::check("dcr_token_scores", logits, dtype, rows, vocab, row_stride, tokens, temperature)) return rc;
    if (top > DCR_MAX_TOP || top > vocab) return set_error(DCR_ERR_INVALID, "dcr_token_scores: top must be at most %u and vocab", DCR_MAX_TOP);
    if (rows && top && (!top_logp || !top_tokens)) return set_error(DCR_ERR_INVALID, "dcr_token_scores: NULL argument");
    if (uintptr_t(logp) % 4 || uintptr_t(entropy) % 4 || uintptr_t(top_logp) % 4 || uintptr_t(top_tokens) % 8 || uintptr_t(stats) % 4)
        return set_error(DCR_ERR_INVALID, "dcr_token_scores: misaligned buffer");
    if (rows == 0 || (!logp && !entropy && !stats && !top)) return DCR_OK;
    if (int rc = check_overlap("dcr_token_scores",
                               {{"logp", logp, rows * 4}, {"entropy", entropy, rows * 4}, {"stats", stats, rows * 12}, {"top_logp", top_logp, rows * top * 4},
                                {"top_tokens", top_tokens, rows * top * 8}},
                               {{"logits", logits, dtype_size(dtype), rows, vocab, row_stride}, {"tokens", tokens, rows * 8}}))
        return rc;
    ScoreArgs A{logits, rows, vocab, row_stride, tokens, logp, entropy, top_logp, top_tokens, stats, top};
    scales_of(temperature, A.inv_temp, A.sc, &A.sc_dn, &A.sc_lo);
    return with_dtype(dtype, [&](auto t) { return scores_launch<decltype(t)>(A, static_cast<cudaStream_t>(stream)); });
}

extern "C" int dcr_token_scores_grad(const void* logits, uint32_t dtype, uint64_t rows, uint64_t vocab, uint64_t row_stride,
                                     const int64_t* tokens, const float* stats, const float* grad_logp, const float* grad_entropy,
                                     float temperature, void* grad, uint64_t grad_stride, void* stream)
{
    if (int rc = dcr::check("dcr_token_scores_grad", logits, dtype, rows, vocab, row_stride, tokens, temperature)) return rc;
    if (rows && (!stats || !grad)) return set_error(DCR_ERR_INVALID, "dcr_token_scores_grad: NULL argument");
    if (grad_stride < vocab || grad_stride >= 1ull << 40) return set_error(DCR_ERR_INVALID, "dcr_token_scores_grad: bad grad_stride");
    if (grad == logits && grad && grad_stride != row_stride)
        return set_error(DCR_ERR_INVALID, "dcr_token_scores_grad: grad in place of logits needs the same stride");
    if (uintptr_t(grad) % dtype_size(dtype) || uintptr_t(stats) % 4 || uintptr_t(grad_logp) % 4 || uintptr_t(grad_entropy) % 4)
        return set_error(DCR_ERR_INVALID, "dcr_token_scores_grad: misaligned buffer");
    if (rows == 0) return DCR_OK;
    if (int rc = check_overlap("dcr_token_scores_grad", {{"grad", grad, dtype_size(dtype), rows, vocab, grad_stride}},
                               {{"logits", grad == logits ? nullptr : logits, dtype_size(dtype), rows, vocab, row_stride}, {"tokens", tokens, rows * 8},
                                {"stats", stats, rows * 12}, {"grad_logp", grad_logp, rows * 4}, {"grad_entropy", grad_entropy, rows * 4}}))
        return rc;
    GradArgs A{logits, grad, rows, vocab, row_stride, grad_stride, tokens, stats, grad_logp, grad_entropy};
    scales_of(temperature, A.inv_temp, A.sc, nullptr, nullptr);
    const uint64_t words = (vocab * dtype_size(dtype) + 15) / 16 + 1;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        return words <= 128 ? grad_launch<T, 128, 1>(A, words, s) : words <= 512 ? grad_launch<T, 128, 4>(A, words, s) : grad_launch<T, 256, 4>(A, words, s);
    });
}
