// Routing of tokens to experts, and its gradient (include/dcr_ops.h).
//
// A warp takes a token, each lane PER consecutive experts.  The k-th largest
// of the lanes' maxima is a bound that at least k keys reach, and few more: the
// keys that reach it go to a lane each, which counts how many are above its
// own.  Where scores are compared (with a bias, or for groups), 32 bits do not
// tell near ones apart: the bound is lowered by what such keys may be off, and
// a token of which two neighbours among the first k, or the last of them and a
// later one, are nearer than that is put in order by scores in 64 bits, a lane
// an expert (settle; about one token in a thousand), and so are groups
// (settle_groups).  Where more keys reach the bound than a warp has lanes, a
// token is decided anew in 64 bits, one expert after another.
//
// The experts' order is a counting sort that keeps the tokens' order: parts of
// the batch, one a block, count what their tokens chose (route_kernel); then
// each block adds up the counts of the parts before its own and places its
// slots (place_kernel).  A small batch takes one block and one launch.
//
// Bound by dependent steps: about 1160 instructions a token of 256 experts in
// groups with a bias (680 without either), issued on two cycles of three by half
// of the warps that an SM holds: 16381 tokens in 31 us, 21 without either, of
// which placing takes 6; their gradient in 6.4 (its 34 MB are 5).  64 tokens over
// 64 experts take 9.2 us, most of it one token's chain.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "ops_internal.h"

namespace dcr {
namespace {

struct RouteArgs {
    const void* logits;
    const float* bias;
    const uint8_t* mask;
    int32_t* chosen;
    float* weights;
    int32_t* offsets;
    int32_t* order;
    int32_t* positions;
    uint32_t* counts;       // [parts][stride]
    uint64_t tokens, row_stride;
    uint32_t experts, stride, parts, per_part;    // stride: of counts, a multiple of 4
    uint32_t k, groups, group_top, group_by, group_size;
    bool sigmoid, renormalise, by_logit;
    float scale;
};

// Order of values as whole numbers: 0 for what cannot be chosen.
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);    // -0 is 0
    return !(v > -INFINITY) ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_of(double v)
{
    const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));
    return !(v > -double(INFINITY)) ? 0ull : b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ float value_of(uint32_t o, float) { return __uint_as_float(o >> 31 ? o & 0x7FFFFFFFu : ~o); }
__device__ __forceinline__ double value_of(uint64_t o, double)
{
    return __longlong_as_double(static_cast<long long>(o >> 63 ? o & ~(1ull << 63) : ~o));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(~0u, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = max(v, uint64_t(__shfl_xor_sync(~0u, static_cast<unsigned long long>(v), o)));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

template <typename V>
__device__ __forceinline__ V sigmoid_of(V x)
{
    const V e = exp_of(x < V(0) ? x : -x);
    return (x < V(0) ? e : V(1)) / (V(1) + e);
}

// The same for keys, off by at most 7 units of 2^-24: e = exp(-|x|) is off by 4
// and 1.5 |x| units of itself (the approximation's 2 and a rounded product),
// which s (1 - s) turns into one at most; the sum's 1, the quotient's 4.
__device__ __forceinline__ float key_sigmoid(float x)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(x) * -1.44269504f));
    return __fdividef(x < 0.0f ? e : 1.0f, 1.0f + e);
}
__device__ __forceinline__ double key_sigmoid(double x) { return sigmoid_of(x); }

// exp(x - m) where m is the largest; equal infinities are 1
template <typename V>
__device__ __forceinline__ V below(V x, V m)
{
    return x == m ? V(1) : exp_of(x - m);
}

// The bias of an expert.
__device__ __forceinline__ float bias_of(const RouteArgs& A, int32_t e) { return A.bias ? A.bias[e] : 0.0f; }

// How far keys of 32 bits may be off: the error of a score in units of 2^-24
// (key_sigmoid's 7, taken as 10; for softmax the exponential's 4, a product's 1,
// those of up to 37 additions and of a difference of up to 60 from the maximum)
// for both of two neighbours, and half a unit of s + bias.
struct Slack {
    float score;
    __device__ __forceinline__ Slack(bool sigmoid, float most) : score(0x1p-24f * (sigmoid ? 20.0f : 256.0f) * most) {}
    // a is the larger one
    __device__ __forceinline__ bool near(float a, float b) const { return a - b <= score + 0x1p-23f * (fabsf(a) + fabsf(b)); }
    // How far a group's sum of two keys may be off, where `size` is the sum of their magnitudes, which may be far larger than
    // their sum's: two scores' errors, half a unit of each key and of the sum, and as much again for what is computed with it.
    __device__ __forceinline__ float of_group(float size) const { return score + 0x1p-22f * size; }
};

// A lane's consecutive values of a row, -inf behind its end; 16 bytes at a
// time where the row lies so and they are all there.
template <int PER, typename T>
__device__ __forceinline__ void load_row(const T* row, uint32_t experts, float (&x)[PER], float empty = -INFINITY)
{
    const uint32_t first = threadIdx.x % 32 * PER;
    if constexpr (PER * sizeof(T) >= 16) {
        if (first + PER <= experts && (uintptr_t(row + first) & 15) == 0) {
            constexpr int N = 16 / sizeof(T);
            uint4 q[PER / N];
#pragma unroll
            for (int i = 0; i < PER / N; ++i) q[i] = reinterpret_cast<const uint4*>(row + first)[i];
            const T* t = reinterpret_cast<const T*>(q);
#pragma unroll
            for (int i = 0; i < PER; ++i) x[i] = to_f32(t[i]);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = first + i < experts ? to_f32(row[first + i]) : empty;
}

// A softmax's maximum and 1 / sum in 64 bits, by the whole warp; nothing for sigmoid.
struct Softmax64 {
    double m, inv;
};
template <int PER, typename T>
__device__ __forceinline__ Softmax64 softmax_64(const T* row, const RouteArgs& A)
{
    Softmax64 f = {0.0, 1.0};
    if (A.sigmoid) return f;
    float x[PER], top = -INFINITY;
    load_row<PER, T>(row, A.experts, x);
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);
    f.m = double(warp_max(top));
    double s = 0.0;
    for (int i = 0; i < PER; ++i) s += x[i] > -INFINITY ? below(double(x[i]), f.m) : 0.0;
    f.inv = 1.0 / warp_sum(s);
    return f;
}
// The order of an expert's key in 64 bits.
template <typename T>
__device__ __forceinline__ uint64_t key_64(const T* row, const RouteArgs& A, const Softmax64& f, int32_t e)
{
    const double x = double(to_f32(row[e]));
    if (!(x > -double(INFINITY))) return 0;
    return order_of((A.sigmoid ? sigmoid_of(x) : below(x, f.m) * f.inv) + double(bias_of(A, e)));
}

// Lanes 0 to n - 1 hold the first `count` experts in the order of 32 bits and
// those behind them that are near to the last: put in order by their scores
// in 64 bits.  The first `count` are the choice.
template <int PER, typename T>
__device__ __noinline__ int32_t settle(const T* row, const RouteArgs& A, int32_t e, uint32_t count, uint32_t n)
{
    const uint32_t lane = threadIdx.x % 32;
    const Softmax64 f = softmax_64<PER>(row, A);
    const uint64_t v = lane < n ? key_64(row, A, f, e) : 0;
    uint32_t rank = 0;
    for (uint32_t i = 0; i < n; ++i) {
        const uint64_t w = __shfl_sync(~0u, static_cast<unsigned long long>(v), i);
        const int32_t other = __shfl_sync(~0u, e, i);
        rank += w > v || (w == v && other < e);
    }
    int32_t out = -1;
    for (uint32_t i = 0; i < n; ++i) {
        const uint32_t r = __shfl_sync(~0u, rank, i);
        const int32_t other = __shfl_sync(~0u, e, i);
        if (r == lane && lane < count) out = other;
    }
    return out;
}

// Of the groups `open`, those of the largest scores in 64 bits join the groups
// `taken` until there are group_top.
template <int PER, typename T>
__device__ __noinline__ uint32_t settle_groups(const T* row, const RouteArgs& A, uint32_t taken, uint32_t open)
{
    const uint32_t lane = threadIdx.x % 32;
    const Softmax64 f = softmax_64<PER>(row, A);
    uint64_t score = 0;
    for (uint32_t rest = open; rest; rest &= rest - 1) {
        const uint32_t g = __ffs(rest) - 1;
        uint64_t a = 0, b = 0;
        for (uint32_t i = lane; i < A.group_size; i += 32) {
            const uint64_t v = key_64(row, A, f, int32_t(g * A.group_size + i));
            b = max(b, min(a, v));
            a = max(a, v);
        }
        const uint64_t top = warp_max(a);
        const uint32_t who = __ffs(__ballot_sync(~0u, a == top)) - 1;
        const uint64_t next = warp_max(lane == who ? b : a);
        if (lane == g) score = next == 0 || A.group_by == 1 ? top : order_of(value_of(top, 0.0) + value_of(next, 0.0));
    }
    while (__popc(taken) < int(A.group_top)) {
        const uint64_t top = warp_max(score);
        if (top == 0) break;
        const uint32_t who = __ffs(__ballot_sync(~0u, score == top)) - 1;
        taken |= 1u << who;
        if (lane == who) score = 0;
    }
    return taken;
}

// The orders of all experts' keys, of type V; 0 for those that cannot be
// chosen, and for those of groups that are not taken.  bias: of PER * 32
// experts, in shared memory; most: the largest score.
template <int PER, typename T, typename V, typename O>
__device__ __forceinline__ void keys_of(const T* row, const float (&x)[PER], const float* bias, const RouteArgs& A, O (&key)[PER], float& most)
{
    constexpr bool k32 = sizeof(V) == 4;
    const uint32_t lane = threadIdx.x % 32, first = lane * PER;
    most = 1.0f;
    if (A.by_logit) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = order_of(V(x[i]));
    } else {
        V m = V(0), inv = V(1);
        if (!A.sigmoid) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);
            m = V(warp_max(top));
            V s = V(0);
#pragma unroll
            for (int i = 0; i < PER; ++i) s += x[i] > -INFINITY ? below(V(x[i]), m) : V(0);
            inv = V(1) / warp_sum(s);
            most = float(inv);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const V v = (A.sigmoid ? key_sigmoid(V(x[i])) : below(V(x[i]), m) * inv) + V(bias[first + i]);
            key[i] = x[i] > -INFINITY ? order_of(v) : O(0);
        }
    }
    if (A.groups > 1) {
        // lane g: the order of group g's score, and the magnitudes that it is the sum of
        O score = 0;
        float size = 0.0f;
        const uint32_t lanes = A.group_size / PER;
        // the sum of two keys that can be chosen is one that can, also where 32 bits do not hold it (64 always do)
        auto join = [&](O a, O b) {
            V sum = value_of(a, V()) + value_of(b, V());
            if constexpr (k32) sum = fmaxf(sum, -FLT_MAX);
            return a == 0 ? O(0) : b == 0 || A.group_by == 1 ? a : order_of(sum);
        };
        auto size_of = [&](O a, O b) {      // of numbers of 32 bits: those of 64 need no bound
            return k32 ? (a == 0 ? 0.0f : fabsf(float(value_of(a, V())))) + (b == 0 ? 0.0f : fabsf(float(value_of(b, V())))) : 0.0f;
        };
        if (lanes * PER == A.group_size && (lanes & (lanes - 1)) == 0) {
            // groups of whole lanes, a power of two of them
            O a = 0, b = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                b = max(b, min(a, key[i]));
                a = max(a, key[i]);
            }
            for (uint32_t o = 1; o < lanes; o <<= 1) {
                const O c = __shfl_xor_sync(~0u, a, o), d = __shfl_xor_sync(~0u, b, o);
                b = max(min(a, c), max(b, d));
                a = max(a, c);
            }
            score = __shfl_sync(~0u, join(a, b), (lane * lanes) & 31);
            size = __shfl_sync(~0u, size_of(a, b), (lane * lanes) & 31);
            if (lane >= A.groups) score = 0;
        } else {
            for (uint32_t g = 0; g < A.groups; ++g) {
                O a = 0, b = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const uint32_t e = first + i;
                    const O v = e >= g * A.group_size && e < (g + 1) * A.group_size ? key[i] : O(0);
                    b = max(b, min(a, v));
                    a = max(a, v);
                }
                const O top = warp_max(a);
                const uint32_t who = __ffs(__ballot_sync(~0u, a == top)) - 1;
                const O next = warp_max(lane == who ? b : a);
                if (lane == g) score = join(top, next), size = size_of(top, next);
            }
        }
        const O group = score;
        uint32_t taken = 0;
        for (uint32_t r = 0; r <= A.group_top; ++r) {
            const O top = warp_max(score);
            if (top == 0) break;
            if (r == A.group_top) {
                if constexpr (k32) {
                    if (!A.by_logit) {
                        // a group may change places if it may be lower than one that is not taken, or higher than one that is
                        // (low is 0 where an infinite error is taken from an infinite score)
                        const float v = value_of(group, 0.0f), err = Slack(A.sigmoid, most).of_group(size);
                        const bool in = taken >> lane & 1, out = group != 0 && !in;
                        const uint32_t low = order_of(v - err), high = order_of(v + err);
                        const uint32_t highest = warp_max(out ? high : 0u), lowest = ~warp_max(in ? ~low : 0u);
                        if (lowest <= highest) {
                            const uint32_t all = __ballot_sync(~0u, in ? low <= highest : out && high >= lowest);
                            taken = settle_groups<PER>(row, A, taken & ~all, all);
                        }
                    }
                }
                break;
            }
            const uint32_t who = __ffs(__ballot_sync(~0u, score == top)) - 1;
            taken |= 1u << who;
            if (lane == who) score = 0;
        }
        uint32_t g = first / A.group_size, within = first - g * A.group_size;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (g > 31 || !(taken >> g & 1)) key[i] = 0;
            if (++within == A.group_size) ++g, within = 0;
        }
    }
}

// The k best experts by keys of 64 bits, one after another: lane j's is the
// j-th (-1: none).  Apart, so that its registers do not weigh on the others.
template <int PER, typename T>
__device__ __noinline__ int32_t choose_again(const T* row, const float* bias, const RouteArgs& A)
{
    const uint32_t lane = threadIdx.x % 32, first = lane * PER;
    float x[PER], most;
    uint64_t key[PER];
    load_row<PER, T>(row, A.experts, x);
    keys_of<PER, T, double>(row, x, bias, A, key, most);
    int32_t mine = -1;
    for (uint32_t r = 0; r < A.k; ++r) {
        uint64_t best = 0;
        int32_t at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint64_t top = warp_max(best);
        if (top == 0) break;
        const uint32_t who = __ffs(__ballot_sync(~0u, best == top)) - 1;    // lanes hold ascending experts: the lowest of equal ones
        const int32_t expert = __shfl_sync(~0u, int32_t(first) + at, who);
        if (lane == r) mine = expert;
        if (lane == who) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i == at) key[i] = 0;
        }
    }
    return mine;
}

// What the warps of a block that route tokens share.
template <int PER, int TH>
struct RouteMemory {
    float bias[PER * 32];
    uint64_t lists[TH / 32][32];
    bool even;      // all biases are the same, and more than -inf
    __device__ __forceinline__ void fill(const RouteArgs& A)
    {
        bool same = true;
        const float first = bias_of(A, 0);
        for (uint32_t e = threadIdx.x; e < PER * 32; e += TH) {
            bias[e] = e < A.experts ? bias_of(A, e) : 0.0f;
            same &= e >= A.experts || bias[e] == first;
        }
        same = __syncthreads_and(same && first > -INFINITY);
        if (threadIdx.x == 0) even = same;
    }
};

// The k best experts: lane j's is the j-th (-1: none).
template <int PER, typename T, int TH>
__device__ __forceinline__ int32_t choose(const float (&x)[PER], const T* row, const RouteArgs& A, RouteMemory<PER, TH>& M)
{
    const uint32_t lane = threadIdx.x % 32, first = lane * PER;
    const float* bias = M.bias;
    uint64_t* list = M.lists[threadIdx.x / 32];
    // a row without a difference (padding, say): the first k, without the comparisons in 64 bits that so many ties would take
    const float one = __shfl_sync(~0u, x[0], 0);
    if (__all_sync(~0u, x[0] == one || first >= A.experts) && M.even && one > -INFINITY) {
        bool even = true;
#pragma unroll
        for (int i = 1; i < PER; ++i) even &= x[i] == one || first + i >= A.experts;
        if (__all_sync(~0u, even)) return lane < A.k ? int32_t(lane) : -1;
    }
    uint32_t key[PER];
    float most;
    keys_of<PER, T, float>(row, x, bias, A, key, most);
    uint32_t best = key[0], bound = 1;
#pragma unroll
    for (int i = 1; i < PER; ++i) best = max(best, key[i]);
    for (uint32_t r = 0; r < A.k; ++r) {
        const uint32_t top = warp_max(best);
        if (top == 0) {     // fewer lanes than k: all that can be chosen
            bound = 1;
            break;
        }
        const uint32_t who = __ffs(__ballot_sync(~0u, best == top)) - 1;
        if (lane == who) best = 0;
        bound = top;
    }
    const Slack slack(A.sigmoid, most);
    if (!A.by_logit && bound > 1) {
        const float b = value_of(bound, 0.0f);
        bound = max(order_of(b - slack.score - 0x1p-21f * fabsf(b)), 1u);   // (infinite - infinite: all)
    }
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = key[i] >= bound;
        const uint32_t all = __ballot_sync(~0u, in), at = n + __popc(all & ((1u << lane) - 1));
        if (in && at < 32) list[at] = uint64_t(key[i]) << 32 | (0xFFFFFFFFu - (first + i));    // the lower expert above
        n += __popc(all);
    }
    if (n > 32) return choose_again<PER, T>(row, bias, A);
    __syncwarp();
    uint64_t mine = lane < n ? list[lane] : 0;
    uint32_t rank = 0;
#pragma unroll 4
    for (uint32_t i = 0; i < n; ++i) rank += list[i] > mine;
    __syncwarp();
    if (lane < n) list[rank] = mine;
    __syncwarp();
    mine = lane < n ? list[lane] : 0;
    __syncwarp();
    const uint32_t count = min(n, A.k);
    const int32_t expert = lane < n ? int32_t(0xFFFFFFFFu - uint32_t(mine)) : -1;
    if (!A.by_logit && n > 1) {
        // each of the first `count` against the next one, those behind them against the last; equal ones are so in any precision
        const uint32_t other = lane < count ? lane + 1 : count - 1;
        const float v = value_of(uint32_t(mine >> 32), 0.0f), u = __shfl_sync(~0u, v, other & 31);
        const int32_t e = __shfl_sync(~0u, expert, other & 31);
        const bool close = lane < n && other < n && slack.near(fmaxf(u, v), fminf(u, v));
        const bool tie = close && !(to_f32(row[e]) == to_f32(row[expert]) && bias_of(A, e) == bias_of(A, expert));
        if (__any_sync(~0u, tie)) return settle<PER, T>(row, A, expert, count, count + __popc(__ballot_sync(~0u, close && lane >= count)));
    }
    return lane < count ? expert : -1;
}

struct Slot {
    int32_t expert;
    float logit;
};

// Weights of the chosen experts from their logits, before the scale; for a
// softmax that is not renormalised m and total are the row's.
__device__ __forceinline__ float weight_of(const Slot& c, bool sigmoid, bool renormalise, float m, float total)
{
    const bool on = c.expert >= 0;
    if (!renormalise) return !on ? 0.0f : sigmoid ? sigmoid_of(c.logit) : below(c.logit, m) / total;
    // relative to the largest, so that a sum of tiny scores keeps its digits
    const float top = warp_max(on ? c.logit : -INFINITY);
    float w = 0.0f;
    if (on && !sigmoid) w = below(c.logit, top);
    if (on && sigmoid) w = c.logit >= 0.0f ? sigmoid_of(c.logit) : expf(c.logit - fminf(top, 0.0f)) / (1.0f + expf(c.logit));
    const float s = warp_sum(w);
    return s > 0.0f ? w / s : 0.0f;
}

template <int PER>
__device__ __forceinline__ void softmax_of(const float (&x)[PER], float& m, float& total)
{
    m = -INFINITY, total = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) total += x[i] > -INFINITY ? below(x[i], m) : 0.0f;
    total = warp_sum(total);
}

// A token by a warp; its experts are counted in `counts`.  Returns lane j's.
template <int PER, typename T, int TH>
__device__ __forceinline__ int32_t route_token(const RouteArgs& A, uint64_t token, RouteMemory<PER, TH>& M, uint32_t* counts)
{
    const uint32_t lane = threadIdx.x % 32;
    const T* row = static_cast<const T*>(A.logits) + token * A.row_stride;
    Slot c = {-1, 0.0f};
    float w = 0.0f;
    float x[PER];
    load_row<PER, T>(row, A.experts, x);
    if (!A.mask || A.mask[token]) {
        c.expert = choose<PER, T>(x, row, A, M);
        if (c.expert >= 0) c.logit = to_f32(row[c.expert]);
        float m = 0.0f, total = 1.0f;
        if (!A.sigmoid && !A.renormalise) {
            load_row<PER, T>(row, A.experts, x);    // again: kept, it would take registers from the choice
            softmax_of(x, m, total);
        }
        w = weight_of(c, A.sigmoid, A.renormalise, m, total) * A.scale;
    }
    if (lane < A.k) {
        A.chosen[token * A.k + lane] = c.expert;
        A.weights[token * A.k + lane] = c.expert < 0 ? 0.0f : w;
        if (c.expert >= 0) atomicAdd(&counts[c.expert], 1u);
    }
    return c.expert;
}

// Exclusive sums of v[0..n) in place, by a whole block; returns the total.
template <int TH>
__device__ __forceinline__ uint32_t scan(uint32_t* v, uint32_t n)
{
    __shared__ uint32_t part[TH / 32];
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t base = 0;
    for (uint32_t at = 0; at < n; at += TH) {
        const uint32_t i = at + threadIdx.x, mine = i < n ? v[i] : 0;
        uint32_t s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(~0u, s, o);
            if (lane >= uint32_t(o)) s += u;
        }
        if (lane == 31) part[warp] = s;
        __syncthreads();
        uint32_t before = base;
        for (uint32_t w = 0; w < TH / 32; ++w) {
            if (w < warp) before += part[w];
            base += part[w];
        }
        __syncthreads();
        if (i < n) v[i] = before + s - mine;
    }
    __syncthreads();
    return base;
}

// Slots begin to end into their rows, in their order; next[e]: the next row of
// expert e.  before: [TH / 32][experts]: what the warps of a round hold of each
// expert, then what lies before each warp's.
template <int TH>
__device__ __forceinline__ void place(const RouteArgs& A, const int32_t* chosen, uint64_t begin, uint64_t end, uint32_t* next, uint16_t* before)
{
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, n = A.experts;
    for (uint64_t at = begin; at < end; at += TH) {
        const uint32_t warps = uint32_t(min((end - at + 31) / 32, uint64_t(TH / 32)));
        for (uint32_t i = threadIdx.x; i < warps * n; i += TH) before[i] = 0;
        __syncthreads();
        const uint64_t slot = at + threadIdx.x;
        const int32_t e = slot < end ? chosen[slot - begin] : -1;
        const uint32_t same = __match_any_sync(~0u, e), first = __popc(same & ((1u << lane) - 1));
        if (e >= 0 && first == 0) before[warp * n + e] = uint16_t(__popc(same));
        __syncthreads();
        uint32_t sum[(DCR_MAX_EXPERTS + TH - 1) / TH];
#pragma unroll
        for (int j = 0; j < int(DCR_MAX_EXPERTS + TH - 1) / TH; ++j) {
            const uint32_t x = threadIdx.x + j * TH;
            sum[j] = 0;
            if (x < n) {
                for (uint32_t w0 = 0; w0 < warps; w0 += 8) {
                    uint32_t v[8];
#pragma unroll
                    for (uint32_t w = 0; w < 8; ++w) v[w] = w0 + w < warps ? before[(w0 + w) * n + x] : 0;
#pragma unroll
                    for (uint32_t w = 0; w < 8; ++w) {
                        if (w0 + w < warps) before[(w0 + w) * n + x] = uint16_t(sum[j]);
                        sum[j] += v[w];
                    }
                }
            }
        }
        __syncthreads();
        if (e >= 0) {
            const uint32_t row = next[e] + before[warp * n + e] + first;
            A.order[row] = int32_t(slot);
            A.positions[slot] = int32_t(row);
        } else if (slot < end) {
            A.positions[slot] = -1;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < int(DCR_MAX_EXPERTS + TH - 1) / TH; ++j)
            if (threadIdx.x + j * TH < n) next[threadIdx.x + j * TH] += sum[j];
        __syncthreads();
    }
}

constexpr int kThreads = 256;
constexpr uint32_t kMaxParts = DCR_ROUTE_PARTS;
// Threads of a block: as many as have the registers that lanes with PER experts take.
template <int PER>
constexpr int kRouteThreads = PER <= 8 ? 1024 : 512;

template <int PER, typename T>
__global__ void __launch_bounds__(kRouteThreads<PER>) route_kernel(const RouteArgs A)
{
    constexpr int TH = kRouteThreads<PER>;
    __shared__ uint32_t counts[PER * 32];
    __shared__ RouteMemory<PER, TH> memory;
    launch_dependents();
    memory.fill(A);
    for (uint32_t e = threadIdx.x; e < A.stride; e += TH) counts[e] = 0;
    __syncthreads();
    const uint64_t begin = uint64_t(blockIdx.x) * A.per_part, end = min(begin + A.per_part, A.tokens);
    for (uint64_t t = begin + threadIdx.x / 32; t < end; t += TH / 32) route_token<PER, T, TH>(A, t, memory, counts);
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < A.stride; e += TH) A.counts[uint64_t(blockIdx.x) * A.stride + e] = counts[e];
}

// Shared memory that place() takes: 32 KB at most.
size_t place_bytes(int threads, uint32_t experts) { return size_t(threads / 32) * experts * sizeof(uint16_t); }

template <int TH>
__global__ void __launch_bounds__(TH) place_kernel(const RouteArgs A)
{
    extern __shared__ uint16_t before[];
    __shared__ uint32_t next[DCR_MAX_EXPERTS], mine[DCR_MAX_EXPERTS];   // all parts' counts, then rows; those of the parts before
    for (uint32_t e = threadIdx.x; e < A.stride; e += TH) next[e] = mine[e] = 0;
    __syncthreads();
    grid_wait();
    // a warp takes the same 128 experts, 4 a lane, of every so many parts
    constexpr uint32_t kAtOnce = 10;
    const uint32_t quads = A.stride / 4, wide = (quads + 31) / 32;
    const uint32_t per = wide <= 1 ? 1 : wide <= 2 ? 2 : wide <= 4 ? 4 : 8, quad = threadIdx.x / 32 % per * 32 + threadIdx.x % 32, step = TH / 32 / per;
    if (quad < quads) {
        uint4 all = make_uint4(0, 0, 0, 0), ours = all;
        for (uint32_t first = threadIdx.x / 32 / per; first < A.parts; first += step * kAtOnce) {
            uint4 v[kAtOnce];
#pragma unroll
            for (uint32_t i = 0; i < kAtOnce; ++i) {
                const uint32_t p = first + i * step;
                v[i] = p < A.parts ? reinterpret_cast<const uint4*>(A.counts)[uint64_t(p) * quads + quad] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (uint32_t i = 0; i < kAtOnce; ++i) {
                all.x += v[i].x, all.y += v[i].y, all.z += v[i].z, all.w += v[i].w;
                if (first + i * step < blockIdx.x) ours.x += v[i].x, ours.y += v[i].y, ours.z += v[i].z, ours.w += v[i].w;
            }
        }
        const uint32_t a[4] = {all.x, all.y, all.z, all.w}, o[4] = {ours.x, ours.y, ours.z, ours.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (a[i]) atomicAdd(&next[quad * 4 + i], a[i]);     // whole numbers: in any order
            if (o[i]) atomicAdd(&mine[quad * 4 + i], o[i]);
        }
    }
    __syncthreads();
    const uint32_t total = scan<TH>(next, A.experts);
    const uint64_t slots = A.tokens * A.k;
    if (blockIdx.x == 0) {
        for (uint32_t e = threadIdx.x; e < A.experts; e += TH) A.offsets[e] = int32_t(next[e]);
        if (threadIdx.x == 0) A.offsets[A.experts] = int32_t(total);
        __syncthreads();
    }
    for (uint64_t r = total + uint64_t(blockIdx.x) * TH + threadIdx.x; r < slots; r += uint64_t(gridDim.x) * TH) A.order[r] = -1;
    for (uint32_t e = threadIdx.x; e < A.experts; e += TH) next[e] += mine[e];
    __syncthreads();
    const uint64_t begin = min(uint64_t(blockIdx.x) * A.per_part * A.k, slots), end = min(begin + uint64_t(A.per_part) * A.k, slots);
    place<TH>(A, A.chosen + begin, begin, end, next, before);
}

// All of it for a batch of few slots, whose choices fit in shared memory.  The
// work goes by tokens, though, and one SM has it all: of 8 experts a token out of
// 64 to 256, one launch takes 6.5 to 7.6 us for 32 tokens, 9.3 to 10.9 for 64 and
// 15 to 18 for 128, two take 7.7 to 8.6 for 129 and about 9 for 1024.  Two are
// faster from about 50 tokens on, and a batch of one expert a token, which this
// bound keeps on one SM up to 1024 tokens, takes 10 to 13 us for 128 and 58 to 76
// for 1024 (8 for 1025).
constexpr uint32_t kOneSlots = 1024;

// What routing and then placing take of the shared memory, one after the other.
template <int PER>
size_t one_bytes(uint32_t experts)
{
    return std::max(sizeof(RouteMemory<PER, kRouteThreads<PER>>), place_bytes(kRouteThreads<PER>, experts));
}

template <int PER, typename T>
__global__ void __launch_bounds__(kRouteThreads<PER>) route_one_kernel(const RouteArgs A)
{
    constexpr int TH = kRouteThreads<PER>;
    extern __shared__ __align__(16) uint8_t shared[];
    __shared__ uint32_t next[PER * 32];
    __shared__ int32_t chosen[kOneSlots];
    RouteMemory<PER, TH>& memory = *reinterpret_cast<RouteMemory<PER, TH>*>(shared);
    uint16_t* before = reinterpret_cast<uint16_t*>(shared);
    memory.fill(A);
    for (uint32_t e = threadIdx.x; e < A.experts; e += TH) next[e] = 0;
    __syncthreads();
    for (uint64_t t = threadIdx.x / 32; t < A.tokens; t += TH / 32) {
        const int32_t expert = route_token<PER, T, TH>(A, t, memory, next);
        if (threadIdx.x % 32 < A.k) chosen[t * A.k + threadIdx.x % 32] = expert;
    }
    __syncthreads();
    const uint32_t total = scan<TH>(next, A.experts), slots = uint32_t(A.tokens) * A.k;
    for (uint32_t e = threadIdx.x; e < A.experts; e += TH) A.offsets[e] = int32_t(next[e]);
    if (threadIdx.x == 0) A.offsets[A.experts] = int32_t(total);
    for (uint32_t r = total + threadIdx.x; r < slots; r += TH) A.order[r] = -1;
    __syncthreads();
    place<TH>(A, chosen, 0, slots, next, before);
}

struct RouteGradArgs {
    const void* logits;
    const int32_t* chosen;
    const float* grad_weights;
    void* grad;
    uint64_t tokens, row_stride, grad_stride;
    uint32_t experts, k;
    bool sigmoid, renormalise;
    float scale;
};

// A warp a token.  With d the derivative by the weights, times the scale:
//   softmax over the chosen: w (d - sum d w);  over all: p (d - sum d p);
//   sigmoid: d s (1 - s), renormalised w (1 - s) (d - sum d w).
template <int PER, typename T>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(const RouteGradArgs A)
{
    __shared__ float rows[kThreads / 32][PER * 32];
    const uint32_t lane = threadIdx.x % 32;
    float* row = rows[threadIdx.x / 32];
    for (uint64_t t = uint64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; t < A.tokens; t += uint64_t(gridDim.x) * (kThreads / 32)) {
        const T* x = static_cast<const T*>(A.logits) + t * A.row_stride;
        Slot c = {-1, 0.0f};
        float d = 0.0f;
        if (lane < A.k) {
            c.expert = A.chosen[t * A.k + lane];
            if (uint32_t(c.expert) >= A.experts) c.expert = -1;
            if (c.expert >= 0) c.logit = to_f32(x[c.expert]), d = A.grad_weights[t * A.k + lane] * A.scale;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) row[i * 32 + lane] = 0.0f;
        __syncwarp();
        if (__any_sync(~0u, c.expert >= 0)) {
            if (A.sigmoid || A.renormalise) {
                const float w = weight_of(c, A.sigmoid, A.renormalise, 0.0f, 1.0f);
                float g = d;
                if (A.renormalise) g = w * (d - warp_sum(d * w));
                else g = w * d;
                if (A.sigmoid) g *= sigmoid_of(-c.logit);
                if (c.expert >= 0) row[c.expert] = g;
                __syncwarp();
            } else {
                float v[PER], m, total;
                load_row<PER, T>(x, A.experts, v);
                softmax_of(v, m, total);
                const float dot = warp_sum(d * weight_of(c, false, false, m, total));
                if (c.expert >= 0) row[c.expert] = d;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float p = v[i] > -INFINITY ? below(v[i], m) / total : 0.0f;
                    v[i] = p * (row[lane * PER + i] - dot);
                }
#pragma unroll
                for (int i = 0; i < PER; ++i) row[lane * PER + i] = v[i];
                __syncwarp();
            }
        }
        T* g = static_cast<T*>(A.grad) + t * A.grad_stride;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * 32 + lane < A.experts) g[i * 32 + lane] = from_f32<T>(row[i * 32 + lane]);
        __syncwarp();
    }
}

// Calls f with the experts a lane holds, as a compile-time number.
template <typename F>
int with_per(uint32_t experts, F f)
{
    if (experts <= 32) return f(std::integral_constant<int, 1>());
    if (experts <= 64) return f(std::integral_constant<int, 2>());
    if (experts <= 128) return f(std::integral_constant<int, 4>());
    if (experts <= 256) return f(std::integral_constant<int, 8>());
    if (experts <= 512) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

int route_launch(RouteArgs A, uint32_t dtype, cudaStream_t s)
{
    const bool one = A.tokens * A.k <= kOneSlots;
    cudaError_t e = cudaSuccess;
    // a part an SM, but no fewer tokens than warps
    A.per_part = uint32_t(std::max<uint64_t>((A.tokens + kMaxParts - 1) / kMaxParts, 16));
    A.parts = uint32_t((A.tokens + A.per_part - 1) / A.per_part);
    with_dtype(dtype, [&](auto t) {
        return with_per(A.experts, [&](auto per) {
            constexpr int PER = decltype(per)::value, TH = kRouteThreads<PER>;
            const LaunchAttrs at(one ? 1 : A.parts, TH, one ? one_bytes<PER>(A.experts) : 0, 1, false, s);
            e = one ? cudaLaunchKernelEx(&at.cfg, route_one_kernel<PER, decltype(t)>, A) : cudaLaunchKernelEx(&at.cfg, route_kernel<PER, decltype(t)>, A);
            return 0;
        });
    });
    if (e != cudaSuccess) return cuda_error(e, "route launch");
    if (one) return DCR_OK;
    const int th = A.experts <= 512 ? 1024 : 512;
    const LaunchAttrs at(A.parts, th, place_bytes(th, A.experts), 1, true, s);
    e = th == 1024 ? cudaLaunchKernelEx(&at.cfg, place_kernel<1024>, A) : cudaLaunchKernelEx(&at.cfg, place_kernel<512>, A);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "route launch");
}

int check_opts(const char* what, uint32_t dtype, uint64_t tokens, uint32_t experts, uint64_t row_stride, const dcr_route_opts* o)
{
    if (!o) return set_error(DCR_ERR_INVALID, "%s: NULL argument", what);
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "%s: unknown dtype %u", what, dtype);
    if (experts == 0 || experts > DCR_MAX_EXPERTS) return set_error(DCR_ERR_INVALID, "%s: experts must be 1 to %u", what, DCR_MAX_EXPERTS);
    if (o->k == 0 || o->k > DCR_MAX_CHOSEN || o->k > experts)
        return set_error(DCR_ERR_INVALID, "%s: k must be 1 to %u and at most the number of experts", what, DCR_MAX_CHOSEN);
    if (o->scoring > DCR_SIGMOID) return set_error(DCR_ERR_INVALID, "%s: unknown scoring %u", what, o->scoring);
    if (!std::isfinite(o->scale)) return set_error(DCR_ERR_INVALID, "%s: scale must be finite", what);
    if (tokens >= 1ull << 31 || tokens * o->k >= 1ull << 31) return set_error(DCR_ERR_INVALID, "%s: tokens * k must be below 2^31", what);
    if (row_stride < experts || row_stride >= 1ull << 40) return set_error(DCR_ERR_INVALID, "%s: bad row_stride", what);
    return DCR_OK;
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_route(const void* logits, uint32_t dtype, uint64_t tokens, uint32_t experts, uint64_t row_stride, const float* bias,
                         const uint8_t* mask, const dcr_route_opts* opts, int32_t* chosen, float* weights, int32_t* offsets, int32_t* order,
                         int32_t* positions, void* workspace, void* stream)
{
    if (int rc = check_opts("dcr_route", dtype, tokens, experts, row_stride, opts)) return rc;
    const dcr_route_opts& o = *opts;
    if (o.groups == 0 || o.groups > DCR_MAX_GROUPS || experts % o.groups)
        return set_error(DCR_ERR_INVALID, "dcr_route: groups must be 1 to %u and divide the experts", DCR_MAX_GROUPS);
    if (o.group_top == 0 || o.group_top > o.groups) return set_error(DCR_ERR_INVALID, "dcr_route: group_top must be 1 to groups");
    if (o.group_by != 1 && o.group_by != 2) return set_error(DCR_ERR_INVALID, "dcr_route: group_by must be 1 or 2");
    if (o.k > experts / o.groups * o.group_top) return set_error(DCR_ERR_INVALID, "dcr_route: the groups taken hold fewer than k experts");
    if (!offsets || (tokens && (!logits || !chosen || !weights || !order || !positions || !workspace)))
        return set_error(DCR_ERR_INVALID, "dcr_route: NULL argument");
    if (uintptr_t(logits) % dtype_size(dtype) || uintptr_t(bias) % 4 || uintptr_t(chosen) % 4 || uintptr_t(weights) % 4 ||
        uintptr_t(offsets) % 4 || uintptr_t(order) % 4 || uintptr_t(positions) % 4 || uintptr_t(workspace) % 16)
        return set_error(DCR_ERR_INVALID, "dcr_route: misaligned buffer");
    const uint64_t slots = tokens * o.k;
    if (int rc = check_overlap("dcr_route",
                               {{"experts", chosen, slots * 4}, {"weights", weights, slots * 4}, {"offsets", offsets, (experts + 1ull) * 4}, {"order", order, slots * 4},
                                {"positions", positions, slots * 4}, {"workspace", workspace, DCR_ROUTE_WORKSPACE(experts)}},
                               {{"logits", logits, dtype_size(dtype), tokens, experts, row_stride}, {"bias", bias, experts * 4ull}, {"mask", mask, tokens}}))
        return rc;
    RouteArgs A{};
    A.logits = logits, A.bias = bias, A.mask = mask, A.chosen = chosen, A.weights = weights, A.offsets = offsets, A.order = order;
    A.positions = positions, A.counts = static_cast<uint32_t*>(workspace), A.tokens = tokens, A.row_stride = row_stride, A.experts = experts;
    A.stride = (experts + 3) / 4 * 4;
    A.k = o.k, A.groups = o.groups, A.group_top = o.group_top, A.group_by = o.group_by, A.group_size = experts / o.groups;
    A.sigmoid = o.scoring == DCR_SIGMOID, A.renormalise = o.renormalise != 0, A.scale = o.scale;
    // one group's scores decide in the same order as the logits
    A.by_logit = !bias && (o.groups == 1 || o.group_by == 1);
    return route_launch(A, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int dcr_route_grad(const void* logits, uint32_t dtype, uint64_t tokens, uint32_t experts, uint64_t row_stride,
                              const int32_t* chosen, const float* grad_weights, const dcr_route_opts* opts, void* grad,
                              uint64_t grad_stride, void* stream)
{
    if (int rc = check_opts("dcr_route_grad", dtype, tokens, experts, row_stride, opts)) return rc;
    if (tokens && (!logits || !chosen || !grad_weights || !grad)) return set_error(DCR_ERR_INVALID, "dcr_route_grad: NULL argument");
    if (grad_stride < experts || grad_stride >= 1ull << 40) return set_error(DCR_ERR_INVALID, "dcr_route_grad: bad grad_stride");
    if (grad == logits && grad && grad_stride != row_stride)
        return set_error(DCR_ERR_INVALID, "dcr_route_grad: grad in place of logits needs the same stride");
    if (uintptr_t(logits) % dtype_size(dtype) || uintptr_t(chosen) % 4 || uintptr_t(grad_weights) % 4 || uintptr_t(grad) % dtype_size(dtype))
        return set_error(DCR_ERR_INVALID, "dcr_route_grad: misaligned buffer");
    if (tokens == 0) return DCR_OK;
    if (int rc = check_overlap("dcr_route_grad", {{"grad", grad, dtype_size(dtype), tokens, experts, grad_stride}},
                               {{"logits", grad == logits ? nullptr : logits, dtype_size(dtype), tokens, experts, row_stride},
                                {"experts", chosen, tokens * opts->k * 4}, {"grad_weights", grad_weights, tokens * opts->k * 4}}))
        return rc;
    const RouteGradArgs A{logits, chosen, grad_weights, grad, tokens, row_stride, grad_stride, experts, opts->k,
                          opts->scoring == DCR_SIGMOID, opts->renormalise != 0, opts->scale};
    const LaunchAttrs at(std::min<uint64_t>((tokens + kThreads / 32 - 1) / (kThreads / 32), 1u << 20), kThreads, 0, 1, false, static_cast<cudaStream_t>(stream));
    cudaError_t e = cudaSuccess;
    with_dtype(dtype, [&](auto t) {
        return with_per(experts, [&](auto per) {
            e = cudaLaunchKernelEx(&at.cfg, route_grad_kernel<decltype(per)::value, decltype(t)>, A);
            return 0;
        });
    });
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "route gradient launch");
}
