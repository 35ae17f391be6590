// Product of two NVFP4 operands, dense or per expert (include/dcr_ops.h), on
// the block-scaled 4-bit tensor-core instruction of sm_103a.
//
// One tile of the output is P (128 rows of one operand, the lanes of tensor
// memory) times Q (BN rows of the other, its columns), summed over K in steps
// of 256 values (128 bytes of codes a row, 16 scales).  Which operand is P
// depends on the call (choose() below): with few tokens the weights are P, so
// that no lane is wasted on tokens that do not exist.
//
// Both operands are read where a refit leaves them, row-major.  The codes
// come by TMA (128-byte swizzle, one box a step).  The instruction wants the
// scales in tensor memory, for 64 values of K as a 32-lane by 4-column patch
// in which lane r, column c holds the four scales of row 32 c + r; the scale
// warps read the rows' scales (16 bytes a row and step), transpose 4 x 4 words
// between the four lanes that hold rows r, 32 + r, 64 + r and 96 + r, and
// leave the patches in shared memory, from where tcgen05.cp takes them.
//
// Warps: 0 TMA, 1 tensor core, 2 tensor memory, 3 tile counts, 4-7 scales,
// from 8 on output.  Sums are held in 32 bits (the instruction's own; their
// error measures as that of 32-bit sums) and rounded once to y's type.
#include <cuda.h>
#include <cuda_fp8.h>

#include "ops_internal.h"

namespace dcr {
namespace {

constexpr int kThreads = 384;
constexpr int kP = 128;             // rows of P
constexpr int kStepBytes = 128;     // codes of a row in one step of K
constexpr int kStep = 256;          // values of K in one step
constexpr int kPatch = 512;         // a scale patch: 32 lanes x 16 bytes
constexpr int64_t kWaitCycles = 2000000000ll;   // a second at the highest clock

__device__ int g_error;             // a wait ran out (dcr_ops_status reads and clears it)

struct MatmulArgs {
    const uint8_t* p_scales;
    const uint8_t* q_scales;
    const float* x_scale;
    const float* w_scale;
    uint32_t x_scale_rows, w_scale_each;   // one scale per row of x / per expert
    uint32_t m, n, k, experts;
    uint32_t p_align, q_align;             // bytes that a row's scales may be read in at once (16, 4 or 1)
    const int32_t* offsets;
    void* y;
    uint64_t y_stride;
    uint32_t y_vec;                        // y rows may be written 32 bytes at once
    uint32_t stall;                        // test only: no tile is ever loaded, so that the waits run out
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t n)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok) : "r"(saddr(b)), "r"(parity) : "memory");
    return ok != 0;
}

// Every wait is bounded: after about a second, or once another warp of the block
// has given up, it returns false and the block winds down.
__device__ __forceinline__ bool mbar_wait_long(uint64_t* b, uint32_t parity, volatile int* dead)
{
    const int64_t t0 = clock64();   // (the global timer takes microseconds to read)
    while (!*dead) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try(b, parity)) return true;
        if (clock64() - t0 > kWaitCycles) {
            *dead = 1;
            atomicExch(&g_error, 1);
        }
    }
    return false;
}

__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, volatile int* dead)
{
    return mbar_try(b, parity) || mbar_wait_long(b, parity, dead);
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        ::"r"(saddr(dst)), "l"(map), "r"(saddr(bar)), "r"(x), "r"(y) : "memory");
}

// Shared-memory descriptors: rows of 128 bytes under the 128-byte swizzle
// (eight rows, 1024 bytes, from group to group), and plain 16-byte rows.
__device__ __forceinline__ uint64_t desc_tile(uint32_t addr)
{
    return uint64_t((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_patch(uint32_t addr)
{
    return uint64_t((addr >> 4) & 0x3FFF) | (8ull << 32) | (1ull << 46);
}

__device__ __forceinline__ void copy_patch(uint32_t tmem, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t add)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p; }"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add) : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t (&v)[16], uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One lane of a converged warp.  The warp that issues the tensor core's
// instructions runs its loop as a whole and elects a lane only around them,
// so that their operands are formed in uniform registers: issued from a loop
// of one lane they took 50 ns each (4096 x 4096 x 14336: 179 us instead of
// 100 without the scales' loads).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float load_cluster(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("{ .reg .b32 a; mapa.shared::cluster.u32 a, %1, %2; ld.shared::cluster.f32 %0, [a]; }"
                 : "=f"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}

// The 16 scales of a row from byte k16 on, or zeros: past the row's end, and
// where `there` is false.  FAST: rows on 16-byte boundaries; one predicated
// load, written so that nothing waits for it before its use (merged from a
// branch, the loads of a group waited for one another: 0.74 us a step instead
// of 0.41).
template <bool FAST>
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, uint32_t k16, uint32_t n16, uint32_t align, bool there)
{
    const uint8_t* p = row + k16;
    if (FAST) {
        uint4 v;
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %5, 0; mov.u32 %0, 0; mov.u32 %1, 0; mov.u32 %2, 0; mov.u32 %3, 0;\n"
            "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4]; }"
            : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"(uint32_t(there)));
        return v;
    }
    uint32_t w[4] = {0, 0, 0, 0};
    if (there) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (align == 4) {
                if (k16 + 4 * i < n16) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k16 + 4 * i + j < n16) w[i] |= uint32_t(p[4 * i + j]) << (8 * j);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A 4 x 4 matrix whose columns lie in the lanes l, l ^ A, l ^ B, l ^ (A | B),
// transposed: `at` is this lane's column.
template <int A, int B, typename V, typename X>
__device__ __forceinline__ void transpose4(V& v0, V& v1, V& v2, V& v3, uint32_t at, X xchg)
{
    const bool b0 = at & 1, b1 = at & 2;
    V t;
    t = xchg(b0 ? v0 : v1, A);
    (b0 ? v0 : v1) = t;
    t = xchg(b0 ? v2 : v3, A);
    (b0 ? v2 : v3) = t;
    t = xchg(b1 ? v0 : v2, B);
    (b1 ? v0 : v2) = t;
    t = xchg(b1 ? v1 : v3, B);
    (b1 ? v1 : v3) = t;
}
__device__ __forceinline__ uint32_t xchg1(uint32_t v, int mask) { return __shfl_xor_sync(~0u, v, mask); }
__device__ __forceinline__ uint4 xchg4(uint4 v, int mask)
{
    return make_uint4(xchg1(v.x, mask), xchg1(v.y, mask), xchg1(v.z, mask), xchg1(v.w, mask));
}

// The scale warps' work.  Lane l of warp w owns row 32 (l / 8) + 8 w + l % 8
// of each 128-row operand.  Scales are loaded for two steps at once: two
// lanes read 32 bytes (a sector) of one row together, then of the other's
// row, and exchange what is not theirs.  kAhead such pairs are in registers,
// the next tile's among them: a pair's load goes out six to eight steps ahead
// of its use.
//   rows(t, v, base, left): tile t's first row of this pair of lanes, of operand v, and how many rows there are from it on
//   put(v): one step's scales of this lane's rows; false ends it
constexpr int kAhead = 4;
template <int NV, bool FAST, typename R, typename F>
__device__ __forceinline__ void stream_scales(uint32_t lane, const uint32_t (&align)[NV], uint32_t n16, uint32_t k0, uint32_t k1,
                                              uint32_t first, uint32_t tiles, uint32_t stride, R rows, F put)
{
    if (first >= tiles) return;
    const uint8_t* base[NV];
    int32_t left[NV];
    uint32_t lt = first, lk = k0;
    auto set_rows = [&] {
#pragma unroll
        for (int v = 0; v < NV; ++v) rows(lt, v, base[v], left[v]);
    };
    set_rows();
    auto load = [&](uint4 (&b)[NV][2]) {
        const uint32_t k = lk + lane % 2;
        const bool there = lt < tiles && k < k1;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                b[v][q] = load_scales<FAST>(base[v] + (q ? n16 : 0), 16 * k, n16, align[v], there && q < left[v]);
        lk += 2;
        if (lk >= k1) {
            lk = k0;
            lt += stride;
            if (lt < tiles) set_rows();
        }
    };
    uint32_t pairs = ((tiles - first + stride - 1) / stride) * ((k1 - k0 + 1) / 2);
    uint32_t k = k0;
    auto use = [&](uint4 (&b)[NV][2]) {
        uint4 one[NV], two[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint4 t = xchg4(lane % 2 ? b[v][0] : b[v][1], 1);
            one[v] = lane % 2 ? t : b[v][0];
            two[v] = lane % 2 ? b[v][1] : t;
        }
        if (!put(one) || (k + 1 < k1 && !put(two))) return false;
        k = k + 2 < k1 ? k + 2 : k0;
        return true;
    };
    uint4 buf[kAhead][NV][2];
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(buf[d]);
    while (true) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
            if (pairs-- == 0 || !use(buf[d])) return;
            load(buf[d]);
        }
    }
}

// One operand's scales of a step into its four patches: the four lanes that
// hold rows r, 32 + r, 64 + r and 96 + r exchange words, so that each writes
// 16 bytes of one patch.
__device__ __forceinline__ void put_patches(uint8_t* at, uint32_t warp, uint4 v, uint32_t lane)
{
    transpose4<8, 16>(v.x, v.y, v.z, v.w, lane / 8, xchg1);
    *reinterpret_cast<uint4*>(at + (lane / 8) * kPatch + 16 * (8 * warp + lane % 8)) = v;
}

// Rows of x that belong to expert e: offsets cut to [0, m], none where they decrease.
__device__ __forceinline__ void expert_rows(const MatmulArgs& A, uint32_t e, uint32_t& lo, uint32_t& hi)
{
    lo = 0, hi = A.m;
    if (A.offsets) {
        lo = uint32_t(min(max(A.offsets[e], 0), int(A.m)));
        hi = max(lo, uint32_t(min(max(A.offsets[e + 1], 0), int(A.m))));
    }
}

// By one warp: token tiles of `tile` rows before each expert, and all of them.
__device__ __forceinline__ void count_tiles(const MatmulArgs& A, uint32_t tile, uint32_t* pref, uint32_t lane)
{
    const uint32_t groups = A.experts ? A.experts : 1;
    uint32_t sum = 0;
    for (uint32_t e0 = 0; e0 < groups; e0 += 32) {
        uint32_t lo = 0, hi = 0;
        if (e0 + lane < groups) expert_rows(A, e0 + lane, lo, hi);
        const uint32_t c = (hi - lo + tile - 1) / tile;
        uint32_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t up = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += up;
        }
        if (e0 + lane < groups) pref[e0 + lane] = sum + inc - c;
        sum += __shfl_sync(~0u, inc, 31);
    }
    if (lane == 0) pref[groups] = sum;
}

// Tile t: its expert, its rows of x from x0 (to x1 at most), its first row of
// the expert's matrix.  nw tiles of tile_w weight rows to each token tile.
struct Tile {
    uint32_t e, x0, x1, w0;
};
__device__ __forceinline__ Tile tile_of(const MatmulArgs& A, const uint32_t* pref, uint32_t t, uint32_t nw, uint32_t tile_x,
                                        uint32_t tile_w)
{
    const uint32_t tt = t / nw;
    uint32_t lo = 0, hi = A.experts ? A.experts - 1 : 0;
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) / 2;
        if (pref[mid] <= tt) lo = mid;
        else hi = mid - 1;
    }
    uint32_t a, b;
    expert_rows(A, lo, a, b);
    return Tile{lo, a + (tt - pref[lo]) * tile_x, b, (t % nw) * tile_w};
}

// ---- few tokens: the weights are P ---------------------------------------------------------------------------------
//
// Bound by reading the weights: 64 experts of 4096 x 6144, 512 tokens, in 138
// us (6.6 TB/s of 6.8); by latency where they are few (6144 x 2048, one token:
// 6.1 us, split in two over K).  Two blocks on an SM, each with three or four
// steps of 18 to 36 KB in flight.

template <int BN>
struct Shape {
    static constexpr int kTileBytes = (kP + BN) * kStepBytes;
    static constexpr int kScaleBytes = 2 * 4 * kPatch;
    static constexpr int kStageBytes = kTileBytes + kScaleBytes;
    static constexpr int kStages = BN == 128 || BN == 64 ? 3 : 4;
    static constexpr int kScaleCols = 32;                         // tensor-memory columns of one stage's scales
    static constexpr int kCols = BN + kStages * kScaleCols;
    static constexpr int kAlloc = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kSmem = kStages * kStageBytes;
    static constexpr int kBlocks = kSmem <= 109 * 1024 && kAlloc <= 256 ? 2 : 1;   // per SM
};

// Behind the stages in shared memory.
template <int NS>
struct Control {
    uint64_t full[NS], scaled[NS], empty[NS], acc_full, acc_empty;
    uint32_t tmem_base;
    int dead;           // a wait ran out: every warp of the block winds down
    uint32_t pref[1];   // token tiles before each expert, and all of them: one entry an expert, and one
};

template <int BN, typename T>
__global__ void __launch_bounds__(kThreads, Shape<BN>::kBlocks)
matmul_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, MatmulArgs A, uint32_t split)
{
    using S = Shape<BN>;
    constexpr int NS = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control<NS>& C = *reinterpret_cast<Control<NS>*>(smem + S::kSmem);
    uint64_t *full = C.full, *scaled = C.scaled, *empty = C.empty, &acc_full = C.acc_full, &acc_empty = C.acc_empty;
    uint32_t* pref = C.pref;
    volatile int& dead = C.dead;

    const uint32_t warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    uint8_t* patches = smem + NS * S::kTileBytes;

    const uint32_t nw = (A.n + kP - 1) / kP;
    const uint32_t groups = A.experts ? A.experts : 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1), mbar_init(&scaled[i], 4), mbar_init(&empty[i], 1);
        mbar_init(&acc_full, 1);
        mbar_init(&acc_empty, 4);
        dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&C.tmem_base)), "r"(S::kAlloc) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        fence_before();
    }
    // The offsets may be read ahead of the wait only because the kernel ahead of a dependent launch is the call's own
    // quantisation, which is itself launched without that attribute: whatever wrote the offsets has ended before it began.
    if (warp == 3) count_tiles(A, BN, pref, lane);
    grid_wait();   // what is read from here on may come from the kernel before
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(~0u, C.tmem_base, 0);
    const uint32_t rank = split > 1 ? cluster_rank() : 0;
    const uint32_t steps = (A.k + kStep - 1) / kStep;
    const uint32_t k0 = uint64_t(steps) * rank / split, k1 = uint64_t(steps) * (rank + 1) / split;

    const uint32_t first = blockIdx.x / split, stride = gridDim.x / split;
    // a split tile's sums are joined once a cluster; the grid has a cluster for every tile that ordered offsets make
    const uint32_t tiles = split > 1 ? min(pref[groups] * nw, stride) : pref[groups] * nw;

    // registers of the launch: 3 warpgroups x 80, as 56 (TMA, tensor core) + 128 (scales) + 56 (output)
    static_assert(S::kBlocks == 2, "80 registers a thread");
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
        uint32_t it = 0;
        bool ok = true;
        if (lane == 0 && !A.stall) {
            for (uint32_t t = first; t < tiles && ok; t += stride) {
                const Tile c = tile_of(A, pref, t, nw, BN, kP);
                const int xr = int(c.x0), wr = int(c.e * A.n + c.w0);
                for (uint32_t k = k0; k < k1; ++k, ++it) {
                    const uint32_t s = it % NS;
                    if (it >= NS && !(ok = mbar_wait(&empty[s], (it / NS - 1) & 1, &dead))) break;
                    uint8_t* at = smem + s * S::kTileBytes;
                    mbar_expect(&full[s], S::kTileBytes);
                    tma_load(at, &map_p, &full[s], int(k * kStepBytes), wr);
                    tma_load(at + kP * kStepBytes, &map_q, &full[s], int(k * kStepBytes), xr);
                }
            }
            // nothing may be in flight into this block's memory when it ends
            volatile int never = 0;
            for (uint32_t i = it > NS ? it - NS : 0; i < it; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, &never);
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = (1u << 7) | (1u << 10) | (uint32_t(BN / 8) << 17) | (8u << 24);
        const uint32_t base = saddr(smem), pbase = saddr(patches);
        uint32_t done = 0, s = 0, phase = 0;
        bool ok = true;
        for (uint32_t t = first; t < tiles && ok; t += stride) {
            if (done > 0) ok = __all_sync(~0u, mbar_wait(&acc_empty, (done - 1) & 1, &dead));
            if (!ok) break;
            fence_after();
            for (uint32_t k = k0; k < k1; ++k) {
                ok = mbar_wait(&full[s], phase, &dead) && mbar_wait(&scaled[s], phase, &dead);
                if (!(ok = __all_sync(~0u, ok))) break;
                fence_after();
                const uint32_t p = base + s * S::kTileBytes;
                const uint32_t tp = tmem + BN + s * S::kScaleCols, tq = tp + 16;
                const uint64_t dp = desc_tile(p), dq = desc_tile(p + kP * kStepBytes), ds = desc_patch(pbase + s * S::kScaleBytes);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        copy_patch(tp + 4 * j, ds + j * (kPatch / 16));
                        copy_patch(tq + 4 * j, ds + (4 + j) * (kPatch / 16));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma(tmem, dp + 2 * j, dq + 2 * j, idesc, tp + 4 * j, tq + 4 * j, k > k0 || j > 0);
                    mma_commit(&empty[s]);
                }
                __syncwarp();
                if (++s == NS) s = 0, phase ^= 1;
            }
            if (elect_one()) mma_commit(&acc_full);
            __syncwarp();
            ++done;
        }
        volatile int never = 0;
        if (done) mbar_wait(&acc_full, (done - 1) & 1, &never);
    }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
        const uint32_t i = 32 * (lane / 8) + 8 * (warp - 4) + (lane % 8 & ~1u);   // the first row of this pair of lanes
        const uint32_t n16 = A.k / 16, align[2] = {A.p_align, A.q_align};
        uint32_t s = 0, phase = 1;   // the first pass over the stages finds them empty
        auto rows = [&](uint32_t t, int v, const uint8_t*& base, int32_t& left) {
            const Tile tl = tile_of(A, pref, t, nw, BN, kP);
            if (v == 0) {
                base = A.p_scales + (uint64_t(tl.e) * A.n + tl.w0 + i) * n16;
                left = int32_t(A.n) - int32_t(tl.w0 + i);
            } else {
                base = A.q_scales + uint64_t(tl.x0 + i) * n16;
                left = i < BN ? int32_t(tl.x1) - int32_t(tl.x0 + i) : 0;
            }
        };
        auto put = [&](const uint4 (&v)[2]) {
            if (!__all_sync(~0u, mbar_wait(&empty[s], phase, &dead))) return false;
            uint8_t* at = patches + s * S::kScaleBytes;
            put_patches(at, warp - 4, v[0], lane);
            put_patches(at + 4 * kPatch, warp - 4, v[1], lane);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&scaled[s]);
            if (++s == NS) s = 0, phase ^= 1;
            return true;
        };
        if (align[0] == 16 && align[1] == 16) stream_scales<2, true>(lane, align, n16, k0, k1, first, tiles, stride, rows, put);
        else stream_scales<2, false>(lane, align, n16, k0, k1, first, tiles, stride, rows, put);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const uint32_t w = warp - 8;
        uint32_t n = 0;
        for (uint32_t t = first; t < tiles; t += stride, ++n) {
            const Tile c = tile_of(A, pref, t, nw, BN, kP);
            if (!__all_sync(~0u, mbar_wait(&acc_full, n & 1, &dead))) break;
            fence_after();
            const uint32_t row = 32 * w + lane;
            const float tw = A.w_scale[A.w_scale_each ? c.e : 0];
            T* y = static_cast<T*>(A.y);
            if (split == 1) {
                const uint32_t nn = c.w0 + row;
#pragma unroll 1
                for (int j = 0; j < BN; j += 16) {
                    if (c.x0 + j >= c.x1) break;
                    uint32_t v[16];
                    tmem_load16(v, tmem + (w << 21) + j);
                    tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t m = c.x0 + j + i;
                        if (m < c.x1 && nn < A.n)
                            y[uint64_t(m) * A.y_stride + nn] =
                                from_f32<T>(__uint_as_float(v[i]) * (A.x_scale[A.x_scale_rows ? m : 0] * tw));
                    }
                }
            } else {
                float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
                for (int j = 0; j < BN; j += 16) {
                    uint32_t v[16];
                    tmem_load16(v, tmem + (w << 21) + j);
                    tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(j + i) * kP + row] = __uint_as_float(v[i]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty);
        }
    }

    __syncwarp();
    if (split > 1) {
        // the cluster's blocks hold the same tile's sums over their parts of K: each adds up, in rank order, the
        // columns (tokens) that fall to it
        cluster_sync();
        if (first < tiles) {
            const Tile c = tile_of(A, pref, first, nw, BN, kP);
            const float tw = A.w_scale[A.w_scale_each ? c.e : 0];
            const uint32_t there = min(c.x1 - c.x0, uint32_t(BN));
            for (uint32_t i = rank * kThreads + threadIdx.x; i < there * kP; i += split * kThreads) {
                const uint32_t m = c.x0 + i / kP, nn = c.w0 + i % kP;
                float sum = 0.0f;
                for (uint32_t q = 0; q < split; ++q) sum += load_cluster(saddr(smem) + 4 * i, q);
                if (nn < A.n)
                    static_cast<T*>(A.y)[uint64_t(m) * A.y_stride + nn] =
                        from_f32<T>(sum * (A.x_scale[A.x_scale_rows ? m : 0] * tw));
            }
        }
        cluster_sync();
    }
    __syncthreads();
    if (warp == 2) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kAlloc));
    }
}

// ---- many tokens: tiles of 128 tokens by 256 weight rows -----------------------------------------------------------
//
// The eight output warps take all sums of a tile into registers before they
// write any, so that the next tile's products begin at once.
// 4096 x 4096 x 14336: 119 us, 4.0 PFLOP/s, with 512 tiles in four rounds of
// 152 (at 3.4 rounds' work).  The products alone take 0.40 us a step of a
// tile, 87 us in all; the scales' loads cost 25 us of the rest, for what they
// take of the bandwidth of shared memory and L1, which the operands' arrival
// (48 KB a step) and reading (48 KB) nearly fill.  64 experts of 6144 x 2048,
// 16384 tokens, 32-bit output: 178 us, 47 of them the output's 403 MB.

struct Wide {
    static constexpr int kThreads = 512;
    static constexpr int kStages = 4;
    static constexpr int kTileBytes = (kP + 256) * kStepBytes;
    static constexpr int kScaleBytes = 3 * 4 * kPatch;              // 128 tokens, 256 weight rows
    static constexpr int kScaleCols = 48;
    static constexpr int kSmem = kStages * (kTileBytes + kScaleBytes);
    static_assert(256 + kStages * kScaleCols <= 512, "tensor memory");
};

__device__ __forceinline__ void tmem_load32(uint32_t* v, uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
          "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]),
          "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}

// 32 bytes to a 32-byte boundary: a whole sector.
__device__ __forceinline__ void store32(void* p, const uint32_t* w)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float, float, float) { return 0; }

template <typename T>
__global__ void __launch_bounds__(Wide::kThreads, 1)
matmul_wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, MatmulArgs A)
{
    using S = Wide;
    constexpr int NS = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control<NS>& C = *reinterpret_cast<Control<NS>*>(smem + S::kSmem);
    uint64_t *full = C.full, *scaled = C.scaled, *empty = C.empty, &acc_full = C.acc_full, &acc_empty = C.acc_empty;
    uint32_t* pref = C.pref;
    volatile int& dead = C.dead;

    const uint32_t warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    uint8_t* patches = smem + NS * S::kTileBytes;
    const uint32_t nw = (A.n + 255) / 256;
    const uint32_t groups = A.experts ? A.experts : 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1), mbar_init(&scaled[i], 4), mbar_init(&empty[i], 1);
        mbar_init(&acc_full, 1);
        mbar_init(&acc_empty, 8);
        C.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&C.tmem_base)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        fence_before();
    }
    grid_wait();
    if (warp == 3) count_tiles(A, kP, pref, lane);
    __syncwarp();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(~0u, C.tmem_base, 0);
    const uint32_t steps = (A.k + kStep - 1) / kStep;
    const uint32_t tiles = pref[groups] * nw, first = blockIdx.x, stride = gridDim.x;

    // registers of the launch: 4 warpgroups x 128, as 56 (TMA, tensor core) + 152 (scales) + 2 x 152 (output)
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            uint32_t it = 0;
            bool ok = true;
            if (lane == 0 && !A.stall) {
                for (uint32_t t = first; t < tiles && ok; t += stride) {
                    const Tile c = tile_of(A, pref, t, nw, kP, 256);
                    const int xr = int(c.x0), wr = int(c.e * A.n + c.w0);
                    for (uint32_t k = 0; k < steps; ++k, ++it) {
                        const uint32_t s = it % NS;
                        if (it >= NS && !(ok = mbar_wait(&empty[s], (it / NS - 1) & 1, &dead))) break;
                        uint8_t* at = smem + s * S::kTileBytes;
                        mbar_expect(&full[s], S::kTileBytes);
                        tma_load(at, &map_x, &full[s], int(k * kStepBytes), xr);
                        tma_load(at + kP * kStepBytes, &map_w, &full[s], int(k * kStepBytes), wr);
                    }
                }
                // nothing may be in flight into this block's memory when it ends
                volatile int never = 0;
                for (uint32_t i = it > NS ? it - NS : 0; i < it; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, &never);
            }
        } else if (warp == 1) {
            constexpr uint32_t idesc = (1u << 7) | (1u << 10) | (uint32_t(256 / 8) << 17) | (8u << 24);
            const uint32_t base = saddr(smem), pbase = saddr(patches);
            uint32_t done = 0, s = 0, phase = 0;
            bool ok = true;
            for (uint32_t t = first; t < tiles && ok; t += stride) {
                if (done > 0) ok = __all_sync(~0u, mbar_wait(&acc_empty, (done - 1) & 1, &dead));
            if (!ok) break;
                fence_after();
                for (uint32_t k = 0; k < steps; ++k) {
                    ok = mbar_wait(&full[s], phase, &dead) && mbar_wait(&scaled[s], phase, &dead);
                if (!(ok = __all_sync(~0u, ok))) break;
                    fence_after();
                    const uint32_t p = base + s * S::kTileBytes;
                    const uint32_t tp = tmem + 256 + s * S::kScaleCols, tq = tp + 16;
                    const uint64_t dp = desc_tile(p), dq = desc_tile(p + kP * kStepBytes), ds = desc_patch(pbase + s * S::kScaleBytes);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            copy_patch(tp + 4 * j, ds + j * (kPatch / 16));
                            copy_patch(tq + 8 * j, ds + (4 + j) * (kPatch / 16));
                            copy_patch(tq + 8 * j + 4, ds + (8 + j) * (kPatch / 16));
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma(tmem, dp + 2 * j, dq + 2 * j, idesc, tp + 4 * j, tq + 8 * j, k > 0 || j > 0);
                        mma_commit(&empty[s]);
                    }
                    __syncwarp();
                    if (++s == NS) s = 0, phase ^= 1;
                }
                if (elect_one()) mma_commit(&acc_full);
                __syncwarp();
                ++done;
            }
            volatile int never = 0;
            if (done) mbar_wait(&acc_full, (done - 1) & 1, &never);
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const uint32_t i = 32 * (lane / 8) + 8 * (warp - 4) + (lane % 8 & ~1u);   // the first row of this pair of lanes
        const uint32_t n16 = A.k / 16, align[3] = {A.p_align, A.q_align, A.q_align};
        uint32_t s = 0, phase = 1;   // the first pass over the stages finds them empty
        auto rows = [&](uint32_t t, int v, const uint8_t*& base, int32_t& left) {
            const Tile tl = tile_of(A, pref, t, nw, kP, 256);
            const uint32_t wi = tl.w0 + i + (v == 2 ? kP : 0);
            base = v == 0 ? A.p_scales + uint64_t(tl.x0 + i) * n16 : A.q_scales + (uint64_t(tl.e) * A.n + wi) * n16;
            left = v == 0 ? int32_t(tl.x1) - int32_t(tl.x0 + i) : int32_t(A.n) - int32_t(wi);
        };
        auto put = [&](const uint4 (&v)[3]) {
            if (!__all_sync(~0u, mbar_wait(&empty[s], phase, &dead))) return false;
            uint8_t* at = patches + s * S::kScaleBytes;
#pragma unroll
            for (int h = 0; h < 3; ++h) put_patches(at + 4 * h * kPatch, warp - 4, v[h], lane);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&scaled[s]);
            if (++s == NS) s = 0, phase ^= 1;
            return true;
        };
        if (align[0] == 16 && align[1] == 16) stream_scales<3, true>(lane, align, n16, 0, steps, first, tiles, stride, rows, put);
        else stream_scales<3, false>(lane, align, n16, 0, steps, first, tiles, stride, rows, put);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        const uint32_t quarter = warp % 4, half = (warp - 8) / 4;
        uint32_t n = 0;
        for (uint32_t t = first; t < tiles; t += stride, ++n) {
            const Tile c = tile_of(A, pref, t, nw, kP, 256);
            if (!__all_sync(~0u, mbar_wait(&acc_full, n & 1, &dead))) break;
            fence_after();
            uint32_t v[128];
#pragma unroll
            for (int j = 0; j < 4; ++j) tmem_load32(v + 32 * j, tmem + (quarter << 21) + 128 * half + 32 * j);
            tmem_load_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty);
            const uint32_t m0 = c.x0 + 32 * quarter, m = m0 + lane, n0 = c.w0 + 128 * half;
            const float sc = m < c.x1 ? A.x_scale[A.x_scale_rows ? m : 0] * A.w_scale[A.w_scale_each ? c.e : 0] : 0.0f;
            T* const y = static_cast<T*>(A.y) + n0;
            constexpr int N = 32 / sizeof(T);   // values of a sector
            if (A.y_vec && n0 + 128 <= A.n) {
                // four lanes write 128 bytes of one of their rows at a time: whole lines, eight to an instruction
#pragma unroll
                for (int j = 0; j < 128; j += 4 * N) {
                    uint32_t u[4][8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            u[q][i] = sizeof(T) == 4 ? __float_as_uint(__uint_as_float(v[j + q * N + i % N]) * sc)
                                                     : pack2(__uint_as_float(v[j + q * N + 2 * i % N]) * sc,
                                                             __uint_as_float(v[j + q * N + (2 * i + 1) % N]) * sc, T());
                        transpose4<1, 2>(u[0][i], u[1][i], u[2][i], u[3][i], lane, xchg1);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t row = m0 + (lane & ~3u) + q;
                        if (row < c.x1) store32(y + uint64_t(row) * A.y_stride + j + N * (lane % 4), u[q]);
                    }
                }
            } else if (m < c.x1) {
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (n0 + j < A.n) y[uint64_t(m) * A.y_stride + j] = from_f32<T>(__uint_as_float(v[j]) * sc);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ---- host ---------------------------------------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

int sm_count()
{
    static const int n = [] {
        int dev = 0, v = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) v = 0;
        return v;
    }();
    return n;
}

// Comes after a call of the runtime's that needs the device's context: on a
// thread whose first call this is there is none before, and the driver's
// function fails.
bool tile_map(CUtensorMap* map, const void* codes, uint64_t rows, uint32_t k, uint32_t box_rows)
{
    const cuuint64_t dims[2] = {k / 2, rows}, strides[1] = {k / 2};
    const cuuint32_t box[2] = {kStepBytes, box_rows}, one[2] = {1, 1};
    EncodeFn fn = encode_fn();
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t scale_align(const void* p, uint32_t k)
{
    const uintptr_t a = uintptr_t(p) | (k / 16);
    return a % 16 == 0 ? 16 : a % 4 == 0 ? 4 : 1;
}

// Shared memory of a kernel whose tile counts take an entry an expert,
// allowed for the most experts in every call: the limit belongs to the kernel,
// not to the call, and another thread may launch it between this and our launch.
template <typename K>
cudaError_t allow_smem(K kernel, size_t without_counts)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(without_counts + 4 * DCR_MAX_EXPERTS));
}

template <int BN, typename T>
int launch(MatmulArgs A, const dcr_nvfp4& x, const dcr_nvfp4& w, uint32_t split, bool dependent, cudaStream_t s)
{
    using S = Shape<BN>;
    const uint64_t groups = A.experts ? A.experts : 1, wrows = groups * A.n;
    A.p_scales = static_cast<const uint8_t*>(w.scales);
    A.q_scales = static_cast<const uint8_t*>(x.scales);
    A.p_align = scale_align(w.scales, A.k);
    A.q_align = scale_align(x.scales, A.k);
    // an expert's rows end in a tile of their own: at most one more tile an expert that has any
    uint64_t xt = (A.m + BN - 1) / BN;
    if (A.experts) xt = A.m / BN + (A.m < groups ? A.m : groups);
    const uint64_t tiles = xt * ((A.n + kP - 1) / kP);
    uint64_t grid = uint64_t(sm_count()) * S::kBlocks;
    if (tiles < grid || split > 1) grid = tiles * split;
    if (grid == 0 || grid >= 1ull << 31) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: matrix too large");
    auto kernel = matmul_kernel<BN, T>;
    const size_t fixed = S::kSmem + sizeof(Control<S::kStages>);
    cudaError_t e = allow_smem(kernel, fixed);
    if (e != cudaSuccess) return cuda_error(e, "NVFP4 product attributes");
    CUtensorMap mp, mq;
    if (!tile_map(&mp, w.codes, wrows, A.k, kP) || !tile_map(&mq, x.codes, A.m, A.k, BN))
        return set_error(DCR_ERR_CUDA, "dcr_nvfp4_matmul: tensor map");
    const LaunchAttrs at(grid, kThreads, fixed + 4 * groups, split, dependent, s);
    e = cudaLaunchKernelEx(&at.cfg, kernel, mp, mq, A, split);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "NVFP4 product launch");
}

template <typename T>
int launch_wide(MatmulArgs A, const dcr_nvfp4& x, const dcr_nvfp4& w, bool dependent, cudaStream_t s)
{
    const uint64_t groups = A.experts ? A.experts : 1, wrows = groups * A.n;
    A.p_scales = static_cast<const uint8_t*>(x.scales);
    A.q_scales = static_cast<const uint8_t*>(w.scales);
    A.p_align = scale_align(x.scales, A.k);
    A.q_align = scale_align(w.scales, A.k);
    uint64_t xt = (A.m + kP - 1) / kP;
    if (A.experts) xt = A.m / kP + (A.m < groups ? A.m : groups);
    const uint64_t tiles = xt * ((A.n + 255) / 256);
    auto kernel = matmul_wide_kernel<T>;
    const size_t fixed = Wide::kSmem + sizeof(Control<Wide::kStages>);
    cudaError_t e = allow_smem(kernel, fixed);
    if (e != cudaSuccess) return cuda_error(e, "NVFP4 product attributes");
    CUtensorMap mx, mw;
    if (!tile_map(&mx, x.codes, A.m, A.k, kP) || !tile_map(&mw, w.codes, wrows, A.k, 256))
        return set_error(DCR_ERR_CUDA, "dcr_nvfp4_matmul: tensor map");
    const LaunchAttrs at(tiles < uint64_t(sm_count()) ? tiles : sm_count(), Wide::kThreads, fixed + 4 * groups, 1, dependent, s);
    e = cudaLaunchKernelEx(&at.cfg, kernel, mx, mw, A);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "NVFP4 product launch");
}

// Which kernel, by the number of tokens (of an expert) and of tiles; measured
// in us, wide against the best of the others, weights not in the L2:
//   64 experts of 4096 x 6144: 512 tokens 138 : 138, 1500 tokens 140 : 143; of 4096 x 2048: 3000 tokens 58 : 70
//   28672 x 4096 (112 wide tiles): 20 tokens 17.8 : 15.6, 37 tokens 17.6 : 18.6, 64 tokens 16.5 : 18.2
//   9728 x 4096, 48 tokens (38 tiles): 11.9 : 10.8;  14336 x 4096, 128 tokens (56 tiles): 14.3 : 16.6
//   2048 x 2048, 600 tokens (40 tiles): 9.6 : 11.4;  4096 x 14336, 300 tokens (48 tiles of 56 steps): 32 : 27
// So: wide from about 16 tokens an expert on; for one matrix from 32 tokens
// on if it gives half of the SMs a tile, and from 96 on if it gives a quarter
// of them one and the sums are not long.  Otherwise the weights are P, Q as
// narrow as the tokens allow, and few tiles are split over K among the
// blocks of a cluster, as long as the clusters find room together (two
// blocks fit an SM, but clusters do not fill every one: 9728 x 4096, 48
// tokens: split 2 11.2, 3 10.8, 4 (304 blocks) 15.5 us).
template <typename T>
int choose(const MatmulArgs& A, const dcr_nvfp4& x, const dcr_nvfp4& w, bool dependent, cudaStream_t s)
{
    const uint64_t groups = A.experts ? A.experts : 1, sms = uint64_t(sm_count());
    const uint64_t each = (A.m + groups - 1) / groups, steps = (A.k + kStep - 1) / kStep;
    const uint64_t wide = ((each + 127) / 128) * ((A.n + 255) / 256) * groups;
    if (A.experts ? each > 16 && wide * 4 >= sms
                  : (each > 32 && wide * 2 >= sms) || (each > 96 && wide * 4 >= sms && steps <= 32))
        return launch_wide<T>(A, x, w, dependent, s);
    const uint64_t bn = each <= 16 ? 16 : each <= 32 ? 32 : each <= 64 ? 64 : 128;
    const uint64_t xt = A.experts ? A.m / bn + (A.m < groups ? A.m : groups) : (A.m + bn - 1) / bn;
    const uint64_t room = sms * 17 / 10 / (xt * ((A.n + 127) / 128)), most = steps / 4 < 8 ? steps / 4 : 8;
    const uint32_t split = uint32_t(room < 1 || most < 1 ? 1 : room < most ? room : most);
    if (bn == 16) return launch<16, T>(A, x, w, split, dependent, s);
    if (bn == 32) return launch<32, T>(A, x, w, split, dependent, s);
    if (bn == 64) return launch<64, T>(A, x, w, split, dependent, s);
    return launch<128, T>(A, x, w, split, dependent, s);
}

}  // namespace

int matmul_launch(const dcr_nvfp4& x, const dcr_nvfp4& w, uint64_t m, uint64_t n, uint64_t k, const int32_t* offsets,
                  uint32_t experts, void* y, uint32_t dtype, uint64_t y_stride, bool dependent, cudaStream_t s)
{
    MatmulArgs A{};
    A.stall = (dtype & DCR_TEST_STALL) != 0;
    dtype &= ~DCR_TEST_STALL;
    A.x_scale = x.scale, A.w_scale = w.scale;
    A.x_scale_rows = x.scale_count > 1, A.w_scale_each = w.scale_count > 1;
    A.m = uint32_t(m), A.n = uint32_t(n), A.k = uint32_t(k), A.experts = experts;
    A.offsets = offsets, A.y = y, A.y_stride = y_stride;
    A.y_vec = uintptr_t(y) % 32 == 0 && y_stride * dtype_size(dtype) % 32 == 0;
    return with_dtype(dtype, [&](auto t) { return choose<decltype(t)>(A, x, w, dependent, s); });
}

namespace {

// What dcr_nvfp4_matmul and dcr_nvfp4_linear refuse alike; 1 if there is nothing to do.
int check(const char* what, const dcr_nvfp4& w, uint64_t m, uint64_t n, uint64_t k, const int32_t* offsets,
          uint32_t experts, const void* y, uint32_t dtype, uint64_t y_stride)
{
    if (dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "%s: unknown dtype %u", what, dtype);
    if (k == 0 || k % 32) return set_error(DCR_ERR_INVALID, "%s: k must be a positive multiple of 32", what);
    if (experts > DCR_MAX_EXPERTS) return set_error(DCR_ERR_INVALID, "%s: more than %u experts", what, DCR_MAX_EXPERTS);
    if ((experts > 0) != (offsets != nullptr))
        return set_error(DCR_ERR_INVALID, "%s: experts and offsets do not go together", what);
    const uint64_t wrows = n * (experts ? experts : 1);
    if (m >= 1ull << 31 || n >= 1ull << 31 || k >= 1ull << 31 || wrows >= 1ull << 31 || y_stride >= 1ull << 40)
        return set_error(DCR_ERR_INVALID, "%s: matrix too large", what);
    if (y_stride < n) return set_error(DCR_ERR_INVALID, "%s: y_stride below n", what);
    if (w.scale_count != 1 && (experts == 0 || w.scale_count != experts))
        return set_error(DCR_ERR_INVALID, "%s: w needs one scale or one per expert", what);
    if (m == 0 || n == 0) return 1;
    if (!w.codes || !w.scales || !w.scale || !y) return set_error(DCR_ERR_INVALID, "%s: NULL argument", what);
    if (uintptr_t(w.codes) % 16 || uintptr_t(y) % dtype_size(dtype) || uintptr_t(w.scale) % 4 || uintptr_t(offsets) % 4)
        return set_error(DCR_ERR_INVALID, "%s: misaligned buffer", what);
    return DCR_OK;
}

}  // namespace
}  // namespace dcr

using namespace dcr;

extern "C" int dcr_nvfp4_matmul(const dcr_nvfp4* x, const dcr_nvfp4* w, uint64_t m, uint64_t n, uint64_t k,
                                const int32_t* offsets, uint32_t experts, void* y, uint32_t dtype, uint64_t y_stride,
                                void* stream)
{
    if (!x || !w) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: NULL argument");
    if (x->scale_count != 1 && x->scale_count != m)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: x needs one scale or one per row");
    if (int rc = dcr::check("dcr_nvfp4_matmul", *w, m, n, k, offsets, experts, y, dtype & ~DCR_TEST_STALL, y_stride))
        return rc > 0 ? DCR_OK : rc;
    if (!x->codes || !x->scales || !x->scale) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: NULL argument");
    if (uintptr_t(x->codes) % 16 || uintptr_t(x->scale) % 4)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: misaligned buffer");
    return matmul_launch(*x, *w, m, n, k, offsets, experts, y, dtype, y_stride, false, static_cast<cudaStream_t>(stream));
}

extern "C" int dcr_nvfp4_linear(const void* x, uint32_t x_dtype, uint64_t x_stride, const dcr_nvfp4* w, uint64_t m,
                                uint64_t n, uint64_t k, const int32_t* offsets, uint32_t experts, void* y, uint32_t dtype,
                                uint64_t y_stride, void* workspace, void* stream)
{
    if (!w) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_linear: NULL argument");
    if (x_dtype > DCR_F16) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_linear: unknown dtype %u", x_dtype);
    if (int rc = dcr::check("dcr_nvfp4_linear", *w, m, n, k, offsets, experts, y, dtype, y_stride)) return rc > 0 ? DCR_OK : rc;
    if (!x || !workspace) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_linear: NULL argument");
    if (x_stride < k || x_stride >= 1ull << 40) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_linear: bad x_stride");
    if (uintptr_t(x) % dtype_size(x_dtype) || uintptr_t(workspace) % 16)
        return set_error(DCR_ERR_INVALID, "dcr_nvfp4_linear: misaligned buffer");
    // k is a multiple of 32: the scales start on a 16-byte boundary, the rows' scales on one of 4
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* scales = codes + m * (k / 2);
    float* scale = reinterpret_cast<float*>(scales + (m * (k / 16) + 3) / 4 * 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = quantize_launch(x, x_dtype, m, k, x_stride, DCR_SCALE_ROW, scale, codes, scales, nullptr, DCR_NONE, nullptr, s))
        return rc;
    return matmul_launch(dcr_nvfp4{codes, scales, scale, m}, *w, m, n, k, offsets, experts, y, dtype, y_stride, true, s);
}

extern "C" int dcr_ops_status(void* stream)
{
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    int err = 0, zero = 0;
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&err, g_error, sizeof(err));
    if (e == cudaSuccess && err) e = cudaMemcpyToSymbol(g_error, &zero, sizeof(zero));
    if (e != cudaSuccess) return cuda_error(e, "dcr_ops_status");
    return err ? set_error(DCR_ERR_TIMEOUT, "an operator's wait on the device gave up; its output is incomplete") : DCR_OK;
}
