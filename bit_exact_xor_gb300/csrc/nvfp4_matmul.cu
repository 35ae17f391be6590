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
// warps read each row's 16 scales as one word of 16 bytes, transpose 4 x 4
// words between the four lanes that hold rows r, 32 + r, 64 + r and 96 + r,
// and leave the patches in shared memory, from where tcgen05.cp takes them.
//
// Warps: 0 TMA, 1 tensor core, 2 tensor memory, 4-7 scales, 8-11 output.
#include <cuda.h>
#include <cuda_fp8.h>

#include "ops_internal.h"

namespace dcr {
namespace {

constexpr int kThreads = 384;
constexpr int kP = 128;             // rows of P
constexpr int kStepBytes = 128;     // codes of a row in one step of K
constexpr int kStep = 256;          // values of K in one step
constexpr int kPatch = 544;         // a scale patch: 512 bytes, and 32 so that four patches start in different banks
constexpr uint64_t kWaitNs = 2000000000ull;

__device__ int g_error;             // a wait ran out (dcr_ops_status reads and clears it)

struct MatmulArgs {
    const uint8_t* p_scales;
    const uint8_t* q_scales;
    const float* x_scale;
    const float* w_scale;
    uint32_t x_scale_rows, w_scale_each;   // one scale per row of x / per expert
    uint32_t m, n, k, experts;
    uint32_t p_align, q_align;             // bytes that a row's scales may be read in at once (16, 8, 4 or 1)
    const int32_t* offsets;
    void* y;
    uint64_t y_stride;
    uint32_t y_vec;                        // y rows may be written 32 bytes at once
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

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Every wait is bounded: after two seconds, or once another warp of the block
// has given up, it returns false and the block winds down.
__device__ __noinline__ bool mbar_wait_long(uint64_t* b, uint32_t parity, volatile int* dead)
{
    const uint64_t t0 = now_ns();
    while (!*dead) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try(b, parity)) return true;
        if (now_ns() - t0 > kWaitNs) {
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

// The 16 scales of a row from byte k16 on; zeros past the row's end.
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, uint32_t k16, uint32_t n16, uint32_t align)
{
    union { uint4 v; uint2 d[2]; uint32_t w[4]; uint8_t b[16]; } u;
    u.v = make_uint4(0, 0, 0, 0);
    const uint8_t* p = row + k16;
    if (align == 16) {
        u.v = *reinterpret_cast<const uint4*>(p);
    } else if (align == 8) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (k16 + 8 * i < n16) u.d[i] = reinterpret_cast<const uint2*>(p)[i];
    } else if (align == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k16 + 4 * i < n16) u.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k16 + 4 * i + j < n16) w |= uint32_t(p[4 * i + j]) << (8 * j);
            u.w[i] = w;
        }
    }
    return u.v;
}

// Lane l of a quad holds four words of one row; afterwards it holds word l of
// the quad's four rows.
__device__ __forceinline__ uint4 transpose4(uint4 v, uint32_t lane)
{
    const bool b0 = lane & 1, b1 = lane & 2;
    uint32_t t;
    t = __shfl_xor_sync(~0u, b0 ? v.x : v.y, 1);
    (b0 ? v.x : v.y) = t;
    t = __shfl_xor_sync(~0u, b0 ? v.z : v.w, 1);
    (b0 ? v.z : v.w) = t;
    t = __shfl_xor_sync(~0u, b1 ? v.x : v.z, 2);
    (b1 ? v.x : v.z) = t;
    t = __shfl_xor_sync(~0u, b1 ? v.y : v.w, 2);
    (b1 ? v.y : v.w) = t;
    return v;
}

template <int BN>
struct Shape {
    static constexpr int kHalves = BN > 128 ? 2 : 1;              // 128-row halves of Q
    static constexpr int kTileBytes = (kP + BN) * kStepBytes;
    static constexpr int kScaleBytes = (1 + kHalves) * 4 * kPatch;
    static constexpr int kStageBytes = kTileBytes + kScaleBytes;
    static constexpr int kStages = BN == 128 || BN == 64 ? 3 : 4;
    static constexpr int kScaleCols = 16 * (1 + kHalves);         // tensor-memory columns of one stage's scales
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

template <int BN, bool XP, typename T>
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

    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint8_t* patches = smem + NS * S::kTileBytes;

    const uint32_t tile_x = XP ? kP : BN, tile_w = XP ? BN : kP;
    const uint32_t nw = (A.n + tile_w - 1) / tile_w;
    const uint32_t groups = A.experts ? A.experts : 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1), mbar_init(&scaled[i], 4), mbar_init(&empty[i], 1);
        mbar_init(&acc_full, 1);
        mbar_init(&acc_empty, 4);
        dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    auto bounds = [&](uint32_t e, uint32_t& lo, uint32_t& hi) {
        lo = 0, hi = A.m;
        if (A.offsets) {
            lo = uint32_t(min(max(A.offsets[e], 0), int(A.m)));
            hi = uint32_t(min(max(A.offsets[e + 1], 0), int(A.m)));
            hi = max(lo, hi);
        }
    };
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&C.tmem_base)), "r"(S::kAlloc) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        fence_before();
    }
    if (warp == 3) {
        uint32_t sum = 0;
        for (uint32_t e0 = 0; e0 < groups; e0 += 32) {
            uint32_t lo = 0, hi = 0;
            if (e0 + lane < groups) bounds(e0 + lane, lo, hi);
            uint32_t c = (hi - lo + tile_x - 1) / tile_x, inc = c;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                uint32_t up = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += up;
            }
            if (e0 + lane < groups) pref[e0 + lane] = sum + inc - c;
            sum += __shfl_sync(~0u, inc, 31);
        }
        if (lane == 0) pref[groups] = sum;
    }
    __syncthreads();
    fence_after();
    grid_wait();   // what is read from here on may come from the kernel before
    const uint32_t tmem = C.tmem_base;
    const uint32_t rank = split > 1 ? cluster_rank() : 0;
    const uint32_t steps = (A.k + kStep - 1) / kStep;
    const uint32_t k0 = uint64_t(steps) * rank / split, k1 = uint64_t(steps) * (rank + 1) / split;

    struct Tile { uint32_t e, x0, x1, w0; };   // expert, its rows of x from x0 (to x1 at most), first row of its matrix
    auto tile_of = [&](uint32_t t) {
        const uint32_t tt = t / nw;
        uint32_t lo = 0, hi = groups - 1;
        while (lo < hi) {
            uint32_t mid = (lo + hi + 1) / 2;
            if (pref[mid] <= tt) lo = mid;
            else hi = mid - 1;
        }
        uint32_t a, b;
        bounds(lo, a, b);
        return Tile{lo, a + (tt - pref[lo]) * tile_x, b, (t % nw) * tile_w};
    };
    const uint32_t first = blockIdx.x / split, stride = gridDim.x / split;
    // a split tile's sums are joined once a cluster; the grid has a cluster for every tile that ordered offsets make
    const uint32_t tiles = split > 1 ? min(pref[groups] * nw, stride) : pref[groups] * nw;

    if (warp == 0) {
        uint32_t it = 0;
        bool ok = true;
        if (lane == 0) {
            for (uint32_t t = first; t < tiles && ok; t += stride) {
                const Tile c = tile_of(t);
                const int xr = int(c.x0), wr = int(c.e * A.n + c.w0);
                for (uint32_t k = k0; k < k1; ++k, ++it) {
                    const uint32_t s = it % NS;
                    if (it >= NS && !(ok = mbar_wait(&empty[s], (it / NS - 1) & 1, &dead))) break;
                    uint8_t* at = smem + s * S::kTileBytes;
                    mbar_expect(&full[s], S::kTileBytes);
                    tma_load(at, &map_p, &full[s], int(k * kStepBytes), XP ? xr : wr);
                    tma_load(at + kP * kStepBytes, &map_q, &full[s], int(k * kStepBytes), XP ? wr : xr);
                }
            }
            // nothing may be in flight into this block's memory when it ends
            volatile int never = 0;
            for (uint32_t i = it > NS ? it - NS : 0; i < it; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, &never);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = (1u << 7) | (1u << 10) | (uint32_t(BN / 8) << 17) | (8u << 24);
            uint32_t it = 0, done = 0;
            bool ok = true;
            for (uint32_t t = first; t < tiles && ok; t += stride) {
                if (done > 0 && !(ok = mbar_wait(&acc_empty, (done - 1) & 1, &dead))) break;
                fence_after();
                for (uint32_t k = k0; k < k1; ++k, ++it) {
                    const uint32_t s = it % NS;
                    if (!(ok = mbar_wait(&full[s], (it / NS) & 1, &dead) && mbar_wait(&scaled[s], (it / NS) & 1, &dead))) break;
                    fence_after();
                    const uint32_t p = saddr(smem + s * S::kTileBytes), q = p + kP * kStepBytes;
                    const uint32_t sc = saddr(patches + s * S::kScaleBytes);
                    const uint32_t tp = tmem + BN + s * S::kScaleCols, tq = tp + 16;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        copy_patch(tp + 4 * j, desc_patch(sc + j * kPatch));
#pragma unroll
                        for (int h = 0; h < S::kHalves; ++h)
                            copy_patch(tq + 4 * (j * S::kHalves + h), desc_patch(sc + (4 + 4 * h + j) * kPatch));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma(tmem, desc_tile(p + 32 * j), desc_tile(q + 32 * j), idesc, tp + 4 * j, tq + 4 * j * S::kHalves,
                            k > k0 || j > 0);
                    mma_commit(&empty[s]);
                }
                mma_commit(&acc_full);
                ++done;
            }
            volatile int never = 0;
            if (done) mbar_wait(&acc_full, (done - 1) & 1, &never);
        }
    } else if (warp >= 4 && warp < 8) {
        // scales, PD steps ahead in registers
        constexpr int PD = 4, NV = 1 + S::kHalves;
        const uint32_t w = warp - 4;
        const uint32_t r = w * 8 + lane / 4, c = lane % 4;   // this lane's row 32 c + r of each 128
        const uint32_t n16 = A.k / 16;
        uint32_t it = 0;
        bool ok = true;
        for (uint32_t t = first; t < tiles && ok; t += stride) {
            const Tile tl = tile_of(t);
            const uint8_t* row[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const uint32_t i = 32 * c + r + (v == 2 ? 128 : 0);
                const bool isx = (v == 0) == XP;
                const bool in = v == 0 || i < BN;
                row[v] = nullptr;
                if (isx) {
                    if (in && tl.x0 + i < tl.x1) row[v] = (v == 0 ? A.p_scales : A.q_scales) + uint64_t(tl.x0 + i) * n16;
                } else {
                    if (in && tl.w0 + i < A.n)
                        row[v] = (v == 0 ? A.p_scales : A.q_scales) + (uint64_t(tl.e) * A.n + tl.w0 + i) * n16;
                }
            }
            auto load = [&](int v, uint32_t k) {
                if (k >= k1 || !row[v]) return make_uint4(0, 0, 0, 0);
                return load_scales(row[v], 16 * k, n16, v == 0 ? A.p_align : A.q_align);
            };
            uint4 buf[PD][NV];
#pragma unroll
            for (int d = 0; d < PD; ++d)
#pragma unroll
                for (int v = 0; v < NV; ++v) buf[d][v] = load(v, k0 + d);
            for (uint32_t kb = k0; kb < k1 && ok; kb += PD) {
#pragma unroll
                for (int d = 0; d < PD; ++d) {
                    if (kb + d < k1 && ok) {
                        const uint32_t s = it % NS;
                        if (it >= NS) ok = mbar_wait(&empty[s], (it / NS - 1) & 1, &dead);
                        ok = __all_sync(~0u, ok);
                        if (ok) {
                            uint8_t* at = patches + s * S::kScaleBytes;
#pragma unroll
                            for (int v = 0; v < NV; ++v) {
                                *reinterpret_cast<uint4*>(at + (4 * v + c) * kPatch + 16 * r) = transpose4(buf[d][v], lane);
                                buf[d][v] = load(v, kb + d + PD);
                            }
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&scaled[s]);
                            ++it;
                        }
                    }
                }
            }
        }
    } else if (warp >= 8) {
        const uint32_t w = warp - 8;
        uint32_t n = 0;
        for (uint32_t t = first; t < tiles; t += stride, ++n) {
            const Tile c = tile_of(t);
            if (!__all_sync(~0u, mbar_wait(&acc_full, n & 1, &dead))) break;
            fence_after();
            const uint32_t row = 32 * w + lane;
            const float tw = A.w_scale[A.w_scale_each ? c.e : 0];
            T* y = static_cast<T*>(A.y);
            if (XP) {
                const uint32_t m = c.x0 + row;
                const bool in = m < c.x1;
                const float sc = in ? A.x_scale[A.x_scale_rows ? m : 0] * tw : 0.0f;
                T* out = y + uint64_t(in ? m : 0) * A.y_stride + c.w0;
#pragma unroll 1
                for (int j = 0; j < BN; j += 16) {
                    uint32_t v[16];
                    tmem_load16(v, tmem + (w << 21) + j);
                    tmem_load_wait();
                    if (in) {
                        if (A.y_vec && c.w0 + j + 16 <= A.n) {
                            alignas(32) T o[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = from_f32<T>(__uint_as_float(v[i]) * sc);
                            const uint4* o4 = reinterpret_cast<const uint4*>(o);
#pragma unroll
                            for (int i = 0; i < int(sizeof(o) / 16); ++i) reinterpret_cast<uint4*>(out + j)[i] = o4[i];
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (c.w0 + j + i < A.n) out[j + i] = from_f32<T>(__uint_as_float(v[i]) * sc);
                        }
                    }
                }
            } else if (split == 1) {
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
        if (first < tiles && !XP) {
            const Tile c = tile_of(first);
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
    return a % 16 == 0 ? 16 : a % 8 == 0 ? 8 : a % 4 == 0 ? 4 : 1;
}

template <int BN, bool XP, typename T>
int launch(MatmulArgs A, const dcr_nvfp4& x, const dcr_nvfp4& w, uint32_t split, bool dependent, cudaStream_t s)
{
    using S = Shape<BN>;
    const dcr_nvfp4 &p = XP ? x : w, &q = XP ? w : x;
    const uint64_t groups = A.experts ? A.experts : 1, wrows = groups * A.n;
    CUtensorMap mp, mq;
    if (!tile_map(&mp, p.codes, XP ? A.m : wrows, A.k, kP) || !tile_map(&mq, q.codes, XP ? wrows : A.m, A.k, BN))
        return set_error(DCR_ERR_CUDA, "dcr_nvfp4_matmul: tensor map");
    A.p_scales = static_cast<const uint8_t*>(p.scales);
    A.q_scales = static_cast<const uint8_t*>(q.scales);
    A.p_align = scale_align(p.scales, A.k);
    A.q_align = scale_align(q.scales, A.k);
    const uint32_t tx = XP ? kP : BN, tw = XP ? BN : kP;
    // an expert's rows end in a tile of their own: at most one more tile an expert that has any
    uint64_t xt = (A.m + tx - 1) / tx;
    if (A.experts) xt = A.m / tx + (A.m < groups ? A.m : groups);
    const uint64_t tiles = xt * ((A.n + tw - 1) / tw);
    uint64_t grid = uint64_t(sm_count()) * S::kBlocks;
    if (tiles < grid || split > 1) grid = tiles * split;
    if (grid == 0 || grid >= 1ull << 31) return set_error(DCR_ERR_INVALID, "dcr_nvfp4_matmul: matrix too large");
    auto kernel = matmul_kernel<BN, XP, T>;
    const int smem = S::kSmem + int(sizeof(Control<S::kStages>) + 4 * groups);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_error(e, "NVFP4 product attributes");
    const LaunchAttrs at(grid, kThreads, size_t(smem), split, dependent, s);
    e = cudaLaunchKernelEx(&at.cfg, kernel, mp, mq, A, split);
    return e == cudaSuccess ? DCR_OK : cuda_error(e, "NVFP4 product launch");
}

// Which kernel: the weights are P, with Q as narrow as the tokens allow, until
// there are enough tokens that 128-token by 256-weight tiles fill the SMs.
// Few tiles are split over K among the blocks of a cluster.
template <typename T>
int choose(const MatmulArgs& A, const dcr_nvfp4& x, const dcr_nvfp4& w, bool dependent, cudaStream_t s)
{
    const uint64_t groups = A.experts ? A.experts : 1, sms = uint64_t(sm_count());
    const uint64_t each = (A.m + groups - 1) / groups;
    const uint64_t wide = ((each + 127) / 128) * ((A.n + 255) / 256) * groups;
    if (each > 64 && wide >= sms / 2) return launch<256, true, T>(A, x, w, 1, dependent, s);
    const uint64_t bn = each <= 16 ? 16 : each <= 32 ? 32 : each <= 64 ? 64 : 128;
    const uint64_t tiles = ((each + bn - 1) / bn) * ((A.n + 127) / 128) * groups;
    const uint32_t steps = (A.k + kStep - 1) / kStep;
    uint32_t split = 1;
    while (split < 8 && tiles * split * 2 <= sms * 2 && steps >= split * 4) split *= 2;
    if (bn == 16) return launch<16, false, T>(A, x, w, split, dependent, s);
    if (bn == 32) return launch<32, false, T>(A, x, w, split, dependent, s);
    if (bn == 64) return launch<64, false, T>(A, x, w, split, dependent, s);
    return launch<128, false, T>(A, x, w, split, dependent, s);
}

}  // namespace

int matmul_launch(const dcr_nvfp4& x, const dcr_nvfp4& w, uint64_t m, uint64_t n, uint64_t k, const int32_t* offsets,
                  uint32_t experts, void* y, uint32_t dtype, uint64_t y_stride, bool dependent, cudaStream_t s)
{
    MatmulArgs A{};
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
    if (int rc = dcr::check("dcr_nvfp4_matmul", *w, m, n, k, offsets, experts, y, dtype, y_stride)) return rc > 0 ? DCR_OK : rc;
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
