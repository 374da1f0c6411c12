// Orthogonalised update of a stack of gradients (mxfp8_muon_update): momentum,
// Frobenius norm, Newton-Schulz products on the tensor cores.
//
// With X the m x n matrix whose rows are the gradient's shorter side, one step is
//   A = X X^T;   R = b A + c A A - beta I;   X <- (a + beta) X + R X
// for any beta (the shift changes nothing but the rounding of R: near the end
// the eigenvalues of A gather around 1, where b A + c A A is about b + c, so
// the last step takes beta = 0.875 (b + c) and the one before half of that, and
// R's largest part, its diagonal, is not rounded).
//
// Precision. The products run on fp16 operands (11 significant bits, eight
// times finer than bf16 at the same rate) scaled by powers of two so that the
// magnitudes that occur neither overflow nor meet fp16's subnormals (A and R end
// at 16, so ||X||_2 at 4: the entry point refuses coefficients that can lead
// there); the accumulators are fp32. Rounding X itself to 11 bits would cost
// more: its error is spread over all directions while every step multiplies a
// small singular value by a = 3.4, so that the error of the first steps grows
// a hundredfold beside what it is to be compared with. The a X term therefore
// takes X from two fp16 planes (22 bits); in R X only R's dominant directions
// see the rounding of X. (Roundings simulated in 64 bits, five steps, on
// normal, heavy-tailed, decaying and low-rank spectra with shorter sides of 96 and
// more: 0.4e-3 .. 1.7e-3 relative error, against 3e-3 .. 27e-3 with one plane and
// 3e-3 .. 59e-3 in bf16. Shorter sides of 8 .. 52: up to 4e-3. Sixteen steps: 5e-3
// as a rule, 1e-2 .. 6e-2 where the map is steep at some singular values; the error
// is about a thousand times that of the same iteration in fp32 throughout. The
// shift in earlier steps too would amplify the noise of directions that u does
// not have: rank 3, eight steps, 1.5e-3 -> 26e-3.)
//
// Kernels of a call: muon_momentum (momentum, partial sums of u^2), muon_scale
// (X0 = u / norm into its two planes, transposed for tall matrices), muon_main:
// persistent CTA pairs over all products of all steps, as one list of 256 x 256
// tiles ordered by product; a tile waits for the product before it of its own
// matrix only, so with several matrices the pairs never drain between
// products. A A^T-type products are symmetric: only tiles on and below the
// diagonal are computed and each is stored twice.
//
// What bounds it (five steps, momentum). Many tiles, 8 x 1408 x 2048: 584 us a
// call, of which muon_main 480 for 599 GFLOP, 1.25 PFLOP/s; its tensor pipe is
// active in 72% of the cycles. The rest is the SM's intake: operands at the full
// rate of the MMA use all of its 64 bytes a clock, and the epilogue's reads of
// earlier products and planes compete with them (without an epilogue the
// same list of products takes 330 us). 32 x 7168 x 2048: 13.7 ms for 15.8 TFLOP.
// Few tiles, 3 x 331 x 1000: 113 us, a chain of 15 products of about 7 us each:
// hand-over 1, first operands 0.85, products 1.75, epilogue 2.2, stores
// and their report 1.3 to 2.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "mxw_experts.h"
#include "mxw_internal.h"
#include "muon_norm.cuh"
#include "mxw_ptx_single.cuh"
#include "../../include/mxfp8_experts.h"

namespace mxw {
namespace {

constexpr int NORM_BLOCKS = 256;     // partial sums per matrix
constexpr int TILE = 256;            // rows of a pair's tile (each CTA: 128); its columns: 256 or 128
constexpr int HALF = TILE / 2;
constexpr int KSTEP = 64;            // contraction columns of a stage (128 bytes)
constexpr int OP_BYTES = HALF * KSTEP * 2;
constexpr int STAGES = 5;
constexpr int EPI0 = 2, EPI_WARPS = 8;
constexpr int SCOUT = EPI0 + EPI_WARPS;  // warp that waits for the products that a tile needs
constexpr int THREADS = 32 * (SCOUT + 1);
constexpr int AHEAD = 4;             // tiles the scout may be ahead
constexpr int SLOT = 32 * 128;       // 32 rows x 64 columns of fp16; two slots per epilogue warp
constexpr int OFF_EPI = STAGES * 2 * OP_BYTES, OFF_BAR = OFF_EPI + 2 * EPI_WARPS * SLOT;
constexpr int SMEM = OFF_BAR + 1024 + 512;
static_assert(SMEM <= 232448, "shared memory of a CTA");
// powers of two that the stored matrices are scaled by
constexpr float SX = 2048.f;         // X
constexpr float SLO = 2048.f;        // lower plane of X, on top of SX
constexpr float SA = 4096.f;         // A and R
// kind::f16: fp16 x fp16 -> fp32, M = 256 across the pair; bits 17-22: N / 8; bit 16: B is MN-major
constexpr uint32_t IDESC = (1u << 4) | (static_cast<uint32_t>(TILE >> 4) << 24);

struct Params {
    int E, m, n, ldm, ldn, steps, tall, tn, T, sym, full;  // columns of a tile; tiles along m; tiles of a symmetric product and of R X
    int parts;           // pieces into which the contraction of X X^T is cut
    float* part;         // [E][sym][parts][2 CTAs][8 warps][tn / 2 columns][32 rows]
    unsigned int* arrived;  // [E][sym][2][8] pieces done
    float a, b, c;
    __half *Xh, *Xl;     // X0's planes
    unsigned int* done;  // [E][3 steps] epilogue warps' shares of tiles stored
    unsigned long long wait_ns;
    int* status;
    int stall;           // test hook: over-declare the first stage's bytes so that its wait runs out
};

struct Maps {
    // X by rows (as the MMA's M and N sides) and by 64 x 64 boxes (its columns as the N side), A likewise, R
    CUtensorMap xk[2], xkn[2], xm[2], a, an, r;
    CUtensorMap exh[2], exl[2], ea, er, eout;  // epilogue: boxes of 32 rows x 64 columns
    CUtensorMap ta, tr, tout;                  // transposed: boxes of 32 x 32
};

// ============================================================== momentum, norm, X0

__device__ __forceinline__ float2 bf16x2_f(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Four values of u at element i (a multiple of 4); FIRST also updates the momentum.
template <bool FIRST>
__device__ __forceinline__ float4 load_u(const MuonArgs& a, size_t i) {
    float4 g;
    if (a.grad_f32) {
        g = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.grad) + i));
    } else {
        const uint2 r = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.grad) + i));
        const float2 lo = bf16x2_f(r.x), hi = bf16x2_f(r.y);
        g = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    if (!a.momentum) return g;
    float4 m = *reinterpret_cast<const float4*>(a.momentum + i);
    if (FIRST) {
        m = make_float4(fmaf(a.mu, m.x, g.x), fmaf(a.mu, m.y, g.y), fmaf(a.mu, m.z, g.z), fmaf(a.mu, m.w, g.w));
        *reinterpret_cast<float4*>(a.momentum + i) = m;
    }
    if (!a.nesterov) return m;
    return make_float4(fmaf(a.mu, m.x, g.x), fmaf(a.mu, m.y, g.y), fmaf(a.mu, m.z, g.z), fmaf(a.mu, m.w, g.w));
}

// One pass: momentum in place, a block's partial sums of u^2 and of (2^100 u)^2:
// where the first has left fp32's normal range below, the second is exact (and
// finite). HBM-bound: 10 bytes
// an element with bf16 gradients, 35 us at 8 x 1408 x 2048 (6.6 TB/s). A block's
// share is contiguous and the partial sums are joined in block order by
// muon_scale: the same bits on every run.
__global__ void __launch_bounds__(256) muon_momentum(const MuonArgs a, float2* part, unsigned int* done, int n_done) {
    griddep_launch_dependents();
    griddep_wait();  // the gradient may come from the kernel before, and a call before may still use the scratch
    const size_t per = static_cast<size_t>(a.N) * a.K, base = blockIdx.y * per;
    float s = 0.f, t = 0.f;
    const size_t share = (per / 4 + NORM_BLOCKS - 1) / NORM_BLOCKS * 4, end = min(per, (blockIdx.x + 1) * share);
    for (size_t i = blockIdx.x * share + 4 * threadIdx.x; i < end; i += 4 * 256) {
        const float4 u = load_u<true>(a, base + i);
        s += (u.x * u.x + u.y * u.y) + (u.z * u.z + u.w * u.w);
        const float4 v = make_float4(u.x * NORM_UP, u.y * NORM_UP, u.z * NORM_UP, u.w * NORM_UP);
        t += (v.x * v.x + v.y * v.y) + (v.z * v.z + v.w * v.w);
    }
    __shared__ float2 red[8];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, d);
        t += __shfl_xor_sync(0xffffffffu, t, d);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(s, t);
    __syncthreads();
    if (threadIdx.x == 0) {
        s = t = 0.f;
        for (int w = 0; w < 8; ++w) {
            s += red[w].x;
            t += red[w].y;
        }
        part[blockIdx.y * NORM_BLOCKS + blockIdx.x] = make_float2(s, t);
    }
    for (int i = (blockIdx.y * NORM_BLOCKS + blockIdx.x) * 256 + threadIdx.x; i < n_done; i += gridDim.y * NORM_BLOCKS * 256)
        done[i] = 0;
}

// X0 in two planes; tall matrices are transposed on the way, 64 x 64 at a time.
// u is formed again from gradient and momentum (a third array of u would cost as
// much to write as this saves). HBM-bound: 10 bytes an element, 41 us at
// 8 x 1408 x 2048 (5.6 TB/s).
__global__ void __launch_bounds__(256) muon_scale(const MuonArgs a, const Params p, const float2* part) {
    __shared__ float t[64][65];
    __shared__ float2 s_norm;
    griddep_launch_dependents();
    griddep_wait();
    const int e = blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    if (threadIdx.x < 32) {
        float s = 0.f, up = 0.f;
#pragma unroll
        for (int i = 0; i < NORM_BLOCKS / 32; ++i) {
            const float2 v = part[e * NORM_BLOCKS + 32 * i + threadIdx.x];
            s += v.x;
            up += v.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, d);
            up += __shfl_xor_sync(0xffffffffu, up, d);
        }
        if (threadIdx.x == 0) s_norm = norm_factors(s, up, a.eps, SX);
    }
    __syncthreads();
    const float pre = s_norm.x, inv = s_norm.y;  // X0 = (u pre) inv
    const size_t base = static_cast<size_t>(e) * a.N * a.K;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = r0 + (threadIdx.x >> 4) + 16 * k, c = c0 + 4 * (threadIdx.x & 15);
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < a.N && c < a.K) u = load_u<false>(a, base + static_cast<size_t>(r) * a.K + c);
        // eps = 0 and a zero matrix: 0 * inf would be NaN
        const float v[4] = {u.x == 0.f && inv == inv ? 0.f : u.x * pre * inv, u.y == 0.f && inv == inv ? 0.f : u.y * pre * inv,
                            u.z == 0.f && inv == inv ? 0.f : u.z * pre * inv, u.w == 0.f && inv == inv ? 0.f : u.w * pre * inv};
        if (p.tall) {
#pragma unroll
            for (int j = 0; j < 4; ++j) t[4 * (threadIdx.x & 15) + j][(threadIdx.x >> 4) + 16 * k] = v[j];
        } else if (r < a.N && c < a.K) {
            const size_t at = (static_cast<size_t>(e) * p.m + r) * p.ldn + c;
            __half h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = __float2half_rn(v[j]);
                l[j] = __float2half_rn((v[j] - __half2float(h[j])) * SLO);
            }
            *reinterpret_cast<uint2*>(p.Xh + at) = *reinterpret_cast<const uint2*>(h);
            *reinterpret_cast<uint2*>(p.Xl + at) = *reinterpret_cast<const uint2*>(l);
        }
    }
    if (!p.tall) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // row of X = column of the gradient
        const int i = (threadIdx.x >> 4) + 16 * k, j0 = 4 * (threadIdx.x & 15);
        if (c0 + i >= a.K || r0 + j0 >= p.ldn) continue;
        const size_t at = (static_cast<size_t>(e) * p.m + c0 + i) * p.ldn + r0 + j0;
        __half h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = t[i][j0 + j];
            h[j] = __float2half_rn(v);
            l[j] = __float2half_rn((v - __half2float(h[j])) * SLO);
        }
        *reinterpret_cast<uint2*>(p.Xh + at) = *reinterpret_cast<const uint2*>(h);
        *reinterpret_cast<uint2*>(p.Xl + at) = *reinterpret_cast<const uint2*>(l);
    }
}

// ============================================================== products

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long ns, int* status) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > ns) {
            *abort_flag = 1;
            atomicOr(status, MXFP8_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long ns, int* status) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, ns, status);
}

__device__ __noinline__ void drain_bar(uint32_t bar, uint32_t parity, unsigned long long ns, int* status) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > ns) {
            atomicOr(status, MXFP8_DEV_WAIT_TIMEOUT);
            return;
        }
}

__device__ __noinline__ bool wait_count(const unsigned int* p, unsigned int target, volatile int* abort_flag, unsigned long long ns,
                                        int* status) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        // (an acquire each time: polled relaxed with one acquire at the end, a
        // question more, 3 x 331 x 1000 takes 117 instead of 113.5 us)
        if (ld_acquire_gpu(p) >= target) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > ns) {
            *abort_flag = 1;
            atomicOr(status, MXFP8_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ void tma_load_3d_plain(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Wait until all but the latest of this thread's committed bulk groups have completed.
__device__ __forceinline__ void bulk_wait_group_but_one() { asm volatile("cp.async.bulk.wait_group 1;" ::: "memory"); }

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t* v) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 t = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}

__device__ __forceinline__ float2 bits_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

__device__ __forceinline__ void tc_mma_f16_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"(mask)
        : "memory");
}

// Descriptor of an operand whose rows are contraction steps (MN-major): 64
// columns of 128 bytes with the 128-byte swizzle, 8-row groups 1024 bytes
// apart, the next 64 columns 8 KB on.
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// A tile of a product. ph 0: A = X X^T, 1: R = b A + c A A - beta I, 2: X <- (a + beta) X + R X.
struct Item {
    int step, ph, e, i, j, k0, ksteps, tile, part;  // first K-step and their number; index and piece of a tile of X X^T
};

template <bool SPLIT>
__device__ __forceinline__ Item get_item(const Params& p, int q) {
    Item it;
    const int first = p.E * p.sym * (SPLIT ? p.parts : 1), sym = p.E * p.sym, per = first + sym + p.E * p.full;
    it.step = q / per;
    q -= it.step * per;
    it.ph = q < first ? 0 : q < first + sym ? 1 : 2;
    q -= it.ph == 0 ? 0 : it.ph == 1 ? first : first + sym;
    it.part = 0;
    if (SPLIT && it.ph == 0) {
        const int t = q / p.parts;
        it.part = q - t * p.parts;
        q = t;
    }
    const int tiles = it.ph == 2 ? p.full : p.sym;
    it.tile = q;
    it.e = q / tiles;
    q -= it.e * tiles;
    if (it.ph == 2) {
        it.j = q / p.T;
        it.i = q - it.j * p.T;
    } else if (p.tn == TILE) {  // row i holds i + 1 tiles on and below the diagonal
        int i = static_cast<int>((sqrtf(8.f * q + 1.f) - 1.f) * 0.5f);
        while (i * (i + 1) / 2 > q) --i;
        while ((i + 1) * (i + 2) / 2 <= q) ++i;
        it.i = i;
        it.j = q - i * (i + 1) / 2;
    } else {                    // 2 i + 2 tiles of half the width
        int i = static_cast<int>((sqrtf(4.f * q + 1.f) - 1.f) * 0.5f);
        while (i * (i + 1) > q) --i;
        while ((i + 1) * (i + 2) <= q) ++i;
        it.i = i;
        it.j = q - i * (i + 1);
    }
    it.ksteps = ((it.ph == 0 ? p.n : p.m) + KSTEP - 1) / KSTEP;
    it.k0 = 0;
    if (SPLIT && it.ph == 0) {
        it.k0 = it.ksteps * it.part / p.parts;
        it.ksteps = it.ksteps * (it.part + 1) / p.parts - it.k0;
    }
    return it;
}

// SPLIT: the contraction of X X^T is cut into pieces (without their code the
// chain of few tiles is 3% shorter: 3 x 331 x 1000 118.4 -> 115.0 us).
template <bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    muon_main(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t bars = sbase + OFF_BAR;
    const uint32_t bar_full = bars, bar_empty = bars + 8 * STAGES, bar_tfull = bar_empty + 8 * STAGES, bar_tempty = bar_tfull + 16,
                   bar_drain = bar_tempty + 16, bar_epi = bar_drain + 8, bar_dep = bar_epi + 8 * EPI_WARPS, bar_dfree = bar_dep + 8 * AHEAD;
    int* flags = reinterpret_cast<int*>(smem + OFF_BAR + 8 * (2 * STAGES + 5 + EPI_WARPS + 2 * AHEAD));  // abort, TMEM base
    volatile int* abort_flag = flags;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 2 * EPI_WARPS);
        }
        mbar_init(bar_drain, 1);
        for (int w = 0; w < EPI_WARPS; ++w) mbar_init(bar_epi + 8 * w, 1);
        for (int i = 0; i < AHEAD; ++i) {
            mbar_init(bar_dep + 8 * i, 1);                // scout: the tile's inputs are there
            mbar_init(bar_dfree + 8 * i, 1 + EPI_WARPS);  // producer and epilogue warps have seen it
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(flags + 1), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(flags[1]);
    griddep_wait();
    const int G = gridDim.x / 2, pair = blockIdx.x / 2;
    const int total = p.steps * p.E * (p.sym * (p.parts + 1) + p.full);

    if (warp == 0) {
        // ------------------------------------------------ loads (both CTAs)
        if (elect_one()) {
            const uint32_t full_leader = mapa_shared(bar_full, 0);
            int c = 0, st = 0;
            uint32_t ph = 1;
            bool ok = true;
            int tile = 0;
            Item next = get_item<SPLIT>(p, pair);
            for (int q = pair; ok && q < total; q += G, ++tile) {
                const Item it = next;
                if (q + G < total) next = get_item<SPLIT>(p, q + G);
                ok = wait_bar(bar_dep + 8 * (tile % AHEAD), (tile / AHEAD) & 1, abort_flag, p.wait_ns, p.status);
                if (!ok) break;
                mbar_arrive(bar_dfree + 8 * (tile % AHEAD));
                const int x = it.step & 1;
                const CUtensorMap* ma = it.ph == 0 ? &maps.xk[x] : it.ph == 1 ? &maps.a : &maps.r;
                const CUtensorMap* mb = it.ph == 0 ? &maps.xkn[x] : it.ph == 1 ? &maps.an : &maps.xm[x];
                const int ra = it.i * TILE + static_cast<int>(rank) * HALF, rb = it.j * p.tn + static_cast<int>(rank) * (p.tn / 2);
                for (int k = 0; k < it.ksteps; ++k, ++c) {
                    ok = wait_bar(bar_empty + 8 * st, ph, abort_flag, p.wait_ns, p.status);
                    if (!ok) break;
                    const uint32_t da = sbase + st * 2 * OP_BYTES, db = da + OP_BYTES, fb = full_leader + 8 * st;
                    if (leader) mbar_arrive_expect_tx(bar_full + 8 * st, 2 * (HALF + p.tn / 2) * KSTEP * 2 + (p.stall && c == 0 ? 16 : 0));
                    const int kc = (it.k0 + k) * KSTEP;
                    tma_load_3d_pair(da, ma, fb, kc, ra, it.e);
                    if (it.ph == 2) {
                        tma_load_3d_pair(db, mb, fb, rb, kc, it.e);
                        if (p.tn == TILE) tma_load_3d_pair(db + OP_BYTES / 2, mb, fb, rb + 64, kc, it.e);
                    } else {
                        tma_load_3d_pair(db, mb, fb, kc, rb, it.e);
                    }
                    if (++st == STAGES) { st = 0; ph ^= 1; }
                }
            }
            if (leader && (!ok || *abort_flag))
                for (int d = 1; d <= min(c, STAGES); ++d)
                    drain_bar(bar_full + 8 * ((c - d) % STAGES), ((c - d) / STAGES) & 1, p.wait_ns, p.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader)
        if (leader && elect_one()) {
            int st = 0, tile = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int q = pair; ok && q < total; q += G, ++tile) {
                const Item it = get_item<SPLIT>(p, q);
                const int buf = tile & 1;
                ok = wait_bar(bar_tempty + 8 * buf, ((tile >> 1) & 1) ^ 1, abort_flag, p.wait_ns, p.status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * TILE;
                const bool mn = it.ph == 2;
                const uint32_t idesc = IDESC | (static_cast<uint32_t>(p.tn >> 3) << 17) | (mn ? 1u << 16 : 0u);
                const uint32_t bstep = mn ? 2048 >> 4 : 32 >> 4;  // 16 contraction rows, or 32 bytes along a row
                for (int k = 0; k < it.ksteps; ++k) {
                    ok = wait_bar(bar_full + 8 * st, ph, abort_flag, p.wait_ns, p.status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t as = sbase + st * 2 * OP_BYTES;
                    const uint64_t ad = desc_kmajor_sw128(as);
                    const uint64_t bd = mn ? desc_mnmajor_sw128(as + OP_BYTES) : desc_kmajor_sw128(as + OP_BYTES);
#pragma unroll
                    for (int kk = 0; kk < KSTEP / 16; ++kk)
                        tc_mma_f16_pair(d, ad + 2 * kk, bd + bstep * kk, idesc, k > 0 || kk > 0 ? 1u : 0u);
                    tc_commit_pair(bar_empty + 8 * st, 0x3);
                    if (++st == STAGES) { st = 0; ph ^= 1; }
                }
                if (!ok) break;
                tc_commit_pair(bar_tfull + 8 * buf, 0x3);
            }
            tc_commit_pair(bar_drain, 0x3);
        }
        __syncwarp();
    } else if (warp == SCOUT) {
        // ------------------------------------------------ scout (both CTAs)
        // Waits, up to AHEAD tiles ahead, until the product before a tile's of the
        // same matrix is complete: a round trip to L2 and a fence that would
        // otherwise stand between two tiles' loads.
        if (lane == 0) {
            int tile = 0;
            for (int q = pair; q < total; q += G, ++tile) {
                const Item it = get_item<SPLIT>(p, q);
                const int gp = 3 * it.step + it.ph;
                if (!wait_bar(bar_dfree + 8 * (tile % AHEAD), ((tile / AHEAD) & 1) ^ 1, abort_flag, p.wait_ns, p.status)) break;
                if (gp) {
                    if (!wait_count(p.done + it.e * 3 * p.steps + gp - 1, 2 * EPI_WARPS * (it.ph == 0 ? p.full : p.sym), abort_flag,
                                    p.wait_ns, p.status))
                        break;
                    asm volatile("fence.proxy.async;" ::: "memory");
                }
                mbar_arrive(bar_dep + 8 * (tile % AHEAD));
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue (8 warps per CTA)
        // A warp owns 32 rows (its TMEM quarter) x half the columns of the CTA's
        // tile, in chunks of 64 columns. What a chunk adds to (A, or X's planes)
        // is loaded by TMA into the warp's two slots (the first chunk's before the
        // products are done), replaced there by the result and stored by TMA:
        // whole 128-byte lines either way. (Measured at the 16B shape, whole call:
        // this 0.60 ms; chunks of 32 columns, 64-byte lines, 0.65; from registers,
        // 8 rows x 64 bytes at a time, 0.78; lane by lane 0.76.) A tile is reported
        // done when its stores have arrived: after the next tile's first chunk
        // where that tile is ready by then.
        const int q4 = warp & 3, h = (warp - EPI0) >> 2;
        const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
        const uint32_t slot = sbase + OFF_EPI + (warp - EPI0) * 2 * SLOT, slot2 = slot + SLOT, bar_in = bar_epi + 8 * (warp - EPI0);
        const uint32_t row_at = lane * 128, sw = lane & 7;  // 16-byte piece k of the lane's row: row_at + ((k ^ sw) << 4)
        const bool odd = lane & 1;
        const int width = p.tn / 2;
        int tile = 0;
        uint32_t in_ph = 0;
        bool ok = true;
        unsigned int* pending = nullptr;  // lane 0: the finished tile that is not reported yet
        auto report = [&]() {
            // (the stores went through the asynchronous proxy and have completed: the
            // reader's proxy fence, in the scout, is the one that is needed)
            red_release_gpu_add(pending, 1);
            pending = nullptr;
        };
        for (int q = pair; q < total; q += G, ++tile) {
            const Item it = get_item<SPLIT>(p, q);
            const int buf = tile & 1;
            const int r0 = it.i * TILE + static_cast<int>(rank) * HALF + q4 * 32, r = r0 + lane;  // row of the product
            const bool last = it.step + 1 == p.steps;
            const float shift = last ? 0.875f * (p.b + p.c) : it.step + 2 == p.steps ? 0.4375f * (p.b + p.c) : 0.f;
            const int cols = it.ph == 2 ? p.n : p.m, x = it.step & 1, c0 = it.j * p.tn + h * width;
            const int chunks = r0 < p.m && c0 < cols ? min(width, cols - c0 + 63) >> 6 : 0;
            const bool mirror = it.ph < 2 && it.j * p.tn < it.i * TILE;
            // the last step reads the upper plane only (its roundings are not amplified)
            const bool low_in = it.ph == 2 && !last, low_out = it.ph == 2 && it.step + 2 < p.steps;
            const bool tall_out = it.ph == 2 && last && p.tall;
            auto load = [&](int c) {
                bulk_wait_group_read<0>();  // the slots' last stores have been read
                if (!it.ph) return;
                mbar_arrive_expect_tx(bar_in, low_in ? 2 * SLOT : SLOT);
                tma_load_3d_plain(slot, it.ph == 1 ? &maps.ea : &maps.exh[x], bar_in, c, r0, it.e);
                if (low_in) tma_load_3d_plain(slot2, &maps.exl[x], bar_in, c, r0, it.e);
            };
            if (lane == 0) {
                const bool ready = mbar_try_wait(bar_tfull + 8 * buf, (tile >> 1) & 1);
                if (pending && (!ready || !chunks)) {  // never wait with a tile unreported
                    bulk_wait_group_all();
                    report();
                }
                ok = wait_bar(bar_dep + 8 * (tile % AHEAD), (tile / AHEAD) & 1, abort_flag, p.wait_ns, p.status);
                if (ok) {
                    mbar_arrive(bar_dfree + 8 * (tile % AHEAD));
                    if (chunks) load(c0);
                    ok = ready || wait_bar(bar_tfull + 8 * buf, (tile >> 1) & 1, abort_flag, p.wait_ns, p.status);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + buf * TILE + h * width;
            const bool split = SPLIT && it.ph == 0;
            const size_t piece = static_cast<size_t>(2 * EPI_WARPS) * width * 32;  // floats of one piece of a tile
            const float* sums = p.part;
            bool finish = true;
            if (split) {
                // this piece's sums, a column of 32 rows (a line) at a time; the warp
                // that brings the last piece of its share goes on with all of them, in
                // order
                const int share = (it.tile * 2 + static_cast<int>(rank)) * EPI_WARPS + warp - EPI0;
                sums = p.part + it.tile * p.parts * piece + static_cast<size_t>(static_cast<int>(rank) * EPI_WARPS + warp - EPI0) * width * 32 + lane;
                float* dst = const_cast<float*>(sums) + it.part * piece;
#pragma unroll 1
                for (int c = 0; c < 64 * chunks; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + c, v);
                    tmem_wait_ld();
                    reg_fence(v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) dst[(c + i) * 32] = __uint_as_float(v[i]);
                }
                __syncwarp();
                if (lane == 0) {
                    if (pending) {
                        bulk_wait_group_all();
                        report();
                    }
                    finish = atom_acq_rel_gpu_add(p.arrived + share, 1) == static_cast<uint32_t>(p.parts - 1);
                    if (finish) p.arrived[share] = 0;  // (the next step's pieces come long after)
                }
                finish = __shfl_sync(0xffffffffu, finish ? 1 : 0, 0) != 0;
            }
#pragma unroll 1
            for (int ch = 0; finish && ch < chunks; ++ch) {
                const int c = c0 + 64 * ch;
                if (lane == 0 && ch) load(c);
                __syncwarp();
                if (it.ph) {
                    if (lane == 0) ok = wait_bar(bar_in, in_ph, abort_flag, p.wait_ns, p.status);
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    (void)mbar_try_wait(bar_in, in_ph);  // complete: makes the loads visible to every lane
                    in_ph ^= 1;
                }
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t v[32];
                    if (split) {
                        const float* src = sums + (64 * ch + 32 * hf) * 32;
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0;
#pragma unroll 1
                        for (int s = 0; s < p.parts; ++s, src += piece)
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __ldcg(src + i * 32));
                    } else {
                        tmem_ld_32x32b_x32(taddr + 64 * ch + 32 * hf, v);
                    }
                    uint32_t u[16], w[16];
                    const uint32_t at = slot + row_at, at2 = slot2 + row_at;
                    if (it.ph) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) ld_shared_v4(at + (((4 * hf + k) ^ sw) << 4), u + 4 * k);
                    }
                    if (low_in) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) ld_shared_v4(at2 + (((4 * hf + k) ^ sw) << 4), w + 4 * k);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = 0;
                    }
                    tmem_wait_ld();
                    reg_fence(v);
                    float f[32];
                    if (it.ph == 0) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]) * (SA / (SX * SX));
                    } else if (it.ph == 1) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 t = bits_half2(u[i]);
                            f[2 * i] = fmaf(p.c / SA, __uint_as_float(v[2 * i]), p.b * t.x);
                            f[2 * i + 1] = fmaf(p.c / SA, __uint_as_float(v[2 * i + 1]), p.b * t.y);
                        }
                        if (!mirror) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (r == c + 32 * hf + i) f[i] -= shift * SA;
                        }
                    } else {
                        const float ax = p.a + shift;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 t = bits_half2(u[i]), l = bits_half2(w[i]);
                            f[2 * i] = fmaf(ax, fmaf(1.f / SLO, l.x, t.x), __uint_as_float(v[2 * i]) * (1.f / SA));
                            f[2 * i + 1] = fmaf(ax, fmaf(1.f / SLO, l.y, t.y), __uint_as_float(v[2 * i + 1]) * (1.f / SA));
                        }
                    }
                    if (it.ph == 2 && last) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            u[i] = pack_bf16x2(__float_as_uint(f[2 * i] * (1.f / SX)), __float_as_uint(f[2 * i + 1] * (1.f / SX)));
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) u[i] = half2_bits(f[2 * i], f[2 * i + 1]);
                    }
                    if (!tall_out) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st_shared_v4(at + (((4 * hf + k) ^ sw) << 4), u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
                    }
                    if (low_out) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 hv = bits_half2(u[i]);
                            w[i] = half2_bits((f[2 * i] - hv.x) * SLO, (f[2 * i + 1] - hv.y) * SLO);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st_shared_v4(at2 + (((4 * hf + k) ^ sw) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    }
                    if (mirror || tall_out) {
                        // transposed, 32 rows (this product's columns) of 64 bytes with
                        // the 64-byte swizzle; lanes r, r + 1 exchange halves: the even
                        // lane stores (r, r + 1) of row 2 i, the odd lane of 2 i + 1
                        const uint32_t base = slot2 + hf * (SLOT / 2), kb = static_cast<uint32_t>(lane & ~1) * 2;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, u[i], 1);
                            const uint32_t y = odd ? __byte_perm(got, u[i], 0x7632) : __byte_perm(u[i], got, 0x5410);
                            const uint32_t row = 2 * i + (odd ? 1 : 0);
                            st_shared_b32(base + row * 64 + (((kb >> 4) ^ ((row >> 1) & 3)) << 4) + (kb & 15), y);
                        }
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    if (!tall_out)
                        tma_store_3d(it.ph == 0 ? &maps.ea : it.ph == 1 ? &maps.er : last ? &maps.eout : &maps.exh[x ^ 1], slot, c, r0, it.e);
                    if (low_out) tma_store_3d(&maps.exl[x ^ 1], slot2, c, r0, it.e);
                    if (mirror || tall_out) {
                        const CUtensorMap* t = it.ph == 0 ? &maps.ta : it.ph == 1 ? &maps.tr : &maps.tout;
                        tma_store_3d(t, slot2, r0, c, it.e);
                        if (c + 32 < cols) tma_store_3d(t, slot2 + SLOT / 2, r0, c + 32, it.e);
                    }
                    bulk_commit_group();
                    if (pending) {  // all stores but this chunk's have arrived
                        bulk_wait_group_but_one();
                        report();
                    }
                }
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(bar_tempty + 8 * buf);
                else mbar_arrive_cluster(tempty_leader + 8 * buf);
                if (finish) pending = p.done + it.e * 3 * p.steps + 3 * it.step + it.ph;
            }
        }
        if (lane == 0) {
            bulk_wait_group_all();
            if (pending) report();
        }
        __syncwarp();
    }
    // All MMAs have completed. Asked once the CTA's own tiles are through, so that
    // the limit bounds what is left of the last one: in the pair's second CTA, whose
    // issuer has nothing else to do, it would otherwise bound the whole call.
    __syncthreads();
    if (warp == 1 && lane == 0) drain_bar(bar_drain, 0, p.wait_ns, p.status);
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ============================================================== host side

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct Layout {
    int m, n, ldm, ldn, tn, T, sym, full, parts;
    size_t norm, done, arrived, xh[2], xl[2], a, r, part, total;
};

constexpr int PAIRS = 76;  // CTA pairs that the tiling reckons with

void layout(int E, int N, int K, Layout* l) {
    l->m = N < K ? N : K;
    l->n = N < K ? K : N;
    l->ldm = (l->m + 63) & ~63;
    l->ldn = (l->n + 63) & ~63;
    // Tiles of 128 columns up to 1 3/4 tiles of 256 a pair: each then takes half
    // the time to compute and store, which shortens the chain of products (5 steps,
    // 256 / 128: 1 x 2048 x 1408, 48 tiles, 249 / 198 us; 4 x 1024 x 1024, 64, 202 / 164;
    // 20 x 512 x 512, 80, 200 / 157; 1 x 2048 x 4096, 128, 383 / 368). With more, the wider
    // ones win: they need three quarters of the operand bytes for the same products
    // (1 x 3000 x 3000, 144, 569 / 640; 4 x 1408 x 2048, 192, 322 / 358).
    l->T = (l->m + TILE - 1) / TILE;
    l->tn = 4LL * E * l->T * ((l->n + TILE - 1) / TILE) <= 7 * PAIRS ? TILE / 2 : TILE;
    const int Tm = (l->m + l->tn - 1) / l->tn, ksteps = (l->n + KSTEP - 1) / KSTEP;
    l->full = l->T * ((l->n + l->tn - 1) / l->tn);
    l->sym = 0;
    for (int i = 0; i < l->T; ++i) l->sym += Tm < (i + 1) * (TILE / l->tn) ? Tm : (i + 1) * (TILE / l->tn);
    // The contraction of X X^T in pieces of sixteen K-steps or more where its tiles
    // occupy less than half of the pairs: the piece that ends last adds them up in
    // order (1 x 129 x 7032 188 -> 142 us; pieces of eight K-steps cost more to
    // join than they save, 3 x 331 x 1000 115 -> 127 us).
    const long long tiles = static_cast<long long>(E) * l->sym;
    l->parts = 1;
    if (2 * tiles <= PAIRS) {
        l->parts = static_cast<int>(PAIRS / tiles);
        if (l->parts > ksteps / 16) l->parts = ksteps / 16;
        if (l->parts > 8) l->parts = 8;
        if (l->parts < 1) l->parts = 1;
    }
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
    const size_t e = E;
    l->norm = take(sizeof(float2) * e * NORM_BLOCKS);
    l->done = take(4 * e * 3 * MXFP8_MUON_MAX_STEPS);  // (done and arrived: zeroed together)
    l->arrived = take(4 * e * l->sym * 2 * EPI_WARPS);
    l->part = take(l->parts > 1 ? 4 * e * l->sym * l->parts * TILE * l->tn : 0);
    for (int i = 0; i < 2; ++i) l->xh[i] = take(2 * e * l->m * l->ldn);
    for (int i = 0; i < 2; ++i) l->xl[i] = take(2 * e * l->m * l->ldn);
    l->a = take(2 * e * l->m * l->ldm);
    l->r = take(2 * e * l->m * l->ldm);
    l->total = at;
}

int map2(CUtensorMap* map, const void* base, int cols, int ld, int rows, int E, int box_rows, int box_cols = KSTEP, bool bf16 = false) {
    const uint64_t d[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(E)};
    const uint64_t s[2] = {2 * static_cast<uint64_t>(ld), 2 * static_cast<uint64_t>(ld) * rows};
    const uint32_t b[3] = {static_cast<uint32_t>(box_cols), static_cast<uint32_t>(box_rows), 1};
    return host_tensor_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, d, s, b,
                           box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace

size_t muon_ws_bytes(int E, int N, int K) {
    Layout l;
    layout(E, N, K, &l);
    return l.total;
}

int launch_muon(const MuonArgs& a) {
    Layout l;
    layout(a.E, a.N, a.K, &l);
    Params p{};
    p.E = a.E; p.m = l.m; p.n = l.n; p.ldm = l.ldm; p.ldn = l.ldn; p.steps = a.steps; p.tall = a.N > a.K;
    p.tn = l.tn; p.T = l.T; p.full = l.full; p.sym = l.sym; p.parts = l.parts;
    p.part = reinterpret_cast<float*>(a.ws + l.part);
    p.arrived = reinterpret_cast<unsigned int*>(a.ws + l.arrived);
    if (static_cast<long long>(a.steps) * a.E * (9LL * p.sym + p.full) > 0x7fffffffLL / 2)
        return host_fail(MXFP8_EINVAL, "E=%d N=%d K=%d steps=%d: too many tiles", a.E, a.N, a.K, a.steps);
    p.a = a.a; p.b = a.b; p.c = a.c;
    p.Xh = reinterpret_cast<__half*>(a.ws + l.xh[0]);
    p.Xl = reinterpret_cast<__half*>(a.ws + l.xl[0]);
    p.done = reinterpret_cast<unsigned int*>(a.ws + l.done);
    p.wait_ns = a.wait_limit_ns;
    p.status = a.status;
    p.stall = a.stall;
    float2* norm = reinterpret_cast<float2*>(a.ws + l.norm);
    const int zeroed = static_cast<int>((l.arrived - l.done) / 4 + static_cast<size_t>(a.E) * l.sym * 2 * EPI_WARPS);
    Maps maps;
    int rc = MXFP8_OK;
    const int E = a.E;
    for (int i = 0; i < 2 && !rc; ++i) {
        rc = map2(&maps.xk[i], a.ws + l.xh[i], l.n, l.ldn, l.m, E, HALF);
        if (!rc) rc = map2(&maps.xkn[i], a.ws + l.xh[i], l.n, l.ldn, l.m, E, p.tn / 2);
        if (!rc) rc = map2(&maps.xm[i], a.ws + l.xh[i], l.n, l.ldn, l.m, E, KSTEP);
        if (!rc) rc = map2(&maps.exh[i], a.ws + l.xh[i], l.n, l.ldn, l.m, E, 32);
        if (!rc) rc = map2(&maps.exl[i], a.ws + l.xl[i], l.n, l.ldn, l.m, E, 32);
    }
    if (!rc) rc = map2(&maps.a, a.ws + l.a, l.m, l.ldm, l.m, E, HALF);
    if (!rc) rc = map2(&maps.an, a.ws + l.a, l.m, l.ldm, l.m, E, p.tn / 2);
    if (!rc) rc = map2(&maps.r, a.ws + l.r, l.m, l.ldm, l.m, E, HALF);
    if (!rc) rc = map2(&maps.ea, a.ws + l.a, l.m, l.ldm, l.m, E, 32);
    if (!rc) rc = map2(&maps.er, a.ws + l.r, l.m, l.ldm, l.m, E, 32);
    if (!rc) rc = map2(&maps.ta, a.ws + l.a, l.m, l.ldm, l.m, E, 32, 32);
    if (!rc) rc = map2(&maps.tr, a.ws + l.r, l.m, l.ldm, l.m, E, 32, 32);
    if (!rc) rc = map2(&maps.eout, a.out, a.K, a.K, a.N, E, 32, 64, true);
    if (!rc) rc = map2(&maps.tout, a.out, a.K, a.K, a.N, E, 32, 32, true);
    if (rc) return rc;

    static std::atomic<int> max_pairs[64];
    int pairs = max_pairs[a.dev].load(std::memory_order_relaxed);
    cudaError_t e;
    if (pairs == 0) {
        e = cudaFuncSetAttribute(muon_main<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(muon_main<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "update kernel: %s", cudaGetErrorString(e));
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(2 * (a.num_sms / 2));
        q.blockDim = dim3(THREADS);
        q.dynamicSmemBytes = SMEM;
        e = cudaOccupancyMaxActiveClusters(&pairs, muon_main<false>, &q);
        if (e != cudaSuccess || pairs < 1) return host_fail(MXFP8_ECUDA, "update kernel: %s", cudaGetErrorString(e));
        max_pairs[a.dev].store(pairs, std::memory_order_relaxed);
    }
    // each kernel a programmatic dependent of the one before
    cudaLaunchConfig_t pre = {};
    cudaLaunchAttribute pdl;
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    pre.attrs = &pdl;
    pre.numAttrs = 1;
    pre.stream = a.stream;
    pre.blockDim = dim3(256);
    pre.gridDim = dim3(NORM_BLOCKS, a.E);
    e = cudaLaunchKernelEx(&pre, muon_momentum, a, norm, p.done, zeroed);
    if (e == cudaSuccess) {
        pre.gridDim = dim3((a.K + 63) / 64, (a.N + 63) / 64, a.E);
        e = cudaLaunchKernelEx(&pre, muon_scale, a, p, static_cast<const float2*>(norm));
    }
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "update kernel: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    const int items = a.E * (p.full > p.sym * p.parts ? p.full : p.sym * p.parts);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (items < pairs ? items : pairs));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    // CTAs wait on one another: all of them resident at once
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1] = pdl;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = p.parts > 1 ? cudaLaunchKernelEx(&cfg, muon_main<true>, maps, p) : cudaLaunchKernelEx(&cfg, muon_main<false>, maps, p);
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "update kernel: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return MXFP8_OK;
}

}  // namespace mxw
