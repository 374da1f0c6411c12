// Orthogonalised update of small matrices (mxfp8_muon_update, shorter side up
// to 128 and longer side up to 2048): one kernel, one cluster per matrix.
//
// The general kernel (muon.cu) hands every product over through global memory,
// 5 to 7 us each, fifteen of them in a row for five steps: for a matrix of a few
// tiles that is all its time. Here the matrix stays on chip. With X the m x n
// matrix (m <= 128), CTA c of the cluster holds the w columns [c w, c w + w),
// w <= 256:
//   A = X X^T     is a sum over the CTAs: each multiplies its slice (M = 128,
//                 N = 128), the partial sums are added through distributed
//                 shared memory, a share of A's columns per CTA, in CTA order,
//                 and the rounded share is written to every CTA;
//   R = b A + c A A - beta I    every CTA computes for itself;
//   X <- (a + beta) X + R X     by columns: nothing to exchange.
// The fp16 slice of X in shared memory serves both products: its rows are the
// contraction of R X (MN-major) and its columns that of X X^T (K-major). The
// a X term takes X in fp32 from TMEM, beside the accumulator. Momentum, norm and
// the two transposes of tall matrices happen on the way in and out. The same
// scaling and shift beta as in the general kernel.
//
// Bound by the latency of the chain: 4 x 128 x 256, five steps, 31 us, 6.6 of
// them to load and normalise and 3.6 to 3.8 a step (three products of 0.3 us,
// the accumulator's way through registers into shared memory after each). 512
// threads on 16 columns at a time: with 32 columns unrolled in each of 256
// threads the same took 36 us, the longer code missing the instruction cache.
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

constexpr int M = 128;               // rows of a CTA's operands
constexpr int MAXW = 256;            // columns of a CTA's slice
constexpr int MAXC = 8;              // CTAs of a cluster
constexpr int THREADS = 512;         // 16 warps: a TMEM quarter (32 rows) and a quarter of the columns each
constexpr int ATOM = M * 128;        // 128 rows of 64 fp16 values, 128-byte swizzle
constexpr float SX = 2048.f, SA = 4096.f;  // as in muon.cu
// shared memory: X's slice; then either u on the way in (fp32, rows padded by
// one) or A, R and the partial sums of A
constexpr int OFF_A = MAXW / 64 * ATOM, OFF_R = OFF_A + 2 * ATOM, OFF_P = OFF_R + 2 * ATOM;
constexpr int OFF_BAR = OFF_A + M * (MAXW + 1) * 4 > OFF_P + M * M * 4 ? OFF_A + M * (MAXW + 1) * 4 : OFF_P + M * M * 4;
constexpr int SMEM = OFF_BAR + 256 + 1024;  // (barrier, TMEM base, 24 pairs of sums; alignment)
constexpr int CH = 16;               // columns that a thread handles at a time (short code: its first pass misses the instruction cache)
static_assert(SMEM <= 232448, "shared memory of a CTA");
constexpr uint32_t IDESC = (1u << 4) | (static_cast<uint32_t>(M >> 4) << 24);  // kind::f16, fp16 x fp16 -> fp32, M = 128
constexpr uint32_t X_COL = 256;      // TMEM: accumulator in columns 0 .. 255, X in fp32 from here on

__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Operand whose rows are contraction steps: 64 columns of 128 bytes a row, 8-row
// groups 1024 bytes apart, the next 64 columns one atom on.
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(ATOM >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// 32 lanes x 16 consecutive 32-bit columns: thread i of the warp holds lane (base lane + i).
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&v)[CH]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[CH]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
          "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void fence16(uint32_t (&v)[CH]) {  // ties loaded registers to a point after the wait
#pragma unroll
    for (int i = 0; i < CH; ++i) asm volatile("" : "+r"(v[i]));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 t = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}

__device__ __forceinline__ void ld_cluster_v4(uint32_t addr, float (&v)[4]) {
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, float a, float b) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

struct Small {
    MuonArgs a;
    int m, n, w, C, tall;
};

// Four values of the gradient from element i on (a multiple of 4).
__device__ __forceinline__ float4 load_grad(const MuonArgs& a, size_t i) {
    if (a.grad_f32) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.grad) + i));
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.grad) + i));
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
}

__device__ __forceinline__ float4 axpy4(float s, const float4& x, const float4& y) {
    return make_float4(fmaf(s, x.x, y.x), fmaf(s, x.y, y.y), fmaf(s, x.z, y.z), fmaf(s, x.w, y.w));
}

__global__ void __launch_bounds__(THREADS, 1) muon_small(const Small p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.C > 1 ? static_cast<int>(cluster_ctarank()) : 0, e = blockIdx.x / p.C;
    const uint32_t bar = sbase + OFF_BAR;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_BAR + 8);
    float2* red = reinterpret_cast<float2*>(smem + OFF_BAR + 32);  // [16] warps' sums of u^2 and (2^100 u)^2
    float2* norms = red + 16;                                      // [8] CTAs' sums
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc_single(smem_u32(tmem_slot), 512);
        tmem_relinquish_single();
    }
    griddep_wait();  // the gradient may come from the kernel before
    const int q4 = warp & 3, h = warp >> 2;         // TMEM quarter, quarter of the columns
    const int row = q4 * 32 + lane, width = p.w / 4;  // this thread's row; columns h * width ..

    // ---- u into shared memory as X's rows, the sum of its squares
    float* u = reinterpret_cast<float*>(smem + OFF_A);
    const int pitch = p.w + 1, col0 = rank * p.w, cols = min(p.w, p.n - col0);
    const size_t base = static_cast<size_t>(e) * p.m * p.n;
    if (p.m < M || cols < p.w) {
        for (int i = threadIdx.x; i < M * pitch; i += THREADS) u[i] = 0.f;
        __syncthreads();
    }
    float sq = 0.f, up = 0.f;
    {
        // four neighbours along the gradient's rows: X's columns, or (tall) X's rows;
        // a warp per line, four lines' loads in flight (the momentum's stores
        // would otherwise hold back the loads behind them)
        constexpr int BATCH = 4, WARPS = THREADS / 32;
        const int groups = (p.tall ? p.m : p.n) / 4, lines = p.tall ? cols : p.m;
        const int g0 = p.tall ? 0 : col0 / 4, ng = p.tall ? groups : min(p.w / 4, groups - g0);
        const size_t first = base + (p.tall ? static_cast<size_t>(col0) * p.m : 4 * static_cast<size_t>(g0)), line = p.tall ? p.m : p.n;
        for (int l0 = warp; l0 < lines; l0 += WARPS * BATCH)
            for (int g = lane; g < ng; g += 32) {
                float4 v[BATCH], mo[BATCH];
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const int l = l0 + WARPS * j;
                    const size_t at = first + l * line + 4 * g;
                    v[j] = l < lines ? load_grad(p.a, at) : make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p.a.momentum && l < lines) mo[j] = *reinterpret_cast<const float4*>(p.a.momentum + at);
                }
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const int l = l0 + WARPS * j;
                    if (l >= lines) continue;
                    if (p.a.momentum) {
                        mo[j] = axpy4(p.a.mu, mo[j], v[j]);
                        *reinterpret_cast<float4*>(p.a.momentum + first + l * line + 4 * g) = mo[j];
                        v[j] = p.a.nesterov ? axpy4(p.a.mu, mo[j], v[j]) : mo[j];
                    }
                    sq += (v[j].x * v[j].x + v[j].y * v[j].y) + (v[j].z * v[j].z + v[j].w * v[j].w);
                    const float4 t = make_float4(v[j].x * NORM_UP, v[j].y * NORM_UP, v[j].z * NORM_UP, v[j].w * NORM_UP);
                    up += (t.x * t.x + t.y * t.y) + (t.z * t.z + t.w * t.w);
                    float* d = p.tall ? u + 4 * g * pitch + l : u + l * pitch + 4 * g;
                    const int st = p.tall ? pitch : 1;
                    d[0] = v[j].x; d[st] = v[j].y; d[2 * st] = v[j].z; d[3 * st] = v[j].w;
                }
            }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, d);
        up += __shfl_xor_sync(0xffffffffu, up, d);
    }
    if (lane == 0) red[warp] = make_float2(sq, up);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (p.C > 1) cluster_sync_all();  // the other CTAs run: their shared memory may be written
    if (threadIdx.x < p.C) {
        float s = 0.f, t = 0.f;
        for (int w = 0; w < THREADS / 32; ++w) {
            s += red[w].x;
            t += red[w].y;
        }
        if (p.C > 1) st_cluster_v2(mapa_shared(smem_u32(norms + rank), threadIdx.x), s, t);
        else norms[0] = make_float2(s, t);
    }
    __syncwarp();
    if (p.C > 1) cluster_sync_all();
    else __syncthreads();
    float total = 0.f, total_up = 0.f;
    for (int c = 0; c < p.C; ++c) {
        total += norms[c].x;
        total_up += norms[c].y;
    }
    const float2 factors = norm_factors(total, total_up, p.a.eps, SX);
    const float pre = factors.x, inv = factors.y;  // X0 = (u pre) inv

    const uint32_t tacc = tmem + (static_cast<uint32_t>(q4 * 32) << 16), tx = tacc + X_COL;
    const uint32_t row_at = row * 128, sw = row & 7;  // 16-byte piece k of the row in an atom: row_at + ((k ^ sw) << 4)
    // offset of 16-byte piece k of columns c .. c + 15 of the thread's row in a matrix of atoms
    auto piece = [&](int c, int k) { return (c >> 6) * ATOM + row_at + ((((c >> 3) & 7) + k) ^ sw) * 16; };
    // those columns as fp16 into X's slice
    auto put_x = [&](int c, const float (&f)[CH]) {
#pragma unroll
        for (int k = 0; k < CH / 8; ++k)
            st_shared_v4(sbase + piece(c, k), half2_bits(f[8 * k], f[8 * k + 1]), half2_bits(f[8 * k + 2], f[8 * k + 3]),
                         half2_bits(f[8 * k + 4], f[8 * k + 5]), half2_bits(f[8 * k + 6], f[8 * k + 7]));
    };
#pragma unroll 1
    for (int c = h * width; c < (h + 1) * width; c += CH) {
        float f[CH];
        uint32_t b[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const float v = u[row * pitch + c + i];
            f[i] = v == 0.f && inv == inv ? 0.f : v * pre * inv;  // (eps = 0 and a zero matrix: 0 * inf would be NaN)
            b[i] = __float_as_uint(f[i]);
        }
        tmem_st_x16(tx + c, b);
        put_x(c, f);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");

    uint32_t phase = 0;
    // All threads: the shared-memory operands are written; one thread issues; all wait for the product.
    auto product = [&](auto issue) {
        fence_proxy_async_shared();
        tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after();
            if (elect_one()) {
                issue();
                tc_commit(bar);
            }
            __syncwarp();
        }
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar, phase))
            if (global_timer_ns() - t0 > p.a.wait_limit_ns) {
                // (no early exit: the CTAs of the cluster meet at its barriers)
                atomicOr(p.a.status, MXFP8_DEV_WAIT_TIMEOUT);
                break;
            }
        phase ^= 1;
        tc_fence_after();
    };
    const uint32_t sa = sbase + OFF_A, sr = sbase + OFF_R;
#pragma unroll 1
    for (int step = 0; step < p.a.steps; ++step) {
        const bool last = step + 1 == p.a.steps;
        const float shift = last ? 0.875f * (p.a.b + p.a.c) : step + 2 == p.a.steps ? 0.4375f * (p.a.b + p.a.c) : 0.f;
        // A: this slice's part
        product([&] {
            for (int k = 0; k < p.w / 16; ++k) {
                const uint64_t d = desc_kmajor_sw128(sbase + (k >> 2) * ATOM) + 2 * (k & 3);
                tc_mma_f16(tmem, d, d, IDESC | (static_cast<uint32_t>(M >> 3) << 17), k > 0 ? 1u : 0u);
            }
        });
        if (p.C == 1) {
#pragma unroll 1
            for (int c = h * (M / 4); c < (h + 1) * (M / 4); c += CH) {
                uint32_t v[CH];
                tmem_ld_x16(tacc + c, v);
                tmem_wait_ld();
                fence16(v);
                constexpr float S = SA / (SX * SX);
#pragma unroll
                for (int k = 0; k < CH / 8; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = half2_bits(__uint_as_float(v[8 * k + 2 * j]) * S, __uint_as_float(v[8 * k + 2 * j + 1]) * S);
                    st_shared_v4(sa + piece(c, k), w[0], w[1], w[2], w[3]);
                }
            }
        } else {
            float* part = reinterpret_cast<float*>(smem + OFF_P);  // [column][row]
#pragma unroll 1
            for (int c = h * (M / 4); c < (h + 1) * (M / 4); c += CH) {
                uint32_t v[CH];
                tmem_ld_x16(tacc + c, v);
                tmem_wait_ld();
                fence16(v);
#pragma unroll
                for (int i = 0; i < CH; ++i) part[(c + i) * M + row] = __uint_as_float(v[i]);
            }
            cluster_sync_all();
            // eight rows of a column of A at a time: its sum over the CTAs, in their
            // order, written to row `column` of A in every CTA (A is symmetric)
            const int per = (M + p.C - 1) / p.C, j1 = min(M, (rank + 1) * per);
            for (int i = rank * per * 16 + threadIdx.x; i < j1 * 16; i += THREADS) {
                const int j = i >> 4, r = (i & 15) * 8;
                float s[8] = {};
                for (int c = 0; c < p.C; ++c) {
                    const uint32_t src = mapa_shared(sbase + OFF_P + (j * M + r) * 4, c);
                    float x[4], y[4];
                    ld_cluster_v4(src, x);
                    ld_cluster_v4(src + 16, y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        s[k] += x[k];
                        s[4 + k] += y[k];
                    }
                }
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = half2_bits(s[2 * k] * (SA / (SX * SX)), s[2 * k + 1] * (SA / (SX * SX)));
                const uint32_t at = sa + (r >> 6) * ATOM + j * 128 + ((((r >> 3) & 7) ^ (j & 7)) << 4);
                for (int c = 0; c < p.C; ++c) st_cluster_v4(mapa_shared(at, c), w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            cluster_sync_all();
        }
        // A A^T = A A
        product([&] {
#pragma unroll
            for (int k = 0; k < M / 16; ++k) {
                const uint64_t d = desc_kmajor_sw128(sa + (k >> 2) * ATOM) + 2 * (k & 3);
                tc_mma_f16(tmem, d, d, IDESC | (static_cast<uint32_t>(M >> 3) << 17), k > 0 ? 1u : 0u);
            }
        });
#pragma unroll 1
        for (int c = h * (M / 4); c < (h + 1) * (M / 4); c += CH) {
            uint32_t v[CH];
            tmem_ld_x16(tacc + c, v);
            tmem_wait_ld();
            fence16(v);
#pragma unroll
            for (int k = 0; k < CH / 8; ++k) {
                const uint4 s = *reinterpret_cast<const uint4*>(smem + OFF_A + piece(c, k));
                const uint32_t in[4] = {s.x, s.y, s.z, s.w};
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&in[j]));
                    const int i = 8 * k + 2 * j;
                    float f0 = fmaf(p.a.c / SA, __uint_as_float(v[i]), p.a.b * t.x);
                    float f1 = fmaf(p.a.c / SA, __uint_as_float(v[i + 1]), p.a.b * t.y);
                    if (c + i == row) f0 -= shift * SA;
                    if (c + i + 1 == row) f1 -= shift * SA;
                    w[j] = half2_bits(f0, f1);
                }
                st_shared_v4(sr + piece(c, k), w[0], w[1], w[2], w[3]);
            }
        }
        // R X: rows of X are the contraction
        product([&] {
#pragma unroll
            for (int k = 0; k < M / 16; ++k)
                tc_mma_f16(tmem, desc_kmajor_sw128(sr + (k >> 2) * ATOM) + 2 * (k & 3), desc_mnmajor(sbase) + 128 * k,
                           IDESC | (1u << 16) | (static_cast<uint32_t>(p.w >> 3) << 17), k > 0 ? 1u : 0u);
        });
#pragma unroll 1
        for (int c = h * width; c < (h + 1) * width; c += CH) {
            uint32_t v[CH], xv[CH];
            tmem_ld_x16(tacc + c, v);
            tmem_ld_x16(tx + c, xv);
            tmem_wait_ld();
            fence16(v);
            fence16(xv);
            float f[CH];
            const float ax = p.a.a + shift;
#pragma unroll
            for (int i = 0; i < CH; ++i) f[i] = fmaf(ax, __uint_as_float(xv[i]), __uint_as_float(v[i]) * (1.f / SA));
            if (!last) {
#pragma unroll
                for (int i = 0; i < CH; ++i) xv[i] = __float_as_uint(f[i]);
                tmem_st_x16(tx + c, xv);
                put_x(c, f);
            } else if (row < p.m && !p.tall) {
                uint16_t* dst = p.a.out + base + static_cast<size_t>(row) * p.n + col0 + c;
#pragma unroll
                for (int i = 0; i < CH; i += 8)
                    if (c + i < cols) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = pack_bf16x2(__float_as_uint(f[i + 2 * j] * (1.f / SX)), __float_as_uint(f[i + 2 * j + 1] * (1.f / SX)));
                        *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            } else if (row < p.m) {
                uint16_t* dst = p.a.out + base + static_cast<size_t>(col0 + c) * p.m + row;
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (c + i < cols) dst[static_cast<size_t>(i) * p.m] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i] * (1.f / SX)));
            }
        }
        if (!last) asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    if (p.C > 1) cluster_sync_all();  // (no CTA leaves while another may still read its shared memory)
    else __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc_single(tmem, 512);
}

}  // namespace

// Every matrix that fits goes this way (5 steps, momentum, us here / general
// kernel): 4 x 128 x 256 31 / 87, 64 x 120 x 120 24 / 115, 256 x 128 x 256 73 / 337,
// 20 x 64 x 1000 64 / 130, and with the largest cluster 1 x 128 x 2048
// 67 / 117, 32 x 128 x 2048 222 / 253; the two meet where many large ones queue for
// the SMs (128 x 128 x 2048 683 / 665, without momentum 622 / 622).
bool muon_fits_small(int N, int K) {
    const int m = N < K ? N : K, n = N < K ? K : N;
    return m <= M && n <= MAXC * MAXW;
}

int launch_muon_small(const MuonArgs& a) {
    Small p{};
    p.a = a;
    p.m = a.N < a.K ? a.N : a.K;
    p.n = a.N < a.K ? a.K : a.N;
    p.tall = a.N > a.K;
    p.C = (p.n + MAXW - 1) / MAXW;
    p.w = ((p.n + p.C - 1) / p.C + 63) & ~63;
    static std::atomic<bool> ready[64];
    cudaError_t e;
    if (!ready[a.dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(muon_small, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "update kernel: %s", cudaGetErrorString(e));
        ready[a.dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.E * p.C);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, muon_small, p);
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "update kernel: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return MXFP8_OK;
}

}  // namespace mxw
