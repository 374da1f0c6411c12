// Tokens sorted by expert and back (include/mxfp8_step.h): the plan of a
// routing, the rows in sorted order (bf16 or quantised to MXFP8), the weighted
// sum back in token order, and the gradients of both.
#include <cuda_fp8.h>

#include "mxw_internal.h"
#include "mxw_ptx.cuh"
#include "mxw_quant.cuh"
#include "mxw_step.h"
#include "../../include/mxfp8_step.h"

namespace mxw {
namespace {

constexpr uint32_t FULL = 0xffffffffu;

// 16 bytes that are read once. (No ld.global.nc in these kernels: they start
// before the kernel that writes their inputs has ended, and that path is for
// data that does not change while a kernel runs.)
__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// ------------------------------------------------------------------ plan

// A counting sort by expert that keeps the order of the pairs, in one cluster:
// every warp counts the experts of its run of pairs (its own row of counters in
// shared memory: no atomics), the warps' and, through distributed shared memory,
// the CTAs' counts become starting rows, and every warp walks its run again and
// hands out rows. match.any gives each lane its place among the lanes with the
// same expert.
constexpr int PLAN_MAX_CTAS = 8;
constexpr int PLAN_SMEM = 200 * 1024;

struct PlanPar {
    const void* ids;
    int pairs, first, local, align, rows;
    int32_t *offs, *slot, *src;
    int* status;
};

__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The local expert of a pair, or -1.
template <class Id>
__device__ __forceinline__ int pair_expert(const Id* ids, int p, int hi, int first, int local) {
    if (p >= hi) return -1;
    const long long e = static_cast<long long>(ids[p]) - first;
    return e >= 0 && e < local ? static_cast<int>(e) : -1;
}

template <class Id>
__global__ void __launch_bounds__(1024) token_plan_kernel(const PlanPar p) {
    extern __shared__ int sm[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* hist = sm;                      // [warps][local]
    int* mine = sm + warps * p.local;    // [local] this CTA's pairs, read by the others
    int* base = mine + p.local;          // [local] first row of the CTA's pairs
    int* ends = base + p.local;          // [local] rows up to the group's end
    __shared__ int part[32];
    const int C = gridDim.x, c = blockIdx.x;  // (the grid is one cluster)
    for (int i = threadIdx.x; i < warps * p.local; i += blockDim.x) hist[i] = 0;
    griddep_launch_dependents();
    griddep_wait();
    __syncthreads();

    const Id* ids = static_cast<const Id*>(p.ids);
    const int per = ((p.pairs + C * warps - 1) / (C * warps) + 31) & ~31;
    const int lo = min(static_cast<long long>(p.pairs), static_cast<long long>(c * warps + warp) * per);
    const int hi = min(p.pairs, lo + per);
    int* count = hist + warp * p.local;
    for (int at = lo; at < hi; at += 32) {
        const int e = pair_expert(ids, at + lane, hi, p.first, p.local);
        const uint32_t same = __match_any_sync(FULL, e);
        if (e >= 0 && lane == __ffs(same) - 1) count[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.local; e += blockDim.x) {
        int run = 0;
        for (int w = 0; w < warps; ++w) {
            const int n = hist[w * p.local + e];
            hist[w * p.local + e] = run;
            run += n;
        }
        mine[e] = run;
    }
    cluster_arrive();
    cluster_wait();
    // experts in runs of `each` a thread: totals over the CTAs, then a scan of the padded sizes
    const int each = (p.local + blockDim.x - 1) / blockDim.x;
    const int e0 = min(p.local, static_cast<int>(threadIdx.x) * each), e1 = min(p.local, e0 + each);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int total = 0, before = 0;
        for (int r = 0; r < C; ++r) {
            const int n = ld_cluster(cluster_map(smem_u32(mine + e), r));
            if (r < c) before += n;
            total += n;
        }
        base[e] = before;
        ends[e] = total;
        sum += (total + p.align - 1) / p.align * p.align;
    }
    cluster_arrive();  // (no CTA leaves before the others have read its counts: waited for at the end)
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(FULL, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int own = lane < warps ? part[lane] : 0;
        int v = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(FULL, v, d);
            if (lane >= d) v += u;
        }
        part[lane] = v - own;
    }
    __syncthreads();
    int row = part[warp] + incl - sum;
    for (int e = e0; e < e1; ++e) {
        const int total = ends[e], end = row + (total + p.align - 1) / p.align * p.align;
        if (c == 0) p.offs[e] = min(end, p.rows);
        base[e] += row;
        ends[e] = end;
        // the group's padding, shared among the CTAs by expert
        if (e % C == c)
            for (int r = row + total; r < min(end, p.rows); ++r) p.src[r] = -1;
        row = end;
    }
    __syncthreads();
    bool dropped = false;
    for (int at = lo; at < hi; at += 32) {
        const int e = pair_expert(ids, at + lane, hi, p.first, p.local);
        const uint32_t same = __match_any_sync(FULL, e);
        int r = -1;
        if (e >= 0) r = base[e] + count[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) count[e] += __popc(same);
        __syncwarp();
        if (r >= p.rows) {
            r = -1;
            dropped = true;
        }
        if (at + lane < hi) p.slot[at + lane] = r;
        if (r >= 0) p.src[r] = at + lane;
    }
    if (__any_sync(FULL, dropped) && lane == 0) atomicOr(p.status, MXFP8_DEV_TOKENS_ROWS);
    const int last = ends[p.local - 1];
    for (long long r = last + static_cast<long long>(c) * blockDim.x + threadIdx.x; r < p.rows; r += C * blockDim.x)
        p.src[r] = -1;
    cluster_wait();
}

// ------------------------------------------------------------------ rows

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int PAD_ROWS = 8;  // rows of the sorted buffers that a warp looks at for padding

struct RowPar {
    int64_t T, rows;
    int H, k, segs;
    const int32_t *slot, *src;
    const uint16_t *tok_in, *sorted_in;
    uint16_t *tok_out, *sorted_out;
    uint8_t *q, *s;
    const float* w;
    float* dw;
    int* status;
};

// An entry of a plan: -1 unless it is in [0, n).
__device__ __forceinline__ int checked(int v, int64_t n, int* status) {
    if (v >= -1 && v < n) return v;
    atomicOr(status, MXFP8_DEV_TOKENS_RANGE);
    return -1;
}

// Slots of token t: lane j holds choices j and j + 32 (-1 where there is none).
struct Slots {
    int lo, hi;
    uint32_t has_lo, has_hi;
};

__device__ __forceinline__ Slots token_slots(const RowPar& p, int64_t t, int lane) {
    Slots s{-1, -1, 0, 0};
    const int32_t* at = p.slot + t * p.k;
    if (lane < p.k) s.lo = checked(at[lane], p.rows, p.status);
    if (lane + 32 < p.k) s.hi = checked(at[lane + 32], p.rows, p.status);
    s.has_lo = __ballot_sync(FULL, s.lo >= 0);
    s.has_hi = p.k > 32 ? __ballot_sync(FULL, s.hi >= 0) : 0;
    return s;
}

__device__ __forceinline__ float2 bf16x2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Bits of the warp's PAD_ROWS rows from r0 on that are padding.
__device__ __forceinline__ uint32_t padding_rows(const RowPar& p, int64_t r0, int lane) {
    bool pad = false;
    if (lane < PAD_ROWS && r0 + lane < p.rows) pad = checked(p.src[r0 + lane], p.T * p.k, p.status) < 0;
    return __ballot_sync(FULL, pad);
}

__device__ __forceinline__ void zero_row(void* row, int bytes, int lane) {
    for (int b = lane * 16; b < bytes; b += 512)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(row) + b) = make_uint4(0, 0, 0, 0);
}

// Each token's columns are read once and written to all of its rows.
constexpr int SEG = 1024;  // columns that a warp moves

__global__ void __launch_bounds__(THREADS) dispatch_kernel(const RowPar p) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t tokens = p.T * p.segs, units = tokens + (p.rows + PAD_ROWS - 1) / PAD_ROWS;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * WARPS) {
        if (u >= tokens) {
            const int64_t r0 = (u - tokens) * PAD_ROWS;
            for (uint32_t pad = padding_rows(p, r0, lane); pad; pad &= pad - 1)
                zero_row(p.sorted_out + (r0 + __ffs(pad) - 1) * p.H, 2 * p.H, lane);
            continue;
        }
        const int64_t t = u / p.segs;
        const int col = static_cast<int>(u - t * p.segs) * SEG + lane * 8;
        const Slots s = token_slots(p, t, lane);
        if (!(s.has_lo | s.has_hi)) continue;
        uint4 v[SEG / 256];
#pragma unroll
        for (int i = 0; i < SEG / 256; ++i)
            if (col + 256 * i < p.H) v[i] = load16(p.tok_in + t * p.H + col + 256 * i);
#pragma unroll 1
        for (int half = 0; half < 2; ++half)
            for (uint32_t has = half ? s.has_hi : s.has_lo; has; has &= has - 1) {
                const int64_t r = __shfl_sync(FULL, half ? s.hi : s.lo, __ffs(has) - 1);
#pragma unroll
                for (int i = 0; i < SEG / 256; ++i)
                    if (col + 256 * i < p.H) *reinterpret_cast<uint4*>(p.sorted_out + r * p.H + col + 256 * i) = v[i];
            }
    }
}

// 16 columns a lane: two neighbouring lanes hold a block of 32.
constexpr int QSEG = 512;

__global__ void __launch_bounds__(THREADS) dispatch_mxfp8_kernel(const RowPar p) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t tokens = p.T * p.segs, units = tokens + (p.rows + PAD_ROWS - 1) / PAD_ROWS;
    const int blocks = p.H / 32;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * WARPS) {
        if (u >= tokens) {
            const int64_t r0 = (u - tokens) * PAD_ROWS;
            for (uint32_t pad = padding_rows(p, r0, lane); pad; pad &= pad - 1) {
                const int64_t r = r0 + __ffs(pad) - 1;
                zero_row(p.q + r * p.H, p.H, lane);
                for (int b = lane; b < blocks; b += 32) p.s[r * blocks + b] = 0;
            }
            continue;
        }
        const int64_t t = u / p.segs;
        const int col = static_cast<int>(u - t * p.segs) * QSEG + lane * 16;
        const Slots sl = token_slots(p, t, lane);
        if (!(sl.has_lo | sl.has_hi)) continue;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (col < p.H) {
            a = load16(p.tok_in + t * p.H + col);
            b = load16(p.tok_in + t * p.H + col + 8);
        }
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, max(w[i] & 0x7fff0000u, (w[i] << 16) & 0x7fff0000u));
        amax = max(amax, __shfl_xor_sync(FULL, amax, 1));
        uint4 q;
        uint8_t sb;
        if (amax >= 0x7f800000u) {  // NaN or infinity in the block
            q = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
            sb = 0xFF;
        } else {
            const int e = block_exponent(amax);
            const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = bf16x2(w[2 * i]), y = bf16x2(w[2 * i + 1]);
                const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(x.x * inv, x.y * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(y.x * inv, y.y * inv), __NV_SATFINITE, __NV_E4M3);
                o[i] = l | (h << 16);
            }
            q = make_uint4(o[0], o[1], o[2], o[3]);
            sb = static_cast<uint8_t>(e + 127);
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half)
            for (uint32_t has = half ? sl.has_hi : sl.has_lo; has; has &= has - 1) {
                const int64_t r = __shfl_sync(FULL, half ? sl.hi : sl.lo, __ffs(has) - 1);
                if (col < p.H) {
                    *reinterpret_cast<uint4*>(p.q + r * p.H + col) = q;
                    if (!(lane & 1)) p.s[r * blocks + (col >> 5)] = sb;
                }
            }
    }
}

// The weighted sum of a token's rows: 8 columns a lane, two runs of 256 columns a
// warp, the rows in ascending order of the choice.
constexpr int CSEG = 512;

template <bool WEIGHTED>
__global__ void __launch_bounds__(THREADS) combine_kernel(const RowPar p) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t units = p.T * p.segs;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * WARPS) {
        const int64_t t = u / p.segs;
        const int col = static_cast<int>(u - t * p.segs) * CSEG + lane * 8;
        const Slots s = token_slots(p, t, lane);
        float w_lo = 1.f, w_hi = 1.f;
        if (WEIGHTED) {
            if (lane < p.k) w_lo = p.w[t * p.k + lane];
            if (lane + 32 < p.k) w_hi = p.w[t * p.k + lane + 32];
        }
        float acc[2][8];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i / 8][i % 8] = 0.f;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            uint32_t has = half ? s.has_hi : s.has_lo;
            while (has) {
                // four rows' loads in flight
                uint4 v[4][2];
                float w[4];
                bool there[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    there[j] = has != 0;
                    const int from = there[j] ? __ffs(has) - 1 : 0;
                    has &= has - 1;
                    const int64_t r = __shfl_sync(FULL, half ? s.hi : s.lo, from);
                    w[j] = __shfl_sync(FULL, half ? w_hi : w_lo, from);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (there[j] && col + 256 * i < p.H)
                            v[j][i] = load16(p.sorted_in + r * p.H + col + 256 * i);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (there[j]) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t x[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const float2 f = bf16x2(x[m]);
                                if (WEIGHTED) {
                                    acc[i][2 * m] = fmaf(w[j], f.x, acc[i][2 * m]);
                                    acc[i][2 * m + 1] = fmaf(w[j], f.y, acc[i][2 * m + 1]);
                                } else {
                                    acc[i][2 * m] += f.x;
                                    acc[i][2 * m + 1] += f.y;
                                }
                            }
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (col + 256 * i < p.H) {
                uint32_t o[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) o[m] = pack_bf16x2(__float_as_uint(acc[i][2 * m]), __float_as_uint(acc[i][2 * m + 1]));
                *reinterpret_cast<uint4*>(p.tok_out + t * p.H + col + 256 * i) = make_uint4(o[0], o[1], o[2], o[3]);
            }
    }
}

// A warp a pair: its row of y against the token's row of dout, and the weighted
// row of dout in y's place. The warps of a CTA hold neighbouring pairs, so that a
// token's row of dout comes from memory once.
__global__ void __launch_bounds__(THREADS) combine_grad_kernel(const RowPar p) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t pairs = p.T * p.k, units = pairs + (p.rows + PAD_ROWS - 1) / PAD_ROWS;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * WARPS) {
        if (u >= pairs) {
            const int64_t r0 = (u - pairs) * PAD_ROWS;
            for (uint32_t pad = padding_rows(p, r0, lane); pad; pad &= pad - 1)
                zero_row(p.sorted_out + (r0 + __ffs(pad) - 1) * p.H, 2 * p.H, lane);
            continue;
        }
        const int64_t r = checked(p.slot[u], p.rows, p.status);
        float dot = 0.f;
        if (r >= 0) {
            const float w = p.w[u];
            const uint16_t* d = p.tok_in + u / p.k * p.H;
            const uint16_t* y = p.sorted_in + r * p.H;
            uint16_t* dy = p.sorted_out + r * p.H;
            for (int c0 = lane * 8; c0 < p.H; c0 += 1024) {
                uint4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 + 256 * i < p.H) {
                        a[i] = *reinterpret_cast<const uint4*>(d + c0 + 256 * i);
                        b[i] = *reinterpret_cast<const uint4*>(y + c0 + 256 * i);  // (dy may be y)
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 + 256 * i < p.H) {
                        const uint32_t av[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, bv[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
                        uint32_t o[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const float2 f = bf16x2(av[m]), g = bf16x2(bv[m]);
                            dot = fmaf(f.x, g.x, dot);
                            dot = fmaf(f.y, g.y, dot);
                            o[m] = pack_bf16x2(__float_as_uint(w * f.x), __float_as_uint(w * f.y));
                        }
                        *reinterpret_cast<uint4*>(dy + c0 + 256 * i) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
            }
        }
#pragma unroll
        for (int d = 16; d; d /= 2) dot += __shfl_xor_sync(FULL, dot, d);
        if (lane == 0) p.dw[u] = dot;
    }
}

int failed(cudaError_t e, const char* what) {
    return host_fail(MXFP8_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Launches `kernel` so that its start overlaps the end of the kernel before it
// (each kernel waits for that one before its first access).
template <class Par>
int launch(void (*kernel)(Par), const Par& p, int64_t units, const TokenArgs& a, const char* what) {
    const int64_t blocks = (units + WARPS - 1) / WARPS;
    if (blocks == 0) return MXFP8_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < (1 << 22) ? blocks : (1 << 22)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? MXFP8_OK : failed(e, what);
}

RowPar row_par(const TokenArgs& a, int seg) {
    RowPar p{};
    p.T = a.T; p.rows = a.rows; p.H = a.H; p.k = a.top_k; p.segs = (a.H + seg - 1) / seg;
    p.slot = a.slot; p.src = a.src; p.tok_in = a.tok_in; p.sorted_in = a.sorted_in;
    p.tok_out = a.tok_out; p.sorted_out = a.sorted_out; p.q = a.q; p.s = a.s; p.w = a.weights; p.dw = a.dweights;
    p.status = a.status;
    return p;
}

int64_t pad_units(const TokenArgs& a) { return (a.rows + PAD_ROWS - 1) / PAD_ROWS; }

}  // namespace

int launch_token_plan(const TokenPlanArgs& a) {
    PlanPar p{a.ids, static_cast<int>(a.pairs), a.first, a.local, a.align, static_cast<int>(a.rows), a.offs, a.slot, a.src, a.status};
    auto kernel = a.id64 ? token_plan_kernel<int64_t> : token_plan_kernel<int32_t>;
    int warps = 32;
    while ((warps + 3) * static_cast<size_t>(a.local) * 4 > PLAN_SMEM) warps /= 2;
    const size_t smem = (warps + 3) * static_cast<size_t>(a.local) * 4;
    // (set before every launch: the attribute belongs to the device that is current)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PLAN_SMEM);
    if (e != cudaSuccess) return failed(e, "token plan: shared memory");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(PLAN_MAX_CTAS);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PLAN_MAX_CTAS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PlanPar>(p));
    return e == cudaSuccess ? MXFP8_OK : failed(e, "token plan kernel");
}

int launch_token_dispatch(const TokenArgs& a) {
    const RowPar p = row_par(a, a.q ? QSEG : SEG);
    return launch(a.q ? dispatch_mxfp8_kernel : dispatch_kernel, p, a.T * p.segs + pad_units(a), a, "dispatch kernel");
}

int launch_token_combine(const TokenArgs& a) {
    const RowPar p = row_par(a, CSEG);
    return launch(a.weights ? combine_kernel<true> : combine_kernel<false>, p, a.T * p.segs, a, "combine kernel");
}

int launch_token_combine_grad(const TokenArgs& a) {
    const RowPar p = row_par(a, a.H);
    return launch(combine_grad_kernel, p, a.T * a.top_k + pad_units(a), a, "combine gradient kernel");
}

}  // namespace mxw
