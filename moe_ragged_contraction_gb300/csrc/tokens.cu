// Tokens sorted by expert and back (include/mxfp8_step.h): the plan of a
// routing, the rows in sorted order (bf16 or quantised to MXFP8), the weighted
// sum back in token order, and the gradients of both.
#include <cuda_fp8.h>

#include <atomic>

#include "mxw_internal.h"
#include "mxw_ptx.cuh"
#include "mxw_quant.cuh"
#include "mxw_step.h"
#include "../../include/mxfp8_step.h"

namespace mxw {
namespace {

constexpr uint32_t FULL = 0xffffffffu;

// 16 bytes that are read once; zeros and no access unless `there` (no branch:
// loads of a group leave together). No ld.global.nc in these kernels: they start
// before the kernel that writes their inputs has ended, and that path is for data
// that does not change while a kernel runs.
__device__ __forceinline__ uint4 load16_if(bool there, const void* p) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(static_cast<uint32_t>(there))
        : "memory");
    return v;
}

// The same through L1, for what neighbouring warps read too.
__device__ __forceinline__ uint4 load16_l1_if(bool there, const void* p) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(static_cast<uint32_t>(there))
        : "memory");
    return v;
}

// ------------------------------------------------------------------ plan

// A counting sort by expert that keeps the order of the pairs, in clusters that do
// not talk to one another. Each CTA of a cluster has a part of the pairs, cut into
// as many segments as there are clusters; the cluster of that number ranks the
// pairs of the segment and gives them rows, and only counts those of the others:
// counting takes some 15 instructions for a warp's 32 pairs, ranking 60, and no
// scratch or hand-over between clusters is needed. In its segment every warp has a run of pairs and a row of
// counters in shared memory (no atomics); the warps' counts and, through
// distributed shared memory, the CTAs' become starting rows.
constexpr int PLAN_MAX_CTAS = 16;
constexpr int PLAN_SMEM = 224 * 1024;
// Pairs up to which one CTA, one cluster sorts: 2040 pairs take 6.9 us on a cluster
// and 7.6 on a CTA, 1536 6.9 / 7.0, 384 5.7 either way; 49152 8.4 on a cluster and
// 8.6 on four, 98304 10.6 / 9.4, 2097152 107 / 45. (More than four clusters of 16 do
// not fit the GPU at once.)
constexpr int PLAN_ONE_CTA = 512, PLAN_ONE_CLUSTER = 65536;

struct PlanPar {
    const void* ids;
    int pairs, first, local, align, rows, groups, C, Q;  // C CTAs in each of Q clusters
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

// (not the .aligned forms: lanes come out of loops of different lengths)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// A warp works on RUN pairs at a time; their experts and ranks stay in shared memory.
constexpr int RUN = 512, LOADS = RUN / 32;

// Writes the local experts (or -1) of the pairs at .. hi (RUN at most) to `kept`,
// with all loads in flight together.
template <class Id>
__device__ __forceinline__ void load_run(const Id* ids, int at, int hi, int first, int local, int lane, int* kept) {
    Id v[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) v[i] = at + 32 * i + lane < hi ? ids[at + 32 * i + lane] : Id(-1);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const long long d = static_cast<long long>(v[i]) - first;
        kept[32 * i + lane] = v[i] >= 0 && d >= 0 && d < local ? static_cast<int>(d) : -1;
    }
}

// Adds the experts of the pairs lo .. hi to `counts`, by the whole CTA.
template <class Id>
__device__ __forceinline__ void count_pairs(const Id* ids, int lo, int hi, const PlanPar& p, int* counts) {
    constexpr int N = 8;
#pragma unroll 1
    for (long long at = lo + static_cast<int>(threadIdx.x); at < hi; at += N * blockDim.x) {
        Id v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = at + i * static_cast<int>(blockDim.x) < hi ? ids[at + i * static_cast<int>(blockDim.x)] : Id(-1);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const long long d = static_cast<long long>(v[i]) - p.first;
            if (v[i] >= 0 && d >= 0 && d < p.local) atomicAdd(counts + d, 1);
        }
    }
}

// Lanes whose e (below 2^(3 groups), or -1) is this lane's. match.any takes the
// longer the more values there are: 262144 pairs, one in eight here, 9.8 us with it
// and 11.2 with ballots; all of 2097152 here, 64 experts, 54 / 45.
__device__ __forceinline__ uint32_t same_expert(int e, int groups) {
    uint32_t m = __ballot_sync(FULL, e >= 0);
    if (__popc(m) <= 8) return __match_any_sync(FULL, e);
#pragma unroll 1
    for (int g = 0; g < groups; ++g, e >>= 3) {
#pragma unroll
        for (int b = 0; b < 3; ++b) m &= ~(__ballot_sync(FULL, e & (1 << b)) ^ static_cast<uint32_t>((e << (31 - b)) >> 31));
    }
    return m;  // (nothing that is used where e is -1)
}

// The place of each lane's pair among the warp's pairs of its expert so far,
// counted on in `count`.
__device__ __forceinline__ int rank_of(int e, int groups, int lane, int* count) {
    const uint32_t same = same_expert(e, groups);
    const int before = e >= 0 ? count[e] : 0;
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) count[e] = before + __popc(same);
    __syncwarp();
    return before + __popc(same & ((1u << lane) - 1));
}

template <class Id>
__global__ void __launch_bounds__(1024) token_plan_kernel(const PlanPar p) {
    extern __shared__ int sm[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* hist = sm;                      // [warps][local]
    int* mine = sm + warps * p.local;    // [local] this CTA's pairs, read by the others
    int* base = mine + p.local;          // [local] first row of the CTA's pairs
    int* full = base + p.local;          // [local] end of the group's pairs
    int* ends = full + p.local;          // [local] end of the group
    int* own = ends + p.local;           // [local] start of the expert's pairs among the segment's, by expert
    int* ahead = own + p.local;          // [2][local] the CTA's pairs ahead of the segment and behind it
    int* kept = ahead + 2 * p.local + warp * RUN;
    uint16_t* sorted = reinterpret_cast<uint16_t*>(ahead + 2 * p.local + warps * RUN);  // [warps * RUN] the segment's pairs by expert
    __shared__ int2 part[32];
    const int C = p.C, c = blockIdx.x % C, q = blockIdx.x / C;
    for (int i = threadIdx.x; i < warps * p.local; i += blockDim.x) hist[i] = 0;
    for (int i = threadIdx.x; i < 2 * p.local; i += blockDim.x) ahead[i] = 0;
    griddep_launch_dependents();
    griddep_wait();
    __syncthreads();

    const Id* ids = static_cast<const Id*>(p.ids);
    const int shares = C * p.Q * warps, per = ((p.pairs + shares - 1) / shares + 31) & ~31;
    const auto at_share = [&](int i) { return static_cast<int>(min(static_cast<long long>(p.pairs), static_cast<long long>(i) * per)); };
    const int seg = (c * p.Q + q) * warps, lo = at_share(seg + warp), hi = at_share(seg + warp + 1);
    const bool once = per <= RUN;  // the first pass's ranks serve the second
    if (p.Q > 1) {
        count_pairs(ids, at_share(c * p.Q * warps), at_share(seg), p, ahead);
        count_pairs(ids, at_share(seg + warps), at_share((c + 1) * p.Q * warps), p, ahead + p.local);
    }
    int* count = hist + warp * p.local;
    // pass 0 counts, pass 1 gives out rows; rolled, so that the code is short: every
    // line of it misses the instruction cache once
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int at = lo; at < hi; at += RUN) {
            const int n = min(RUN, hi - at);
            if (pass == 1 && once) {
#pragma unroll 1
                for (int k = lane; k < n; k += 32) {
                    const int v = kept[k], e = v & 2047;
                    int row = -1;
                    if (v >= 0) {
                        const int place = count[e] + (v >> 11);
                        sorted[own[e] + place] = static_cast<uint16_t>(warp * per + k);
                        row = base[e] + place;
                        if (row >= p.rows) row = -1;
                    }
                    p.slot[at + k] = row;
                }
                continue;
            }
            load_run(ids, at, hi, p.first, p.local, lane, kept);
            __syncwarp();
            if (!once && pass == 0) {
#pragma unroll 1
                for (int k = lane; k < n; k += 32)
                    if (kept[k] >= 0) atomicAdd(count + kept[k], 1);  // (counts only: the order does not matter)
                continue;
            }
#pragma unroll 1
            for (int k = lane; k - lane < n; k += 32) {
                const int e = kept[k], rank = rank_of(e, p.groups, lane, count);
                if (once) {
                    if (e >= 0) kept[k] = rank << 11 | e;  // (rank < 512, local <= 2048)
                } else if (k < n) {
                    int row = e >= 0 ? base[e] + rank : -1;
                    if (row >= p.rows) row = -1;
                    if (row >= 0) p.src[row] = at + k;
                    p.slot[at + k] = row;
                }
            }
        }
        if (pass == 1) break;
        __syncthreads();
        for (int e = threadIdx.x; e < p.local; e += blockDim.x) {
            int run = 0;
#pragma unroll 1
            for (int w = 0; w < warps; w += 8) {
                int n[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] = hist[(w + i) * p.local + e];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    hist[(w + i) * p.local + e] = run;
                    run += n[i];
                }
            }
            full[e] = run;
            mine[e] = run + ahead[e] + ahead[p.local + e];
        }
        cluster_arrive();
        cluster_wait();
        // experts in runs of `each` a thread: totals over the CTAs, then a scan of the padded sizes
        const int each = (p.local + blockDim.x - 1) / blockDim.x;
        const int e0 = min(p.local, static_cast<int>(threadIdx.x) * each), e1 = min(p.local, e0 + each);
        int sum = 0, here = 0;
#pragma unroll 1
        for (int e = e0; e < e1; ++e) {
            int n[PLAN_MAX_CTAS], total = 0, before = 0;
#pragma unroll
            for (int r = 0; r < PLAN_MAX_CTAS; ++r) n[r] = r < C ? ld_cluster(cluster_map(smem_u32(mine + e), r)) : 0;
#pragma unroll
            for (int r = 0; r < PLAN_MAX_CTAS; ++r) {
                if (r < c) before += n[r];
                total += n[r];
            }
            base[e] = before + ahead[e];
            ends[e] = total;
            sum += (total + p.align - 1) / p.align * p.align;
            here += full[e];
        }
        cluster_arrive();  // (no CTA leaves before the others have read its counts: waited for at the end)
        int2 incl = make_int2(sum, here);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(FULL, incl.x, d), y = __shfl_up_sync(FULL, incl.y, d);
            if (lane >= d) {
                incl.x += x;
                incl.y += y;
            }
        }
        if (lane == 31) part[warp] = incl;
        __syncthreads();
        int row = incl.x - sum, at = incl.y - here;
        for (int w = 0; w < warp && e0 < p.local; ++w) {
            row += part[w].x;
            at += part[w].y;
        }
#pragma unroll 1
        for (int e = e0; e < e1; ++e) {
            const int total = ends[e], n = full[e], end = row + (total + p.align - 1) / p.align * p.align;
            if (blockIdx.x == 0) p.offs[e] = min(end, p.rows);
            base[e] += row;
            full[e] = row + total;
            ends[e] = end;
            own[e] = at;
            ahead[e] = n;  // (the segment's pairs from here on)
            row = end;
            at += n;
        }
        __syncthreads();
    }
    if (once) {
        // src by expert: a warp's stores are neighbours
        __syncthreads();
        const int first = seg * per;
#pragma unroll 1
        for (int e = warp; e < p.local; e += warps)
            for (int i = lane; i < min(ahead[e], p.rows - base[e]); i += 32) p.src[base[e] + i] = first + sorted[own[e] + i];
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e < p.local; e += blockDim.x)
            if (full[e] > p.rows) atomicOr(p.status, MXFP8_DEV_TOKENS_ROWS);  // (that many pairs were dropped)
    // padding: a warp an expert, and the rows behind the last group
    for (int e = blockIdx.x * warps + warp; e < p.local; e += gridDim.x * warps)
        for (int r = full[e] + lane; r < min(ends[e], p.rows); r += 32) p.src[r] = -1;
    for (long long r = ends[p.local - 1] + static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; r < p.rows; r += gridDim.x * blockDim.x)
        p.src[r] = -1;
    cluster_wait();
}

// ------------------------------------------------------------------ rows

// What bounds these kernels is DRAM in calls of many tokens with some 1000 columns
// or more (92% to 99% of the copy rate); with short rows it is what a unit takes
// whatever its width: a chain of two loads, and lanes without columns (17613 tokens of
// 96 columns to MXFP8: 12.8 us for 2.2 of bytes; sum of 54484 tokens of 240 columns:
// 20.7 for 5.5). They have no arithmetic to speak of. A unit of work is a warp's: some columns of
// a token, or a pair. CTAs of four warps: a CTA
// lives as long as its longest unit, and tokens have from none to top_k rows here
// (with eight warps: 16B dispatch 76.9 us against 74.1, combine on the 671B rank
// 162 / 158, its gradient 225 / 220; with two 75.1, 157, 233).
constexpr int THREADS = 128, WARPS = THREADS / 32;
constexpr int PAD_CTAS = 4096;

struct RowPar {
    int64_t T, rows;
    int H, k, seg, segs;  // seg: columns of a unit
    int words;            // rows of scales are whole aligned words
    int pad, pad_ctas;    // zero_padding's rows, and its CTAs
    int each;             // pairs of a warp (gradient of the sum)
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

// Warps that share a row of padding: each writes 2 KB of it or more.
__host__ __device__ inline int pad_parts(int bytes) { return bytes <= 2048 ? 1 : bytes <= 4096 ? 2 : 4; }
static_assert(WARPS % 4 == 0, "pad_parts");

// Zeros on the padding among the `cta`th p.pad * (WARPS / parts) rows (of `bytes`,
// and of scales): a CTA's work, p.pad rows for each `parts` warps.
__device__ __forceinline__ void zero_padding(const RowPar& p, uint32_t cta, int lane, uint8_t* out, int bytes, uint8_t* scales, int blocks) {
    const int parts = pad_parts(bytes), warp = threadIdx.x >> 5, part = (warp & (parts - 1)) * 32 + lane;
    const int64_t r0 = (static_cast<int64_t>(cta) * (WARPS / parts) + warp / parts) * p.pad;
    bool pad = false;
    if (lane < p.pad && r0 + lane < p.rows) pad = checked(p.src[r0 + lane], p.T * p.k, p.status) < 0;
#pragma unroll 1
    for (uint32_t rows = __ballot_sync(FULL, pad); rows; rows &= rows - 1) {
        const int64_t r = r0 + __ffs(rows) - 1;
        uint8_t* row = out + r * bytes;
#pragma unroll 4
        for (int b = part * 16; b < bytes; b += parts * 512) *reinterpret_cast<uint4*>(row + b) = make_uint4(0, 0, 0, 0);
        if (p.words)
            for (int b = 4 * part; b < blocks; b += parts * 128) *reinterpret_cast<uint32_t*>(scales + r * blocks + b) = 0;
        else
            for (int b = part; b < blocks; b += parts * 32) scales[r * blocks + b] = 0;
    }
}

// Each token's columns are read once and written to all of its rows, SEG at a time.
// 16384 tokens of 2048 columns to 6 rows each: 74 us, 6.4 TB/s; 32768 of 7168, 32 of
// 256 experts here: 156 us.
constexpr int SEG = 1024;

__global__ void __launch_bounds__(THREADS) dispatch_kernel(const RowPar p) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t tokens = static_cast<uint32_t>(p.T) * p.segs, first_pad = (tokens + WARPS - 1) / WARPS;
    const uint32_t ctas = first_pad + p.pad_ctas;
    for (uint32_t cta = blockIdx.x; cta < ctas; cta += gridDim.x) {
        if (cta >= first_pad) {
            zero_padding(p, cta - first_pad, lane, reinterpret_cast<uint8_t*>(p.sorted_out), 2 * p.H, nullptr, 0);
            continue;
        }
        const uint32_t u = cta * WARPS + (threadIdx.x >> 5);
        if (u >= tokens) continue;
        const int64_t t = u / static_cast<uint32_t>(p.segs);
        const int seg = static_cast<int>(u - static_cast<uint32_t>(t) * p.segs) * p.seg, end = min(p.H, seg + p.seg);
        const Slots s = token_slots(p, t, lane);
        if (!(s.has_lo | s.has_hi)) continue;
#pragma unroll 1
        for (int c = seg; c < end; c += SEG) {  // (the same for all lanes)
            const int col = c + lane * 8;
            uint4 v[SEG / 256];
#pragma unroll
            for (int i = 0; i < SEG / 256; ++i) v[i] = load16_if(col + 256 * i < end, p.tok_in + t * p.H + col + 256 * i);
#pragma unroll 1
            for (int half = 0; half < 2; ++half)
#pragma unroll 1
                for (uint32_t has = half ? s.has_hi : s.has_lo; has; has &= has - 1) {
                    const int64_t r = __shfl_sync(FULL, half ? s.hi : s.lo, __ffs(has) - 1);
                    uint16_t* out = p.sorted_out + r * p.H + col;
#pragma unroll
                    for (int i = 0; i < SEG / 256; ++i)
                        if (col + 256 * i < end) *reinterpret_cast<uint4*>(out + 256 * i) = v[i];
                }
        }
    }
}

// As dispatch_kernel, with a token's columns quantised once for all of its rows:
// 16 columns a lane in each of RUNS runs of 512, so that two neighbouring lanes
// hold a block of 32. Scales go out in words of four. 32768 tokens of 7168 columns,
// 32 of 256 experts here: 106 us, 6.4 TB/s. RUNS is 4, or 1 for rows of up to 512
// columns (49809 tokens of 128: 35 us, 54 with 4, all of it instructions).
__device__ __forceinline__ void quantise16(const uint4& a, const uint4& b, uint4& q, uint32_t& sb) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, max(w[i] & 0x7fff0000u, (w[i] << 16) & 0x7fff0000u));
    amax = max(amax, __shfl_xor_sync(FULL, amax, 1));
    if (amax >= 0x7f800000u) {  // NaN or infinity in the block
        q = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
        sb = 0xFF;
        return;
    }
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
    sb = e + 127;
}

template <int RUNS>
__global__ void __launch_bounds__(THREADS, 8) dispatch_mxfp8_kernel(const RowPar p) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t tokens = static_cast<uint32_t>(p.T) * p.segs, first_pad = (tokens + WARPS - 1) / WARPS;
    const int blocks = p.H / 32;
    const uint32_t ctas = first_pad + p.pad_ctas;
    for (uint32_t cta = blockIdx.x; cta < ctas; cta += gridDim.x) {
        if (cta >= first_pad) {
            zero_padding(p, cta - first_pad, lane, p.q, p.H, p.s, blocks);
            continue;
        }
        const uint32_t u = cta * WARPS + (threadIdx.x >> 5);
        if (u >= tokens) continue;
        const int64_t t = u / static_cast<uint32_t>(p.segs);
        const int seg = static_cast<int>(u - static_cast<uint32_t>(t) * p.segs) * p.seg, end = min(p.H, seg + p.seg);
        const Slots sl = token_slots(p, t, lane);
        if (!(sl.has_lo | sl.has_hi)) continue;
#pragma unroll 1
        for (int c = seg; c < end; c += 512 * RUNS) {  // (the same for all lanes)
            const int col = c + lane * 16;
            uint4 v[RUNS][2], q[RUNS];
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                v[i][0] = load16_if(col + 512 * i < end, p.tok_in + t * p.H + col + 512 * i);
                v[i][1] = load16_if(col + 512 * i < end, p.tok_in + t * p.H + col + 512 * i + 8);
            }
            uint32_t mine = 0, word = 0;
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                uint32_t sb;
                quantise16(v[i][0], v[i][1], q[i], sb);
                mine |= sb << (8 * i);
            }
            // lanes 0 .. 15: the scales of four neighbouring blocks (run lane / 4, lanes 8 (lane % 4) + 0, 2, 4, 6)
#pragma unroll
            for (int m = 0; m < 4; ++m) word |= ((__shfl_sync(FULL, mine, 8 * (lane & 3) + 2 * m) >> (8 * (lane >> 2 & 3))) & 0xff) << (8 * m);
#pragma unroll 1
            for (int half = 0; half < 2; ++half)
#pragma unroll 1
                for (uint32_t has = half ? sl.has_hi : sl.has_lo; has; has &= has - 1) {
                    const int64_t r = __shfl_sync(FULL, half ? sl.hi : sl.lo, __ffs(has) - 1);
                    uint8_t* out = p.q + r * p.H + col;
                    uint8_t* scales = p.s + r * blocks + c / 32;
#pragma unroll
                    for (int i = 0; i < RUNS; ++i)
                        if (col + 512 * i < end) *reinterpret_cast<uint4*>(out + 512 * i) = q[i];
                    if (p.words) {
                        if (lane < 4 * RUNS && c + 128 * lane < end) *reinterpret_cast<uint32_t*>(scales + 4 * lane) = word;
                    } else if (!(lane & 1)) {
#pragma unroll
                        for (int i = 0; i < RUNS; ++i)
                            if (col + 512 * i < end) scales[16 * i + lane / 2] = static_cast<uint8_t>(mine >> (8 * i));
                    }
                }
        }
    }
}

__device__ __forceinline__ void words(const uint4& v, uint32_t (&w)[4]) {
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}

// Rows and weights of the next G choices of a token that have a row: the lowest
// set bits of `has`, which are taken from it.
template <int G>
struct Group {
    int row[G];
    float w[G];      // 0 where there is none
    int choice[G];   // -1 where there is none
};

template <int G, bool WEIGHTED>
__device__ __forceinline__ Group<G> next_group(uint32_t& has, int slot, float w) {
    Group<G> g;
#pragma unroll
    for (int j = 0; j < G; ++j) {
        const int from = __ffs(has) - 1;
        has &= has - 1;
        g.choice[j] = from;
        g.row[j] = __shfl_sync(FULL, slot, from & 31);
        const float v = WEIGHTED ? __shfl_sync(FULL, w, from & 31) : 1.f;
        g.w[j] = from >= 0 ? v : 0.f;
    }
    return g;
}

// acc += w * row over a group's rows, 8 columns a lane at col + 256 u
template <int G, int U, bool WEIGHTED>
__device__ __forceinline__ void add_rows(const RowPar& p, const Group<G>& g, int col, int end, float (&acc)[U][8]) {
    uint4 v[G][U];
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[j][u] = load16_if(g.choice[j] >= 0 && col + 256 * u < end, p.sorted_in + static_cast<int64_t>(g.row[j]) * p.H + col + 256 * u);
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t x[4];
            words(v[j][u], x);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 f = bf16x2(x[m]);
                acc[u][2 * m] = WEIGHTED ? fmaf(g.w[j], f.x, acc[u][2 * m]) : acc[u][2 * m] + f.x;
                acc[u][2 * m + 1] = WEIGHTED ? fmaf(g.w[j], f.y, acc[u][2 * m + 1]) : acc[u][2 * m + 1] + f.y;
            }
        }
}

// The sum of a token's rows over the columns of a unit, G rows of U vectors in
// flight: with six 16-byte loads a lane and 32 warps an SM latency is covered.
template <int G, int U, bool WEIGHTED>
__device__ __forceinline__ void combine_token(const RowPar& p, int64_t t, int seg, int lane, const Slots& s, float w_lo, float w_hi) {
    const int end = min(p.H, seg + p.seg);
#pragma unroll 1
    for (int c0 = seg; c0 < end; c0 += 256 * U) {  // (the same for all lanes: they exchange slots)
        const int c = c0 + lane * 8;
        float acc[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < 8; ++m) acc[u][m] = 0.f;
        for (uint32_t has = s.has_lo; has;) add_rows<G, U, WEIGHTED>(p, next_group<G, WEIGHTED>(has, s.lo, w_lo), c, end, acc);
        for (uint32_t has = s.has_hi; has;) add_rows<G, U, WEIGHTED>(p, next_group<G, WEIGHTED>(has, s.hi, w_hi), c, end, acc);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + 256 * u < end) {
                uint32_t o[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) o[m] = pack_bf16x2(__float_as_uint(acc[u][2 * m]), __float_as_uint(acc[u][2 * m + 1]));
                *reinterpret_cast<uint4*>(p.tok_out + t * p.H + c + 256 * u) = make_uint4(o[0], o[1], o[2], o[3]);
            }
    }
}

// A token with one row or none: 8 vectors in flight, no sums to keep.
template <bool WEIGHTED>
__device__ __forceinline__ void combine_one(const RowPar& p, int64_t t, int seg, int lane, const Slots& s, float w_lo, float w_hi) {
    const int end = min(p.H, seg + p.seg), from = __ffs(s.has_lo | s.has_hi) - 1;
    const bool some = from >= 0;
    const int64_t row = __shfl_sync(FULL, s.has_lo ? s.lo : s.hi, from & 31);
    const float w = WEIGHTED ? __shfl_sync(FULL, s.has_lo ? w_lo : w_hi, from & 31) : 1.f;
    const uint16_t* in = p.sorted_in + (some ? row * p.H : 0);
    uint16_t* out = p.tok_out + t * p.H;
#pragma unroll 1
    for (int c = seg + lane * 8; c < end; c += 256 * 8) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = load16_if(some && c + 256 * u < end, in + c + 256 * u);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (c + 256 * u < end) {
                uint32_t x[4];
                words(v[u], x);
                // 0 + w x, as in the sums of more rows (where it turns a product of -0 into 0)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 f = bf16x2(x[m]);
                    x[m] = pack_bf16x2(__float_as_uint(fmaf(w, f.x, 0.f)), __float_as_uint(fmaf(w, f.y, 0.f)));
                }
                *reinterpret_cast<uint4*>(out + c + 256 * u) = some ? make_uint4(x[0], x[1], x[2], x[3]) : make_uint4(0, 0, 0, 0);
            }
    }
}

// The way by the number n of the token's rows, so that six to eight loads are in
// flight at any n (one way with six rows: k = 8 53.3 us against 51.2; without the
// way for one row: 671B rank 174 / 162; without that of four rows of one vector in
// units of 256 columns: 512 tokens, 4 rows of 2048 columns 3.6 / 3.1, 54484 tokens of
// 240 columns 21.3 / 18.9). 16384 tokens, 6 rows of 2048 columns: 74
// us, 6.3 TB/s.
template <bool WEIGHTED>
__global__ void __launch_bounds__(THREADS, 8) combine_kernel(const RowPar p) {
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t units = static_cast<uint32_t>(p.T) * p.segs;
    for (uint32_t u = blockIdx.x * WARPS + (threadIdx.x >> 5); u < units; u += gridDim.x * WARPS) {
        const int64_t t = u / static_cast<uint32_t>(p.segs);
        const int seg = static_cast<int>(u - static_cast<uint32_t>(t) * p.segs) * p.seg;
        const Slots s = token_slots(p, t, lane);
        float w_lo = 1.f, w_hi = 1.f;
        if (WEIGHTED) {
            if (lane < p.k) w_lo = p.w[t * p.k + lane];
            if (lane + 32 < p.k) w_hi = p.w[t * p.k + lane + 32];
        }
        const int n = __popc(s.has_lo) + __popc(s.has_hi);
        if (p.seg == 256 && n <= 4) combine_token<4, 1, WEIGHTED>(p, t, seg, lane, s, w_lo, w_hi);
        else if (n <= 1) combine_one<WEIGHTED>(p, t, seg, lane, s, w_lo, w_hi);
        else if (n <= 3) combine_token<3, 2, WEIGHTED>(p, t, seg, lane, s, w_lo, w_hi);
        else if (n <= 6) combine_token<6, 1, WEIGHTED>(p, t, seg, lane, s, w_lo, w_hi);
        else combine_token<8, 1, WEIGHTED>(p, t, seg, lane, s, w_lo, w_hi);
    }
}

// A pair's row of y against the token's row of dout, and the weighted row of dout
// to the pair's row of dy; this thread's part of the product.
template <int GRAD_VECS>
__device__ __forceinline__ float grad_row(const RowPar& p, int64_t pair, int64_t row, float w, int from, int step) {
    const uint16_t* d = p.tok_in + static_cast<int64_t>(static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.k)) * p.H;
    const int64_t off = row * p.H;
    float dot = 0.f;
#pragma unroll 1
    for (int c = from; c < p.H; c += step * GRAD_VECS) {
        uint4 a[GRAD_VECS], b[GRAD_VECS];
#pragma unroll
        for (int v = 0; v < GRAD_VECS; ++v) {
            b[v] = load16_if(c + step * v < p.H, p.sorted_in + off + c + step * v);
            a[v] = load16_l1_if(c + step * v < p.H, d + c + step * v);
        }
#pragma unroll
        for (int v = 0; v < GRAD_VECS; ++v) {
            uint32_t x[4], y[4], o[4];
            words(a[v], x);
            words(b[v], y);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 f = bf16x2(x[m]), q = bf16x2(y[m]);
                dot = fmaf(f.x, q.x, dot);
                dot = fmaf(f.y, q.y, dot);
                o[m] = pack_bf16x2(__float_as_uint(w * f.x), __float_as_uint(w * f.y));
            }
            // (dy may be y: every row has one owner, which has read these columns)
            if (c + step * v < p.H) *reinterpret_cast<uint4*>(p.sorted_out + off + c + step * v) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
#pragma unroll
    for (int v = 16; v; v /= 2) dot += __shfl_xor_sync(FULL, dot, v);
    return dot;
}

// The gradient of the weighted sum. How a CTA's warps take pairs:
//   LIST   it lists those of PAIRS neighbouring pairs that have a row, a warp takes
//          one at a time, LOADS = 8 loads of each of the two rows in flight: where
//          most pairs have none and rows more than 2048 columns (671B rank: 223 us, WARP
//          239; 2560 columns 87 / 100. Shorter rows end sooner than a list pays: 1024
//          columns 44, WARP 38; 512 38 / 25; at 1536 and 2048 LIST is 5% ahead)
//   WARP   a warp a pair, 4 loads of each row in flight (1 for rows of up to 256
//          columns), twice the warps: where most have one (16B: 137 us, LIST 143; 512 tokens 6.3 / 15). Several pairs
//          (`each`) one after the other where rows are short, so that there are not
//          more CTAs than the GPU can start (321264 pairs of 392 columns, one in four
//          here: 65 us, 146 with a pair a warp; 16B 134 / 136)
//   TEAM   all warps one pair, for so few that latency counts (64 pairs: 3.8 us, WARP 5.7)
// Neighbouring pairs share their token's row of dout in L1. 32768 tokens of 7168
// columns, 32 of 256 experts: 220 us, 6.8 TB/s.
enum Share { LIST, WARP, TEAM };
constexpr int PAIRS = 64;

template <Share SHARE, int LOADS>
__global__ void __launch_bounds__(THREADS, SHARE == LIST ? 4 : 8) combine_grad_kernel(const RowPar p) {
    const int per = SHARE == LIST ? PAIRS : SHARE == WARP ? WARPS * p.each : 1;  // pairs of a CTA at a time
    __shared__ int list[PAIRS], rows[PAIRS], counts[2];
    __shared__ float sums[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t pairs = p.T * p.k;
    const uint32_t lists = static_cast<uint32_t>((pairs + per - 1) / per),
                   units = lists + p.pad_ctas;
    for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
        if (u >= lists) {
            zero_padding(p, u - lists, lane, reinterpret_cast<uint8_t*>(p.sorted_out), 2 * p.H, nullptr, 0);
            continue;
        }
        const int64_t first = static_cast<int64_t>(u) * per;
        if (SHARE == LIST) {
            __syncthreads();  // (the list before is done with)
            int r = -1, at = 0;
            if (threadIdx.x < PAIRS) {
                if (first + threadIdx.x < pairs) {
                    r = checked(p.slot[first + threadIdx.x], p.rows, p.status);
                    if (r < 0) p.dw[first + threadIdx.x] = 0.f;
                }
                const uint32_t has = __ballot_sync(FULL, r >= 0);
                at = __popc(has & ((1u << lane) - 1));
                if (lane == 0) counts[warp] = __popc(has);
            }
            __syncthreads();
            if (r >= 0) {
                if (warp) at += counts[0];
                list[at] = threadIdx.x;
                rows[at] = r;
            }
            __syncthreads();
            for (int i = warp; i < counts[0] + counts[1]; i += WARPS) {
                const float dot = grad_row<LOADS>(p, first + list[i], rows[i], p.w[first + list[i]], lane * 8, 256);
                if (lane == 0) p.dw[first + list[i]] = dot;
            }
        } else if (SHARE == WARP) {
            // a lane a pair for what there is to know of it, then one after the other
            const int64_t pair = first + warp * p.each + lane;
            int r = -1;
            float w = 0.f, mine = 0.f;
            const bool real = lane < p.each && pair < pairs;
            if (real) {
                r = checked(p.slot[pair], p.rows, p.status);
                w = p.w[pair];
            }
#pragma unroll 1
            for (uint32_t has = __ballot_sync(FULL, r >= 0); has; has &= has - 1) {
                const int i = __ffs(has) - 1;
                const float dot = grad_row<LOADS>(p, pair - lane + i, __shfl_sync(FULL, r, i), __shfl_sync(FULL, w, i), lane * 8, 256);
                if (lane == i) mine = dot;
            }
            if (real) p.dw[pair] = mine;
        } else {
            const int r = checked(p.slot[first], p.rows, p.status);
            float dot = r >= 0 ? grad_row<LOADS>(p, first, r, p.w[first], threadIdx.x * 8, 8 * THREADS) : 0.f;
            __syncthreads();  // (the sums of the pair before have been read)
            if (lane == 0) sums[warp] = dot;
            __syncthreads();
            dot = 0.f;
#pragma unroll
            for (int v = 0; v < WARPS; ++v) dot += sums[v];
            if (threadIdx.x == 0) p.dw[first] = dot;
        }
    }
}

int failed(cudaError_t e, const char* what) {
    return host_fail(MXFP8_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Launches `kernel` so that its start overlaps the end of the kernel before it
// (each kernel waits for that one before its first access).
template <class... Par, class... Arg>
int launch(void (*kernel)(Par...), int64_t ctas, const TokenArgs& a, const char* what, const Arg&... arg) {
    if (ctas == 0) return MXFP8_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < (1 << 22) ? ctas : (1 << 22)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, arg...);
    return e == cudaSuccess ? MXFP8_OK : failed(e, what);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Columns of a unit: as many as leave units enough for the warps to even out. A
// unit's start is a chain of two loads: 256 columns everywhere took 402 us for the
// sum on the 671B rank, whole tokens everywhere 10.6 us for its 8 tokens; here 149
// and 2.1. Tokens of few choices are alike and need fewer units to even out (10539
// tokens of 2728 columns, one row each: 33 us with 40000 units, 20.6 with 20000; two
// rows 37.7 / 34.9; 30000 of 4096 columns, two rows 112 / 114). With more choices it
// depends: three rows of 2048 columns 49.1 / 45.1, of 4096 149 / 151, the sum on the 671B
// rank 149 / 158.
int unit_columns(const TokenArgs& a) {
    int seg = 256;
    while (seg < a.H && a.T * ceil_div(a.H, 2 * seg) >= (seg == 256 || a.top_k <= 2 ? 20000 : 40000)) seg *= 2;
    return seg;
}

// Quantising wants longer units, 2048 columns (one trip of its loop) where that
// leaves some 5000 (2048 tokens on the 671B rank: 512 columns 22.6 us, whole tokens
// 15.1, here 10.4).
int unit_columns_mxfp8(const TokenArgs& a) {
    int seg = 512;
    while (seg < a.H && a.T * ceil_div(a.H, 2 * seg) >= 5000) seg *= 2;
    return seg;
}

RowPar row_par(const TokenArgs& a, int seg) {
    RowPar p{};
    p.T = a.T; p.rows = a.rows; p.H = a.H; p.k = a.top_k; p.seg = seg; p.segs = (a.H + seg - 1) / seg;
    p.slot = a.slot; p.src = a.src; p.tok_in = a.tok_in; p.sorted_in = a.sorted_in;
    p.tok_out = a.tok_out; p.sorted_out = a.sorted_out; p.q = a.q; p.s = a.s; p.w = a.weights; p.dw = a.dweights;
    p.status = a.status;
    p.words = a.q && a.H % 128 == 0 && (reinterpret_cast<uintptr_t>(a.s) & 3) == 0;
    // padding: a row for each group of warps while that gives few CTAs, else up to 32
    // (always 1: dispatch on the 671B rank 137 us against 108; always 32: 512 tokens 12.8 / 5.2)
    const int groups = WARPS / pad_parts(a.q ? a.H : 2 * a.H);
    p.pad = 1;
    while (p.pad < 32 && ceil_div(a.rows, groups * p.pad) > PAD_CTAS) p.pad *= 2;
    p.pad_ctas = static_cast<int>(ceil_div(a.rows, groups * p.pad));
    return p;
}

}  // namespace

// The plan kernels' attributes on the device that is current, set once, and the
// CTAs of a cluster there: 16 where a cluster of 16 full SMs has room, else the
// portable 8.
static cudaError_t plan_device(int dev, int* ctas) {
    static std::atomic<int> known[64];
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        for (const void* f : {reinterpret_cast<const void*>(token_plan_kernel<int32_t>), reinterpret_cast<const void*>(token_plan_kernel<int64_t>)}) {
            cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, PLAN_SMEM);
            if (e != cudaSuccess) return e;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(PLAN_MAX_CTAS);
        cfg.blockDim = dim3(1024);
        cfg.dynamicSmemBytes = PLAN_SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = PLAN_MAX_CTAS;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, token_plan_kernel<int64_t>, &cfg);
        if (e != cudaSuccess) return e;
        n = clusters > 0 ? PLAN_MAX_CTAS : 8;
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *ctas = n;
    return cudaSuccess;
}

int launch_token_plan(const TokenPlanArgs& a) {
    PlanPar p{a.ids, static_cast<int>(a.pairs), a.first, a.local, a.align, static_cast<int>(a.rows), 0, 1, 1, a.offs, a.slot, a.src, a.status};
    while ((1 << (3 * p.groups)) < a.local) ++p.groups;
    auto kernel = a.id64 ? token_plan_kernel<int64_t> : token_plan_kernel<int32_t>;
    // (few of either: 8 warps start sooner. 2 pairs, 4 experts: 3.4 us, 4.3 with 32; 64 pairs, 32 experts 4.3 / 4.7;
    // with more experts 32 clear and scan faster: 48 pairs, 64 experts 5.5 / 5.2; 64 pairs, 256 experts 8.3 / 6.7)
    int warps = a.pairs <= 64 && a.local <= 64 ? 8 : 32;
    const auto bytes = [&] { return (warps + 7) * static_cast<size_t>(a.local) * 4 + warps * RUN * 6; };
    while (bytes() > PLAN_SMEM) warps /= 2;
    cudaError_t e = cudaSuccess;
    if (a.pairs > PLAN_ONE_CTA || bytes() > 48 * 1024) {
        e = plan_device(a.dev, &p.C);
        if (e != cudaSuccess) return failed(e, "token plan: kernel attributes");
        if (a.pairs <= PLAN_ONE_CTA) p.C = 1;
        p.Q = a.pairs > PLAN_ONE_CLUSTER ? 4 : 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.C * p.Q);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = bytes();
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const PlanPar>(p));
    return e == cudaSuccess ? MXFP8_OK : failed(e, "token plan kernel");
}

int launch_token_dispatch(const TokenArgs& a) {
    const RowPar p = row_par(a, a.q ? unit_columns_mxfp8(a) : unit_columns(a));
    return launch(!a.q ? dispatch_kernel : a.H <= 512 ? dispatch_mxfp8_kernel<1> : dispatch_mxfp8_kernel<4>, ceil_div(a.T * p.segs, WARPS) + p.pad_ctas, a, "dispatch kernel", p);
}

int launch_token_combine(const TokenArgs& a) {
    const RowPar p = row_par(a, unit_columns(a));
    return launch(a.weights ? combine_kernel<true> : combine_kernel<false>, ceil_div(a.T * p.segs, WARPS), a, "combine kernel", p);
}

int launch_token_combine_grad(const TokenArgs& a) {
    RowPar p = row_par(a, a.H);
    const int64_t pairs = a.T * a.top_k, sms = a.num_sms;
    const auto go = [&](auto kernel, int per) { return launch(kernel, ceil_div(pairs, per) + p.pad_ctas, a, "combine gradient kernel", p); };
    if (pairs <= 2 * sms) return go(combine_grad_kernel<TEAM, 4>, 1);
    if (a.H <= 2048 || 2 * a.rows >= pairs || pairs <= PAIRS * 4 * sms) {
        p.each = 1;
        while (p.each < 32 && 2 * p.each * a.H <= 8192 && pairs >= 16384 * static_cast<int64_t>(p.each)) p.each *= 2;
        return go(a.H <= 256 ? combine_grad_kernel<WARP, 1> : combine_grad_kernel<WARP, 4>, WARPS * p.each);
    }
    return go(combine_grad_kernel<LIST, 8>, PAIRS);
}

}  // namespace mxw
