// A whole mixture-of-experts layer for a few tokens (mxfp8_moe_layer): router,
// choice of experts, gated MLPs on MXFP8 weights, weighted sum.
//
// The layer reads each chosen expert's weights once and does little with them
// (2 x tokens multiply-adds per weight byte), so it is bound by HBM: the design
// keeps one stream of weights running through every SM from the routing to the
// last product. The weights go straight from HBM to the tensor cores: TMA puts
// E4M3 tiles of 128 rows x 128 columns into shared memory and the block-scaled
// tcgen05 MMA multiplies them with their E8M0 scales, so no thread touches a
// weight. The tokens are the N side of the MMA (16 .. 256 columns). The
// activations keep their precision as two E4M3 pieces per value, each 32-block
// of a piece with its own power-of-two scale (two columns per token): a bf16
// value has 8 significant bits and each piece holds 4, so x is represented
// exactly down to 2^-17 of its block's largest value, and the fp32 inner
// activations h to about 9 bits.
//
// Two kernels per call:
//   moe_logits  : router logits (partial sums over slices of H), x as pieces,
//                 counters to zero.
//   moe_experts : persistent, one CTA per SM (a programmatic dependent of
//                 moe_logits). Chooses the experts, then works off
//                 one queue of tiles: up/gate tiles (64 gate and the same 64 up
//                 rows, h = silu(g) u on drain), then down tiles (128 rows), by
//                 expert. A CTA takes the next tile when its weight producer has
//                 finished with the last one, so that SMs with a slower path to
//                 memory take fewer; the producer runs ahead of the products (the
//                 weights of the first down tiles arrive while h is finished).
//                 Where the tiles are fewer than the SMs, each is cut into parts
//                 along the contraction, summed in order by the part that ends
//                 last. No atomics on data: bit-reproducible whoever computes
//                 what. Last, when all tiles are done, the weighted sum over
//                 each token's experts.
//
// Measured, bytes of the chosen experts' weights over the whole call's time:
// 64 experts of H = 2048, I = 1408, top 6, all here: 64 tokens 571 MB in 112 us
// (5.1 TB/s; DRAM reads are exactly the weights), 8 tokens 312 MB in 66 us, 1
// token 53.5 MB in 33 us (28 on one box); 32 of 256 experts here, H = 7168, I = 2048,
// top 8: 128 tokens 1.44 GB in 220 to 243 us. A fixed chain of 15 to 16 us
// stands beside the stream: launches, routing (4 us at one token, 9 at 128),
// lists, the hand-over of h, the last sum. Small layers are that chain alone
// (H = 256: 15 us on the GPU, 17 with the host's launches).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include <atomic>

#include "mxw_experts.h"
#include "mxw_internal.h"
#include "mxw_ptx_single.cuh"
#include "../../include/mxfp8_experts.h"

namespace mxw {
namespace {

constexpr int PIECES = 2;            // E4M3 pieces per activation
constexpr int STEP = 128;            // columns of a K-step
constexpr int TILE = 128;            // weight rows of a tile
constexpr int A_BYTES = TILE * STEP;
constexpr int MAX_ST = 12;           // pipeline stages
constexpr int THREADS = 288;         // warps: 0 weight producer, 1 MMA issuer, 2, 3, 8 loaders, 4 .. 7 epilogue
constexpr int LOADERS = 3;
constexpr int BLOCK = 2;             // K-steps that a loader takes at a time (rings of 6 stages or more; else 1)
constexpr int SMEM = 221184;         // leaves room beside a moe_logits<1, 2> block: moe_experts' CTAs start under it (all of
                                     // it instead: 92.4 -> 95.2 us for 16 tokens of the 671B rank, equal from 64 tokens on)
constexpr uint32_t TMEM_ALL = 512;
// the largest lists, masks and stages still leave a ring of a stage per loader (launch_moe lays them out)
static_assert((SMEM - 1024 - (512 + MXFP8_MOE_MAX_TOKENS * MXFP8_MOE_MAX_TOPK * 10 + MXFP8_MOE_MAX_EXPERTS * 24 + 256 + 2 * 8 * TILE * 4 +
                              LOADERS * 1024 + 1024)) / (A_BYTES + PIECES * MXFP8_MOE_MAX_TOKENS * STEP + 512 * 3) >= LOADERS,
              "pipeline stages");
// counters: tokens claimed and chosen for, units claimed, down units done
constexpr int C_CLAIM = 0, C_CHOSEN = 1, C_QUEUE = 2, C_DONE = 3, C_H = 4;
constexpr int MAX_PARTS = 8;         // pieces of a tile's contraction
constexpr int NQ = 4;                // queue entries in flight in a CTA
constexpr int EPI_BAR = 1;           // named barriers: the epilogue warps; the lists are made; the pairs are placed
constexpr int LIST_BAR = 2, PLACE_BAR = 3;
// kind::mxf8f6f4, E4M3 x E4M3, both K-major, E8M0 scales, M = 128
constexpr uint32_t IDESC = (1u << 23) | (static_cast<uint32_t>(TILE >> 4) << 24);

struct Params {
    const uint16_t *x, *router;
    const float* bias;
    const uint8_t *s13, *s2;
    int T, experts, first, local, H, I, top_k, score, renormalize;
    float scale;
    uint16_t* out;
    int32_t* user_ids;
    float* user_weights;
    // scratch
    unsigned int* counters;  // C_* below; then h tiles done per chosen expert; then parts done per up/gate tile
    float* logits;           // [ksplit][T][experts]
    int32_t* ids;            // [T][top_k]
    float* weights;
    uint8_t *xq, *sx;        // [T][2][Hp], [T][2][Hp / 32]
    uint8_t *hq, *sh;        // [slots][2][Ip], [slots][2][sh_stride]
    float* y;                // [slots][Hp]
    float *part_up, *part_down;  // [unit][T][128]
    int Hp, Ip, sh_stride, ksplit, slots, n_counters;
    int up_tiles, down_tiles, up_steps, down_steps;
    uint32_t off_lists, off_mask, off_epi, off_rows, off_ring;
    unsigned long long wait_ns;
    int* status;
    int stall;               // test hook: over-declare the first stage's bytes so that its wait runs out
};

__device__ __forceinline__ float bf16_f(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// E8M0 scale of a block whose largest magnitude has the bits `amax`: the
// smallest 2^e with amax <= 448 * 2^e (448 = 1.75 * 2^8); 255 for NaN / infinity.
__device__ __forceinline__ uint32_t block_scale(uint32_t amax) {
    if (amax >= 0x7F800000u) return 255u;
    const int s = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(s > 0 ? s : 0);
}

// One warp, one 32-block: lane l's value v as two E4M3 pieces (returned in the
// low and second byte) and the pieces' scales s0, s1 (the same in all lanes).
__device__ __forceinline__ uint32_t split_block(float v, uint32_t& s0, uint32_t& s1) {
    s0 = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
    if (s0 == 255u) {
        s1 = 255u;
        return 0x7F7Fu;
    }
    const float inv0 = __uint_as_float((254u - s0) << 23);
    const __nv_fp8_storage_t q0 = __nv_cvt_float_to_fp8(v * inv0, __NV_SATFINITE, __NV_E4M3);
    const float scale0 = __uint_as_float(s0 ? s0 << 23 : 0x400000u);
    const float r = v - __half2float(__half(__nv_cvt_fp8_to_halfraw(q0, __NV_E4M3))) * scale0;
    s1 = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(r) & 0x7FFFFFFFu));
    const float inv1 = __uint_as_float((254u - s1) << 23);
    const __nv_fp8_storage_t q1 = __nv_cvt_float_to_fp8(r * inv1, __NV_SATFINITE, __NV_E4M3);
    return static_cast<uint32_t>(q0) | (static_cast<uint32_t>(q1) << 8);
}

// ============================================================== logits

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 32-blocks of a row at a time: lane l holds columns 4 l .. 4 l + 3 of the
// 128, eight lanes a block; v becomes the pieces' bytes, s0 and s1 their scales.
__device__ __forceinline__ void split_rows(const Params& p, int first, int stride) {
    const int lane = threadIdx.x & 31, per = p.Hp / STEP;
    for (int i = first; i < p.T * per; i += stride) {
        const int t = i / per, b = i - t * per, h = b * STEP + 4 * lane;
        uint2 raw = make_uint2(0, 0);
        if (h < p.H) raw = __ldg(reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(t) * p.H + h));
        float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u), __uint_as_float(raw.y << 16),
                      __uint_as_float(raw.y & 0xFFFF0000u)};
        uint32_t s[PIECES];
#pragma unroll
        for (int pc = 0; pc < PIECES; ++pc) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            s[pc] = block_scale(m);
            if (pc && s[0] == 255u) s[pc] = 255u;
            const float inv = __uint_as_float((254u - min(s[pc], 254u)) << 23), up = __uint_as_float(s[pc] ? s[pc] << 23 : 0x400000u);
            uint32_t q = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_fp8_storage_t f = __nv_cvt_float_to_fp8(v[j] * inv, __NV_SATFINITE, __NV_E4M3);
                q |= static_cast<uint32_t>(f) << (8 * j);
                v[j] -= __half2float(__half(__nv_cvt_fp8_to_halfraw(f, __NV_E4M3))) * up;
            }
            *reinterpret_cast<uint32_t*>(p.xq + (static_cast<size_t>(t) * PIECES + pc) * p.Hp + h) = s[pc] == 255u ? 0x7F7F7F7Fu : q;
        }
        if ((lane & 7) == 0) {
#pragma unroll
            for (int pc = 0; pc < PIECES; ++pc)
                p.sx[(static_cast<size_t>(t) * PIECES + pc) * (p.Hp / 32) + 4 * b + (lane >> 3)] = static_cast<uint8_t>(s[pc]);
        }
    }
}

// Block (expert group, token tile, H slice): 16 MF tokens x 8 NF experts, each
// of 8 warps a share of the slice, joined in shared memory in warp order. A
// thread's 16 bytes hold eight consecutive values of a row: the same
// assignment of columns to the MMA's K on both sides, so the sum is the dot
// product whatever the order. The blocks after those split x into pieces and
// zero the counters. Latency-bound: 6.7 us at 64 tokens, 64 experts, H = 2048
// with a cold L2.
template <int MF, int NF>
__global__ void __launch_bounds__(256) moe_logits(const Params p) {
    __shared__ float red[8][16 * MF][8 * NF];
    griddep_launch_dependents();
    griddep_wait();  // x may come from the kernel before, and a call before may still use the scratch
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tg = lane & 3;
    const int ge = (p.experts + 8 * NF - 1) / (8 * NF), gt = (p.T + 16 * MF - 1) / (16 * MF);
    if (static_cast<int>(blockIdx.x) >= ge * gt * p.ksplit) {
        const int b = blockIdx.x - ge * gt * p.ksplit, nb = gridDim.x - ge * gt * p.ksplit;
        split_rows(p, b * 8 + warp, nb * 8);
        for (int i = b * 256 + threadIdx.x; i < p.n_counters; i += nb * 256) p.counters[i] = 0;
        return;
    }
    const int bz = blockIdx.x / (ge * gt), by = (blockIdx.x - bz * ge * gt) / ge, bx = blockIdx.x - (bz * gt + by) * ge;
    const int e0 = bx * 8 * NF, t0 = by * 16 * MF;
    const long long chunks = p.H / 32, nw = 8LL * p.ksplit, wi = bz * 8 + warp;
    const int c0 = static_cast<int>(chunks * wi / nw), c1 = static_cast<int>(chunks * (wi + 1) / nw);
    float acc[MF][NF][4] = {};
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
        uint4 a[MF][2], b[NF];
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = t0 + 16 * i + 8 * h + g;
                a[i][h] = t < p.T ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.H + 32 * c + 8 * tg))
                                  : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int e = e0 + 8 * j + g;
            b[j] = e < p.experts ? __ldg(reinterpret_cast<const uint4*>(p.router + static_cast<size_t>(e) * p.H + 32 * c + 8 * tg))
                                 : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                mma_bf16(acc[i][j], a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, b[j].x, b[j].y);
                mma_bf16(acc[i][j], a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, b[j].z, b[j].w);
            }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[warp][16 * i + g + 8 * (r >> 1)][8 * j + 2 * tg + (r & 1)] = acc[i][j][r];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * MF * 8 * NF; o += 256) {
        const int t = t0 + o / (8 * NF), e = e0 + o % (8 * NF);
        if (t < p.T && e < p.experts) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) s += red[w][o / (8 * NF)][o % (8 * NF)];
            p.logits[(static_cast<size_t>(bz) * p.T + t) * p.experts + e] = s;
        }
    }
}

// ============================================================== routing

// Order-preserving map of a float to an unsigned integer; NaN below everything, 0 is free for "taken".
__device__ __forceinline__ uint32_t sort_key(float v) {
    if (v != v) return 1u;
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 -> +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The CTA: logits of n tokens from t on (sums of the slices, in order) into shared memory.
__device__ __forceinline__ void gather_logits(const Params& p, int t, int n, float* score) {
    const float* src = p.logits + static_cast<size_t>(t) * p.experts;
    const size_t slice = static_cast<size_t>(p.T) * p.experts;
#pragma unroll 2
    for (int i = threadIdx.x; i < n * p.experts; i += THREADS) {
        float v[8], s = 0.f;  // (at most 8 slices: all loads in flight together)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < p.ksplit ? __ldcg(src + k * slice + i) : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
        score[i] = s;
    }
}

struct Choice {
    int id;        // lane k < top_k: the k-th chosen expert and its weight
    float weight;
};

// One warp: the choice for one token from its logits (score: [experts], shared; key: [experts], shared scratch).
// Lane l holds experts l, l + 32, ... (Loops, not registers: unrolled for eight experts a lane this took
// 13 us longer, all of it misses of the instruction cache.)
__device__ __noinline__ Choice choose(const Params& p, float* score, uint32_t* key) {
    const int lane = threadIdx.x & 31;
    const unsigned full = 0xffffffffu;
    float m = -CUDART_INF_F;
    for (int e = lane; e < p.experts; e += 32) m = fmaxf(m, score[e]);
    if (p.score == MXFP8_SCORE_SOFTMAX) {
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(full, m, d));
        float sum = 0.f;
        for (int e = lane; e < p.experts; e += 32) sum += (score[e] = expf(score[e] - m));
        sum = warp_sum(sum);
        for (int e = lane; e < p.experts; e += 32) score[e] /= sum;
    } else {
        for (int e = lane; e < p.experts; e += 32) score[e] = 1.f / (1.f + expf(-score[e]));
    }
    uint32_t best = 0;
    int at = 0x7fffffff;
    auto scan = [&]() {
        best = 0;
        at = 0x7fffffff;
        for (int e = lane; e < p.experts; e += 32) {
            const uint32_t v = key[e];
            if (v > best) { best = v; at = e; }
        }
    };
    for (int e = lane; e < p.experts; e += 32) key[e] = sort_key(score[e] + (p.bias ? p.bias[e] : 0.f));
    scan();
    float total = 0.f, mine = 0.f;
    int my_id = 0;
    __syncwarp();
    for (int k = 0; k < p.top_k; ++k) {
        const uint32_t top = __reduce_max_sync(full, best);
        const int e = static_cast<int>(__reduce_min_sync(full, best == top ? static_cast<uint32_t>(at) : 0x7fffffffu));
        const float s = score[e];
        total += s;
        if (lane == k) { mine = s; my_id = e; }
        if ((e & 31) == lane) {
            key[e] = 0;
            scan();
        }
    }
    __syncwarp();
    return Choice{my_id, (p.renormalize ? mine / total : mine) * p.scale};
}

// ============================================================== experts

// Bounded waits. The polling loops are kept out of line: a CTA's first pass
// through its code misses the instruction cache all along, so the roles' code
// is kept short.
__device__ __noinline__ bool wait_bar_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long ns,
                                           int* status) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (mbar_try_wait_suspend(bar, parity, 20000)) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > ns) {
            *abort_flag = 1;
            atomicOr(status, MXFP8_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long ns,
                                         int* status) {
    return mbar_try_wait(bar, parity) || wait_bar_slow(bar, parity, abort_flag, ns, status);
}

__device__ __noinline__ void drain_bar(uint32_t bar, uint32_t parity, unsigned long long ns, int* status) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > ns) {
            atomicOr(status, MXFP8_DEV_WAIT_TIMEOUT);
            return;
        }
}

// Bounded wait until *p >= target: an acquire each time, no pause (polled relaxed
// with one acquire at the end: 16B, 64 tokens 119.7 -> 121.5 us).
__device__ __noinline__ bool wait_count(const unsigned int* p, unsigned int target, volatile int* abort_flag,
                                           unsigned long long ns, int* status) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (ld_acquire_gpu(p) >= target) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > ns) {
            *abort_flag = 1;
            atomicOr(status, MXFP8_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

// One warp: h = silu(gate) up of 32 inner rows of one token, as two pieces and their scales.
__device__ __noinline__ void store_h(const Params& p, int slot, int i0, float gate, float up) {
    const int lane = threadIdx.x & 31;
    const float h = gate / (1.f + expf(-gate)) * up;
    uint32_t s0, s1;
    const uint32_t pc = split_block(h, s0, s1);
    uint8_t* d = p.hq + static_cast<size_t>(slot) * PIECES * p.Ip + i0 + lane;
    d[0] = static_cast<uint8_t>(pc);
    d[p.Ip] = static_cast<uint8_t>(pc >> 8);
    if (lane < PIECES)
        p.sh[(static_cast<size_t>(slot) * PIECES + lane) * p.sh_stride + (i0 >> 5)] = static_cast<uint8_t>(lane ? s1 : s0);
}

// Per-CTA lists in shared memory.
struct Lists {
    float* wts;          // [slots] weight of entry (token, k)
    uint16_t* eid;       // [slots] local expert of the entry, 0xffff: none
    uint16_t* slot_of;   // [slots] position of the entry among the local pairs sorted by expert
    uint16_t* entry_of;  // [slots] entry of a position
    uint16_t* act_of;    // [local] chosen-expert index of a local expert
    uint16_t* count;     // [chosen] tokens of a chosen expert
    uint16_t* act;       // [local] local expert of a chosen-expert index
    uint16_t* off;       // [local] first position of a chosen expert
    int* info;           // chosen experts, most tokens of one
};

// Parts into which a phase's tiles are cut along the contraction: enough to
// give every CTA one, at least four K-steps each. Handing a partial sum over
// costs several K-steps' time, so tiles that outnumber half the CTAs stay whole.
__device__ __forceinline__ int parts_of(int tiles, int steps, int G) {
    return 2 * tiles > G ? 1 : max(1, min(min(G / max(tiles, 1), steps / 4), MAX_PARTS));
}

// A unit of the queue: K-steps [k0, k1) of a tile.
struct Seg {
    int phase, tile, a, rt, part, parts, k0, k1, steps;
};

template <bool PARTS>
struct Queue {
    int nact, up_parts, down_parts, up_units, units;
    const Params& p;

    __device__ __forceinline__ Queue(const Params& p_, int G, int nact_) : nact(nact_), p(p_) {
        up_parts = PARTS ? parts_of(nact * p.up_tiles, p.up_steps, G) : 1;
        down_parts = PARTS ? parts_of(nact * p.down_tiles, p.down_steps, G) : 1;
        up_units = nact * p.up_tiles * up_parts;
        units = up_units + nact * p.down_tiles * down_parts;
    }

    __device__ __forceinline__ Seg get(int u) const {
        Seg g;
        g.phase = u >= up_units;
        const int v = g.phase ? u - up_units : u, tiles = g.phase ? p.down_tiles : p.up_tiles;
        g.parts = PARTS ? (g.phase ? down_parts : up_parts) : 1;
        g.steps = g.phase ? p.down_steps : p.up_steps;
        g.tile = v;
        g.part = g.k0 = 0;
        g.k1 = g.steps;
        if (PARTS && g.parts > 1) {
            g.tile = v / g.parts;
            g.part = v - g.tile * g.parts;
            g.k0 = g.steps * g.part / g.parts;
            g.k1 = g.steps * (g.part + 1) / g.parts;
        }
        g.a = static_cast<uint32_t>(g.tile) / static_cast<uint32_t>(tiles);
        g.rt = g.tile - g.a * tiles;
        return g;
    }
};

// PARTS: tiles may be cut along the contraction (see cuts()).
template <bool PARTS>
__global__ void __launch_bounds__(THREADS, 1)
    moe_experts(const __grid_constant__ CUtensorMap tm13, const __grid_constant__ CUtensorMap tm2, const Params p) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x, cta = blockIdx.x;

    const uint32_t bar_w = sbase, bar_act = bar_w + 8 * MAX_ST, bar_empty = bar_act + 8 * MAX_ST,
                   bar_tfull = bar_empty + 8 * MAX_ST, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
    const uint32_t bar_qf = bar_drain + 8, bar_qe = bar_qf + 8 * NQ;
    int* flags = reinterpret_cast<int*>(smem + 8 * (3 * MAX_ST + 5 + 2 * NQ));  // abort, TMEM base, epilogue unit x2, chosen, most, wait ok, token, last part, queue
    volatile int* abort_flag = flags;
    Lists L;
    L.wts = reinterpret_cast<float*>(smem + p.off_lists);
    L.eid = reinterpret_cast<uint16_t*>(L.wts + p.slots);
    L.slot_of = L.eid + p.slots;
    L.entry_of = L.slot_of + p.slots;
    L.act_of = L.entry_of + p.slots;
    L.count = L.act_of + p.local;
    L.act = L.count + p.local;
    L.off = L.act + p.local;
    L.info = flags + 4;

    if (threadIdx.x == 0) {
        for (int s = 0; s < MAX_ST; ++s) {
            mbar_init(bar_w + 8 * s, 1);      // weight producer (with its bytes)
            mbar_init(bar_act + 8 * s, 1);    // the K-step's loader
            mbar_init(bar_empty + 8 * s, 1);  // the MMAs' commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 4);
        }
        mbar_init(bar_drain, 1);
        for (int i = 0; i < NQ; ++i) {
            mbar_init(bar_qf + 8 * i, 1);            // weight producer: the entry is written
            mbar_init(bar_qe + 8 * i, 2 + LOADERS);  // MMA issuer, loaders, epilogue have read it
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm13);
        tma_prefetch_desc(&tm2);
    }
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + p.off_mask);  // [local][4] tokens of a local expert
    for (int i = threadIdx.x; i < 4 * p.local; i += THREADS) mask[i] = 0;
    if (warp == 1) {
        tmem_alloc_single(smem_u32(flags + 1), TMEM_ALL);
        tmem_relinquish_single();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(flags[1]);
    griddep_launch_dependents();  // (what follows in the stream may get ready; it waits for this grid's end)
    griddep_wait();               // logits, pieces of x, zeroed counters

    // ---- routing. Up to 8 tokens: every CTA chooses for all of them (one warp
    // each). More: CTAs claim a token each and wait until all are chosen for.
    // (Waits are only ever for work that a running CTA has claimed, here and
    // below: the kernel ends however few of its CTAs are resident at a time.)
    unsigned int first_unit = 0;
    if (threadIdx.x == 0) first_unit = atomicAdd(p.counters + C_QUEUE, 1u);
    if (warp == 0) first_unit = __shfl_sync(0xffffffffu, first_unit, 0);
    {
        // entry (token, k) of the routing: its expert if it lives here, its weight,
        // and the token's bit in the expert's mask. Bit counts are then the experts'
        // sizes and the pairs' ranks, whatever the order in which the bits were set.
        auto enter = [&](int t, int k, int e, float w) {
            const int i = t * p.top_k + k;
            const bool here = e >= p.first && e < p.first + p.local;
            L.eid[i] = here ? static_cast<uint16_t>(e - p.first) : 0xffff;
            L.wts[i] = w;
            if (here) atomicOr(mask + 4 * (e - p.first) + (t >> 5), 1u << (t & 31));
        };
        float* scores = reinterpret_cast<float*>(smem + p.off_ring);  // [tokens in hand][experts], then as many keys
        auto tell_user = [&](int t, const Choice& c) {
            if (p.user_ids) p.user_ids[t * p.top_k + lane] = c.id;
            if (p.user_weights) p.user_weights[t * p.top_k + lane] = c.weight;
        };
        if (p.T <= 8) {
            gather_logits(p, 0, p.T, scores);
            __syncthreads();
            if (warp < p.T) {
                const Choice c = choose(p, scores + warp * p.experts, reinterpret_cast<uint32_t*>(scores) + (p.T + warp) * p.experts);
                if (lane < p.top_k) {
                    enter(warp, lane, c.id, c.weight);
                    if (cta == 0) tell_user(warp, c);
                }
            }
        } else {
            for (;;) {
                if (threadIdx.x == 0) flags[7] = static_cast<int>(atomicAdd(p.counters + C_CLAIM, 1u));
                __syncthreads();
                const int t = flags[7];
                if (t >= p.T) break;
                gather_logits(p, t, 1, scores);
                __syncthreads();
                if (warp == 0) {
                    const Choice c = choose(p, scores, reinterpret_cast<uint32_t*>(scores) + p.experts);
                    if (lane < p.top_k) {
                        p.ids[t * p.top_k + lane] = c.id;
                        p.weights[t * p.top_k + lane] = c.weight;
                        tell_user(t, c);
                    }
                    __syncwarp();
                    if (lane == 0) red_release_gpu_add(p.counters + C_CHOSEN, 1);
                }
            }
            if (threadIdx.x == 0) flags[6] = wait_count(p.counters + C_CHOSEN, p.T, abort_flag, p.wait_ns, p.status) ? 1 : 0;
            __syncthreads();
            if (flags[6])
                for (int i = threadIdx.x; i < p.slots; i += THREADS) {
                    const int t = i / p.top_k;
                    enter(t, i - t * p.top_k, __ldcg(p.ids + i), __ldcg(p.weights + i));
                }
        }
        fence_proxy_async_shared();  // the ring's space held the scores
        __syncthreads();
        // ---- the (token, expert) pairs sorted by expert, in token order. Warp 0
        // lists the chosen experts and goes on to load their weights; the others
        // place the pairs.
        if (warp == 0) {
            int chosen = 0, first = 0, most = 0;
            for (int b = 0; b < p.local; b += 32) {
                const int e = b + lane;
                int n = 0;
                if (e < p.local) {
                    const uint4 m = *reinterpret_cast<const uint4*>(mask + 4 * e);
                    n = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
                }
                const unsigned have = __ballot_sync(0xffffffffu, n > 0);
                int incl = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += v;
                }
                if (n > 0) {
                    const int a = chosen + __popc(have & ((1u << lane) - 1));
                    L.act[a] = static_cast<uint16_t>(e);
                    L.act_of[e] = static_cast<uint16_t>(a);
                    L.off[a] = static_cast<uint16_t>(first + incl - n);
                    L.count[a] = static_cast<uint16_t>(n);
                }
                chosen += __popc(have);
                first += __shfl_sync(0xffffffffu, incl, 31);
                most = max(most, __reduce_max_sync(0xffffffffu, n));
            }
            if (lane == 0) {
                L.info[0] = chosen;
                L.info[1] = most;
            }
            __syncwarp();
            named_bar_arrive(LIST_BAR, THREADS);
        } else {
            named_bar_sync(LIST_BAR, THREADS);
            for (int i = threadIdx.x - 32; i < p.slots; i += THREADS - 32)
                if (p.T <= 8 || flags[6]) {
                    const int e = L.eid[i];
                    if (e == 0xffff) continue;
                    const int t = i / p.top_k;
                    const uint32_t* m = mask + 4 * e;
                    int s = L.off[L.act_of[e]] + __popc(m[t >> 5] & ((1u << (t & 31)) - 1));
                    for (int w = 0; w < (t >> 5); ++w) s += __popc(m[w]);
                    L.slot_of[i] = static_cast<uint16_t>(s);
                    L.entry_of[s] = static_cast<uint16_t>(i);
                }
            named_bar_sync(PLACE_BAR, THREADS - 32);
        }
    }
    const int nact = L.info[0];
    // MMA width for the expert with the most tokens; ring of K-step stages
    const int nmax = max(16, (PIECES * L.info[1] + 15) & ~15);
    const uint32_t nblk = (nmax + 127) / 128;
    const uint32_t sf_stage = 512 * (1 + nblk);
    const uint32_t ab_stage = A_BYTES + nmax * STEP;
    const int S = min(MAX_ST, static_cast<int>((SMEM - 1024 - p.off_ring) / (ab_stage + sf_stage)));
    const uint32_t ring = sbase + p.off_ring, sf_ring = ring + S * ab_stage;
    const uint32_t sf_cols = 4 * (1 + nblk);
    const int nbuf = 2 * nmax + S * static_cast<int>(sf_cols) <= 512 ? 2 : 1;  // accumulators
    const uint32_t sf_tmem = tmem + nbuf * nmax;
    const Queue<PARTS> queue(p, G, nact);
    volatile int* entry = flags + 9;  // [NQ] units; -1: no more

    // Reader's side of the queue: the next entry (-1 at the end), or -2 after an abort.
    auto read_entry = [&](int i) {
        if (!wait_bar(bar_qf + 8 * (i % NQ), (i / NQ) & 1, abort_flag, p.wait_ns, p.status)) return -2;
        const int u = entry[i % NQ];
        mbar_arrive(bar_qe + 8 * (i % NQ));
        return u;
    };

    if (warp == 0) {
        // ------------------------------------------------ weight producer
        if (elect_one()) {
            const uint64_t once = l2_evict_first();  // weights leave L2 first: it keeps the code, x, h and partial sums
            int c = 0, st = 0, put = 0;
            uint32_t ph = 1;
            bool ok = true;
            // units come from the counter shared by all; each is published while the
            // unit before is copied
            auto publish = [&](int u) {
                if (!wait_bar(bar_qe + 8 * (put % NQ), ((put / NQ) & 1) ^ 1, abort_flag, p.wait_ns, p.status)) return false;
                entry[put % NQ] = u < queue.units ? u : -1;
                mbar_arrive(bar_qf + 8 * (put % NQ));
                ++put;
                return true;
            };
            int u = static_cast<int>(first_unit);
            ok = publish(u);
            while (ok && u < queue.units) {
                const int un = static_cast<int>(atomicAdd(p.counters + C_QUEUE, 1u));
                const Seg g = queue.get(u);
                const int e = L.act[g.a];
                const int kp = min(g.k0 + 3, g.k1 - 1);  // (the counter's answer is back by then)
                for (int k = g.k0; ok && k < g.k1; ++k) {
                    if (k == kp) ok = publish(un);
                    if (!ok) break;
                    ok = wait_bar(bar_empty + 8 * st, ph, abort_flag, p.wait_ns, p.status);
                    if (!ok) break;
                    const uint32_t dst = ring + st * ab_stage, bar = bar_w + 8 * st;
                    mbar_arrive_expect_tx(bar, A_BYTES + (p.stall && c == 0 ? 16 : 0));
                    if (g.phase) tma_load_3d(dst, &tm2, bar, k * STEP, g.rt * TILE, e, once);
                    else tma_load_4d(dst, &tm13, bar, k * STEP, g.rt * (TILE / 2), 0, e, once);
                    ++c;
                    if (++st == S) { st = 0; ph ^= 1; }
                }
                u = un;
            }
            if (!ok || *abort_flag)  // every copy in flight lands before the CTA exits
                for (int d = 1; d <= min(c, S); ++d) drain_bar(bar_w + 8 * ((c - d) % S), ((c - d) / S) & 1, p.wait_ns, p.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // One elected thread runs the whole loop: with a fresh election for each
        // instruction, and descriptors rebuilt for it, a K-step took 820 cycles to
        // issue (measured); this form takes 340, below the 700 in which a K-step's
        // weights arrive.
        if (elect_one()) {
            int st = 0, tile = 0;
            uint32_t ph = 0;
            bool ok = true;
            while (ok) {
                const int u = read_entry(tile);
                if (u < 0) break;
                const Seg g = queue.get(u);
                const int K = g.phase ? p.I : p.H;
                const int n = max(16, (PIECES * L.count[g.a] + 15) & ~15);
                const uint32_t idesc = IDESC | (static_cast<uint32_t>(n >> 3) << 17);
                const int buf = nbuf == 2 ? tile & 1 : 0, use = nbuf == 2 ? tile >> 1 : tile;
                ok = wait_bar(bar_tempty + 8 * buf, (use & 1) ^ 1, abort_flag, p.wait_ns, p.status);
                if (!ok) break;
                const uint32_t d = tmem + buf * nmax;
                for (int k = g.k0; k < g.k1; ++k) {
                    ok = wait_bar(bar_act + 8 * st, ph, abort_flag, p.wait_ns, p.status) &&
                         wait_bar(bar_w + 8 * st, ph, abort_flag, p.wait_ns, p.status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sf = sf_ring + st * sf_stage, sft = sf_tmem + st * sf_cols;
                    tc_cp_32x128b_warpx4(sft, desc_sf_block(sf));
                    tc_cp_32x128b_warpx4(sft + 4, desc_sf_block(sf + 512));
                    if (n > 128) tc_cp_32x128b_warpx4(sft + 8, desc_sf_block(sf + 1024));
                    const uint64_t ad = desc_kmajor_sw128(ring + st * ab_stage);
                    const uint64_t bd = desc_kmajor_sw128(ring + st * ab_stage + A_BYTES);
                    const int nk = min(4, (K - k * STEP) >> 5);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // (descriptors count in 16 bytes: 32 bytes on per slice)
                        if (kk < nk)
                            tc_mma_mxf8(d, ad + 2 * kk, bd + 2 * kk,
                                        idesc | (static_cast<uint32_t>(kk) << 29) | (static_cast<uint32_t>(kk) << 4), sft,
                                        sft + 4, k > g.k0 || kk > 0 ? 1u : 0u);
                    tc_commit(bar_empty + 8 * st);
                    if (++st == S) { st = 0; ph ^= 1; }
                }
                if (!ok) break;
                tc_commit(bar_tfull + 8 * buf);
                ++tile;
            }
            tc_commit(bar_drain);
            drain_bar(bar_drain, 0, p.wait_ns, p.status);
        }
        __syncwarp();
    } else if (warp < 4 || warp >= 8) {
        // ------------------------------------------------ loaders: token columns and scales
        // Loader i takes blocks i, i + 3, ... of two K-steps of a tile (an even one
        // and the next): lane l reads the scale words of weight rows l, l + 32,
        // l + 64, l + 96 into registers, one of its blocks (6 K-steps) ahead, so
        // that their HBM latency is hidden; the token rows and their scales come
        // from L2 by asynchronous copies. Every block is handed over before the
        // next is begun: a loader that waits for another CTA's h holds nothing
        // back. A loader's consecutive blocks start at most S K-steps apart (one
        // K-step a block in rings of fewer than 6), which keeps its waits on the
        // stages' parity unambiguous: when it asks for K-step c - S, it has seen
        // c - 2 S done, and c, still to be handed over by itself, cannot be.
        const int ldr = warp < 4 ? warp - 2 : warp - 6;
        const int bs = S >= LOADERS * BLOCK ? BLOCK : 1;
        uint32_t* rows = reinterpret_cast<uint32_t*>(smem + p.off_rows) + ldr * 256;  // source row of each column
        struct Block {
            Seg g;
            int k0, k1, st;  // K-steps of the tile, and the first one's stage
            uint32_t ph;     // parity of the stage's last use
        };
        Seg seg;
        seg.k0 = seg.k1 = 0;
        int kpos = 0, spos = 0, turn = 0, got = 0;
        uint32_t sph = 1;
        // The loader's next block: 1 found, 0 no more, 2 not yet known (the next
        // unit is not published; only when not told to wait).
        auto next_block = [&](Block& b, bool wait) {
            for (;;) {
                if (kpos >= seg.k1) {
                    int u = -3;
                    if (lane == 0 && (wait || mbar_try_wait(bar_qf + 8 * (got % NQ), (got / NQ) & 1))) u = read_entry(got);
                    u = __shfl_sync(0xffffffffu, u, 0);
                    if (u == -3) return 2;
                    if (u < 0) return 0;
                    ++got;
                    seg = queue.get(u);
                    kpos = seg.k0;
                }
                b.k0 = kpos;
                b.k1 = min(seg.k1, (kpos & ~(bs - 1)) + bs);
                b.st = spos;
                b.ph = sph;
                kpos = b.k1;
                spos += b.k1 - b.k0;
                if (spos >= S) { spos -= S; sph ^= 1; }
                const bool mine = turn == ldr;
                if (++turn == LOADERS) turn = 0;
                if (mine) {
                    b.g = seg;
                    return 1;
                }
            }
        };
        auto fetch = [&](const Block& b, uint32_t (&v)[4][BLOCK]) {
            const uint8_t* plane = b.g.phase ? p.s2 : p.s13;
            const int R = b.g.phase ? p.H : 2 * p.I, K32 = (b.g.phase ? p.I : p.H) / 32;
            const int k = b.k0 & ~(BLOCK - 1), nw = min(BLOCK, b.g.steps - k);  // words (K-steps), fewer at a row's end
            const size_t base = static_cast<size_t>(L.act[b.g.a]) * R;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                // (rows past the matrix are not stored: any row's scales will do)
                const int wr = b.g.phase ? min(b.g.rt * TILE + 32 * h + lane, p.H - 1)
                                         : (h >> 1) * p.I + min(b.g.rt * (TILE / 2) + 32 * (h & 1) + lane, p.I - 1);
                const size_t at = (base + wr) * K32 + 4 * k;
                if (((K32 | static_cast<int>(reinterpret_cast<uintptr_t>(plane))) & 7) == 0) {  // (the planes: 4-byte aligned)
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(plane + at));
                    v[h][0] = u.x; v[h][1] = u.y;
                } else {
                    // rows of any length: aligned words, shifted together (the plane
                    // is a whole number of words)
                    const size_t end = static_cast<size_t>(p.local) * R * K32, w0 = at & ~size_t(3);
                    uint32_t u[BLOCK + 1];
#pragma unroll
                    for (int i = 0; i <= BLOCK; ++i)
                        u[i] = i <= nw && w0 + 4 * i < end ? __ldg(reinterpret_cast<const uint32_t*>(plane + w0) + i) : 0u;
#pragma unroll
                    for (int i = 0; i < BLOCK; ++i) v[h][i] = __funnelshift_r(u[i], u[i + 1], static_cast<uint32_t>(at & 3) * 8);
                }
            }
        };
        bool ok = true;
        Block cur, b;
        uint32_t nxt[4][BLOCK];
        int tab_a = -1, tab_phase = -1;
        bool have = false;
        for (;;) {
            uint32_t sc[4][BLOCK];
            cur = b;
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int i = 0; i < BLOCK; ++i) sc[h][i] = nxt[h][i];
            // waits for the next unit only with no block in hand
            const int more = next_block(b, !have);
            if (more == 1) fetch(b, nxt);
            if (!have) {
                if (more == 0) break;
                have = true;
                continue;
            }
            const int phase = cur.g.phase, nt = L.count[cur.g.a], n = PIECES * nt;
            const uint8_t* act = phase ? p.hq : p.xq;
            const uint8_t* sact = phase ? p.sh : p.sx;
            const int stride = phase ? p.Ip : p.Hp, sstride = phase ? p.sh_stride : p.Hp / 32;
            if (tab_a != cur.g.a || tab_phase != phase) {
                if (phase) {  // this expert's h
                    if (lane == 0) ok = wait_count(p.counters + C_H + cur.g.a, p.up_tiles, abort_flag, p.wait_ns, p.status);
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (!ok) break;
                }
                const int off = L.off[cur.g.a];
                __syncwarp();
                for (int r = lane; r < n; r += 32) {
                    const int pc = r >= nt ? 1 : 0, j = r - pc * nt;
                    rows[r] = (phase ? off + j : L.entry_of[off + j] / p.top_k) * PIECES + pc;
                }
                __syncwarp();
                tab_a = cur.g.a;
                tab_phase = phase;
            }
            const int nb = cur.k1 - cur.k0;
            int st = cur.st;
            uint32_t ph = cur.ph;
            const int st0 = st;
            auto hand = [&](int i) {
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_act + 8 * (st0 + i < S ? st0 + i : st0 + i - S));
            };
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
                if (i >= nb) break;
                // the stage's last use has been multiplied
                if (lane == 0) ok = wait_bar(bar_empty + 8 * st, ph, abort_flag, p.wait_ns, p.status);
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
                const int k = cur.k0 + i;
                const bool odd = k & 1;
                const uint32_t sf = sf_ring + st * sf_stage, bsm = ring + st * ab_stage + A_BYTES;
                // one 16-byte store: this K-step's scale words of rows l, l + 32, l + 64, l + 96
                st_shared_v4(sf + lane * 16, odd ? sc[0][1] : sc[0][0], odd ? sc[1][1] : sc[1][0], odd ? sc[2][1] : sc[2][0],
                             odd ? sc[3][1] : sc[3][0]);
                for (int r = lane; r < n; r += 32)
                    cp_async_4(sf + 512 + 512 * (r >> 7) + (r & 31) * 16 + ((r >> 5) & 3) * 4,
                               sact + static_cast<size_t>(rows[r]) * sstride + 4 * k);
                const uint32_t chunk = lane & 7;  // lane l takes 16-byte piece l % 8 of rows l / 8, l / 8 + 4, ...
                for (int r = lane >> 3; r < n; r += 4)
                    cp_async_16(bsm + r * 128 + ((chunk ^ (r & 7)) << 4),
                                act + static_cast<size_t>(rows[r]) * stride + k * STEP + chunk * 16);
                cp_async_commit();
                if (++st == S) { st = 0; ph ^= 1; }
            }
            if (!ok) break;
            if (nb == 2) {
                cp_async_wait<1>();
                hand(0);
            }
            cp_async_wait<0>();
            hand(nb - 1);
            if (more == 0) break;
            have = more == 1;
        }
        cp_async_wait<0>();
    } else {
        // ------------------------------------------------ epilogue (4 warps)
        // Thread = TMEM lane = weight row of the tile. Columns: piece 0 of every
        // token, then piece 1; their sum is the product.
        const int q = warp - 4, row = threadIdx.x - 128;
        float* xch = reinterpret_cast<float*>(smem + p.off_epi);  // [2][8 tokens][128 rows]
        int tile = 0;
        for (;;) {
            const int buf = nbuf == 2 ? tile & 1 : 0, use = nbuf == 2 ? tile >> 1 : tile;
            if (q == 0 && lane == 0) {
                int u = read_entry(tile);
                if (u >= 0 && !wait_bar(bar_tfull + 8 * buf, use & 1, abort_flag, p.wait_ns, p.status)) u = -2;
                flags[2 + (tile & 1)] = u;
            }
            named_bar_sync(EPI_BAR, 128);
            const int unit = flags[2 + (tile & 1)];
            if (unit < 0) break;
            const Seg g = queue.get(unit);
            const int nt = L.count[g.a], off = L.off[g.a];
            const bool whole = !PARTS || g.parts == 1;
            ++tile;
            tc_fence_after();
            const uint32_t d = tmem + buf * nmax + (static_cast<uint32_t>(q * 32) << 16);
            float* part = g.phase ? p.part_down + static_cast<size_t>(unit - queue.up_units) * p.T * TILE
                                  : p.part_up + static_cast<size_t>(unit) * p.T * TILE;
            for (int j0 = 0; j0 < nt; j0 += 8) {
                uint32_t v0[8], v1[8];
                tmem_ld_32x32b_x8(d + j0, v0);
                tmem_ld_32x32b_x8(d + nt + j0, v1);
                tmem_wait_ld();
                reg_fence8(v0);
                reg_fence8(v1);
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(v0[j]) + __uint_as_float(v1[j]);
                if (!whole) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j0 + j < nt) part[(j0 + j) * TILE + row] = v[j];
                } else if (g.phase) {
                    const int n = g.rt * TILE + row;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j0 + j < nt && n < p.H)
                            p.y[static_cast<size_t>(off + j0 + j) * p.Hp + n] = v[j] * L.wts[L.entry_of[off + j0 + j]];
                } else {
                    float* x = xch + ((j0 >> 3) & 1) * 8 * TILE;
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j * TILE + row] = v[j];
                    named_bar_sync(EPI_BAR, 128);
                    // (token, half of the 64 inner rows) pairs, dealt to the warps
#pragma unroll 1
                    for (int o = q; o < 2 * min(8, nt - j0); o += 4) {
                        const int j = o >> 1, i = 32 * (o & 1) + lane, i0 = g.rt * (TILE / 2) + 32 * (o & 1);
                        if (i0 < p.I) store_h(p, off + j0 + j, i0, x[j * TILE + i], x[j * TILE + TILE / 2 + i]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_tempty + 8 * buf);
            if (g.phase) {
                named_bar_sync(EPI_BAR, 128);
                if (q == 0 && lane == 0) red_release_gpu_add(p.counters + C_DONE, 1);
            } else {
                bool finish = whole;
                if (!whole) {
                    // the part that ends last sums all of them, in order
                    named_bar_sync(EPI_BAR, 128);
                    if (q == 0 && lane == 0)
                        flags[8] = atom_acq_rel_gpu_add(p.counters + C_H + p.local + g.tile, 1) == static_cast<uint32_t>(g.parts - 1) ? 1 : 0;
                    named_bar_sync(EPI_BAR, 128);
                    finish = flags[8] != 0;
                    for (int o = q; finish && o < 2 * nt; o += 4) {
                        const int j = o >> 1, i = 32 * (o & 1) + lane, i0 = g.rt * (TILE / 2) + 32 * (o & 1);
                        if (i0 >= p.I) continue;
                        const float* src = p.part_up + static_cast<size_t>(g.tile * g.parts) * p.T * TILE + static_cast<size_t>(j) * TILE + i;
                        const size_t piece = static_cast<size_t>(p.T) * TILE;
                        float vg[MAX_PARTS], vu[MAX_PARTS], gate = 0.f, up = 0.f;  // (all loads in flight together)
#pragma unroll
                        for (int c = 0; c < MAX_PARTS; ++c) {
                            vg[c] = c < g.parts ? __ldcg(src + c * piece) : 0.f;
                            vu[c] = c < g.parts ? __ldcg(src + c * piece + TILE / 2) : 0.f;
                        }
#pragma unroll
                        for (int c = 0; c < MAX_PARTS; ++c) {
                            gate += vg[c];
                            up += vu[c];
                        }
                        store_h(p, off + j, i0, gate, up);
                    }
                }
                if (finish) {
                    named_bar_sync(EPI_BAR, 128);
                    if (q == 0 && lane == 0) red_release_gpu_add(p.counters + C_H + g.a, 1);
                }
            }
        }
    }

    // ---- once every product is in y or a partial: the weighted sum, a share per CTA
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_single(tmem, TMEM_ALL);
    if (threadIdx.x == 0) {
        bool ok = !*abort_flag;
        if (ok) ok = wait_count(p.counters + C_DONE, queue.units - queue.up_units, abort_flag, p.wait_ns, p.status);
        flags[6] = ok ? 1 : 0;
    }
    __syncthreads();
    if (!flags[6]) return;
    const int half = p.H / 2;
    for (int o = cta * THREADS + threadIdx.x; o < p.T * half; o += G * THREADS) {
        const int t = o / half, n = 2 * (o - t * half), rt = n / TILE, r = n - rt * TILE;
        float y0 = 0.f, y1 = 0.f;
        // four of the token's experts at a time, their loads in flight together
        for (int k0 = 0; k0 < p.top_k; k0 += 4) {
            float2 v[4];
            int e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = t * p.top_k + k0 + j;
                e[j] = k0 + j < p.top_k ? L.eid[i] : 0xffff;
                v[j] = make_float2(0.f, 0.f);
                if (e[j] != 0xffff && (!PARTS || queue.down_parts == 1))
                    v[j] = __ldcg(reinterpret_cast<const float2*>(p.y + static_cast<size_t>(L.slot_of[i]) * p.Hp + n));
            }
            if (PARTS && queue.down_parts > 1) {
                // the parts of each down tile, in order; then the expert's weight
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (e[j] == 0xffff) continue;
                    const int i = t * p.top_k + k0 + j, a = L.act_of[e[j]];
                    const float* src = p.part_down + static_cast<size_t>(a * p.down_tiles + rt) * queue.down_parts * p.T * TILE +
                                       static_cast<size_t>(L.slot_of[i] - L.off[a]) * TILE + r;
                    float2 z[MAX_PARTS];
#pragma unroll
                    for (int c = 0; c < MAX_PARTS; ++c)
                        z[c] = c < queue.down_parts ? __ldcg(reinterpret_cast<const float2*>(src + static_cast<size_t>(c) * p.T * TILE))
                                                    : make_float2(0.f, 0.f);
#pragma unroll
                    for (int c = 0; c < MAX_PARTS; ++c) {
                        v[j].x += z[c].x;
                        v[j].y += z[c].y;
                    }
                    v[j].x *= L.wts[i];
                    v[j].y *= L.wts[i];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y0 += v[j].x;
                y1 += v[j].y;
            }
        }
        reinterpret_cast<uint32_t*>(p.out)[static_cast<size_t>(t) * half + (n >> 1)] = pack_bf16x2(__float_as_uint(y0), __float_as_uint(y1));
    }
}

// ============================================================== host side

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct Layout {
    int ksplit, Hp, Ip, sh_stride, up_tiles, down_tiles, up_steps, down_steps, slots, local_slots, n_counters, mf, nf;
    size_t counters, logits, ids, weights, xq, sx, hq, sh, y, part_up, part_down, total;
};

void layout(int T, int experts, int local, int H, int I, int top_k, int sms, Layout* l) {
    // Logits: tiles of 16 tokens x 16 experts, H in up to 8 slices so that about 300
    // blocks share them, each of their 8 warps at least one 32-column chunk. Tiles
    // of 32 x 32, which read x and the router half as often, where the small ones
    // are so many that they would get fewer slices (whole call, 32 x 32 / 16 x 16: H = 7168,
    // 256 experts, 128 tokens 248 / 254 us, 32 tokens 157.6 / 155.0; H = 2048, 64
    // experts, 64 tokens 111.6 / 110.2).
    auto tiles_of = [&](int mf, int nf) { return ((experts + 8 * nf - 1) / (8 * nf)) * ((T + 16 * mf - 1) / (16 * mf)); };
    constexpr int BLOCKS = 300, SLICES = 8;
    const bool wide = T > 16 && tiles_of(1, 2) > BLOCKS / SLICES;
    l->mf = wide ? 2 : 1;
    l->nf = wide ? 4 : 2;
    int ks = BLOCKS / tiles_of(l->mf, l->nf);
    if (ks > SLICES) ks = SLICES;
    if (ks > H / 256) ks = H / 256;
    l->ksplit = ks < 1 ? 1 : ks;
    l->Hp = (H + STEP - 1) / STEP * STEP;
    l->Ip = (I + STEP - 1) / STEP * STEP;
    l->sh_stride = (l->Ip / 32 + 127) & ~127;  // a line of its own for each row: read through L1 while others are written
    l->up_tiles = (I + TILE / 2 - 1) / (TILE / 2);
    l->down_tiles = (H + TILE - 1) / TILE;
    l->up_steps = l->Hp / STEP;
    l->down_steps = l->Ip / STEP;
    l->slots = T * top_k;
    l->local_slots = top_k < local ? T * top_k : T * local;
    l->n_counters = C_H + local + local * l->up_tiles;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
    l->counters = take(4 * static_cast<size_t>(l->n_counters));
    l->logits = take(4 * static_cast<size_t>(l->ksplit) * T * experts);
    l->ids = take(4 * static_cast<size_t>(l->slots));
    l->weights = take(4 * static_cast<size_t>(l->slots));
    l->xq = take(static_cast<size_t>(T) * PIECES * l->Hp);
    l->sx = take(static_cast<size_t>(T) * PIECES * (l->Hp / 32));
    l->hq = take(static_cast<size_t>(l->local_slots) * PIECES * l->Ip);
    l->sh = take(static_cast<size_t>(l->local_slots) * PIECES * l->sh_stride);
    l->y = take(4 * static_cast<size_t>(l->local_slots) * l->Hp);
    l->part_up = take(4 * static_cast<size_t>(sms) * T * TILE);  // (parts are only made up to one per SM)
    l->part_down = take(4 * static_cast<size_t>(sms) * T * TILE);
    l->total = at;
}

// Whether a call takes the form of moe_experts that can cut tiles along the
// contraction: where a contraction of 32 K-steps or more (4096 columns) is
// expected to meet fewer tiles than CTAs. Which experts are chosen is known on
// the GPU only; here their number is taken as if all were equally likely, and
// what is cut, if anything, is decided there (parts_of). H = 7168, I = 2048, 32
// experts of 256, 1 / 2 / 4 tokens: 19.0 / 24.2 / 52.9 us in this form, 18.8 / 27.2 /
// 51.8 without cuts, by what the routing leaves here; one expert of I = 128, 64
// tokens: 51.3 / 74.1. Elsewhere the cuts' code alone costs up to 5 us (H = 2048, I =
// 1408, 64 experts, 128 tokens: 127.7 / 122.5).
bool cuts(const MoeArgs& a, const Layout& l) {
    const long long pairs = static_cast<long long>(a.T) * a.top_k * a.local / a.experts;
    const long long chosen = pairs < 1 ? 1 : pairs < a.local ? pairs : a.local;
    return (l.up_steps >= 32 && chosen * l.up_tiles <= a.num_sms) || (l.down_steps >= 32 && chosen * l.down_tiles <= a.num_sms);
}

}  // namespace

size_t moe_ws_bytes(int T, int experts, int local, int H, int I, int top_k, int sms) {
    Layout l;
    layout(T, experts, local, H, I, top_k, sms, &l);
    return l.total;
}

int launch_moe(const MoeArgs& a) {
    Layout l;
    layout(a.T, a.experts, a.local, a.H, a.I, a.top_k, a.num_sms, &l);
    if (static_cast<long long>(a.local) * l.up_tiles * l.up_steps > 0x7fffffffLL / 2 ||
        static_cast<long long>(a.local) * l.down_tiles * l.down_steps > 0x7fffffffLL / 2)
        return host_fail(MXFP8_EINVAL, "local=%d experts of H=%d, I=%d: too many tiles", a.local, a.H, a.I);
    Params p{};
    p.x = a.x; p.router = a.router; p.bias = a.bias; p.s13 = a.s13; p.s2 = a.s2;
    p.T = a.T; p.experts = a.experts; p.first = a.first; p.local = a.local; p.H = a.H; p.I = a.I; p.top_k = a.top_k;
    p.score = a.score; p.renormalize = a.renormalize; p.scale = a.scale;
    p.out = a.out; p.user_ids = a.ids; p.user_weights = a.weights;
    p.counters = reinterpret_cast<unsigned int*>(a.ws + l.counters);
    p.logits = reinterpret_cast<float*>(a.ws + l.logits);
    p.ids = reinterpret_cast<int32_t*>(a.ws + l.ids);
    p.weights = reinterpret_cast<float*>(a.ws + l.weights);
    p.xq = a.ws + l.xq; p.sx = a.ws + l.sx; p.hq = a.ws + l.hq; p.sh = a.ws + l.sh;
    p.y = reinterpret_cast<float*>(a.ws + l.y);
    p.part_up = reinterpret_cast<float*>(a.ws + l.part_up);
    p.part_down = reinterpret_cast<float*>(a.ws + l.part_down);
    p.Hp = l.Hp; p.Ip = l.Ip; p.sh_stride = l.sh_stride; p.ksplit = l.ksplit; p.slots = l.slots; p.n_counters = l.n_counters;
    p.up_tiles = l.up_tiles; p.down_tiles = l.down_tiles; p.up_steps = l.up_steps; p.down_steps = l.down_steps;
    p.off_lists = 512;
    p.off_mask = (p.off_lists + l.slots * 10 + a.local * 8 + 127) & ~127u;
    p.off_epi = (p.off_mask + a.local * 16 + 127) & ~127u;
    p.off_rows = p.off_epi + 2 * 8 * TILE * 4;
    p.off_ring = (p.off_rows + LOADERS * 1024 + 1023) & ~1023u;
    p.wait_ns = a.wait_limit_ns;
    p.status = a.status;
    p.stall = a.stall;

    CUtensorMap m13, m2;
    // w13 as [local][2][I][H]: one box holds 64 gate rows and the same 64 up rows
    const uint32_t b13[4] = {STEP, TILE / 2, 2, 1}, b2[3] = {STEP, TILE, 1};
    const uint64_t H = a.H, I = a.I, E = a.local;
    const uint64_t d13[4] = {H, I, 2, E}, st13[3] = {H, I * H, 2 * I * H}, d2[3] = {I, H, E}, st2[2] = {I, H * I};
    int rc = host_tensor_map(&m13, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.w13, d13, st13, b13, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    rc = host_tensor_map(&m2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.w2, d2, st2, b2, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;

    static std::atomic<bool> ready[64];
    cudaError_t e;
    if (!ready[a.dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(moe_experts<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_experts<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "expert layer kernel: %s", cudaGetErrorString(e));
        ready[a.dev].store(true, std::memory_order_relaxed);
    }
    const int lblocks = ((a.experts + 8 * l.nf - 1) / (8 * l.nf)) * ((a.T + 16 * l.mf - 1) / (16 * l.mf)) * l.ksplit;
    int sblocks = (a.T * (l.Hp / STEP) + 7) / 8;  // one 128-column piece of a row per warp, up to 304 blocks
    if (sblocks > 304) sblocks = 304;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.stream = a.stream;
    cfg.gridDim = dim3(lblocks + sblocks);
    cfg.blockDim = dim3(256);
    e = l.mf == 2 ? cudaLaunchKernelEx(&cfg, moe_logits<2, 4>, p) : cudaLaunchKernelEx(&cfg, moe_logits<1, 2>, p);
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "router kernel: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    cfg.gridDim = dim3(a.num_sms);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    e = cuts(a, l) ? cudaLaunchKernelEx(&cfg, moe_experts<true>, m13, m2, p) : cudaLaunchKernelEx(&cfg, moe_experts<false>, m13, m2, p);
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "expert layer kernel: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return MXFP8_OK;
}

}  // namespace mxw
