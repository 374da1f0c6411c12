// A whole mixture-of-experts layer for a few tokens (mxfp8_moe_layer): router,
// choice of experts, gated MLPs on MXFP8 weights, weighted sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "mxw_experts.h"
#include "mxw_internal.h"
#include "../../include/mxfp8_experts.h"

namespace mxw {
namespace {

__device__ __forceinline__ float bf16_f(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__device__ __forceinline__ float e8m0_f(uint8_t s) {
    return s == 255 ? CUDART_NAN_F : __uint_as_float(s == 0 ? 0x00400000u : static_cast<uint32_t>(s) << 23);
}

__device__ __forceinline__ float e4m3_f(uint8_t q) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// One block per token: logits, scores, the top-k (ties to the lower index).
__global__ void __launch_bounds__(256) route_simple(const MoeArgs a, int32_t* ids, float* wts) {
    __shared__ float score[MXFP8_MOE_MAX_EXPERTS];
    __shared__ float key[MXFP8_MOE_MAX_EXPERTS];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = warp; e < a.experts; e += 8) {
        float s = 0.f;
        for (int h = lane; h < a.H; h += 32) s += bf16_f(a.x[t * a.H + h]) * bf16_f(a.router[static_cast<size_t>(e) * a.H + h]);
        s = warp_sum(s);
        if (lane == 0) score[e] = s;
    }
    __syncthreads();
    if (warp != 0) return;
    if (a.score == MXFP8_SCORE_SOFTMAX) {
        float m = -CUDART_INF_F, sum = 0.f;
        for (int e = lane; e < a.experts; e += 32) m = fmaxf(m, score[e]);
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        for (int e = lane; e < a.experts; e += 32) sum += (score[e] = expf(score[e] - m));
        sum = warp_sum(sum);
        for (int e = lane; e < a.experts; e += 32) score[e] /= sum;
    } else {
        for (int e = lane; e < a.experts; e += 32) score[e] = 1.f / (1.f + expf(-score[e]));
    }
    for (int e = lane; e < a.experts; e += 32) {
        const float v = score[e] + (a.bias ? a.bias[e] : 0.f);
        key[e] = v != v ? -CUDART_INF_F : v;
    }
    __syncwarp();
    uint32_t taken[MXFP8_MOE_MAX_EXPERTS / 32 / 32] = {0};
    float total = 0.f;
    for (int k = 0; k < a.top_k; ++k) {
        float best = -CUDART_INF_F;
        int at = 0x7fffffff;
        for (int i = 0; i * 32 + lane < a.experts; ++i)
            if (!((taken[i >> 5] >> (i & 31)) & 1) && (at == 0x7fffffff || key[i * 32 + lane] > best)) {
                best = key[i * 32 + lane];
                at = i * 32 + lane;
            }
        for (int d = 16; d > 0; d >>= 1) {
            const float ob = __shfl_xor_sync(0xffffffffu, best, d);
            const int oa = __shfl_xor_sync(0xffffffffu, at, d);
            if (ob > best || (ob == best && oa < at)) { best = ob; at = oa; }
        }
        if ((at & 31) == lane) taken[at >> 10] |= 1u << ((at >> 5) & 31);
        total += score[at];
        if (lane == 0) { ids[t * a.top_k + k] = at; wts[t * a.top_k + k] = score[at]; }
    }
    __syncwarp();
    if (lane < a.top_k) wts[t * a.top_k + lane] = a.renormalize ? wts[t * a.top_k + lane] / total * a.scale : wts[t * a.top_k + lane] * a.scale;
}

__device__ __forceinline__ float row_dot(const uint8_t* q, const uint8_t* s, int n, const float* v32, const uint16_t* v16, int lane) {
    float acc = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float v = v32 ? v32[i] : bf16_f(v16[i]);
        acc += e4m3_f(q[i]) * e8m0_f(s[i >> 5]) * v;
    }
    return warp_sum(acc);
}

// One warp per (token, chosen expert, inner row): h = silu(g) u.
__global__ void __launch_bounds__(256) up_simple(const MoeArgs a, const int32_t* ids, float* h) {
    const int slot = blockIdx.y, i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int e = ids[slot] - a.first;
    if (i >= a.I || e < 0 || e >= a.local) return;
    const uint16_t* x = a.x + static_cast<size_t>(slot / a.top_k) * a.H;
    const size_t rg = static_cast<size_t>(e) * 2 * a.I + i, ru = rg + a.I;
    const float g = row_dot(a.w13 + rg * a.H, a.s13 + rg * (a.H / 32), a.H, nullptr, x, lane);
    const float u = row_dot(a.w13 + ru * a.H, a.s13 + ru * (a.H / 32), a.H, nullptr, x, lane);
    if (lane == 0) h[static_cast<size_t>(slot) * a.I + i] = g / (1.f + expf(-g)) * u;
}

// One warp per (token, output row): the weighted sum over its experts.
__global__ void __launch_bounds__(256) down_simple(const MoeArgs a, const int32_t* ids, const float* wts, const float* h) {
    const int t = blockIdx.y, n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (n >= a.H) return;
    float y = 0.f;
    for (int k = 0; k < a.top_k; ++k) {
        const int slot = t * a.top_k + k, e = ids[slot] - a.first;
        if (e < 0 || e >= a.local) continue;
        const size_t r = static_cast<size_t>(e) * a.H + n;
        y += wts[slot] * row_dot(a.w2 + r * a.I, a.s2 + r * (a.I / 32), a.I, h + static_cast<size_t>(slot) * a.I, nullptr, lane);
    }
    if (lane == 0) a.out[static_cast<size_t>(t) * a.H + n] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

}  // namespace

size_t moe_ws_bytes(int T, int, int, int, int I, int top_k, int) {
    return static_cast<size_t>(T) * top_k * (8 + static_cast<size_t>(I) * 4) + 256;
}

int launch_moe(const MoeArgs& a) {
    const int slots = a.T * a.top_k;
    float* h = reinterpret_cast<float*>(a.ws);
    int32_t* ids = a.ids ? a.ids : reinterpret_cast<int32_t*>(h + static_cast<size_t>(slots) * a.I);
    float* wts = a.weights ? a.weights : h + static_cast<size_t>(slots) * (a.I + 1);
    route_simple<<<a.T, 256, 0, a.stream>>>(a, ids, wts);
    up_simple<<<dim3((a.I + 7) / 8, slots), 256, 0, a.stream>>>(a, ids, h);
    down_simple<<<dim3((a.H + 7) / 8, a.T), 256, 0, a.stream>>>(a, ids, wts, h);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "expert layer kernel: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return MXFP8_OK;
}

}  // namespace mxw
