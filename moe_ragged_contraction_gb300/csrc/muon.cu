// Orthogonalised update of a stack of gradients (mxfp8_muon_update): momentum,
// Frobenius norm, Newton-Schulz products.
#include <cuda_bf16.h>

#include "mxw_experts.h"
#include "mxw_internal.h"
#include "../../include/mxfp8_experts.h"

namespace mxw {
namespace {

constexpr int NORM_BLOCKS = 64;

// u (fp32) and the momentum; per-block partial sums of u^2.
__global__ void __launch_bounds__(256) momentum_simple(const MuonArgs a, float* u, float* part) {
    const size_t per = static_cast<size_t>(a.N) * a.K, base = blockIdx.y * per;
    float s = 0.f;
    for (size_t i = blockIdx.x * 256 + threadIdx.x; i < per; i += NORM_BLOCKS * 256) {
        const float g = a.grad_f32 ? static_cast<const float*>(a.grad)[base + i]
                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(a.grad)[base + i]);
        float v = g;
        if (a.momentum) {
            const float m = a.mu * a.momentum[base + i] + g;
            a.momentum[base + i] = m;
            v = a.nesterov ? g + a.mu * m : m;
        }
        u[base + i] = v;
        s += v * v;
    }
    __shared__ float red[256];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if (threadIdx.x < d) red[threadIdx.x] += red[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) part[blockIdx.y * NORM_BLOCKS + blockIdx.x] = red[0];
}

__global__ void __launch_bounds__(256) normalise_simple(const MuonArgs a, float* u, const float* part) {
    const size_t per = static_cast<size_t>(a.N) * a.K, base = blockIdx.y * per;
    float s = 0.f;
    for (int i = 0; i < NORM_BLOCKS; ++i) s += part[blockIdx.y * NORM_BLOCKS + i];
    const float inv = 1.f / (sqrtf(s) + a.eps);
    for (size_t i = blockIdx.x * 256 + threadIdx.x; i < per; i += NORM_BLOCKS * 256)
        u[base + i] = isfinite(s) ? u[base + i] * inv : __int_as_float(0x7fffffff);
}

// C[i][j] = alpha * sum_k A(i,k) B(j,k) + beta * D[i][j]; element (i,k) of an
// operand at i * si + k * sk; C, D row-major with ldc. out16: bf16 result.
struct Gemm {
    const float *A, *B, *D;
    float* C;
    uint16_t* out16;
    int m, n, k;
    size_t sai, sak, sbj, sbk, ldc, batch_a, batch_b, batch_c;
    float alpha, beta;
};

__global__ void __launch_bounds__(256) gemm_simple(const Gemm g) {
    __shared__ float As[16][65], Bs[16][65];
    const float* A = g.A + blockIdx.z * g.batch_a;
    const float* B = g.B + blockIdx.z * g.batch_b;
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < g.k; k0 += 16) {
        for (int l = threadIdx.x; l < 1024; l += 256) {
            const int r = l >> 4, k = l & 15;
            As[k][r] = i0 + r < g.m && k0 + k < g.k ? A[(i0 + r) * g.sai + (k0 + k) * g.sak] : 0.f;
            Bs[k][r] = j0 + r < g.n && k0 + k < g.k ? B[(j0 + r) * g.sbj + (k0 + k) * g.sbk] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += As[k][ty * 4 + i] * Bs[k][tx * 4 + j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = i0 + ty * 4 + i, c = j0 + tx * 4 + j;
            if (r >= g.m || c >= g.n) continue;
            const size_t at = blockIdx.z * g.batch_c + r * g.ldc + c;
            const float v = g.alpha * acc[i][j] + (g.D ? g.beta * g.D[at] : 0.f);
            if (g.out16) g.out16[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            else g.C[at] = v;
        }
}

}  // namespace

size_t muon_ws_bytes(int E, int N, int K) {
    const size_t m = N < K ? N : K, per = static_cast<size_t>(N) * K;
    return 4 * static_cast<size_t>(E) * (2 * per + 2 * m * m + NORM_BLOCKS) + 256;
}

int launch_muon(const MuonArgs& a) {
    const size_t per = static_cast<size_t>(a.N) * a.K;
    const int m = a.N < a.K ? a.N : a.K, n = a.N < a.K ? a.K : a.N;
    const bool tall = a.N > a.K;
    const size_t mm = static_cast<size_t>(m) * m;
    float* X = reinterpret_cast<float*>(a.ws);
    float* Y = X + a.E * per;
    float* A = Y + a.E * per;
    float* B = A + a.E * mm;
    float* part = B + a.E * mm;
    momentum_simple<<<dim3(NORM_BLOCKS, a.E), 256, 0, a.stream>>>(a, X, part);
    normalise_simple<<<dim3(NORM_BLOCKS, a.E), 256, 0, a.stream>>>(a, X, part);
    const size_t si = tall ? 1 : a.K, sk = tall ? a.K : 1;  // X(i, k): row i of the shorter side, column k of the longer
    auto run = [&](const Gemm& g) {
        gemm_simple<<<dim3((g.n + 63) / 64, (g.m + 63) / 64, a.E), 256, 0, a.stream>>>(g);
    };
    for (int s = 0; s < a.steps; ++s) {
        const size_t sm = m;
        run(Gemm{X, X, nullptr, A, nullptr, m, m, n, si, sk, si, sk, sm, per, per, mm, 1.f, 0.f});
        run(Gemm{A, A, A, B, nullptr, m, m, m, sm, 1, sm, 1, sm, mm, mm, mm, a.c, a.b});
        uint16_t* out = s + 1 == a.steps ? a.out : nullptr;
        if (!tall)
            run(Gemm{B, X, X, Y, out, m, n, m, sm, 1, sk, si, static_cast<size_t>(a.K), mm, per, per, 1.f, a.a});
        else
            run(Gemm{X, B, X, Y, out, n, m, m, sk, si, sm, 1, static_cast<size_t>(a.K), per, mm, per, 1.f, a.a});
        float* t = X;
        X = Y;
        Y = t;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "update kernel: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return MXFP8_OK;
}

}  // namespace mxw
