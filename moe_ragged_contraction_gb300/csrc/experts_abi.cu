// Entry points of include/mxfp8_experts.h: argument checks, scratch, launch.
#include <cmath>

#include "mxw_experts.h"
#include "mxw_internal.h"
#include "../../include/mxfp8_experts.h"

namespace {

using mxw::host_fail;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// SMs the scratch of a call is sized for before a device is known.
constexpr int MAX_SMS = 160;

bool moe_sizes(int T, int experts, int first, int local, int H, int I, int top_k) {
    return T >= 0 && T <= MXFP8_MOE_MAX_TOKENS && experts >= 1 && experts <= MXFP8_MOE_MAX_EXPERTS && first >= 0 &&
           local >= 1 && local <= experts && first <= experts - local && H >= 32 && H % 32 == 0 && H <= 32768 &&
           I >= 32 && I % 32 == 0 && I <= 32768 && top_k >= 1 && top_k <= experts && top_k <= MXFP8_MOE_MAX_TOPK;
}

int moe(const uint16_t* x, int T, const uint16_t* router, const float* bias, const uint8_t* w13, const uint8_t* s13,
        const uint8_t* w2, const uint8_t* s2, int experts, int first, int local, int H, int I, int top_k, int score,
        int renormalize, float scale, uint16_t* out, int32_t* ids, float* weights, void* ws, size_t ws_bytes,
        bool use_cache, void* stream) {
    if (!moe_sizes(T, experts, first, local, H, I, top_k))
        return host_fail(MXFP8_EINVAL,
                         "unsupported sizes T=%d experts=%d first=%d local=%d H=%d I=%d top_k=%d (T <= %d, experts <= "
                         "%d, H and I multiples of 32 up to 32768, top_k <= min(experts, %d))",
                         T, experts, first, local, H, I, top_k, MXFP8_MOE_MAX_TOKENS, MXFP8_MOE_MAX_EXPERTS,
                         MXFP8_MOE_MAX_TOPK);
    if (score != MXFP8_SCORE_SOFTMAX && score != MXFP8_SCORE_SIGMOID)
        return host_fail(MXFP8_EINVAL, "score=%d: 0 (softmax) or 1 (sigmoid)", score);
    if (!std::isfinite(scale)) return host_fail(MXFP8_EINVAL, "scale is not finite");
    if (T == 0) return MXFP8_OK;
    if (!x || !router || !w13 || !s13 || !w2 || !s2 || !out) return host_fail(MXFP8_EINVAL, "null pointer argument");
    if (misaligned(x, 16) || misaligned(router, 16) || misaligned(w13, 16) || misaligned(w2, 16) || misaligned(out, 16))
        return host_fail(MXFP8_EALIGN, "x, router, w13, w2 and out must be 16-byte aligned");
    if (misaligned(s13, 4) || misaligned(s2, 4) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4))
        return host_fail(MXFP8_EALIGN, "s13, s2, bias, topk_ids and topk_weights must be 4-byte aligned");
    const size_t need = mxw::moe_ws_bytes(T, experts, local, H, I, top_k, MAX_SMS);
    if (!use_cache) {
        if (!ws) return host_fail(MXFP8_EINVAL, "null workspace");
        if (misaligned(ws, 256)) return host_fail(MXFP8_EALIGN, "workspace must be 256-byte aligned");
        if (ws_bytes < need) return host_fail(MXFP8_ENOWS, "workspace of %zu bytes, need %zu", ws_bytes, need);
    }
    mxw::MoeArgs a{};
    int rc = mxw::host_device(&a.dev, &a.num_sms);
    if (rc) return rc;
    if (a.num_sms > MAX_SMS) a.num_sms = MAX_SMS;
    a.stream = static_cast<cudaStream_t>(stream);
    mxw::LaunchLock launches;
    if (use_cache) {
        rc = mxw::host_workspace(a.dev, a.stream, need, &ws, &launches);
        if (rc) return rc;
    }
    a.x = x; a.router = router; a.bias = bias; a.w13 = w13; a.s13 = s13; a.w2 = w2; a.s2 = s2;
    a.T = T; a.experts = experts; a.first = first; a.local = local; a.H = H; a.I = I; a.top_k = top_k;
    a.score = score; a.renormalize = renormalize ? 1 : 0; a.scale = scale;
    a.out = out; a.ids = ids; a.weights = weights;
    a.ws = static_cast<uint8_t*>(ws);
    a.wait_limit_ns = mxw::host_wait_limit_ns();
    a.stall = mxw::host_take_stall();
    const cudaError_t e = mxw::device_status_address(a.dev, &a.status);
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "device status: %s", cudaGetErrorString(e));
    return mxw::launch_moe(a);
}

bool muon_sizes(int E, int N, int K) {
    return E >= 0 && E <= MXFP8_MAX_EXPERTS && N >= 1 && N <= 32768 && K >= 1 && K <= 32768;
}

// Scratch of an update. Matrices that stay on chip need none: a nominal amount is
// asked for, as 0 stands for invalid sizes.
constexpr size_t MUON_SMALL_WS = 512;

size_t muon_need(int E, int N, int K) { return mxw::muon_fits_small(N, K) ? MUON_SMALL_WS : mxw::muon_ws_bytes(E, N, K); }

// Largest |k0 + k1 t + k2 t^2| on [0, T].
double quadratic_max(double k0, double k1, double k2, double T) {
    double m = std::fmax(std::fabs(k0), std::fabs(k0 + (k1 + k2 * T) * T));
    const double t = -k1 / (2 * k2);
    if (t > 0 && t < T) m = std::fmax(m, std::fabs(k0 + (k1 + k2 * t) * t));
    return m;
}

// Largest |a s + b s^3 + c s^5| on [0, S].
double step_max(double a, double b, double c, double S) {
    auto f = [&](double s) { const double t = s * s; return std::fabs(s * (a + t * (b + t * c))); };
    double m = f(S);
    // the derivative a + 3 b t + 5 c t^2 vanishes; with c = 0 at t = -a / (3 b)
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
        const double q = -(3 * b + std::copysign(std::sqrt(d), b)) / 2;  // (the root without cancellation, the other from their product)
        for (const double t : {q / (5 * c), a / q})
            if (t > 0 && t < S * S) m = std::fmax(m, f(std::sqrt(t)));
    }
    return m;
}

// Whether the iteration stays in the range of the kernels' fp16 operands for
// every matrix. X0's singular values fill [0, 1]; a step takes s to a s + b s^3
// + c s^5, so that A's largest eigenvalue and R's largest value (R = b A + c A A
// - beta I) are known beforehand. Both are stored times 4096 and end at 16; the
// limit of 14 and the share added to each step's largest value (four roundings
// to 11 bits of R's terms) leave room for what the roundings add.
constexpr double MUON_LIMIT = 14.0;

bool muon_in_range(double a, double b, double c, int steps) {
    double S = 1.0;
    for (int k = 0; k < steps; ++k) {
        const double T = S * S, beta = (b + c) * (k + 1 == steps ? 0.875 : k + 2 == steps ? 0.4375 : 0.0);
        const double r = quadratic_max(-beta, b, c, T);
        if (!(T <= MUON_LIMIT) || !(r <= MUON_LIMIT)) return false;
        S = step_max(a, b, c, S) + S * (std::fabs(b) * T + 2 * std::fabs(c) * T * T + r) / 1024;
    }
    return true;
}

int muon(const void* grad, int grad_type, float* momentum, int E, int N, int K, float mu, int nesterov, int steps,
         float a_, float b_, float c_, float eps, uint16_t* out, void* ws, size_t ws_bytes, bool use_cache,
         void* stream) {
    if (!muon_sizes(E, N, K))
        return host_fail(MXFP8_EINVAL, "unsupported sizes E=%d N=%d K=%d (E <= %d, N and K in [1, 32768])", E, N, K,
                         MXFP8_MAX_EXPERTS);
    if (grad_type != MXFP8_GRAD_BF16 && grad_type != MXFP8_GRAD_F32)
        return host_fail(MXFP8_EINVAL, "grad_type=%d: 0 (bf16) or 1 (fp32)", grad_type);
    if (steps < 1 || steps > MXFP8_MUON_MAX_STEPS)
        return host_fail(MXFP8_EINVAL, "steps=%d out of range [1, %d]", steps, MXFP8_MUON_MAX_STEPS);
    if (!(std::fabs(a_) <= 16.f) || !(std::fabs(b_) <= 16.f) || !(std::fabs(c_) <= 16.f))
        return host_fail(MXFP8_EINVAL, "coefficients %g, %g, %g: finite and at most 16 in magnitude", a_, b_, c_);
    if (!muon_in_range(a_, b_, c_, steps))
        return host_fail(MXFP8_EINVAL,
                         "coefficients %g, %g, %g with %d steps leave the range of the products' operands: the eigenvalues of A "
                         "or R can exceed %g",
                         a_, b_, c_, steps, MUON_LIMIT);
    if (!std::isfinite(mu) || !std::isfinite(eps) || eps < 0.f)
        return host_fail(MXFP8_EINVAL, "mu=%g must be finite and eps=%g finite and >= 0", mu, eps);
    if ((K % 8) != 0) return host_fail(MXFP8_EALIGN, "K=%d must be a multiple of 8 (16-byte output rows)", K);
    if (E == 0) return MXFP8_OK;
    if (!grad || !out) return host_fail(MXFP8_EINVAL, "null pointer argument");
    if (misaligned(grad, 16) || misaligned(momentum, 16) || misaligned(out, 16))
        return host_fail(MXFP8_EALIGN, "grad, momentum and out must be 16-byte aligned");
    const bool small = mxw::muon_fits_small(N, K);
    const size_t need = muon_need(E, N, K);
    if (!use_cache) {
        if (!ws) return host_fail(MXFP8_EINVAL, "null workspace");
        if (misaligned(ws, 256)) return host_fail(MXFP8_EALIGN, "workspace must be 256-byte aligned");
        if (ws_bytes < need) return host_fail(MXFP8_ENOWS, "workspace of %zu bytes, need %zu", ws_bytes, need);
    }
    mxw::MuonArgs a{};
    int rc = mxw::host_device(&a.dev, &a.num_sms);
    if (rc) return rc;
    a.stream = static_cast<cudaStream_t>(stream);
    mxw::LaunchLock launches;
    if (use_cache && !small) {
        rc = mxw::host_workspace(a.dev, a.stream, need, &ws, &launches);
        if (rc) return rc;
    }
    a.grad = grad; a.grad_f32 = grad_type == MXFP8_GRAD_F32; a.momentum = momentum;
    a.E = E; a.N = N; a.K = K; a.nesterov = nesterov ? 1 : 0; a.steps = steps;
    a.mu = mu; a.a = a_; a.b = b_; a.c = c_; a.eps = eps;
    a.out = out;
    a.ws = static_cast<uint8_t*>(ws);
    a.wait_limit_ns = mxw::host_wait_limit_ns();
    a.stall = mxw::host_take_stall();
    const cudaError_t e = mxw::device_status_address(a.dev, &a.status);
    if (e != cudaSuccess) return host_fail(MXFP8_ECUDA, "device status: %s", cudaGetErrorString(e));
    return small ? mxw::launch_muon_small(a) : mxw::launch_muon(a);
}

}  // namespace

extern "C" {

int mxfp8_moe_layer(const uint16_t* x, int T, const uint16_t* router, const float* bias, const uint8_t* w13,
                    const uint8_t* s13, const uint8_t* w2, const uint8_t* s2, int experts, int first, int local, int H,
                    int I, int top_k, int score, int renormalize, float scale, uint16_t* out, int32_t* topk_ids,
                    float* topk_weights, void* stream) {
    return moe(x, T, router, bias, w13, s13, w2, s2, experts, first, local, H, I, top_k, score, renormalize, scale, out,
               topk_ids, topk_weights, nullptr, 0, true, stream);
}

int mxfp8_moe_layer_ws(const uint16_t* x, int T, const uint16_t* router, const float* bias, const uint8_t* w13,
                       const uint8_t* s13, const uint8_t* w2, const uint8_t* s2, int experts, int first, int local,
                       int H, int I, int top_k, int score, int renormalize, float scale, uint16_t* out,
                       int32_t* topk_ids, float* topk_weights, void* workspace, size_t workspace_bytes, void* stream) {
    return moe(x, T, router, bias, w13, s13, w2, s2, experts, first, local, H, I, top_k, score, renormalize, scale, out,
               topk_ids, topk_weights, workspace, workspace_bytes, false, stream);
}

size_t mxfp8_moe_layer_workspace_bytes(int T, int experts, int local, int H, int I, int top_k) {
    if (!moe_sizes(T, experts, 0, local, H, I, top_k)) return 0;
    return mxw::moe_ws_bytes(T, experts, local, H, I, top_k, MAX_SMS);
}

int mxfp8_muon_update(const void* grad, int grad_type, float* momentum, int E, int N, int K, float mu, int nesterov,
                      int steps, float a, float b, float c, float eps, uint16_t* out, void* stream) {
    return muon(grad, grad_type, momentum, E, N, K, mu, nesterov, steps, a, b, c, eps, out, nullptr, 0, true, stream);
}

int mxfp8_muon_update_ws(const void* grad, int grad_type, float* momentum, int E, int N, int K, float mu, int nesterov,
                         int steps, float a, float b, float c, float eps, uint16_t* out, void* workspace,
                         size_t workspace_bytes, void* stream) {
    return muon(grad, grad_type, momentum, E, N, K, mu, nesterov, steps, a, b, c, eps, out, workspace, workspace_bytes,
                false, stream);
}

size_t mxfp8_muon_update_workspace_bytes(int E, int N, int K) {
    if (!muon_sizes(E, N, K) || E < 1 || (K % 8) != 0) return 0;
    return muon_need(E, N, K);
}

}  // extern "C"
