// Entry points of include/mxfp8_step.h: argument checks, scratch, launch.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "mxw_internal.h"
#include "mxw_step.h"
#include "../../include/mxfp8_step.h"

namespace {

using mxw::host_fail;

constexpr int MAX_H = 32768;
constexpr int64_t MAX_ELEMENTS = int64_t(1) << 42;  // of one call: no device holds as many
constexpr int64_t MAX_ROWS = (int64_t(1) << 31) - 1;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

bool routing(int64_t T, int top_k) {
    return T >= 0 && top_k >= 1 && top_k <= MXFP8_TOKENS_MAX_TOPK && T <= MXFP8_TOKENS_MAX_PAIRS / top_k;
}

int bad_routing(int64_t T, int top_k) {
    return host_fail(MXFP8_EINVAL, "unsupported sizes T=%lld top_k=%d (T >= 0, top_k in [1, %d], at most %d pairs)",
                     static_cast<long long>(T), top_k, MXFP8_TOKENS_MAX_TOPK, MXFP8_TOKENS_MAX_PAIRS);
}

// Checks what the row operators have in common and fills `a`.
int token_args(mxw::TokenArgs& a, int64_t T, int64_t rows, int H, int top_k, int unit, const int32_t* slot,
               const int32_t* src, bool needs_src, void* stream) {
    if (!routing(T, top_k)) return bad_routing(T, top_k);
    if (rows < 0 || rows > MAX_ROWS) return host_fail(MXFP8_EINVAL, "rows=%lld out of range", static_cast<long long>(rows));
    if (H < 1 || H > MAX_H) return host_fail(MXFP8_EINVAL, "H=%d out of range [1, %d]", H, MAX_H);
    if (T > (MAX_ELEMENTS >> 2) / H || rows > (MAX_ELEMENTS >> 2) / H)
        return host_fail(MXFP8_EINVAL, "T=%lld or rows=%lld of H=%d columns are more than any device holds", static_cast<long long>(T),
                         static_cast<long long>(rows), H);
    if (H % unit) return host_fail(unit == 32 ? MXFP8_EINVAL : MXFP8_EALIGN, "H=%d must be a multiple of %d", H, unit);
    if ((T && !slot) || (needs_src && rows && !src)) return host_fail(MXFP8_EINVAL, "null plan");
    if (misaligned(slot, 4) || misaligned(src, 4)) return host_fail(MXFP8_EALIGN, "slot and src must be 4-byte aligned");
    a.T = T; a.rows = rows; a.H = H; a.top_k = top_k; a.slot = slot; a.src = src;
    a.stream = static_cast<cudaStream_t>(stream);
    return MXFP8_OK;
}

// A buffer of n elements: null only where it is empty.
int buffer(const void* p, int64_t n, uintptr_t align, const char* name) {
    if (n && !p) return host_fail(MXFP8_EINVAL, "null %s", name);
    if (misaligned(p, align)) return host_fail(MXFP8_EALIGN, "%s must be %d-byte aligned", name, static_cast<int>(align));
    return MXFP8_OK;
}

int device(int* dev, int* sms, int** status) {
    const int rc = mxw::host_device(dev, sms);
    if (rc) return rc;
    const cudaError_t e = mxw::device_status_address(*dev, status);
    return e == cudaSuccess ? MXFP8_OK : host_fail(MXFP8_ECUDA, "device status: %s", cudaGetErrorString(e));
}

// Whether an output overlaps another output, or a gradient other than its own
// (which it may equal).
struct Span {
    uintptr_t lo, hi;
    int i;
    bool out;
};

bool overlapping(const void* const* grads, const int64_t* sizes, const int32_t* types, int n, void* const* outs, bool* memory) {
    std::unique_ptr<Span[]> s(new (std::nothrow) Span[2 * static_cast<size_t>(n)]);
    *memory = s != nullptr;
    if (!s) return false;
    size_t m = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t bytes = sizes[i] * (types[i] == MXFP8_GRAD_F32 ? 4 : 2);
        if (!bytes) continue;
        const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = outs ? reinterpret_cast<uintptr_t>(outs[i]) : g;
        s[m++] = {o, o + bytes, i, true};
        if (o != g) s[m++] = {g, g + bytes, i, false};
    }
    const auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    if (!std::is_sorted(s.get(), s.get() + m, before)) std::sort(s.get(), s.get() + m, before);
    uintptr_t outs_end = 0, all_end = 0;  // ends of the spans so far
    for (size_t k = 0; k < m; ++k) {
        if (s[k].lo < (s[k].out ? all_end : outs_end)) return true;
        all_end = std::max(all_end, s[k].hi);
        if (s[k].out) outs_end = std::max(outs_end, s[k].hi);
    }
    return false;
}

int grads(const void* const* g, const int64_t* sizes, const int32_t* types, int n, bool clip, float max_norm, float eps,
          const float* norm_in, float* norm, void* const* outs, void* ws, size_t ws_bytes, bool use_cache, void* stream) {
    if (n < 0 || n > MXFP8_GRAD_MAX_TENSORS) return host_fail(MXFP8_EINVAL, "n=%d out of range [0, %d]", n, MXFP8_GRAD_MAX_TENSORS);
    if (n && (!g || !sizes || !types)) return host_fail(MXFP8_EINVAL, "null array");
    if (!clip && !norm) return host_fail(MXFP8_EINVAL, "null norm");
    if (clip && !(max_norm >= 0.f && std::isfinite(max_norm) && eps >= 0.f && std::isfinite(eps)))
        return host_fail(MXFP8_EINVAL, "max_norm=%g and eps=%g must be finite and >= 0", max_norm, eps);
    if (norm_in && norm && norm != norm_in) return host_fail(MXFP8_EINVAL, "norm must be NULL or norm_in where norm_in is given");
    if (misaligned(norm, 4) || misaligned(norm_in, 4)) return host_fail(MXFP8_EALIGN, "norm must be 4-byte aligned");
    int64_t bytes = 0;
    for (int i = 0; i < n; ++i) {
        if (types[i] != MXFP8_GRAD_BF16 && types[i] != MXFP8_GRAD_F32)
            return host_fail(MXFP8_EINVAL, "types[%d]=%d: 0 (bf16) or 1 (fp32)", i, types[i]);
        const int item = types[i] == MXFP8_GRAD_F32 ? 4 : 2;
        if (sizes[i] < 0 || sizes[i] > MAX_ELEMENTS || (bytes += sizes[i] * item) > 4 * MAX_ELEMENTS)
            return host_fail(MXFP8_EINVAL, "sizes[%d]=%lld out of range", i, static_cast<long long>(sizes[i]));
        if (sizes[i] && (!g[i] || (outs && !outs[i]))) return host_fail(MXFP8_EINVAL, "null tensor %d", i);
        if (sizes[i] && (misaligned(g[i], item) || (outs && misaligned(outs[i], item))))
            return host_fail(MXFP8_EALIGN, "tensor %d is not aligned to its elements", i);
    }
    if (clip) {
        bool memory;
        if (overlapping(g, sizes, types, n, outs, &memory)) return host_fail(MXFP8_EINVAL, "an output overlaps another output or gradient");
        if (!memory) return host_fail(MXFP8_ECUDA, "no host memory for the list of tensors");
    }
    const size_t need = mxw::grad_ws_bytes(n);
    if (!use_cache) {
        if (!ws) return host_fail(MXFP8_EINVAL, "null workspace");
        if (misaligned(ws, 256)) return host_fail(MXFP8_EALIGN, "workspace must be 256-byte aligned");
        if (ws_bytes < need) return host_fail(MXFP8_ENOWS, "workspace of %zu bytes, need %zu", ws_bytes, need);
    }
    int dev;
    mxw::GradArgs a{};
    int rc = mxw::host_device(&dev, &a.num_sms);
    if (rc) return rc;
    a.stream = static_cast<cudaStream_t>(stream);
    mxw::LaunchLock launches;
    if (use_cache) {
        rc = mxw::host_workspace(dev, a.stream, need, &ws, &launches);
        if (rc) return rc;
    }
    a.grads = g; a.sizes = sizes; a.types = types; a.outs = outs; a.n = n;
    a.clip = clip; a.max_norm = max_norm; a.eps = eps; a.norm_in = norm_in; a.norm = norm;
    a.ws = static_cast<double*>(ws);
    return mxw::launch_grads(a);
}

}  // namespace

extern "C" {

int64_t mxfp8_token_plan_rows(int64_t T, int top_k, int local, int align) {
    if (!routing(T, top_k) || local < 1 || local > MXFP8_MAX_EXPERTS || align < 1 || align > MXFP8_TOKENS_MAX_ALIGN) return -1;
    const int64_t pairs = T * top_k, used = pairs < local ? pairs : local;
    const int64_t rows = (pairs + used * (align - 1)) / align * align;
    return rows <= MAX_ROWS ? rows : -1;
}

int mxfp8_token_plan(const void* ids, int id_type, int64_t T, int top_k, int first, int local, int align, int64_t rows,
                     int32_t* offs, int32_t* slot, int32_t* src, void* stream) {
    if (!routing(T, top_k)) return bad_routing(T, top_k);
    if (id_type != MXFP8_ID_I32 && id_type != MXFP8_ID_I64) return host_fail(MXFP8_EINVAL, "id_type=%d: 0 (int32) or 1 (int64)", id_type);
    if (first < 0 || local < 1 || local > MXFP8_MAX_EXPERTS || align < 1 || align > MXFP8_TOKENS_MAX_ALIGN)
        return host_fail(MXFP8_EINVAL, "unsupported first=%d local=%d align=%d (local in [1, %d], align in [1, %d])", first, local, align,
                         MXFP8_MAX_EXPERTS, MXFP8_TOKENS_MAX_ALIGN);
    if (rows < 0 || rows > MAX_ROWS || rows % align)
        return host_fail(MXFP8_EINVAL, "rows=%lld: a multiple of align=%d below 2^31", static_cast<long long>(rows), align);
    int rc = buffer(ids, T, id_type == MXFP8_ID_I64 ? 8 : 4, "ids");
    if (!rc) rc = buffer(offs, local, 4, "offs");
    if (!rc) rc = buffer(slot, T, 4, "slot");
    if (!rc) rc = buffer(src, rows, 4, "src");
    int sms;
    mxw::TokenPlanArgs a{};
    if (!rc) rc = device(&a.dev, &sms, &a.status);
    if (rc) return rc;
    a.ids = ids; a.id64 = id_type == MXFP8_ID_I64; a.first = first; a.local = local; a.align = align;
    a.pairs = T * top_k; a.rows = rows; a.offs = offs; a.slot = slot; a.src = src;
    a.stream = static_cast<cudaStream_t>(stream);
    return mxw::launch_token_plan(a);
}

int mxfp8_token_dispatch(const uint16_t* x, int64_t T, int H, int top_k, const int32_t* slot, const int32_t* src,
                         int64_t rows, uint16_t* out, void* stream) {
    mxw::TokenArgs a{};
    int dev;
    int rc = token_args(a, T, rows, H, top_k, 8, slot, src, true, stream);
    if (!rc) rc = buffer(x, T, 16, "x");
    if (!rc) rc = buffer(out, rows, 16, "out");
    if (!rc) rc = device(&dev, &a.num_sms, &a.status);
    if (rc) return rc;
    a.tok_in = x; a.sorted_out = out;
    return mxw::launch_token_dispatch(a);
}

int mxfp8_token_dispatch_mxfp8(const uint16_t* x, int64_t T, int H, int top_k, const int32_t* slot, const int32_t* src,
                               int64_t rows, uint8_t* q, uint8_t* s, void* stream) {
    mxw::TokenArgs a{};
    int dev;
    int rc = token_args(a, T, rows, H, top_k, 32, slot, src, true, stream);
    if (!rc) rc = buffer(x, T, 16, "x");
    if (!rc) rc = buffer(q, rows, 16, "q");
    if (!rc) rc = buffer(s, rows, 1, "s");
    if (!rc) rc = device(&dev, &a.num_sms, &a.status);
    if (rc || rows == 0) return rc;
    a.tok_in = x; a.q = q; a.s = s;
    return mxw::launch_token_dispatch(a);
}

int mxfp8_token_dispatch_grad(const uint16_t* dxs, int64_t rows, int64_t T, int H, int top_k, const int32_t* slot,
                              uint16_t* dx, void* stream) {
    mxw::TokenArgs a{};
    int dev;
    int rc = token_args(a, T, rows, H, top_k, 8, slot, nullptr, false, stream);
    if (!rc) rc = buffer(dxs, rows, 16, "dxs");
    if (!rc) rc = buffer(dx, T, 16, "dx");
    if (!rc) rc = device(&dev, &a.num_sms, &a.status);
    if (rc) return rc;
    a.sorted_in = dxs; a.tok_out = dx;
    return mxw::launch_token_combine(a);
}

int mxfp8_token_combine(const uint16_t* y, int64_t rows, const float* weights, int64_t T, int H, int top_k,
                        const int32_t* slot, uint16_t* out, void* stream) {
    mxw::TokenArgs a{};
    int dev;
    int rc = token_args(a, T, rows, H, top_k, 8, slot, nullptr, false, stream);
    if (!rc) rc = buffer(y, rows, 16, "y");
    if (!rc) rc = buffer(weights, T, 4, "weights");
    if (!rc) rc = buffer(out, T, 16, "out");
    if (!rc) rc = device(&dev, &a.num_sms, &a.status);
    if (rc || T == 0) return rc;
    a.sorted_in = y; a.weights = weights; a.tok_out = out;
    return mxw::launch_token_combine(a);
}

int mxfp8_token_combine_grad(const uint16_t* dout, const uint16_t* y, const float* weights, int64_t T, int H, int top_k,
                             const int32_t* slot, const int32_t* src, int64_t rows, uint16_t* dy, float* dweights,
                             void* stream) {
    mxw::TokenArgs a{};
    int dev;
    int rc = token_args(a, T, rows, H, top_k, 8, slot, src, true, stream);
    if (!rc) rc = buffer(dout, T, 16, "dout");
    if (!rc) rc = buffer(y, rows, 16, "y");
    if (!rc) rc = buffer(weights, T, 4, "weights");
    if (!rc) rc = buffer(dy, rows, 16, "dy");
    if (!rc) rc = buffer(dweights, T, 4, "dweights");
    if (!rc) rc = device(&dev, &a.num_sms, &a.status);
    if (rc) return rc;
    a.tok_in = dout; a.sorted_in = y; a.weights = weights; a.sorted_out = dy; a.dweights = dweights;
    return mxw::launch_token_combine_grad(a);
}

size_t mxfp8_grad_workspace_bytes(int n) { return n < 0 || n > MXFP8_GRAD_MAX_TENSORS ? 0 : mxw::grad_ws_bytes(n); }

int mxfp8_grad_norm(const void* const* g, const int64_t* sizes, const int32_t* types, int n, float* norm, void* stream) {
    return grads(g, sizes, types, n, false, 0.f, 0.f, nullptr, norm, nullptr, nullptr, 0, true, stream);
}

int mxfp8_grad_norm_ws(const void* const* g, const int64_t* sizes, const int32_t* types, int n, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream) {
    return grads(g, sizes, types, n, false, 0.f, 0.f, nullptr, norm, nullptr, workspace, workspace_bytes, false, stream);
}

int mxfp8_clip_grads(const void* const* g, const int64_t* sizes, const int32_t* types, int n, float max_norm,
                     float eps, const float* norm_in, float* norm, void* const* outs, void* stream) {
    return grads(g, sizes, types, n, true, max_norm, eps, norm_in, norm, outs, nullptr, 0, true, stream);
}

int mxfp8_clip_grads_ws(const void* const* g, const int64_t* sizes, const int32_t* types, int n, float max_norm,
                        float eps, const float* norm_in, float* norm, void* const* outs, void* workspace,
                        size_t workspace_bytes, void* stream) {
    return grads(g, sizes, types, n, true, max_norm, eps, norm_in, norm, outs, workspace, workspace_bytes, false, stream);
}

}  // extern "C"
