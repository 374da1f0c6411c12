// Global norm of many gradients and clipping (include/mxfp8_step.h).
//
// The tensors' bytes, cut into chunks of CHUNK bytes from the 16-byte boundary
// at or below each tensor's start, are one list that the CTAs share. A table of
// the tensors travels as a kernel parameter: nothing is copied to the device and
// a captured call keeps its own.
#include "mxw_internal.h"
#include "mxw_ptx.cuh"
#include "mxw_step.h"
#include "../../include/mxfp8_step.h"

namespace mxw {
namespace {

constexpr uint32_t FULL = 0xffffffffu;
constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int VECS = 8;                        // 16-byte vectors of a thread in a chunk
constexpr int CHUNK = THREADS * VECS * 16;     // bytes
constexpr int MAX_CTAS = 160 * 8;              // partial sums of one launch
constexpr int FEW = 64, MANY = 1024;           // tensors of one launch (parameters: 1.9 or 29.7 KB of 32)

template <int N>
struct Table {
    const void* in[N];
    void* out[N];
    int64_t bytes[N];
    uint32_t chunk0[N];  // first chunk of the tensor
    uint8_t f32[N];
    uint32_t chunks;
    int n;
};

// A thread's share of one chunk of a tensor: VECS vectors, some of which may
// reach over the tensor's ends.
struct Piece {
    const uint8_t *lo, *hi, *at;  // tensor's first and last byte + 1, the thread's first vector
    ptrdiff_t to_out;             // from an input's address to its output's
    bool f32;
};

template <int N>
__device__ __forceinline__ Piece piece(const Table<N>& t, uint32_t chunk) {
    int a = 0, b = t.n;  // the last tensor whose chunk0 is <= chunk (empty tensors share it with the next one)
    while (b - a > 1) {
        const int m = (a + b) / 2;
        if (t.chunk0[m] <= chunk) a = m; else b = m;
    }
    Piece p;
    p.lo = static_cast<const uint8_t*>(t.in[a]);
    p.hi = p.lo + t.bytes[a];
    const uint8_t* base = p.lo - (reinterpret_cast<uintptr_t>(p.lo) & 15);
    p.at = base + static_cast<int64_t>(chunk - t.chunk0[a]) * CHUNK + threadIdx.x * 16;
    p.to_out = static_cast<uint8_t*>(t.out[a]) - p.lo;
    p.f32 = t.f32[a] != 0;
    return p;
}

__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// The vector at `at`, with zeros for what lies outside the tensor.
__device__ __forceinline__ uint4 load_vector(const Piece& p, const uint8_t* at) {
    if (at >= p.lo && at + 16 <= p.hi) return load16(at);
    uint32_t w[4] = {0, 0, 0, 0};
    if (at < p.hi) {  // (a vector that starts below lo belongs to the tensor's first chunk and reaches into it)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t* e = at + 2 * i;  // (halves: elements are aligned to their size)
            if (e >= p.lo && e < p.hi) w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(e)) << (16 * (i & 1));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_vector(const Piece& p, const uint8_t* at, const uint4& v) {
    uint8_t* to = const_cast<uint8_t*>(at) + p.to_out;
    if (at >= p.lo && at + 16 <= p.hi && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
        *reinterpret_cast<uint4*>(to) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (at + 2 * i >= p.lo && at + 2 * i < p.hi)
            *reinterpret_cast<uint16_t*>(to + 2 * i) = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Sum of squares of a thread's vectors, in fp32 where that holds it to a few
// 2^-24: not near overflow, and so large that what underflow takes from a square
// (2^-150 at most) is nothing beside it. Elsewhere (and for NaN) the elements
// are summed again in 64 bits.
__device__ __forceinline__ double squares(const uint4 (&v)[VECS], bool f32) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            any |= w[j];
            if (f32) {
                const float x = __uint_as_float(w[j]);
                s[j] = fmaf(x, x, s[j]);
            } else {
                const float x = lo_bf16(w[j]), y = hi_bf16(w[j]);
                s[j] = fmaf(x, x, s[j]);
                s[j] = fmaf(y, y, s[j]);
            }
        }
    }
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (sum >= 0x1p-80f && sum <= 0x1p120f) return sum;
    if ((any & 0x7fff7fffu) == 0 && (!f32 || (any & 0x7fffffffu) == 0)) return 0.0;  // zeros of either sign
    double d = 0.0;
#pragma unroll 1
    for (int i = 0; i < VECS; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double x = f32 ? __uint_as_float(w[j]) : lo_bf16(w[j]), y = f32 ? 0.f : hi_bf16(w[j]);
            d += x * x + y * y;
        }
    }
    return d;
}

// The block's sum, in thread 0; fixed order.
__device__ __forceinline__ double block_sum(double d, double* part) {
#pragma unroll
    for (int i = 16; i; i /= 2) d += __shfl_down_sync(FULL, d, i);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
    __syncthreads();
    d = 0.0;
    if (threadIdx.x == 0)
#pragma unroll
        for (int i = 0; i < WARPS; ++i) d += part[i];
    return d;
}

template <int N>
__global__ void __launch_bounds__(THREADS) squares_kernel(const __grid_constant__ Table<N> t, double* partial) {
    __shared__ double part[WARPS];
    griddep_launch_dependents();
    griddep_wait();
    double d = 0.0;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Piece p = piece(t, c);
        uint4 v[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i) v[i] = load_vector(p, p.at + i * (THREADS * 16));
        d += squares(v, p.f32);
    }
    d = block_sum(d, part);
    if (threadIdx.x == 0) partial[blockIdx.x] = d;
}

struct Total {
    const double* partial;  // of `count` CTAs
    int count;
    const float* norm_in;   // or the norm itself
    float* norm;            // receives it (or nullptr)
    float max_norm, eps;
};

// sqrt of the sum of the partial sums, the same in every thread and CTA.
__device__ __forceinline__ double global_norm(const Total& t, double* part) {
    if (t.norm_in) return *t.norm_in;
    double d = 0.0;
    for (int i = threadIdx.x; i < t.count; i += THREADS) d += t.partial[i];
    d = block_sum(d, part);
    if (threadIdx.x == 0) part[0] = d;
    __syncthreads();
    return sqrt(part[0]);
}

__global__ void __launch_bounds__(THREADS) norm_kernel(const Total t) {
    __shared__ double part[WARPS];
    griddep_launch_dependents();
    griddep_wait();
    const double norm = global_norm(t, part);
    if (threadIdx.x == 0) *t.norm = static_cast<float>(norm);
}

template <int N>
__global__ void __launch_bounds__(THREADS) scale_kernel(const __grid_constant__ Table<N> t, const Total total, int in_place) {
    __shared__ double part[WARPS];
    griddep_launch_dependents();
    griddep_wait();
    const double norm = global_norm(total, part);
    if (total.norm && blockIdx.x == 0 && threadIdx.x == 0) *total.norm = static_cast<float>(norm);
    double c = total.max_norm / (norm + total.eps);
    if (c >= 1.0) c = 1.0;  // (a NaN stays one)
    if (c == 1.0 && in_place) return;
    // two factors where fp32 would hold the one with fewer bits
    const float second = c < 0x1p-100 ? 0x1p-100f : 1.f;
    const float first = static_cast<float>(c / second);
    for (uint32_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
        const Piece p = piece(t, chunk);
        uint4 v[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i) v[i] = load_vector(p, p.at + i * (THREADS * 16));
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = p.f32 ? __float_as_uint(__uint_as_float(w[j]) * first * second)
                             : pack_bf16x2(__float_as_uint(lo_bf16(w[j]) * first * second),
                                           __float_as_uint(hi_bf16(w[j]) * first * second));
            store_vector(p, p.at + i * (THREADS * 16), make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

int failed(cudaError_t e, const char* what) {
    return host_fail(MXFP8_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

template <class... Par, class... Arg>
cudaError_t start(void (*kernel)(Par...), unsigned ctas, cudaStream_t stream, const Arg&... arg) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, arg...);
}

// The tensors from `from` on that fit one table.
template <int N>
void fill(Table<N>& t, const GradArgs& a, int from) {
    t.n = a.n - from < N ? a.n - from : N;
    uint32_t chunks = 0;
    for (int i = 0; i < t.n; ++i) {
        const int g = from + i;
        t.in[i] = a.grads[g];
        t.out[i] = a.outs ? a.outs[g] : const_cast<void*>(a.grads[g]);
        t.f32[i] = a.types[g] == MXFP8_GRAD_F32;
        t.bytes[i] = a.sizes[g] * (t.f32[i] ? 4 : 2);
        t.chunk0[i] = chunks;
        if (t.bytes[i]) chunks += static_cast<uint32_t>((t.bytes[i] + (reinterpret_cast<uintptr_t>(t.in[i]) & 15) + CHUNK - 1) / CHUNK);
    }
    t.chunks = chunks;
}

int ctas_for(uint32_t chunks, int sms) {
    const int most = sms * 8 < MAX_CTAS ? sms * 8 : MAX_CTAS;
    return chunks < static_cast<uint32_t>(most) ? static_cast<int>(chunks) : most;
}

template <int N>
int run(const GradArgs& a) {
    Table<N> t;
    int count = 0;  // partial sums so far
    cudaError_t e = cudaSuccess;
    if (!a.norm_in)
        for (int from = 0; from < a.n; from += N) {
            fill(t, a, from);
            if (t.chunks == 0) continue;
            const int ctas = ctas_for(t.chunks, a.num_sms);
            e = start(squares_kernel<N>, ctas, a.stream, t, a.ws + count);
            if (e != cudaSuccess) return failed(e, "sum of squares kernel");
            count += ctas;
        }
    Total total{a.ws, count, a.norm_in, a.norm_in ? nullptr : a.norm, a.max_norm, a.eps};
    if (a.clip)
        for (int from = 0; from < a.n; from += N) {
            if (a.n > N || a.norm_in) fill(t, a, from);
            if (t.chunks == 0) continue;
            e = start(scale_kernel<N>, ctas_for(t.chunks, a.num_sms), a.stream, t, total, a.outs ? 0 : 1);
            if (e != cudaSuccess) return failed(e, "scaling kernel");
            total.norm = nullptr;  // (written once)
        }
    if (total.norm) {
        e = start(norm_kernel, 1, a.stream, total);
        if (e != cudaSuccess) return failed(e, "norm kernel");
    }
    return MXFP8_OK;
}

}  // namespace

size_t grad_ws_bytes(int n) {
    const size_t launches = n <= FEW ? 1 : (static_cast<size_t>(n) + MANY - 1) / MANY;
    return launches * MAX_CTAS * sizeof(double);
}

int launch_grads(const GradArgs& a) { return a.n <= FEW ? run<FEW>(a) : run<MANY>(a); }

}  // namespace mxw
