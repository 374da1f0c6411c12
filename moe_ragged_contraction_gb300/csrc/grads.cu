// Global norm of many gradients and clipping (include/mxfp8_step.h).
//
// The tensors' bytes, cut into chunks of CHUNK bytes from the 16-byte boundary
// at or below the start of what is written (of what is read, where nothing is),
// are one list that the CTAs share. A table of the tensors travels as a kernel
// parameter: nothing is copied to the device and a captured call keeps its own.
// Where outputs lie otherwise than their inputs the stores are the whole vectors
// and the loads the pieces (15.9M fp32 elements in views of one buffer to tensors of
// their own: 40 us, with the loads whole 95).
//
// Bound by DRAM. 416M bf16 elements: sum 119 us (7.0 TB/s), scaled beside them 253
// more (6.6 TB/s); in place within the limit 5 more.
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
constexpr int SUM_CTAS = 4, SCALE_CTAS = 5;    // resident on an SM
constexpr int MAX_CTAS = 160 * SUM_CTAS;       // partial sums of one launch
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
    ptrdiff_t to_out;             // from an input's address to its output's: there vectors are aligned
    bool f32;
    bool whole;                   // all of the chunk's vectors, and 2 bytes around, lie inside the tensor
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
    const uint8_t* begin = p.lo - (reinterpret_cast<uintptr_t>(t.out[a]) & 15) + static_cast<int64_t>(chunk - t.chunk0[a]) * CHUNK;
    p.at = begin + threadIdx.x * 16;
    p.to_out = static_cast<uint8_t*>(t.out[a]) - p.lo;
    p.f32 = t.f32[a] != 0;
    p.whole = begin >= p.lo + 2 && begin + CHUNK + 2 <= p.hi;
    return p;
}

__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// 16 bytes at an address of lower alignment. (What two threads read is in L1.)
template <class T>
__device__ __forceinline__ uint4 load16_by(const uint8_t* p) {
    uint4 v;
    T* w = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i) w[i] = reinterpret_cast<const T*>(p)[i];
    return v;
}

// The same at an odd number of halves, from the five words around.
__device__ __forceinline__ uint4 load16_halves(const uint8_t* p) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p - 2);
    uint32_t x[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) x[i] = w[i];
    return make_uint4(__byte_perm(x[0], x[1], 0x5432), __byte_perm(x[1], x[2], 0x5432), __byte_perm(x[2], x[3], 0x5432), __byte_perm(x[3], x[4], 0x5432));
}

// The vector at `at`, element by element, with zeros for what lies outside the tensor.
__device__ __forceinline__ uint4 load_vector(const Piece& p, const uint8_t* at) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (at < p.hi && at + 16 > p.lo) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t* e = at + 2 * i;  // (halves: elements are aligned to their size)
            if (e >= p.lo && e < p.hi) w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(e)) << (16 * (i & 1));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ALIGNED: inputs lie like their outputs, vectors are aligned in both.
template <bool ALIGNED>
__device__ __forceinline__ void load_piece(const Piece& p, uint4 (&v)[VECS]) {
    constexpr int STEP = THREADS * 16;
    const int odd = ALIGNED ? 0 : static_cast<int>(p.to_out & 15);
    if (!p.whole) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const uint8_t* at = p.at + i * STEP;
            v[i] = odd == 0 && at >= p.lo && at + 16 <= p.hi ? load16(at) : load_vector(p, at);
        }
    } else if (odd == 0) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) v[i] = load16(p.at + i * STEP);
    } else if (odd == 8) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) v[i] = load16_by<uint2>(p.at + i * STEP);
    } else if ((odd & 3) == 0) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) v[i] = load16_by<uint32_t>(p.at + i * STEP);
    } else {
#pragma unroll
        for (int i = 0; i < VECS; ++i) v[i] = load16_halves(p.at + i * STEP);
    }
}

__device__ __forceinline__ void store_vector(const Piece& p, const uint8_t* at, const uint4& v) {
    uint8_t* to = const_cast<uint8_t*>(at) + p.to_out;
    if (p.whole || (at >= p.lo && at + 16 <= p.hi)) {
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
template <bool F32>
__device__ __forceinline__ float squares_fp32(const uint4 (&v)[VECS]) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = F32 ? __uint_as_float(w[j]) : lo_bf16(w[j]);
            s[j] = fmaf(x, x, s[j]);
            if (!F32) s[j] = fmaf(hi_bf16(w[j]), hi_bf16(w[j]), s[j]);
        }
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __noinline__ double squares_fp64(uint4 v, bool f32) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    double d = 0.0;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const double x = f32 ? __uint_as_float(w[j]) : lo_bf16(w[j]), y = f32 ? 0.f : hi_bf16(w[j]);
        d += x * x + y * y;
    }
    return d;
}

__device__ __forceinline__ double squares(const uint4 (&v)[VECS], bool f32) {
    const float sum = f32 ? squares_fp32<true>(v) : squares_fp32<false>(v);
    if (sum >= 0x1p-80f && sum <= 0x1p120f) return sum;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i) any |= v[i].x | v[i].y | v[i].z | v[i].w;
    if ((any & (f32 ? 0x7fffffffu : 0x7fff7fffu)) == 0) return 0.0;  // zeros of either sign
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < VECS; ++i) d += squares_fp64(v[i], f32);
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
__global__ void __launch_bounds__(THREADS, SUM_CTAS) squares_kernel(const __grid_constant__ Table<N> t, double* partial) {
    __shared__ double part[WARPS];
    griddep_launch_dependents();
    griddep_wait();
    double d = 0.0;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Piece p = piece(t, c);
        uint4 v[VECS];
        load_piece<true>(p, v);
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
    float2* factor;         // receives the factor (norm_kernel), or holds it (scale_kernel); nullptr: neither
};

// The factor min(1, max_norm / (norm + eps)) as a product of two: fp32 would hold
// a very small one with fewer bits.
__device__ __forceinline__ float2 clip_factor(const Total& t, double norm) {
    double c = t.max_norm / (norm + t.eps);
    if (c >= 1.0) c = 1.0;  // (a NaN stays one)
    const float second = c < 0x1p-100 ? 0x1p-100f : 1.f;
    return make_float2(static_cast<float>(c / second), second);
}

// The norm, from the partial sums or the caller, in thread 0.
__device__ __forceinline__ double global_norm(const Total& t, double* part) {
    if (t.norm_in) return *t.norm_in;
    double d = 0.0;
    for (int i = threadIdx.x; i < t.count; i += THREADS) d += t.partial[i];
    d = block_sum(d, part);
    return threadIdx.x == 0 ? sqrt(d) : 0.0;
}

__global__ void __launch_bounds__(THREADS) norm_kernel(const Total t) {
    __shared__ double part[WARPS];
    griddep_launch_dependents();
    griddep_wait();
    const double norm = global_norm(t, part);
    if (threadIdx.x) return;
    if (t.norm) *t.norm = static_cast<float>(norm);
    if (t.factor) *t.factor = clip_factor(t, norm);
}

template <bool F32>
__device__ __forceinline__ void scale_piece(const Piece& p, const uint4 (&v)[VECS], float first, float second) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = F32 ? __float_as_uint(__uint_as_float(w[j]) * first * second)
                       : pack_bf16x2(__float_as_uint(lo_bf16(w[j]) * first * second), __float_as_uint(hi_bf16(w[j]) * first * second));
        store_vector(p, p.at + i * (THREADS * 16), make_uint4(w[0], w[1], w[2], w[3]));
    }
}

template <int N>
__global__ void __launch_bounds__(THREADS, SCALE_CTAS) scale_kernel(const __grid_constant__ Table<N> t, const Total total, int in_place) {
    __shared__ double part[WARPS];
    __shared__ float2 factor;
    griddep_launch_dependents();
    griddep_wait();
    // (fp64 steps by one thread: a division by all took longer than the scaling)
    if (total.factor) {
        if (threadIdx.x == 0) factor = *total.factor;
    } else {
        const double norm = global_norm(total, part);
        if (threadIdx.x == 0) {
            factor = clip_factor(total, norm);
            if (total.norm && blockIdx.x == 0) *total.norm = static_cast<float>(norm);
        }
    }
    __syncthreads();
    const float2 f = factor;
    if (f.x == 1.f && f.y == 1.f && in_place) return;
    // (the last chunks first: the sum of squares has read them last)
    for (uint32_t k = blockIdx.x; k < t.chunks; k += gridDim.x) {
        const Piece p = piece(t, t.chunks - 1 - k);
        uint4 v[VECS];
        load_piece<false>(p, v);
        if (p.f32) scale_piece<true>(p, v, f.x, f.y); else scale_piece<false>(p, v, f.x, f.y);
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

// The tensors from `from` on that fit one table; outs: with their outputs.
template <int N>
void fill(Table<N>& t, const GradArgs& a, int from, bool outs) {
    t.n = a.n - from < N ? a.n - from : N;
    uint32_t chunks = 0;
    for (int i = 0; i < t.n; ++i) {
        const int g = from + i;
        t.in[i] = a.grads[g];
        t.out[i] = outs ? a.outs[g] : const_cast<void*>(a.grads[g]);
        t.f32[i] = a.types[g] == MXFP8_GRAD_F32;
        t.bytes[i] = a.sizes[g] * (t.f32[i] ? 4 : 2);
        t.chunk0[i] = chunks;
        if (t.bytes[i]) chunks += static_cast<uint32_t>((t.bytes[i] + (reinterpret_cast<uintptr_t>(t.out[i]) & 15) + CHUNK - 1) / CHUNK);
    }
    t.chunks = chunks;
}

int ctas_for(uint32_t chunks, int sms) {
    const int most = sms * SUM_CTAS < MAX_CTAS ? sms * SUM_CTAS : MAX_CTAS;
    return chunks < static_cast<uint32_t>(most) ? static_cast<int>(chunks) : most;
}

// Scaling, from MANY_CHUNKS an SM on: the norm is worked out once beforehand and
// two chunks are a CTA's; in place, where there is mostly nothing to scale, a
// grid of IN_PLACE_CTAS an SM ends sooner. With fewer chunks every CTA of a
// resident grid works the norm out: a launch less.
constexpr unsigned MANY_CHUNKS = 8, OUT_CHUNKS = 2, IN_PLACE_CTAS = 16;

template <int N>
int run(const GradArgs& a) {
    Table<N> t;
    t.n = 0;
    t.chunks = 0;
    int count = 0;  // partial sums so far
    cudaError_t e = cudaSuccess;
    if (!a.norm_in)
        for (int from = 0; from < a.n; from += N) {
            fill(t, a, from, false);
            if (t.chunks == 0) continue;
            const int ctas = ctas_for(t.chunks, a.num_sms);
            e = start(squares_kernel<N>, ctas, a.stream, t, a.ws + count);
            if (e != cudaSuccess) return failed(e, "sum of squares kernel");
            count += ctas;
        }
    Total total{a.ws, count, a.norm_in, a.norm_in ? nullptr : a.norm, a.max_norm, a.eps, nullptr};
    uint64_t chunks = 0;
    if (a.clip)
        for (int from = 0; from < a.n; from += N) {
            fill(t, a, from, a.outs != nullptr);
            chunks += t.chunks;
        }
    const bool once = chunks > static_cast<uint64_t>(a.num_sms) * MANY_CHUNKS;
    if (once || (total.norm && (!a.clip || chunks == 0))) {
        if (a.clip) total.factor = reinterpret_cast<float2*>(a.ws + count);
        e = start(norm_kernel, 1, a.stream, total);
        if (e != cudaSuccess) return failed(e, "norm kernel");
        total.norm = nullptr;
    }
    if (a.clip)
        for (int from = 0; from < a.n; from += N) {
            if (a.n > N) fill(t, a, from, a.outs != nullptr);
            if (t.chunks == 0) continue;
            unsigned ctas = ctas_for(t.chunks, a.num_sms);
            if (once) ctas = a.outs ? (t.chunks + OUT_CHUNKS - 1) / OUT_CHUNKS : t.chunks < a.num_sms * IN_PLACE_CTAS ? t.chunks : a.num_sms * IN_PLACE_CTAS;
            e = start(scale_kernel<N>, ctas, a.stream, t, total, a.outs ? 0 : 1);
            if (e != cudaSuccess) return failed(e, "scaling kernel");
            total.norm = nullptr;  // (written once)
        }
    return MXFP8_OK;
}

}  // namespace

size_t grad_ws_bytes(int n) {
    const size_t launches = n <= FEW ? 1 : (static_cast<size_t>(n) + MANY - 1) / MANY;
    return (launches * MAX_CTAS + 1) * sizeof(double);  // (the partial sums, the norm)
}

int launch_grads(const GradArgs& a) { return a.n <= FEW ? run<FEW>(a) : run<MANY>(a); }

}  // namespace mxw
