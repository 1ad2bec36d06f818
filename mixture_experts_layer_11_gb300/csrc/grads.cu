// grads.cu -- the global norm of a list of gradients, and clipping by it.
//
//   N = sqrt(sum_i sum_j g_i[j]^2),   out_i = g_i * min(1, max_norm / N)
//
// Two passes over the list, one launch each (per kGradTable tensors): sums of
// squares, one partial per block; then every block adds the partials (in index
// order, so the norm does not depend on timing) and scales its chunks.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGradThreads = 512;
constexpr int kGradChunk = 16384;      // elements of one unit of work
constexpr int kGradTable = 128;        // tensors one launch takes
constexpr int kGradBlocksPerSm = 4;    // 2048 threads

// The tensors of one launch, in its parameters.  Tensor i's chunks are
// [first[i], first[i+1]).  Its chunk boundaries lie kGradChunk elements apart
// counted from the 16-byte boundary at or before the source, so that every
// chunk but the first starts aligned wherever the tensor starts.
struct GradTable {
    const void* src[kGradTable];
    void* dst[kGradTable];
    int64_t n[kGradTable];
    int64_t first[kGradTable + 1];
    uint8_t bf16[kGradTable];
    int count;
};

struct Chunk {
    const void* src;
    void* dst;
    int n;       // elements
    bool bf16;
};

__device__ __forceinline__ Chunk find_chunk(const GradTable& t, int64_t c) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (t.first[m] <= c) lo = m; else hi = m;
    }
    const int es = t.bf16[lo] ? 2 : 4;
    const int skew = (int)((reinterpret_cast<uintptr_t>(t.src[lo]) & 15) / es);
    int64_t a = (c - t.first[lo]) * kGradChunk - skew, b = a + kGradChunk;
    if (a < 0) a = 0;
    if (b > t.n[lo]) b = t.n[lo];
    return {(const uint8_t*)t.src[lo] + a * es, (uint8_t*)t.dst[lo] + a * es, (int)(b - a),
            t.bf16[lo] != 0};
}

// Sum of squares over the whole range of fp32 inputs: values whose squares
// leave fp32's range are scaled by a power of two first and kept in sums of
// their own.  A group of values goes by its largest magnitude: what the others
// lose then is below 2^-40 of that value's square.
struct SquareSum {
    float mid = 0.f, low = 0.f, high = 0.f;
    double total = 0.0;
    template <int N> __device__ __forceinline__ void add(const float (&v)[N]) {
        float m = 0.f;
        #pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));   // NaN: not seen here
        if (m > 0x1p56f) {
            #pragma unroll
            for (int i = 0; i < N; ++i) { const float s = v[i] * 0x1p-80f; high = fmaf(s, s, high); }
        } else if (m < 0x1p-40f && m > 0.f) {
            #pragma unroll
            for (int i = 0; i < N; ++i) { const float s = v[i] * 0x1p80f; low = fmaf(s, s, low); }
        } else {
            #pragma unroll
            for (int i = 0; i < N; ++i) mid = fmaf(v[i], v[i], mid);
        }
    }
    // into 64 bits, after each chunk (at most 48 values a thread)
    __device__ __forceinline__ void flush() {
        total += (double)mid;
        if (low != 0.f) total += (double)low * 0x1p-160;
        if (high != 0.f) total += (double)high * 0x1p160;
        mid = low = high = 0.f;
    }
};

template <typename T> struct Vec;   // 16 bytes of T as floats
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t w[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// elements before the first 16-byte boundary of a chunk
template <typename T> __device__ __forceinline__ int head_of(const void* p, int n) {
    const int h = (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
    return h < n ? h : n;
}

template <typename T>
__device__ __forceinline__ void square_chunk(const Chunk& c, SquareSum& sum) {
    constexpr int N = Vec<T>::N;
    const T* p = (const T*)c.src;
    const int head = head_of<T>(p, c.n);
    const int nv = (c.n - head) / N;
    const uint4* q = (const uint4*)(p + head);
    constexpr int U = kGradChunk / N / kGradThreads;   // vectors a thread of a full chunk
    if (nv == U * kGradThreads) {
        uint4 u[U];
        #pragma unroll
        for (int i = 0; i < U; ++i) u[i] = __ldg(q + threadIdx.x + i * kGradThreads);
        #pragma unroll
        for (int i = 0; i < U; ++i) {
            float v[N];
            Vec<T>::unpack(u[i], v);
            sum.add(v);
        }
    } else {
        for (int i = threadIdx.x; i < nv; i += kGradThreads) {
            float v[N];
            Vec<T>::unpack(__ldg(q + i), v);
            sum.add(v);
        }
    }
    const int rest = c.n - nv * N;   // head and tail, fewer than 2 N
    if ((int)threadIdx.x < rest) {
        const int i = (int)threadIdx.x < head ? (int)threadIdx.x : nv * N + (int)threadIdx.x;
        const float v[1] = {to_f32<T>(p[i])};
        sum.add(v);
    }
    sum.flush();
}

// sum over the block, the same on every thread
__device__ __forceinline__ double block_sum(double v, double* buf) {
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    #pragma unroll
    for (int i = 0; i < kGradThreads / 32; ++i) s += buf[i];
    return s;
}

__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm)
    grad_square_kernel(const __grid_constant__ GradTable t, double* __restrict__ partial) {
    __shared__ double buf[kGradThreads / 32];
    SquareSum sum;
    const int64_t chunks = t.first[t.count];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Chunk k = find_chunk(t, c);
        if (k.bf16) square_chunk<__nv_bfloat16>(k, sum);
        else square_chunk<float>(k, sum);
    }
    const double s = block_sum(sum.total, buf);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// the norm from the partials; block 0 of a call's first launch writes it down
__device__ __forceinline__ float finish_norm(const double* partial, int np, double* buf,
                                             float* norm, int32_t* status, bool writer) {
    double s = 0.0;
    for (int i = threadIdx.x; i < np; i += kGradThreads) s += partial[i];
    const float n = (float)sqrt(block_sum(s, buf));
    if (writer && threadIdx.x == 0) {
        *norm = n;
        if (!isfinite(n)) report(status, MOE_ERR_NONFINITE);
    }
    return n;
}

__global__ void __launch_bounds__(kGradThreads)
    grad_norm_kernel(const double* __restrict__ partial, int np, float* norm, int32_t* status) {
    __shared__ double buf[kGradThreads / 32];
    finish_norm(partial, np, buf, norm, status, true);
}

template <typename T> __device__ __forceinline__ void scale_chunk(const Chunk& c, float f) {
    constexpr int N = Vec<T>::N;
    const T* p = (const T*)c.src;
    T* o = (T*)c.dst;
    const int head = head_of<T>(p, c.n);
    const bool vec = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    if (!vec) {   // the two sides never meet a 16-byte boundary together
        for (int i = threadIdx.x; i < c.n; i += kGradThreads) o[i] = from_f32<T>(to_f32<T>(p[i]) * f);
        return;
    }
    const int nv = (c.n - head) / N;
    const uint4* q = (const uint4*)(p + head);
    uint4* r = (uint4*)(o + head);
    constexpr int U = kGradChunk / N / kGradThreads;
    auto scaled = [&](uint4 u) {
        float v[N];
        Vec<T>::unpack(u, v);
        #pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= f;
        return Vec<T>::pack(v);
    };
    if (nv == U * kGradThreads) {
        uint4 u[U];
        #pragma unroll
        for (int i = 0; i < U; ++i) u[i] = q[threadIdx.x + i * kGradThreads];
        #pragma unroll
        for (int i = 0; i < U; ++i) r[threadIdx.x + i * kGradThreads] = scaled(u[i]);
    } else {
        for (int i = threadIdx.x; i < nv; i += kGradThreads) r[i] = scaled(q[i]);
    }
    const int rest = c.n - nv * N;
    if ((int)threadIdx.x < rest) {
        const int i = (int)threadIdx.x < head ? (int)threadIdx.x : nv * N + (int)threadIdx.x;
        o[i] = from_f32<T>(to_f32<T>(p[i]) * f);
    }
}

__global__ void __launch_bounds__(kGradThreads)
    grad_scale_kernel(const __grid_constant__ GradTable t, const double* __restrict__ partial,
                      int np, float max_norm, float* norm, int first_launch, int32_t* status) {
    __shared__ double buf[kGradThreads / 32];
    const float n = finish_norm(partial, np, buf, norm, status, first_launch && blockIdx.x == 0);
    // a norm within the bound, or none (infinite, NaN): the gradients as they are
    const float f = isfinite(n) && n > max_norm ? max_norm / n : 1.f;
    const int64_t chunks = t.first[t.count];
    for (int64_t c = chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const Chunk k = find_chunk(t, c);
        if (f == 1.f && k.src == k.dst) continue;
        if (k.bf16) scale_chunk<__nv_bfloat16>(k, f);
        else scale_chunk<float>(k, f);
    }
}

int grad_blocks(int64_t chunks) {
    const int64_t most = (int64_t)device_sm_count() * kGradBlocksPerSm;
    return (int)(chunks < most ? (chunks > 0 ? chunks : 1) : most);
}

// tensors [from, from + kGradTable) of the list
GradTable make_table(const moe_grad* g, int from, int n) {
    GradTable t;
    t.count = n - from < kGradTable ? n - from : kGradTable;
    int64_t c = 0;
    for (int i = 0; i < t.count; ++i) {
        const moe_grad& x = g[from + i];
        const bool half = x.dtype == MOE_BF16;
        const int64_t skew = (int64_t)((reinterpret_cast<uintptr_t>(x.grad) & 15) / (half ? 2 : 4));
        t.src[i] = x.grad;
        t.dst[i] = x.out ? x.out : const_cast<void*>(x.grad);
        t.n[i] = x.n;
        t.bf16[i] = half;
        t.first[i] = c;
        c += x.n ? (x.n + skew + kGradChunk - 1) / kGradChunk : 0;
    }
    t.first[t.count] = c;
    return t;
}

}  // namespace

size_t grad_workspace(int n) {
    const int launches = n > 0 ? (n + kGradTable - 1) / kGradTable : 1;
    return (size_t)launches * device_sm_count() * kGradBlocksPerSm * sizeof(double);
}

cudaError_t launch_grad_norm(int n, const moe_grad* g, bool clip, float max_norm, float* norm,
                             void* ws, int32_t* status, cudaStream_t st) {
    double* partial = (double*)ws;
    int np = 0;
    for (int i = 0; i < n; i += kGradTable) {
        const GradTable t = make_table(g, i, n);
        const int blocks = grad_blocks(t.first[t.count]);
        grad_square_kernel<<<blocks, kGradThreads, 0, st>>>(t, partial + np);
        np += blocks;
    }
    if (!clip || n == 0) {
        grad_norm_kernel<<<1, kGradThreads, 0, st>>>(partial, np, norm, status);
        return cudaGetLastError();
    }
    for (int i = 0; i < n; i += kGradTable) {
        const GradTable t = make_table(g, i, n);
        grad_scale_kernel<<<grad_blocks(t.first[t.count]), kGradThreads, 0, st>>>(
            t, partial, np, max_norm, norm, i == 0, status);
    }
    return cudaGetLastError();
}

}  // namespace moe
