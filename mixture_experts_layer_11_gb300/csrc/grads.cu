// grads.cu -- the global norm of a list of gradients, and clipping by it.
//
//   N = sqrt(sum_i sum_j g_i[j]^2),   out_i = g_i * min(1, max_norm / N)
//
// Memory bounds both passes over the list: sums of squares, one partial a block,
// added in index order (so that the norm does not depend on timing); then the
// scaling.  The second pass needs the first's result, so the gradients are read
// twice, except for what the L2 still holds.  Measured on a GB300 (device time in
// a graph): the norm of 537 M fp32 gradients 297 us, 7.2 TB/s; with clipping of
// 1.07 G into other buffers 1.82 ms (12.9 GB, 7.1 TB/s), of 38 M 70 us, of 211
// tensors of odd sizes and both types (112 MB) 57 us, of the 66 thousand of a tiny
// layer 6.5 us (two launches, the second set up during the first).
#include <limits.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGradThreads = 256;
constexpr int kGradBlocksPerSm = 4;    // at 64 registers: 128 KB of loads in flight an SM
constexpr int kScaleBlocksPerSm = 3;   // of the second pass: 80 registers, none spilled
constexpr int kGradVecs = 8;           // 16-byte vectors a thread has in flight
constexpr int kChunkBytes = kGradThreads * kGradVecs * 16;   // one unit of work

// The tensors of one launch, in its parameters.  Tensor i's chunks are
// [first[i], first[i+1]); a list has at most kGradMostBytes, far fewer than 2^31
// chunks.  Its chunk boundaries lie kChunkBytes apart counted
// from the 16-byte boundary at or before the source, so that every chunk but
// the first starts aligned wherever the tensor starts.
template <int CAP> struct GradTable {
    const void* src[CAP];
    void* dst[CAP];
    int64_t n[CAP];
    int32_t first[CAP + 1];
    uint8_t bf16[CAP];
    int count;
};

struct Chunk {
    const void* src;
    void* dst;
    int n;       // elements
    bool bf16;
};

// Chunk c, which tensor i holds.
template <int CAP> __device__ __forceinline__ Chunk chunk_of(const GradTable<CAP>& t, int i, int c) {
    const int shift = t.bf16[i] ? 1 : 2;
    const int skew = (int)(reinterpret_cast<uintptr_t>(t.src[i]) & 15) >> shift;
    int64_t a = ((int64_t)(c - t.first[i]) * kChunkBytes >> shift) - skew;
    int64_t b = a + (kChunkBytes >> shift);
    if (a < 0) a = 0;
    if (b > t.n[i]) b = t.n[i];
    return {(const uint8_t*)t.src[i] + (a << shift), (uint8_t*)t.dst[i] + (a << shift), (int)(b - a),
            t.bf16[i] != 0};
}

template <int CAP> __device__ __forceinline__ int find_tensor(const GradTable<CAP>& t, int c) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (t.first[m] <= c) lo = m; else hi = m;
    }
    return lo;
}

// Sum of squares over the whole range of fp32 inputs: values whose squares would
// leave it are scaled by a power of two first and go to 64 bits.  Four values go by
// their largest magnitude: between 2^-60 and 2^40 its square is 2^-120 at least, of
// which the others' squares, rounded to 2^-150, lose less than 2^-28, and a sum of
// 2^47 such squares stays finite.  Gradients below 1e-18 take the other way: 537 M in
// 787 us, against 295 (bf16 777, against 153).  The common sum is kept as an unevaluated
// pair of fp32 (each chunk's sum added exactly, by the error of an addition being
// an fp32 number itself), since 64-bit additions run at a small fraction of the
// rate here.
__device__ __noinline__ double rare_squares(float a, float b, float c, float d, float scale) {
    a *= scale; b *= scale; c *= scale; d *= scale;
    const double s = fmaf(a, a, fmaf(b, b, fmaf(c, c, d * d)));
    return s * (scale < 1.f ? 0x1p160 : 0x1p-200);
}

struct SquareSum {
    float high = 0.f, low = 0.f;
    double rare = 0.0;
    __device__ __forceinline__ void add(float a, float b, float c, float d, float& sum) {
        const float m = fmaxf(fmaxf(fabsf(a), fabsf(b)), fmaxf(fabsf(c), fabsf(d)));   // no NaN
        if (m <= 0x1p40f && (m >= 0x1p-60f || m == 0.f))
            sum = fmaf(a, a, fmaf(b, b, fmaf(c, c, fmaf(d, d, sum))));
        else
            rare += rare_squares(a, b, c, d, m > 1.f ? 0x1p-80f : 0x1p100f);
    }
    // the sum of one chunk's squares (at most 64 in vectors and one beside them a thread)
    __device__ __forceinline__ void flush(float sum) {
        const float s = __fadd_rn(high, sum), b = __fsub_rn(s, high);
        low = __fadd_rn(low, __fadd_rn(__fsub_rn(high, __fsub_rn(s, b)), __fsub_rn(sum, b)));
        high = s;
    }
    __device__ __forceinline__ double total() const { return (double)high + (double)low + rare; }
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
    float s = 0.f;
    uint4 u[kGradVecs];
    #pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int j = threadIdx.x + i * kGradThreads;
        u[i] = j < nv ? __ldcg(q + j) : make_uint4(0u, 0u, 0u, 0u);
    }
    const int rest = c.n - nv * N;   // head and tail, fewer than 2 N
    if ((int)threadIdx.x < rest) {
        const int i = (int)threadIdx.x < head ? (int)threadIdx.x : nv * N + (int)threadIdx.x;
        sum.add(to_f32<T>(p[i]), 0.f, 0.f, 0.f, s);
    }
    #pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        float v[N];
        Vec<T>::unpack(u[i], v);
        #pragma unroll
        for (int j = 0; j < N; j += 4) sum.add(v[j], v[j + 1], v[j + 2], v[j + 3], s);
    }
    sum.flush(s);
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

// It begins while the kernel before it may still write the gradients: they are read
// past the L1, and not through the non-coherent path, after the wait.
template <int CAP>
__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm)
    grad_square_kernel(const __grid_constant__ GradTable<CAP> t, double* partial, int* ticket) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ double buf[kGradThreads / 32];
    SquareSum sum;
    const int chunks = t.first[t.count];
    int c = blockIdx.x;
    for (int i = c < chunks ? find_tensor(t, c) : 0; c < chunks; c += gridDim.x) {
        while (c >= t.first[i + 1]) ++i;
        const Chunk k = chunk_of(t, i, c);
        if (k.bf16) square_chunk<__nv_bfloat16>(k, sum);
        else square_chunk<float>(k, sum);
    }
    const double s = block_sum(sum.total(), buf);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
    if (threadIdx.x == 0 && blockIdx.x == 0) *ticket = 0;   // of grad_scale_kernel
}

// the norm from the partials; block 0 of a call's first launch writes it down
__device__ __forceinline__ float finish_norm(const double* partial, int np, double* buf,
                                             float* norm, int32_t* status, bool writer) {
    double s = 0.0;
    for (int i = threadIdx.x; i < np; i += kGradThreads) s += __ldcg(partial + i);
    const float n = (float)sqrt(block_sum(s, buf));
    if (writer && threadIdx.x == 0) {
        *norm = n;
        if (!isfinite(n)) report(status, MOE_ERR_NONFINITE);
    }
    return n;
}

__global__ void __launch_bounds__(kGradThreads)
    grad_norm_kernel(const double* partial, int np, float* norm, int32_t* status) {
    __shared__ double buf[kGradThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    finish_norm(partial, np, buf, norm, status, true);
}

// out = grad * f * f2; f2 is 1, or 2^-126 where the factor alone would not be a normal
// number: that happens next to never, so the vectors' path goes without it.
template <typename T>
__device__ __forceinline__ void scale_chunk(const Chunk& c, float f, float f2) {
    constexpr int N = Vec<T>::N;
    const T* p = (const T*)c.src;
    T* o = (T*)c.dst;
    const int head = head_of<T>(p, c.n);
    const bool vec = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
    if (!vec || f2 != 1.f) {   // the two sides never meet a 16-byte boundary together, or as above
        for (int i = threadIdx.x; i < c.n; i += kGradThreads) o[i] = from_f32<T>(to_f32<T>(p[i]) * f * f2);
        return;
    }
    const int nv = (c.n - head) / N;
    const uint4* q = (const uint4*)(p + head);
    uint4* r = (uint4*)(o + head);
    uint4 u[kGradVecs];
    #pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int j = threadIdx.x + i * kGradThreads;
        if (j < nv) u[i] = __ldcs(q + j);
    }
    #pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int j = threadIdx.x + i * kGradThreads;
        float v[N];
        Vec<T>::unpack(u[i], v);
        #pragma unroll
        for (int n = 0; n < N; ++n) v[n] *= f;
        if (j < nv) __stcs(r + j, Vec<T>::pack(v));
    }
    const int rest = c.n - nv * N;
    if ((int)threadIdx.x < rest) {
        const int i = (int)threadIdx.x < head ? (int)threadIdx.x : nv * N + (int)threadIdx.x;
        o[i] = from_f32<T>(to_f32<T>(p[i]) * f);
    }
}

// Chunks by a ticket, the list's last ones first: what the sums read last is still
// in the L2.  (Where each block has chunks of its own, blocks drift apart, and
// reads and writes all over the list cost memory bandwidth: 2.09 ms against 1.82
// for 1.07 G fp32 gradients.)  np > 0: the block adds the partials itself; np ==
// 0: the norm is there.
template <int CAP>
__global__ void __launch_bounds__(kGradThreads, kScaleBlocksPerSm)
    grad_scale_kernel(const __grid_constant__ GradTable<CAP> t, const double* partial, int np,
                      float max_norm, float* norm, int writes_norm, int in_place, int* ticket,
                      int32_t* status) {
    __shared__ double buf[kGradThreads / 32];
    __shared__ int next[2];
    int c = t.first[t.count] - 1 - (int)blockIdx.x;
    int i = c >= 0 ? find_tensor(t, c) : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float n = np > 0 ? finish_norm(partial, np, buf, norm, status, writes_norm && blockIdx.x == 0)
                           : __ldcg(norm);
    // a norm within the bound, or none (infinite, NaN): the gradients as they are
    float f = isfinite(n) && n > max_norm ? max_norm / n : 1.f;
    // Below fp32's normal range the factor would lose bits that the products, up to
    // max_norm, have: 2^126 of it at first (n > 2^-23 then, max_norm < 4).
    float f2 = 1.f;
    if (f < 0x1p-126f && max_norm > 0.f) {
        f = (max_norm * 0x1p63f) / (n * 0x1p-63f);
        f2 = 0x1p-126f;
    }
    if (f == 1.f && in_place) return;
    for (int turn = 0; c >= 0; turn ^= 1) {
        if (threadIdx.x == 0) next[turn] = (int)gridDim.x + atomicAdd(ticket, 1);
        while (c < t.first[i]) --i;
        const Chunk k = chunk_of(t, i, c);
        if (f != 1.f || k.src != k.dst) {
            if (k.bf16) scale_chunk<__nv_bfloat16>(k, f, f2);
            else scale_chunk<float>(k, f, f2);
        }
        __syncthreads();
        c = t.first[t.count] - 1 - next[turn];
    }
}

int grad_blocks(int64_t chunks) {
    const int64_t most = (int64_t)device_sm_count() * kGradBlocksPerSm;
    return (int)(chunks < most ? (chunks > 0 ? chunks : 1) : most);
}

// Tensors [from, from + CAP) of the list.
template <int CAP> void make_table(GradTable<CAP>& t, const moe_grad* g, int from, int n) {
    int32_t c = 0;
    t.count = n - from < CAP ? n - from : CAP;
    for (int i = 0; i < t.count; ++i) {
        const moe_grad& x = g[from + i];
        const bool half = x.dtype == MOE_BF16;
        const int64_t bytes = x.n * (half ? 2 : 4) + (int64_t)(reinterpret_cast<uintptr_t>(x.grad) & 15);
        t.src[i] = x.grad;
        t.dst[i] = x.out ? x.out : const_cast<void*>(x.grad);
        t.n[i] = x.n;
        t.bf16[i] = half;
        t.first[i] = c;
        c += x.n ? (int32_t)((bytes + kChunkBytes - 1) / kChunkBytes) : 0;
    }
    t.first[t.count] = c;
}

// A launch that may begin while the kernel before it in the stream ends; every
// kernel here waits for that one's end before it touches memory.
template <typename... A, typename... B>
cudaError_t launch_after(void (*kern)(A...), int blocks, cudaStream_t st, const B&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kGradThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int CAP>
cudaError_t launch(int n, const moe_grad* g, bool clip, float max_norm, float* norm, double* partial,
                   int* tickets, int32_t* status, cudaStream_t st) {
    GradTable<CAP> t;
    int np = 0, in_place = 1;
    int64_t chunks = 0;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < n; i += CAP) {
        make_table(t, g, i, n);
        const int blocks = grad_blocks(t.first[t.count]);
        e = launch_after(grad_square_kernel<CAP>, blocks, st, t, partial + np, tickets + i / CAP);
        if (e != cudaSuccess) return e;
        np += blocks;
        chunks += t.first[t.count];
        for (int j = 0; j < t.count; ++j) in_place &= t.n[j] == 0 || t.src[j] == t.dst[j];
    }
    // Few chunks: their blocks add the partials themselves, which spares a launch.
    const bool fused = clip && chunks > 0 && chunks <= grad_blocks(INT32_MAX);
    if (!fused) {
        e = launch_after(grad_norm_kernel, 1, st, (const double*)partial, np, norm, status);
        if (!clip) return e;
        np = 0;
    }
    int writes_norm = fused;   // the first launch
    for (int i = 0; i < n && e == cudaSuccess; i += CAP) {
        if (n > CAP) make_table(t, g, i, n);
        const int have = t.first[t.count], most = device_sm_count() * kScaleBlocksPerSm;
        if (have == 0) continue;
        e = launch_after(grad_scale_kernel<CAP>, have < most ? have : most, st, t,
                         (const double*)partial, np, max_norm, norm, writes_norm, in_place,
                         tickets + i / CAP, status);
        writes_norm = 0;
    }
    return e;
}

}  // namespace

// Tables of two sizes: launches copy their parameters, 29 KB for the larger.
constexpr int kSmallTable = 64, kLargeTable = 1000;

namespace {
int64_t grad_launches(int n) { return n > 0 ? (n + (int64_t)kLargeTable - 1) / kLargeTable : 1; }
int64_t grad_partials(int n) { return grad_launches(n) * device_sm_count() * kGradBlocksPerSm; }
}  // namespace

// partial sums, then a ticket for each launch
size_t grad_workspace(int n) {
    return (size_t)grad_partials(n) * sizeof(double) + (size_t)grad_launches(n) * sizeof(int);
}

cudaError_t launch_grad_norm(int n, const moe_grad* g, bool clip, float max_norm, float* norm,
                             void* ws, int32_t* status, cudaStream_t st) {
    double* partial = (double*)ws;
    int* tickets = (int*)(partial + grad_partials(n));
    return n <= kSmallTable
               ? launch<kSmallTable>(n, g, clip, max_norm, norm, partial, tickets, status, st)
               : launch<kLargeTable>(n, g, clip, max_norm, norm, partial, tickets, status, st);
}

}  // namespace moe
