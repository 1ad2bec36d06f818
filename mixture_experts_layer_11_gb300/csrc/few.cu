// few.cu -- one whole MoE layer for a few tokens (T <= MOE_FEW_MAX_TOKENS):
// router, top-k gate, experts, combine and residual, for decode steps.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kFewMax = MOE_FEW_MAX_TOKENS;
constexpr int kMaxSlots = kFewMax * 16;   // T * k

// 16 bytes of T as floats
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// ---- router logits -----------------------------------------------------------------
// L[t,e] = <x_t, Wg_e> + beta_e in fp32.  A block computes kLogitE experts x TT
// tokens; its warps split d (16 bytes a lane and step), their sums are added in
// warp order.
constexpr int kLogitE = 4;
constexpr int kLogitThreads = 256;

template <typename T, int TT>
__global__ void __launch_bounds__(kLogitThreads)
    few_logits_kernel(int tokens, int d, int E, const T* __restrict__ x, const T* __restrict__ Wg,
                      const float* __restrict__ beta, float* __restrict__ logits) {
    constexpr int N = Vec<T>::N, W = kLogitThreads / 32, V = kLogitE * TT;
    __shared__ float part[W][V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.x * kLogitE, t0 = blockIdx.y * TT;
    float acc[kLogitE][TT] = {};
    for (int i = threadIdx.x * N; i < d; i += kLogitThreads * N) {
        float g[kLogitE][N];
        #pragma unroll
        for (int a = 0; a < kLogitE; ++a)   // experts and tokens past the end: the last one again
            Vec<T>::load(Wg + (int64_t)(e0 + a < E ? e0 + a : E - 1) * d + i, g[a]);
        #pragma unroll
        for (int b = 0; b < TT; ++b) {
            float v[N];
            Vec<T>::load(x + (int64_t)(t0 + b < tokens ? t0 + b : tokens - 1) * d + i, v);
            #pragma unroll
            for (int a = 0; a < kLogitE; ++a)
                #pragma unroll
                for (int n = 0; n < N; ++n) acc[a][b] = fmaf(g[a][n], v[n], acc[a][b]);
        }
    }
    #pragma unroll
    for (int a = 0; a < kLogitE; ++a)
        #pragma unroll
        for (int b = 0; b < TT; ++b) {
            float v = acc[a][b];
            #pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
            if (lane == 0) part[warp][a * TT + b] = v;
        }
    __syncthreads();
    const int a = threadIdx.x / TT, b = threadIdx.x % TT;
    if (a < kLogitE && e0 + a < E && t0 + b < tokens) {
        float v = 0.f;
        #pragma unroll
        for (int w = 0; w < W; ++w) v += part[w][threadIdx.x];
        logits[(int64_t)(t0 + b) * E + e0 + a] = v + (beta ? beta[e0 + a] : 0.f);
    }
}

// ---- gate and dispatch ------------------------------------------------------------
// Every block of the expert kernels works the gate out for itself from the
// logits (64 x 256 of them at most): that takes it less time than waiting for
// one block to do it.  Rows are the (token, slot) pairs sorted by expert, then
// by token.
struct Plan {
    unsigned long long tokens[256];   // bit t: token t goes to this expert
    int off[257];                     // first row of each expert
    int act[256];                     // experts with tokens, ascending
    int nact;
    int warp_sum[32];
    float w[kMaxSlots];               // [t * k + j]
    short pos[kMaxSlots];             // row of slot (t, j)
    uint8_t e_of[kMaxSlots];          // expert of slot (t, j)
};

// the largest of (value, lower expert first) over the warp
__device__ __forceinline__ void warp_best(float& v, int& e) {
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float v2 = __shfl_xor_sync(kFull, v, o);
        const int e2 = __shfl_xor_sync(kFull, e, o);
        if (v2 > v || (v2 == v && e2 < e)) { v = v2; e = e2; }
    }
}

// Called by all threads of a block of at least 256.
__device__ void make_plan(Plan& p, const float* logits, int tokens, int E, int k, int renorm,
                          int32_t* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int e = threadIdx.x; e < 256; e += blockDim.x) p.tokens[e] = 0ull;
    __syncthreads();
    for (int t = warp; t < tokens; t += warps) {
        float L[8];
        bool bad = false;
        float m = -INFINITY;
        #pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int e = lane + 32 * q;
            L[q] = -INFINITY;
            if (e < E) {
                const float v = __ldcg(logits + (int64_t)t * E + e);
                if (!isfinite(v)) bad = true;
                if (!isnan(v)) L[q] = v;   // a NaN ranks below every number
            }
            m = fmaxf(m, L[q]);
        }
        if (__any_sync(kFull, bad) && lane == 0) report(status, MOE_ERR_NONFINITE);
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        float z = 0.f;
        #pragma unroll
        for (int q = 0; q < 8; ++q)
            if (lane + 32 * q < E) z += expf(L[q] - m);
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
        uint32_t taken = 0u;
        float mine = 0.f, sum = 0.f;
        for (int j = 0; j < k; ++j) {
            // an expert not yet taken always beats (-inf, 256)
            float v = -INFINITY;
            int e = 256;
            #pragma unroll
            for (int q = 7; q >= 0; --q) {
                const int c = lane + 32 * q;
                if (c < E && !(taken >> q & 1u) && (L[q] >= v)) { v = L[q]; e = c; }
            }
            warp_best(v, e);
            if ((e & 31) == lane) taken |= 1u << (e >> 5);
            const float pr = expf(v - m) / z;
            sum += pr;
            if (lane == j) mine = pr;
            if (lane == 0) {
                atomicOr(&p.tokens[e], 1ull << t);
                p.e_of[t * k + j] = (uint8_t)e;
            }
        }
        if (lane < k) p.w[t * k + lane] = renorm ? mine / sum : mine;
    }
    __syncthreads();
    // exclusive prefix sums over the experts of (rows, has rows), in one word
    const int e = threadIdx.x;
    int n = 0, v = 0;
    if (e < 256) {
        n = __popcll(p.tokens[e]);
        v = n | (n > 0 ? 1 << 16 : 0);
        const int own = v;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) p.warp_sum[warp] = v;
        v -= own;
    }
    __syncthreads();
    if (e < 256) {
        for (int q = 0; q < warp; ++q) v += p.warp_sum[q];
        p.off[e] = v & 0xffff;
        if (n > 0) p.act[v >> 16] = e;
        if (e == 255) { p.off[256] = (v & 0xffff) + n; p.nact = (v >> 16) + (n > 0); }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * k; i += blockDim.x) {
        const int ee = p.e_of[i], t = i / k;
        p.pos[i] = (short)(p.off[ee] + __popcll(p.tokens[ee] & ((1ull << t) - 1ull)));
    }
    __syncthreads();
}

// ---- experts ----------------------------------------------------------------------
// One warp per output feature of one expert, over the expert's rows one after
// another: out[row][i] = <W[e][i], in_row> (+ bias), then GELU for the first
// product.
template <typename T, bool FIRST>
__global__ void __launch_bounds__(256)
    few_product_kernel(int tokens, int E, int k, int renorm, const float* __restrict__ logits, int K,
                       int M, const T* __restrict__ in, const float* __restrict__ hidden,
                       const T* __restrict__ W, const T* __restrict__ bias, float* __restrict__ out,
                       int32_t* status) {
    constexpr int N = Vec<T>::N;
    __shared__ Plan p;
    make_plan(p, logits, tokens, E, k, renorm, FIRST && blockIdx.x == 0 && blockIdx.y == 0 ? status : nullptr);
    if ((int)blockIdx.y >= p.nact) return;
    const int e = p.act[blockIdx.y], lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= M) return;
    const T* wr = W + ((int64_t)e * M + i) * K;
    unsigned long long left = p.tokens[e];
    for (int r = p.off[e]; r < p.off[e + 1]; ++r) {
        const int t = __ffsll((long long)left) - 1;
        left &= left - 1;
        float acc = 0.f;
        for (int c = lane * N; c < K; c += 32 * N) {
            float a[N];
            Vec<T>::load(wr + c, a);
            #pragma unroll
            for (int n = 0; n < N; ++n)
                acc = fmaf(a[n], FIRST ? to_f32<T>(in[(int64_t)t * K + c + n])
                                       : hidden[(int64_t)r * K + c + n], acc);
        }
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
        if (lane == 0) {
            if (bias) acc += to_f32<T>(bias[(int64_t)e * M + i]);
            out[(int64_t)r * M + i] = FIRST ? gelu_f(acc) : acc;
        }
    }
}

// y_t = residual_t + sum_j w_tj Y[pos_tj], j ascending
template <typename T>
__global__ void __launch_bounds__(256)
    few_combine_kernel(int tokens, int d, int E, int k, int renorm, const float* __restrict__ logits,
                       const float* __restrict__ Y, const T* residual, T* y) {
    __shared__ Plan p;
    make_plan(p, logits, tokens, E, k, renorm, nullptr);
    const int c = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (c >= d) return;
    float v = 0.f;
    for (int j = 0; j < k; ++j) v = fmaf(p.w[t * k + j], Y[(int64_t)p.pos[t * k + j] * d + c], v);
    if (residual) v += to_f32<T>(residual[(int64_t)t * d + c]);
    y[(int64_t)t * d + c] = from_f32<T>(v);
}

size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

struct FewLayout {
    size_t logits, hidden, rows, total;
};
FewLayout few_layout(const moe_shape& s) {
    FewLayout l;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t a = at; at += pad256(n); return a; };
    l.logits = take(sizeof(float) * s.T * s.E);
    l.hidden = take(sizeof(float) * s.T * s.k * s.f);
    l.rows = take(sizeof(float) * s.T * s.k * s.d);
    l.total = at;
    return l;
}

template <typename T>
cudaError_t run(const moe_shape& s, const moe_layer_params& p, const T* x, const T* residual, T* y,
                uint8_t* ws, int32_t* status, cudaStream_t st) {
    const FewLayout l = few_layout(s);
    float* logits = (float*)(ws + l.logits);
    float* hidden = (float*)(ws + l.hidden);
    float* rows = (float*)(ws + l.rows);
    const int t = (int)s.T;
    const unsigned ge = (unsigned)((s.E + kLogitE - 1) / kLogitE);
    if (t == 1)
        few_logits_kernel<T, 1><<<dim3(ge, 1), kLogitThreads, 0, st>>>(
            t, s.d, s.E, x, (const T*)p.Wg, p.logit_bias, logits);
    else
        few_logits_kernel<T, 8><<<dim3(ge, (unsigned)((t + 7) / 8)), kLogitThreads, 0, st>>>(
            t, s.d, s.E, x, (const T*)p.Wg, p.logit_bias, logits);
    const int most = t * s.k < s.E ? t * s.k : s.E;
    few_product_kernel<T, true><<<dim3((s.f + 7) / 8, most), 256, 0, st>>>(
        t, s.E, s.k, s.renorm, logits, s.d, s.f, x, nullptr, (const T*)p.W1, (const T*)p.b1, hidden,
        status);
    few_product_kernel<T, false><<<dim3((s.d + 7) / 8, most), 256, 0, st>>>(
        t, s.E, s.k, s.renorm, logits, s.f, s.d, nullptr, hidden, (const T*)p.W2, (const T*)p.b2,
        rows, status);
    few_combine_kernel<T><<<dim3((s.d + 255) / 256, t), 256, 0, st>>>(
        t, s.d, s.E, s.k, s.renorm, logits, rows, residual, y);
    return cudaGetLastError();
}

}  // namespace

size_t few_workspace(const moe_shape& s) { return few_layout(s).total; }

cudaError_t launch_layer_few(const moe_shape& s, const moe_layer_params& p, const void* x,
                             const void* residual, void* y, void* ws, int32_t* status,
                             cudaStream_t st) {
    if (s.dtype == MOE_BF16)
        return run<__nv_bfloat16>(s, p, (const __nv_bfloat16*)x, (const __nv_bfloat16*)residual,
                                  (__nv_bfloat16*)y, (uint8_t*)ws, status, st);
    return run<float>(s, p, (const float*)x, (const float*)residual, (float*)y, (uint8_t*)ws, status,
                      st);
}

}  // namespace moe
