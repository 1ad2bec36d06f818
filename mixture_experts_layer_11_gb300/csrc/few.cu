// few.cu -- one whole MoE layer for a few tokens (T <= MOE_FEW_MAX_TOKENS), for
// decode steps, in two launches:
//
//   few_logits_kernel   L = x Wg^T + beta
//   few_direct_kernel   one token, or up to four of a small layer, or
//   few_experts_kernel  everything else:
//     gate of L;  a = GELU(W1[e] x_t + b1[e]) for every chosen (t, e);
//     y_t = residual_t + sum_j w_tj (W2[e_j] a_tj + b2[e_j])
//
// The weights of the chosen experts are nearly all the bytes, and with at most 64
// tokens a weight meets at most 64 of them: memory bounds the layer (64 flop a
// byte in bf16 against 290 that the GPU has), and beside it the latencies between
// its dependent steps.  So both expert kernels stream every chosen weight once, in
// equal shares over all SMs, and do all the rest of the layer in the same launch:
// what a step waits for is a counter in memory, not a launch.  The second launch may
// begin during the first, so that a block is set up as soon as its SM is free.  (A block
// of the large kernel needs an SM's whole shared memory and nearly all its registers, so
// that it never shares one with a block of the logits kernel.)
//
// Measured on a GB300 (device time of both launches in a graph, weights from HBM):
//   bf16, d = 4096, f = 1024, 128 experts, top-8:  64 tokens (all 2.1 GB of weights)
//     339 us, 6.2 TB/s; one token (134 MB) 35 us, 3.9 TB/s
//   bf16, d = 2048, f = 8192, 16 experts, top-2:   13 tokens (0.87 GB) 153 us, 5.7 TB/s
//   bf16, d = 768, f = 3072, 8 experts, top-2:     64 tokens (76 MB) 41 us; one 13 us
//   fp32, d = 768, f = 3072, 64 experts, top-1, skewed: 33 tokens (38 or 57 MB) 53 to 56 us
// At the large sizes memory bounds it (its streams alone run at 6.7 to 6.9 TB/s);
// about 25 us are the logits, the gate, the hand-over between the products and
// the adding of split tiles, which bound the small sizes.
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kFewMax = MOE_FEW_MAX_TOKENS;
constexpr int kMaxSlots = kFewMax * 16;   // T * k

// These kernels begin while the kernel before them may still write what they read
// after their wait.  So nothing is read through the non-coherent path, whose data
// must not change while a kernel runs: no ld.global.nc, no const __restrict__ pointer
// that would let the compiler choose it.

// 16 bytes of T as floats
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
        unpack(*reinterpret_cast<const uint4*>(p), v);
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
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
        unpack(*reinterpret_cast<const uint4*>(p), v);
    }
};

// The warp's sums of V values (a power of two): each step sends half of what a lane
// holds and keeps the sums of the rest, so that V values take V + log2(32 / V)
// exchanges. Lane l returns the sum of value `which`; the lanes that hold the same
// one have the same.
template <int V> __device__ __forceinline__ float warp_sums(float (&v)[V], int& which) {
    const int lane = threadIdx.x & 31;
    which = 0;
    int o = 16;
    #pragma unroll
    for (int n = V; n > 1; n /= 2, o /= 2) {
        const bool up = lane & o;
        which += up ? n / 2 : 0;
        #pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(kFull, send, o);
        }
    }
    #pragma unroll
    for (int q = 16 / V; q > 0; q /= 2) v[0] += __shfl_xor_sync(kFull, v[0], q);
    return v[0];
}

// ---- GELU ------------------------------------------------------------------------------
// x Phi(x) with a small relative error in both tails, as hidden activations are held to
// more than bf16's precision each: 1 + erf(x / sqrt 2) would lose nearly all of it below -5.
// Phi(-|x|) = R(|x|) phi(x) with the Mills ratio R; R / t, t = 1 / (1 + p |x|), is a
// smooth function of t, here the polynomial with the least relative error for |x| <=
// 13.2, beyond which phi is below 2^-126 and taken as 0.

// One value, to 2^-21: degree 7 (2^-24), p = 0.3041, phi's factor in the polynomial; the
// rounding errors of the exponent enter as a factor 1 + ln 2 * low.
__device__ __forceinline__ float gelu_one(float x) {
    const float a = fminf(fabsf(x), 16.f), t = rcp_approx(fmaf(0.3041f, a, 1.0f));
    float r = 0.036699917f;
    r = fmaf(t, r, -0.1545382f);
    r = fmaf(t, r, 0.190735817f);
    r = fmaf(t, r, -0.0419697948f);
    r = fmaf(t, r, 0.123010464f);
    r = fmaf(t, r, 0.102595039f);
    r = fmaf(t, r, 0.122191094f);
    r = fmaf(t, r, 0.121275641f);
    constexpr float c = -0.72134752f, c_low = -9.62981495e-9f;   // -log2(e) / 2 in two parts
    const float s = a * a, power = s * c;
    const float low = fmaf(fmaf(a, a, -s), c, fmaf(s, c_low, fmaf(s, c, -power)));
    float e = ex2_approx(power);
    e = fmaf(e * low, 0.693147181f, e);
    const float q = t * r * e;                         // Phi(-|x|)
    return x * (x >= 0.f ? 1.0f - q : q);
}
// One copy of it for the expert kernel, whose instructions run once or twice a launch (33
// fp32 tokens of the skewed layer: 55.9 us so, inlined 56.6, with CUDA's normcdff 57.7).
__device__ __noinline__ float gelu_call(float x) { return gelu_one(x); }

// Two values, for hidden activations of 16 bits: degree 6 (2^-21), p = 0.2638.  Off by at
// most 2^-18.4 for |x| <= 8 and 2^-16.5 for |x| <= 13 (the rounding of the exponent).
__device__ __forceinline__ uint64_t gelu_two(float x0, float x1) {
    const float t0 = rcp_approx(fmaf(0.2638f, fabsf(x0), 1.0f));
    const float t1 = rcp_approx(fmaf(0.2638f, fabsf(x1), 1.0f));
    const uint64_t x = f2_pack(x0, x1), t = f2_pack(t0, t1);
    // log2 of phi: -x^2 log2(e) / 2 - log2(sqrt(2 pi))
    const uint64_t arg = f2_fma(f2_mul(x, x), f2_pack(-0.72134752f, -0.72134752f),
                                f2_pack(-1.32574806f, -1.32574806f));
    float a0, a1;
    f2_unpack(arg, a0, a1);
    const uint64_t phi = f2_pack(ex2_approx(a0), ex2_approx(a1));
    uint64_t r = f2_pack(-0.174574688f, -0.174574688f);
    r = f2_fma(t, r, f2_pack(0.51463443f, 0.51463443f));
    r = f2_fma(t, r, f2_pack(-0.197119161f, -0.197119161f));
    r = f2_fma(t, r, f2_pack(0.376498967f, 0.376498967f));
    r = f2_fma(t, r, f2_pack(0.200137436f, 0.200137436f));
    r = f2_fma(t, r, f2_pack(0.2703242f, 0.2703242f));
    r = f2_fma(t, r, f2_pack(0.263412178f, 0.263412178f));
    const uint64_t q = f2_mul(f2_mul(t, r), phi);                                 // Phi(-|x|)
    const uint64_t w = f2_fma(q, f2_pack(-2.0f, -2.0f), f2_pack(1.0f, 1.0f));     // 1 - 2q
    const uint64_t st = f2_pack(x0 >= 0.f ? 1.0f : 0.0f, x1 >= 0.f ? 1.0f : 0.0f);
    return f2_mul(x, f2_fma(st, w, q));
}

// ---- router logits -----------------------------------------------------------------
// L[t,e] = <x_t, Wg_e> + beta_e in fp32.  A block computes EE experts x TT tokens;
// its warps split d (16 bytes a lane and step), their sums are added in warp order.
// Small blocks, so that Wg streams to as many SMs as there are; it also clears the
// expert kernel's counters.
constexpr int kLogitThreads = 256;

template <typename T, int EE, int TT>
__global__ void __launch_bounds__(kLogitThreads)
    few_logits_kernel(int tokens, int d, int E, const T* x, const T* Wg, const float* beta,
                      float* logits, int* counters, int words) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < words; i += kLogitThreads) counters[i] = 0;
    constexpr int N = Vec<T>::N, W = kLogitThreads / 32, V = EE * TT;
    __shared__ float part[W][V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.x * EE, t0 = blockIdx.y * TT;
    float acc[V] = {};
    #pragma unroll 2
    for (int i = threadIdx.x * N; i < d; i += kLogitThreads * N) {
        float g[EE][N];
        #pragma unroll
        for (int a = 0; a < EE; ++a)   // experts and tokens past the end: the last one again
            Vec<T>::load(Wg + (int64_t)(e0 + a < E ? e0 + a : E - 1) * d + i, g[a]);
        #pragma unroll
        for (int b = 0; b < TT; ++b) {
            float v[N];
            Vec<T>::load(x + (int64_t)(t0 + b < tokens ? t0 + b : tokens - 1) * d + i, v);
            #pragma unroll
            for (int a = 0; a < EE; ++a)
                #pragma unroll
                for (int n = 0; n < N; ++n)
                    acc[a * TT + b] = fmaf(g[a][n], v[n], acc[a * TT + b]);
        }
    }
    int which;
    const float sum = warp_sums(acc, which);
    if (lane % (32 / V) == 0) part[warp][which] = sum;
    __syncthreads();
    const int a = threadIdx.x / TT, b = threadIdx.x % TT;
    if (a < EE && e0 + a < E && t0 + b < tokens) {
        float v = 0.f;
        #pragma unroll
        for (int w = 0; w < W; ++w) v += part[w][threadIdx.x];
        logits[(int64_t)(t0 + b) * E + e0 + a] = v + (beta ? beta[e0 + a] : 0.f);
    }
}

// ---- gate ---------------------------------------------------------------------------
// One warp: the k experts with the largest logits (equal ones by their index) and
// their softmax weights.  Lane l holds experts l, l + 32, ...
template <int EPL>
__device__ __forceinline__ void gate(const float* L, int E, int k, int renorm, uint8_t* e_of,
                                     float* w, int32_t* status) {
    const int lane = threadIdx.x & 31;
    auto value = [](uint32_t x) { return __uint_as_float(x & 0x80000000u ? x & 0x7fffffffu : ~x); };
    uint32_t key[EPL], high = 0u;   // ordered as the logits; 0: not an expert, or taken
    bool bad = false;
    #pragma unroll
    for (int q = 0; q < EPL; ++q) {
        const int e = lane + 32 * q;
        key[q] = 0u;
        if (e < E) {
            float l = __ldcg(L + e);
            if (!isfinite(l)) bad = true;
            if (isnan(l)) l = -INFINITY;                   // ranks below every number
            const uint32_t u = __float_as_uint(l + 0.f);   // one zero
            key[q] = u & 0x80000000u ? ~u : u | 0x80000000u;
        }
        high = key[q] > high ? key[q] : high;
    }
    if (__any_sync(kFull, bad) && lane == 0) report(status, MOE_ERR_NONFINITE);
    const float m = value(__reduce_max_sync(kFull, high));
    float z = 0.f;
    #pragma unroll
    for (int q = 0; q < EPL; ++q)
        if (lane + 32 * q < E) z += expf(value(key[q]) - m);
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
    int my_e = 0;
    uint32_t my_key = 0u;
    #pragma unroll 1
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
        int at = lane;
        #pragma unroll
        for (int q = 1; q < EPL; ++q)
            if (key[q] > best) { best = key[q]; at = lane + 32 * q; }
        const uint32_t top = __reduce_max_sync(kFull, best);
        at = (int)__reduce_min_sync(kFull, best == top ? (unsigned)at : 256u);
        #pragma unroll
        for (int q = 0; q < EPL; ++q)
            if (at == lane + 32 * q) key[q] = 0u;
        if (lane == j) { my_e = at; my_key = top; }
    }
    float pr = lane < k ? expf(value(my_key) - m) / z : 0.f;
    if (renorm) {
        float sum = pr;
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        pr /= sum;
    }
    if (lane < k) {
        e_of[lane] = (uint8_t)my_e;
        w[lane] = pr;
    }
}

// The block's warps, a token each in turn.
__device__ __forceinline__ void gate_tokens(const float* logits, int tokens, int E, int k, int renorm,
                                            uint8_t* e_of, float* w, int32_t* status) {
    #pragma unroll 1
    for (int t = threadIdx.x >> 5; t < tokens; t += blockDim.x >> 5) {
        if (E <= 32) gate<1>(logits + t * E, E, k, renorm, e_of + t * k, w + t * k, status);
        else if (E <= 128) gate<4>(logits + t * E, E, k, renorm, e_of + t * k, w + t * k, status);
        else gate<8>(logits + t * E, E, k, renorm, e_of + t * k, w + t * k, status);
    }
}

// ---- a handful of tokens on the CUDA cores -------------------------------------------
// With at most kDirectTokens tokens an expert's weights meet one to four rows: a
// dot product per weight row and token, lanes along K, weights straight from
// memory to registers.  Compared with the tensor-core kernel below this spares
// the way through shared and tensor memory and the adding of partial tiles, and
// its code is short (a launch's instructions come from the L2 cache the first
// time: measured 25 clocks for each).  Blocks take tasks by a ticket: the first
// product's, then the second's, which wait until all of the first's are done.  A
// task waits only for tasks that running blocks hold, so blocks need not be
// resident together.
constexpr int kDirectTokens = 4;
// With two to four tokens, up to so many weights (each token's counted): measured
// on 8 experts, top-2, against the kernel below: d = 256, f = 1024, 4 tokens 14.8
// against 19.9 us in bf16 and 14.0 against 22.7 in fp32; d = 512, f = 2048, 4 tokens
// (17 M weights) 19.5 against 20.4 and 25.1 against 27.6; d = 768, f = 3072, 2 tokens
// (19 M) 24.3 against 23.1 and 28 against 32.7, 3 tokens (28 M) 28.5 against 24.2
// and 36.6 against 34.6.  Over ten more layers (1 to 128 experts, top-1 to top-8, the L2
// flushed) this kernel was the faster one below the limits, but for one by 1 us; above
// them as fast or slower, by up to 43 us (4 tokens, top-8 of 128 experts of 4096 x 1024),
// unless tokens share experts (one expert of 1024 x 4096: 5 to 7 us faster).
template <typename T> constexpr int64_t direct_weights() {
    return int64_t(sizeof(T) == 2 ? 17 : 24) << 20;
}
constexpr int kDirectThreads = 256;
// 64, 80 or 128 registers a thread
template <int TT> constexpr int direct_blocks_per_sm() { return TT == 1 ? 4 : TT == 2 ? 3 : 2; }

struct DirectArgs {
    int d, f, E, k, renorm, tokens;
    int split1, split2;        // warps that share a group of weight rows
    const float* logits;
    const void *x, *W1, *b1, *W2, *b2, *residual;
    void* y;
    float* hidden;             // [T k][f]: gate weight times GELU
    int* ticket;
    int* done;
    int32_t* status;
    uint64_t limit_ns;
};

__device__ __forceinline__ int load_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// Writes of the block's other threads that a barrier has ordered before these two
// are published with them, as the calling thread's own are.
__device__ __forceinline__ int add_acq_rel(int* p, int v) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void add_release(int* p, int v) {
    asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// 16 bytes of T, streamed past L1
__device__ __forceinline__ uint4 stream16(const void* p) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}

// TT tokens at most, RW weight rows a warp, U steps of loads in flight
template <typename T, int TT, int RW, int U>
__global__ void __launch_bounds__(kDirectThreads, direct_blocks_per_sm<TT>())
    few_direct_kernel(const __grid_constant__ DirectArgs g) {
    constexpr int N = Vec<T>::N, W = kDirectThreads / 32;
    __shared__ uint8_t e_of[TT * 16], act[TT * 16], slot[TT * 16][TT];
    __shared__ float w[TT * 16];
    __shared__ float part[W][RW * TT];
    __shared__ int nact, next;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slots = g.tokens * g.k;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int claimed = 0;
    if (threadIdx.x == 0) claimed = atomicAdd(g.ticket, 1);
    gate_tokens(g.logits, g.tokens, g.E, g.k, g.renorm, e_of, w, blockIdx.x == 0 ? g.status : nullptr);
    __syncthreads();
    // the distinct experts in the order of their first slots, and each one's slot
    // (255: none) of every token
    if (warp == 0) {
        int count = 0;
        for (int i0 = 0; i0 < slots; i0 += 32) {
            const int i = i0 + lane;
            bool first = i < slots;
            for (int j = 0; first && j < i / g.k * g.k; ++j) first = e_of[j] != e_of[i];
            const uint32_t b = __ballot_sync(kFull, first);
            if (first) {
                const int a = count + __popc(b & ((1u << lane) - 1u));
                act[a] = e_of[i];
                for (int t = 0; t < TT; ++t) {
                    int s = 255;
                    for (int j = 0; t < g.tokens && j < g.k; ++j)
                        if (e_of[t * g.k + j] == e_of[i]) s = t * g.k + j;
                    slot[a][t] = (uint8_t)s;
                }
            }
            count += __popc(b);
        }
        if (lane == 0) {
            nact = count;
            next = claimed;
        }
    }
    __syncthreads();
    const int S1 = g.split1, S2 = g.split2;
    const int n1 = ((g.f + RW - 1) / RW + W / S1 - 1) / (W / S1);   // tasks an expert
    const int total1 = nact * n1;
    const int total = total1 + ((g.d + RW - 1) / RW + W / S2 - 1) / (W / S2);
    bool ready = false;
    for (int task = next; task < total; task = next) {
        if (threadIdx.x == 0) claimed = atomicAdd(g.ticket, 1);
        const bool one = task < total1;
        const int a1 = one ? task / n1 : 0;
        const int S = one ? S1 : S2, M = one ? g.f : g.d, K = one ? g.d : g.f;
        const int row0 = ((one ? task - a1 * n1 : task - total1) * (W / S) + warp / S) * RW;
        const int nk = (K + 32 * N - 1) / (32 * N);      // steps of 32 lanes along K
        const int steps = one ? nk : nact * nk;
        const T* Wm = (const T*)(one ? g.W1 : g.W2);
        float acc[RW * TT] = {};
        int c = warp % S;
        int a = one ? a1 : c / nk, ck = one ? c : c % nk;
        bool more = row0 < M && c < steps;
        // every warp passes the wait below once, in the block's first task of the second product
        while (more || (!one && !ready)) {
            uint4 wv[U][RW];
            int at[U], ex[U];
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = (ck * 32 + lane) * N;
                ex[u] = a;
                at[u] = more && c < steps && i < K ? i : -1;
                #pragma unroll
                for (int r = 0; r < RW; ++r) {
                    const int row = row0 + r < M ? row0 + r : M - 1;
                    wv[u][r] = at[u] >= 0 ? stream16(Wm + ((int64_t)act[a] * M + row) * K + i)
                                          : make_uint4(0u, 0u, 0u, 0u);
                }
                c += S;
                ck += S;
                while (!one && ck >= nk && a < nact) { ck -= nk; ++a; }
                if (a >= nact) { a = nact - 1; ck = 0; }
            }
            if (!one && !ready) {   // (the weights are on their way meanwhile)
                if (threadIdx.x == 0) {
                    const uint64_t t0 = globaltimer_ns();
                    while (load_acquire(g.done) < total1)
                        if (globaltimer_ns() - t0 > g.limit_ns) {
                            report(g.status, MOE_ERR_TIMEOUT);
                            break;
                        }
                }
                __syncthreads();
                ready = true;
            }
            #pragma unroll
            for (int u = 0; u < U; ++u) {
                float wf[RW][N];
                #pragma unroll
                for (int r = 0; r < RW; ++r) Vec<T>::unpack(wv[u][r], wf[r]);
                #pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (at[u] < 0 || (TT > 1 && slot[ex[u]][t] == 255)) continue;
                    float v[N];
                    if (one) {
                        Vec<T>::load((const T*)g.x + (int64_t)t * K + at[u], v);
                    } else {
                        const float* h = g.hidden + (int64_t)slot[ex[u]][t] * K + at[u];
                        #pragma unroll
                        for (int n = 0; n < N; n += 4) {
                            const float4 q = __ldcg(reinterpret_cast<const float4*>(h + n));
                            v[n] = q.x; v[n + 1] = q.y; v[n + 2] = q.z; v[n + 3] = q.w;
                        }
                    }
                    #pragma unroll
                    for (int r = 0; r < RW; ++r)
                        #pragma unroll
                        for (int n = 0; n < N; ++n)
                            acc[r * TT + t] = fmaf(wf[r][n], v[n], acc[r * TT + t]);
                }
            }
            more = more && c < steps;
        }
        // biases of the second product, a slot a lane
        if (!one && g.b2 && warp % S == 0)
            for (int t = 0; t < TT; ++t)
                if (t < g.tokens && lane < g.k)
                    #pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (row0 + r < M) {
                            const float v = w[t * g.k + lane] *
                                            to_f32<T>(((const T*)g.b2)[(int64_t)e_of[t * g.k + lane] * M + row0 + r]);
                            #pragma unroll
                            for (int q = 0; q < TT; ++q)
                                if (q == t) acc[r * TT + q] += v;
                        }
        int which;
        const float sum = warp_sums(acc, which);
        if (lane % (32 / (RW * TT)) == 0) part[warp][which] = sum;
        __syncthreads();
        // thread (group of warps, row, token): the warps' sums in order
        if ((int)threadIdx.x < W / S * RW * TT) {
            const int grp = threadIdx.x / (RW * TT), rt = threadIdx.x % (RW * TT);
            const int t = rt % TT;
            const int row = ((one ? task - a1 * n1 : task - total1) * (W / S) + grp) * RW + rt / TT;
            float v = 0.f;
            for (int q = 0; q < S; ++q) v += part[grp * S + q][rt];
            if (row < M && t < g.tokens) {
                if (one) {
                    const int s = slot[a1][t];
                    if (s != 255) {
                        if (g.b1) v += to_f32<T>(((const T*)g.b1)[(int64_t)act[a1] * M + row]);
                        g.hidden[(int64_t)s * M + row] = w[s] * gelu_one(v);
                    }
                } else {
                    const int64_t o = (int64_t)t * M + row;
                    if (g.residual) v += to_f32<T>(((const T*)g.residual)[o]);
                    ((T*)g.y)[o] = from_f32<T>(v);
                }
            }
        }
        if (threadIdx.x == 0) next = claimed;
        __syncthreads();
        if (one && threadIdx.x == 0) add_release(g.done, 1);
    }
}

// ---- experts ----------------------------------------------------------------------
// Both products with the weights as the 128-row operand and the tokens as the
// narrow one: D[128 output features][rows] = W tile x activations^T, K blocks of 128
// bytes.  One block an SM:
//   warp 0  takes shares (below) and loads their weights by TMA, 16 KB a K block,
//           the second product's right behind the first's;
//   warp 1  loads the activations: all tokens' K block of x (columns of tokens that
//           are not the expert's are left unused), then the expert's hidden rows;
//   warp 2  (bf16) issues the MMAs, into one of two accumulators;
//   8 (fp32) or 12 warps  take the accumulators out: GELU and hidden rows, or the gate-
//           weighted sum over the experts of an output tile in shared memory.  fp32: they do
//           the products themselves.
// In bf16 hidden activations are stored as two bf16 numbers each, high and low
// part, and enter the second product as two columns: they are held to 2^-16 of each,
// for no more than twice the narrow operand's bytes.  (few_direct_kernel holds them in
// fp32, as this kernel does in fp32.)
constexpr int kTileM = 128;          // weight rows (output features) of a tile
constexpr int kBlockBytes = 128;     // one K block of a row: 64 bf16 or 32 fp32
constexpr int kABytes = kTileM * kBlockBytes;
constexpr int kMaxAStages = 12, kMaxBStages = 8;
constexpr int kWarpsBeforeEpilogue = 4;
// Times that decide whether the first product's units are cut: a K block of
// weights when all blocks stream (16 KB of each of 152 at 6.8 TB/s), when few do
// (measured: 60 GB/s an SM), and adding the parts of cut units.
constexpr float kBlockNs = 366.f, kLoneBlockNs = 280.f, kJoinNs = 2000.f;
// Copies and MMAs in flight end by themselves: waits for them at a block's end have
// a bound of their own, however short the caller's is.
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr uint64_t kTakeOverNs = 20000;   // a share without a block for so long is taken over

template <typename T> struct Kind;
template <> struct Kind<__nv_bfloat16> {
    static constexpr bool kTensor = true;
    static constexpr int kBox = 16;             // activation rows a TMA box takes
    static constexpr int kRowsPerSlot = 2;      // hidden rows of a slot: high and low part
    static constexpr int kBlock = 64;           // elements of a K block
    // threads (64 tokens of 8 experts of 768 x 3072: 128 43.9 us, 256 41.6, 384 41.0)
    static constexpr int kEpilogue = 384;
};
template <> struct Kind<float> {
    static constexpr bool kTensor = false;
    static constexpr int kBox = 8;
    static constexpr int kRowsPerSlot = 1;
    static constexpr int kBlock = 32;
    static constexpr int kEpilogue = 256;
};
template <typename T> constexpr int few_threads() {
    return kWarpsBeforeEpilogue * 32 + Kind<T>::kEpilogue;
}

constexpr int kMaxBlocks = 512;

// In the workspace, zeroed by the logits kernel.
struct Counters {
    int done;                    // finished units (few_direct_kernel: tasks) of the first product
    int ticket;                  // few_direct_kernel: tasks handed out
    int claimed[2];              // shares of each product that a block has taken
    int sums;                    // summing tasks handed out
    int gated;                   // tokens whose gate is in `slots`
    int claim[2][kMaxBlocks];    // 1: the share is taken
    int joined[kMaxBlocks];      // per share: parts of the unit that starts in it and ends in another
    // then per output tile: parts written
};

struct FewArgs {
    int tokens, d, f, E, k, renorm;
    int tiles1, tiles2, KB1, KB2;         // of the two products: output tiles, K blocks
    int slices;                           // summing tasks an output tile
    int a_stages, b_ring;                 // shared-memory rings: weights (stages), activations (bytes)
    const float* logits;
    float2* slots;         // [T k]: expert (as bits) and gate weight
    const void *b1, *b2, *residual;
    void* y;
    void* hidden;          // [T k kRowsPerSlot][f]
    float *part1, *part2;  // [shares][2][T][128] partial sums of the two products
    Counters* cnt;
    int* tiles_done;       // per output tile
    int32_t* status;
    uint64_t limit_ns;
};

// ---- dispatch -----------------------------------------------------------------------
// Every block of the expert kernel sorts the (token, slot) pairs (1024 of them at
// most) for itself: rows by expert, then by token.  With few tokens each also works out
// the gate, which takes it less time than to wait for another block's result; with more
// the blocks share it out (gate_plan).
struct Sorted {
    unsigned long long tokens[256];   // bit t: token t goes to this expert
    int off[257];                     // first row of each expert
    int act[256];                     // experts with tokens, ascending
    int cost[257];                    // prefix sums over act of block_cost()
    int most;                         // largest block_cost()
    int most_rows;                    // largest number of rows of an expert
    int nact;
    float w[kMaxSlots];               // gate weight of slot (t, j)
    float row_w[kMaxSlots];           // gate weight of each row
    uint8_t e_of[kMaxSlots];          // expert of slot (t, j)
    uint8_t row_token[kMaxSlots];     // token of each row
};

// Relative time of one K block with `rows` activation rows: the bytes of the
// weights (4), unless fp32 products take longer.  Of ten such tables these shares
// took the least time over 44 fp32 layers of 6 to 64 tokens (geometric mean 99.0 us;
// 4, 6, 12, 24: 100.4; 4, 8, 18, 34: 101.0).
constexpr int kMaxCost = 25;
template <typename T> __device__ __forceinline__ int block_cost(int rows) {
    return sizeof(T) == 2 ? 1 : rows <= 8 ? 4 : rows <= 16 ? 7 : rows <= 32 ? 13 : kMaxCost;
}

// One block's consecutive K blocks of one (expert, tile).
struct Seg {
    int a, m;         // active expert, tile
    int kb0, kb1;     // K blocks
    int c0, c1;       // blocks that hold the unit's first and last K block
};

// A share of a product.  The K blocks of a product lie one after another on a line,
// each as long as its cost: in the first product an expert's tiles follow one
// another, in the second an output tile's experts.  The line is cut into equal
// shares, one a block, and a K block is the share's in which it begins; so every
// block works for the same time, and a share may begin and end inside a unit (an
// expert's tile).
enum : int { kFirst = 0, kSecond = 1, kSum = 2, kEnd = 3 };
struct Walk {
    int phase;
    int me;                // the share's (kSum: the task's) number
    int tiles, KB;         // of the product
    int shares, size, longer;    // the first `longer` shares are size + 1 long
    bool whole;            // first product: shares of whole units, counted in units
    int end;
    int a, m, kb;          // next K block

    __device__ int start(int share) const { return share * size + (share < longer ? share : longer); }
    __device__ int line(const Sorted& p, int a_, int m_, int kb_) const {   // where a K block begins
        const int c = p.cost[a_ + 1] - p.cost[a_];
        return phase == kFirst ? p.cost[a_] * tiles * KB + (m_ * KB + kb_) * c
                               : (m_ * p.cost[p.nact] + p.cost[a_]) * KB + kb_ * c;
    }
    __device__ int holder(const Sorted& p, int a_, int m_, int kb_) const {   // the share it is in
        const int x = line(p, a_, m_, kb_), cut = longer * (size + 1);
        return x < cut ? x / (size + 1) : longer + (x - cut) / size;
    }
    template <typename T> __device__ void cut(const FewArgs& g, const Sorted& p, int product) {
        phase = product;
        tiles = product == kFirst ? g.tiles1 : g.tiles2;
        KB = product == kFirst ? g.KB1 : g.KB2;
        const int grid = (int)gridDim.x, nact = p.nact;
        const int units = nact * tiles;
        whole = false;
        if (product == kFirst) {
            // whole units: full rounds, and one of `rest` blocks that share the memory's
            // bandwidth; cut units: all blocks all the time, and the adding of parts
            const int full = units / grid, rest = units - full * grid;
            const float ns = kBlockNs * (float)p.most / (float)block_cost<T>(1);
            const float last = rest ? fmaxf(1.25f * ns * (float)rest / (float)grid, kLoneBlockNs * ns / kBlockNs) : 0.f;
            whole = (float)KB * ((float)full * ns + last) <=
                    (float)(KB * tiles) * (float)p.cost[nact] / (float)(grid * block_cost<T>(1)) * kBlockNs + kJoinNs;
        }
        const int total = whole ? units : p.cost[nact] * tiles * KB;
        // no share is shorter than a K block: each holds the beginning of one
        shares = whole || p.most == 1 ? total : total / p.most;
        shares = shares < grid ? shares : grid;
        size = total / shares;
        longer = total - size * shares;
    }
    __device__ void begin(const Sorted& p, int share) {
        me = share;
        a = m = kb = 0;
        int x = start(share);
        end = start(share + 1);
        if (whole) {
            a = x / tiles;
            m = x - a * tiles;
            return;
        }
        // the first K block that begins at or after x
        const int nact = p.nact, per = phase == kFirst ? tiles * KB : KB;   // K blocks an expert
        if (phase == kSecond) {
            m = x / (per * p.cost[nact]);
            x -= m * per * p.cost[nact];
        }
        int lo = 0, hi = nact;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cost[mid] * per <= x) lo = mid; else hi = mid;
        }
        a = lo;
        const int c = p.cost[a + 1] - p.cost[a];
        kb = x - p.cost[a] * per;
        if (c > 1) kb = (kb + c - 1) / c;
        if (phase == kFirst) {
            m = kb / KB;
            kb -= m * KB;
        }
        wrap(p);
    }
    __device__ void wrap(const Sorted& p) {   // past the end of a unit, an expert, a tile
        if (kb >= KB) {
            kb = 0;
            if (phase == kFirst) ++m; else ++a;
        }
        if (phase == kFirst && m >= tiles) { m = 0; ++a; }
        if (phase == kSecond && a >= p.nact) { a = 0; ++m; }
    }
    __device__ bool next(const Sorted& p, Seg& s) {
        if (whole) {
            if (a * tiles + m >= end) return false;
        } else if ((phase == kFirst ? a >= p.nact : m >= tiles) || line(p, a, m, kb) >= end) {
            return false;
        }
        s.a = a;
        s.m = m;
        s.kb0 = kb;
        s.kb1 = KB;
        s.c0 = s.c1 = me;
        if (!whole) {
            const int c = p.cost[a + 1] - p.cost[a];
            int n = end - line(p, a, m, kb);
            if (c > 1) n = (n + c - 1) / c;
            if (kb + n < KB) s.kb1 = kb + n;
            if (kb > 0) s.c0 = holder(p, a, m, 0);
            if (s.kb1 < KB) s.c1 = holder(p, a, m, KB - 1);
        }
        kb = s.kb1;
        wrap(p);
        return true;
    }
};

// The sorted rows, and how the two products are cut.
struct Plan : Sorted {
    Walk first, second;
};

// The gate of all tokens.  More tokens than the block's warps do in two turns are
// shared out, one to a block (measured for 64 tokens: 10 us for a block that does
// them all, 4 so); a block that another's result does not reach soon, because
// that block is not running, does them all.
__device__ __forceinline__ void gate_plan(Sorted& p, const FewArgs& g) {
    __shared__ int there;
    const int tokens = g.tokens, k = g.k, warps = blockDim.x >> 5;
    int32_t* status = blockIdx.x == 0 ? g.status : nullptr;
    if (tokens > 2 * warps && (int)gridDim.x >= tokens) {
        const int t = (int)blockIdx.x;
        if (t < tokens && threadIdx.x < 32) {
            gate_tokens(g.logits + t * g.E, 1, g.E, k, g.renorm, p.e_of, p.w, g.status);
            __syncwarp();
            if ((int)threadIdx.x < k)
                __stcg(&g.slots[t * k + threadIdx.x],
                       make_float2(__int_as_float(p.e_of[threadIdx.x]), p.w[threadIdx.x]));
            __syncwarp();
            if (threadIdx.x == 0) add_release(&g.cnt->gated, 1);
        }
        if (threadIdx.x == 0) {
            const uint64_t t0 = globaltimer_ns();
            int n;
            do n = load_acquire(&g.cnt->gated);
            while (n < tokens && globaltimer_ns() - t0 < kTakeOverNs);
            there = n >= tokens;
        }
        __syncthreads();
        if (there) {
            for (int i = threadIdx.x; i < tokens * k; i += blockDim.x) {
                const float2 v = __ldcg(&g.slots[i]);
                p.e_of[i] = (uint8_t)__float_as_int(v.x);
                p.w[i] = v.y;
            }
            return;
        }
    }
    gate_tokens(g.logits, tokens, g.E, k, g.renorm, p.e_of, p.w, status);
}

// Called by all threads of a block of at least 256.
template <typename T>
__device__ __forceinline__ void make_plan(Plan& p, const FewArgs& g) {
    const int tokens = g.tokens, k = g.k, E = g.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < E; e += blockDim.x) p.tokens[e] = 0ull;
    gate_plan(p, g);
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * k; i += blockDim.x)
        atomicOr(&p.tokens[p.e_of[i]], 1ull << (i / k));
    __syncthreads();
    if (warp == 0) {
        // Prefix sums over the experts, `per` of them a lane: (rows, has rows) in one
        // word, and cost.  (Loops, not unrolled: short code is fast code here.)
        const int per = (E + 31) >> 5, e0 = lane * per;
        int v = 0, c = 0, rows = 0;
        #pragma unroll 1
        for (int e = e0; e < e0 + per; ++e) {
            const int n = e < E ? __popcll(p.tokens[e]) : 0;
            if (n == 0) continue;
            v += n | 1 << 16;
            c += block_cost<T>(n);
            rows = n > rows ? n : rows;
        }
        const int own_v = v, own_c = c;
        #pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, v, o), uc = __shfl_up_sync(kFull, c, o);
            if (lane >= o) { v += u; c += uc; }
        }
        v -= own_v;
        c -= own_c;
        #pragma unroll 1
        for (int e = e0; e < e0 + per && e < E; ++e) {
            const int n = __popcll(p.tokens[e]);
            p.off[e] = v & 0xffff;
            if (n == 0) continue;
            p.act[v >> 16] = e;
            p.cost[v >> 16] = c;
            v += n | 1 << 16;
            c += block_cost<T>(n);
        }
        rows = (int)__reduce_max_sync(kFull, (unsigned)rows);
        if (lane == 31) {
            p.off[E] = v & 0xffff;
            p.nact = v >> 16;
            p.cost[v >> 16] = c;
            p.most_rows = rows;
            p.most = block_cost<T>(rows);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * k; i += blockDim.x) {
        const int e = p.e_of[i], t = i / k;
        const int r = p.off[e] + __popcll(p.tokens[e] & ((1ull << t) - 1ull));
        p.row_token[r] = (uint8_t)t;
        p.row_w[r] = p.w[i];
    }
    if (lane == 0 && warp >= 6 && warp < 8) {
        Walk& w = warp == 6 ? p.first : p.second;
        w.template cut<T>(g, p, warp - 6);
        if ((int)blockIdx.x < w.shares) w.begin(p, (int)blockIdx.x);
    }
    __syncthreads();
}

struct FewCtrl {
    uint64_t a_full[kMaxAStages], a_empty[kMaxAStages];
    uint64_t b_full[2][kMaxBStages];   // of each product
    uint64_t t_full[2], t_empty[2], drain;
    uint64_t q_full[2], q_empty[2];
    Walk queue[2];         // what the block's roles work on next
    uint32_t tmem;
    int abort_flag;
    int last;
};

constexpr int kAccCols = 128;   // columns of one of the two accumulators

__device__ __forceinline__ void few_abort(FewCtrl& c, int32_t* status) {
    *(volatile int*)&c.abort_flag = 1;
    report(status, MOE_ERR_TIMEOUT);
}

__device__ __forceinline__ void fence_proxy_async_all() {
    asm volatile("fence.proxy.async;" ::: "memory");
}
template <int N> __device__ __forceinline__ void epilogue_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// Columns of this thread's TMEM lane: four in a row, or any two.
__device__ __forceinline__ void tmem_ld4(uint32_t addr, float (&v)[4]) {
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    #pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld_pair(uint32_t addr0, uint32_t addr1, float& a, float& b) {
    uint32_t r0, r1;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r0) : "r"(addr0));
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r1) : "r"(addr1));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    a = __uint_as_float(r0);
    b = __uint_as_float(r1);
}

// a barrier that also says whether `ok` holds on every thread: the epilogue goes
// on or gives up as one
template <int N> __device__ __forceinline__ bool epilogue_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, %2, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(N)
        : "memory");
    return r != 0;
}

// The activations' ring.  A K block's slot is as large as the product needs, so
// each product has its own number of slots in the same memory, and its own
// barriers for their filling.  What empties a slot is the K block's weights'
// stage being emptied (one completion for both): there are no more slots than
// stages, so that the stage is not in use again before the slot's next K block.
struct Ring {
    uint32_t base, full;   // shared addresses of the slots and their barriers
    int slots, bytes;
    int slot;
    uint32_t parity;
    __device__ void set(FewCtrl& c, const FewArgs& g, uint8_t* memory, int product, int rows, int box) {
        base = smem_u32(memory);
        full = smem_u32(c.b_full[product]);
        bytes = (rows + box - 1) / box * box * kBlockBytes;
        slots = g.b_ring / bytes;
        slots = slots < kMaxBStages ? slots : kMaxBStages;
        slots = slots < g.a_stages ? slots : g.a_stages;
        slot = 0;
        parity = 0;
    }
    __device__ uint32_t at() const { return base + slot * bytes; }
    __device__ uint32_t bar() const { return full + slot * 8; }
    __device__ void step() {
        if (++slot == slots) { slot = 0; parity ^= 1; }
    }
};

// A role's view of the queue of shares.
struct Reader {
    int slot = 0;
    uint32_t parity = 0;
    __device__ void step() {
        if (++slot == 2) { slot = 0; parity ^= 1; }
    }
};

// 16 bytes of shared memory at a 32-bit address
__device__ __forceinline__ ulonglong2 lds16(uint32_t at) {
    ulonglong2 v;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(at) : "memory");
    return v;
}

// fp32 products on the CUDA cores: 8 warps, a lane holding 4 weight rows and NC
// activation rows.  With more than NC rows the warps split them into `groups`
// (1, 2, 4 or 8) and K into 8 / groups; sums run over even and odd k apart, as
// packed pairs.  The result goes to red[K slice][row][128].  One 16-byte chunk of
// the K block a turn, all its loads first, and the turns not unrolled: five copies
// of this loop share the instruction cache, and each runs for a few microseconds
// (33 tokens on 64 experts of 768 x 3072: 57.9 us, unrolled 62.2; 8 tokens on 16
// of 2048 x 8192: 226 us against 237, of which the products cost 5).
template <int NC, int GROUPS>
__device__ __forceinline__ bool products_f32(const FewArgs& g, FewCtrl& c, const Seg& s, bool first,
                                             int rows, const uint8_t* row_token,
                                             uint32_t a_ring, int& as, uint32_t& ap, Ring& b, int ew, int lane,
                                             float* red) {
    const int grp = ew % GROUPS, slice = ew / GROUPS;
    uint32_t brow[NC];
    #pragma unroll
    for (int j = 0; j < NC; ++j) {
        int r = grp * NC + j;
        r = r < rows ? r : rows - 1;
        const uint32_t q = first ? row_token[r] : r;
        brow[j] = q * 128 + ((q & 7) << 4);   // the row with its swizzle
    }
    uint64_t acc[4][NC];
    #pragma unroll
    for (int q = 0; q < 4; ++q)
        #pragma unroll
        for (int j = 0; j < NC; ++j) acc[q][j] = 0ull;
    for (int kb = s.kb0; kb < s.kb1; ++kb) {
        if (!mbar_wait_warp(smem_u32(&c.a_full[as]), ap, g.limit_ns, &c.abort_flag) ||
            !mbar_wait_warp(b.bar(), b.parity, g.limit_ns, &c.abort_flag))
            return false;
        const uint32_t A = a_ring + as * kABytes + (lane << 7) + ((lane & 7) << 4);
        const uint32_t B = b.at();
        #pragma unroll 1
        for (int i = 0; i < GROUPS; ++i) {
            const uint32_t ch = (slice * GROUPS + i) << 4;   // 16-byte chunk of the K block
            ulonglong2 a[4];
            #pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = lds16((A ^ ch) + q * 4096);
            ulonglong2 x[NC];
            #pragma unroll
            for (int j = 0; j < NC; ++j) x[j] = lds16(B + (brow[j] ^ ch));
            #pragma unroll
            for (int j = 0; j < NC; ++j)
                #pragma unroll
                for (int q = 0; q < 4; ++q) acc[q][j] = f2_fma(a[q].x, x[j].x, acc[q][j]);
            #pragma unroll
            for (int j = 0; j < NC; ++j)
                #pragma unroll
                for (int q = 0; q < 4; ++q) acc[q][j] = f2_fma(a[q].y, x[j].y, acc[q][j]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.a_empty[as]));
        if (++as == g.a_stages) { as = 0; ap ^= 1; }
        b.step();
    }
    #pragma unroll
    for (int j = 0; j < NC; ++j)
        #pragma unroll
        for (int q = 0; q < 4; ++q) {
            float e, o;
            f2_unpack(acc[q][j], e, o);
            red[((slice * GROUPS + grp) * NC + j) * kTileM + lane + 32 * q] = e + o;
        }
    return true;
}

// Adds the parts that shares wrote of a unit, in their order: to = (p[c0 + 1] + ... + p[c1]),
// + p[c0] with `own`.  Four float4 and two parts at a time, so that their loads overlap (33
// fp32 tokens on 64 experts: 57.3 us with one value and one part at a time, 55.6 so).  A function of
// its own, since a launch runs it about once: one copy to fetch, not two.
template <int NT>
__device__ __noinline__ void add_parts(const float* part1, int tokens, int c0, int c1, bool own,
                                       int rows, int tid, float4* to) {
    const int n = rows * (kTileM / 4), parts = c1 - c0 + (own ? 1 : 0);
    const int64_t slot = (int64_t)tokens * (kTileM / 4);
    const float4* base = reinterpret_cast<const float4*>(part1) + c0 * 2 * slot;
    auto part = [&](int x) {   // the x-th to be added; a share that a unit starts in uses its second slot
        return x >= parts ? nullptr : x < c1 - c0 ? base + (x + 1) * 2 * slot : base + slot;
    };
    #pragma unroll 1
    for (int i = tid; i < n; i += 4 * NT) {
        float4 v[4];
        #pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        #pragma unroll 1
        for (int x = 0; x < parts; x += 2) {
            const float4* p0 = part(x);
            const float4* p1 = part(x + 1);
            float4 w[2][4];
            #pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at = i + u * NT;
                w[0][u] = at < n ? __ldcg(p0 + at) : make_float4(0.f, 0.f, 0.f, 0.f);
                w[1][u] = p1 && at < n ? __ldcg(p1 + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            #pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[u].x = v[u].x + w[0][u].x + w[1][u].x;
                v[u].y = v[u].y + w[0][u].y + w[1][u].y;
                v[u].z = v[u].z + w[0][u].z + w[1][u].z;
                v[u].w = v[u].w + w[0][u].w + w[1][u].w;
            }
        }
        #pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * NT < n) to[i + u * NT] = v[u];
    }
}

template <typename T>
__global__ void __launch_bounds__(few_threads<T>(), 1)
    few_experts_kernel(const __grid_constant__ CUtensorMap mapW1, const __grid_constant__ CUtensorMap mapX,
                       const __grid_constant__ CUtensorMap mapW2, const __grid_constant__ CUtensorMap mapH,
                       const __grid_constant__ FewArgs g) {
    using K = Kind<T>;
    constexpr int BOX = K::kBox, RPS = K::kRowsPerSlot;
    extern __shared__ __align__(1024) uint8_t few_smem[];
    uint8_t* a_ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(few_smem) + 1023) & ~(uintptr_t)1023);
    uint8_t* b_ring = a_ring + (size_t)g.a_stages * kABytes;
    float* yacc = reinterpret_cast<float*>(b_ring + g.b_ring);  // [T][128]
    float* red = yacc + g.tokens * kTileM;      // fp32 only
    __shared__ Plan plan;
    __shared__ FewCtrl c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        const int consumers = K::kTensor ? 1 : K::kEpilogue / 32;
        #pragma unroll 1
        for (int i = 0; i < g.a_stages; ++i) {
            mbar_init(smem_u32(&c.a_full[i]), 1);
            mbar_init(smem_u32(&c.a_empty[i]), consumers);
        }
        #pragma unroll 1
        for (int i = 0; i < 2 * kMaxBStages; ++i) {
            mbar_init(smem_u32(&c.b_full[i / kMaxBStages][i % kMaxBStages]), 1);
        }
        #pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c.t_full[i]), 1);
            mbar_init(smem_u32(&c.t_empty[i]), K::kEpilogue / 32);
            mbar_init(smem_u32(&c.q_full[i]), 1);
            mbar_init(smem_u32(&c.q_empty[i]), K::kEpilogue / 32 + (K::kTensor ? 2 : 1));
        }
        mbar_init(smem_u32(&c.drain), 1);
        c.abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&mapW1);
        tma_prefetch_map(&mapX);
        tma_prefetch_map(&mapW2);
        tma_prefetch_map(&mapH);
    }
    if (K::kTensor && warp == 2) {
        tmem_alloc(smem_u32(&c.tmem), 2 * kAccCols);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (on its way while the plan is made)
    int taken = threadIdx.x == 0 ? atomicCAS(&g.cnt->claim[kFirst][blockIdx.x], 0, 1) : 0;
    make_plan<T>(plan, g);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = K::kTensor ? c.tmem : 0u;
    Walk walk;
    Seg s;
    Reader q;
    // B, MMA: the next entry of the queue, by one thread
    auto take = [&]() {
        if (!mbar_wait_bounded(smem_u32(&c.q_full[q.slot]), q.parity, g.limit_ns, &c.abort_flag)) {
            few_abort(c, g.status);
            return false;
        }
        walk = c.queue[q.slot];
        mbar_arrive(smem_u32(&c.q_empty[q.slot]));
        q.step();
        return walk.phase != kEnd;
    };

    if (warp == 0) {
        // ---- shares, and weights: one box of 128 rows a K block ------------------------
        // Block b takes share b of each product.  It goes on to the second product (whose
        // products wait for the whole of the first) and to the summing (which waits for
        // all parts) only when every share before has a block that works on it, and
        // takes over one that has none for long: the block it is meant for may wait
        // for an SM that this kernel, or another, holds.  So nothing waits for a block
        // that does not run, and blocks need not be resident together.
        if (lane == 0) {
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto post = [&](const Walk& w) {
                if (!mbar_wait_bounded(smem_u32(&c.q_empty[q.slot]), q.parity ^ 1, g.limit_ns,
                                       &c.abort_flag)) {
                    few_abort(c, g.status);
                    return false;
                }
                c.queue[q.slot] = w;
                mbar_arrive(smem_u32(&c.q_full[q.slot]));
                q.step();
                return true;
            };
            #pragma unroll 1
            for (int product = kFirst; product <= kSecond && ok; ++product) {
                walk = product == kFirst ? plan.first : plan.second;
                const CUtensorMap* map = product == kFirst ? &mapW1 : &mapW2;
                int* claim = g.cnt->claim[product];
                if (product == kSecond) taken = atomicCAS(&claim[blockIdx.x], 0, 1);
                int share = (int)blockIdx.x < walk.shares && taken == 0 ? (int)blockIdx.x : -1;
                while (ok) {
                    if (share >= 0) {
                        atomicAdd(&g.cnt->claimed[product], 1);
                        if (share != (int)blockIdx.x) walk.begin(plan, share);
                        ok = post(walk);
                        while (ok && walk.next(plan, s)) {
                            const int e = plan.act[s.a];
                            for (int kb = s.kb0; kb < s.kb1; ++kb) {
                                if (!mbar_wait_bounded(smem_u32(&c.a_empty[st]), ph ^ 1, g.limit_ns,
                                                       &c.abort_flag)) {
                                    few_abort(c, g.status);
                                    ok = false;
                                    break;
                                }
                                mbar_arrive_expect_tx(smem_u32(&c.a_full[st]), kABytes);
                                tma_load_3d(smem_u32(a_ring + st * kABytes), map,
                                            smem_u32(&c.a_full[st]), kb * K::kBlock, s.m * kTileM, e);
                                if (issued < g.a_stages) ++issued;
                                if (++st == g.a_stages) { st = 0; ph ^= 1; }
                            }
                        }
                    }
                    share = -1;
                    const uint64_t t0 = globaltimer_ns();
                    uint64_t t1 = t0;
                    while (ok && load_acquire(&g.cnt->claimed[product]) < walk.shares) {
                        const uint64_t now = globaltimer_ns();
                        if (now - t1 > kTakeOverNs) {
                            for (int i = 0; i < walk.shares && share < 0; ++i)
                                if (load_acquire(&claim[i]) == 0 && atomicCAS(&claim[i], 0, 1) == 0)
                                    share = i;
                            if (share >= 0) break;
                            t1 = globaltimer_ns();
                        }
                        if (now - t0 > g.limit_ns || *(volatile int*)&c.abort_flag) {
                            few_abort(c, g.status);
                            ok = false;
                        }
                    }
                    if (share < 0) break;
                }
            }
            while (ok) {
                walk.phase = kSum;
                walk.me = atomicAdd(&g.cnt->sums, 1);
                if (walk.me >= g.tiles2 * g.slices) break;
                ok = post(walk);
            }
            walk.phase = kEnd;
            if (ok) post(walk);
            // copies in flight land before the block ends
            for (int i = 0; i < issued; ++i) {
                if (--st < 0) { st = g.a_stages - 1; ph ^= 1; }
                mbar_wait_bounded(smem_u32(&c.a_full[st]), ph, kDrainNs, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- activations: all tokens' K block of x, or the expert's hidden rows -------
        if (lane == 0) {
            Ring r;
            r.set(c, g, b_ring, kFirst, g.tokens, BOX);
            int issued = 0, st = 0;        // st, ph: weights' stage to wait for next
            uint32_t ph = 0;
            bool second = false, ok = true;
            auto emptied = [&]() {         // the oldest K block not yet waited for
                ok = mbar_wait_bounded(smem_u32(&c.a_empty[st]), ph, g.limit_ns, &c.abort_flag);
                if (!ok) {   // its copy may still be in flight: it stays among the issued ones
                    few_abort(c, g.status);
                    return;
                }
                if (++st == g.a_stages) { st = 0; ph ^= 1; }
                --issued;
            };
            while (ok && take()) {
                if (walk.phase == kSum) continue;
                bool more = walk.next(plan, s);
                if (walk.phase == kSecond && !second) {
                    while (ok && issued > 0) emptied();   // the first product's slots are free
                    if (!ok) break;                       // (or their ring is the one to drain)
                    second = true;
                    r.set(c, g, b_ring, kSecond, plan.most_rows * RPS, BOX);
                    // All hidden rows are written.  (One counter for all experts: the
                    // shares are equal, so that waiting for some of them first gains nothing,
                    // and each further poll would cost a round trip to the L2.)
                    const uint64_t t0 = globaltimer_ns();
                    while (ok && load_acquire(&g.cnt->done) < plan.nact * g.tiles1)
                        ok = !*(volatile int*)&c.abort_flag && globaltimer_ns() - t0 <= g.limit_ns;
                    if (!ok) {
                        few_abort(c, g.status);
                        break;
                    }
                    fence_proxy_async_all();
                }
                for (; ok && more; more = walk.next(plan, s)) {
                    const int e = plan.act[s.a];
                    const int row0 = second ? plan.off[e] * RPS : 0;
                    const int rows = second ? (plan.off[e + 1] - plan.off[e]) * RPS : g.tokens;
                    const int boxes = (rows + BOX - 1) / BOX;
                    const CUtensorMap* map = second ? &mapH : &mapX;
                    for (int kb = s.kb0; kb < s.kb1; ++kb) {
                        if (issued == r.slots) emptied();
                        if (!ok) break;
                        mbar_arrive_expect_tx(r.bar(), boxes * BOX * kBlockBytes);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(r.at() + i * BOX * kBlockBytes, map, r.bar(), kb * K::kBlock,
                                        row0 + i * BOX);
                        ++issued;
                        r.step();
                    }
                }
            }
            // copies in flight land before the block ends
            for (int i = 0; i < issued; ++i) {
                if (--r.slot < 0) { r.slot = r.slots - 1; r.parity ^= 1; }
                mbar_wait_bounded(r.bar(), r.parity, kDrainNs, nullptr);
            }
        }
        __syncwarp();
    } else if (K::kTensor && warp == 2) {
        // ---- tensor core: D[128 weight rows][activation rows], one accumulator a segment --
        if (lane == 0) {
            // One thread: between two K blocks it does as little as it can (the low words
            // of the operands' descriptors move by the stage; the high words are alike).
            Ring r;
            r.set(c, g, b_ring, kFirst, g.tokens, BOX);
            int as = 0, acc = 0;
            uint32_t ap = 0, tp = 0;
            bool second = false, ok = true;
            const uint64_t a0 = smem_desc_sw128(smem_u32(a_ring), 16, 1024);
            const uint64_t b0 = smem_desc_sw128(r.base, 16, 1024);
            const uint32_t a_full = smem_u32(c.a_full), a_empty = smem_u32(c.a_empty);
            while (ok && take()) {
                if (walk.phase == kSum) continue;
                if (walk.phase == kSecond && !second) {
                    second = true;
                    r.set(c, g, b_ring, kSecond, plan.most_rows * RPS, BOX);
                }
                while (ok && walk.next(plan, s)) {
                    const int e = plan.act[s.a];
                    const int rows = second ? (plan.off[e + 1] - plan.off[e]) * RPS : g.tokens;
                    const uint32_t idesc = idesc_bf16_f32(kTileM, (rows + 15) & ~15, false, false);
                    const uint32_t d_tmem = tmem + acc * kAccCols;
                    if (!mbar_wait_bounded(smem_u32(&c.t_empty[acc]), tp ^ 1, g.limit_ns, &c.abort_flag)) {
                        few_abort(c, g.status);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint32_t more = 0;
                    for (int n = s.kb1 - s.kb0; n > 0; --n) {
                        if (!mbar_wait_bounded(a_full + as * 8, ap, g.limit_ns, &c.abort_flag) ||
                            !mbar_wait_bounded(r.bar(), r.parity, g.limit_ns, &c.abort_flag)) {
                            few_abort(c, g.status);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = a0 + as * (kABytes >> 4);
                        const uint64_t bd = b0 + r.slot * (r.bytes >> 4);
                        #pragma unroll
                        for (int kk = 0; kk < K::kBlock / 16; ++kk) {
                            tc_mma_bf16(d_tmem, ad + kk * 2, bd + kk * 2, idesc, more);
                            more = 1;
                        }
                        tc_commit(a_empty + as * 8);
                        if (++as == g.a_stages) { as = 0; ap ^= 1; }
                        r.step();
                    }
                    if (!ok) break;
                    tc_commit(smem_u32(&c.t_full[acc]));
                    if (++acc == 2) { acc = 0; tp ^= 1; }
                }
            }
            // every MMA issued has completed before TMEM is freed
            tc_commit(smem_u32(&c.drain));
            mbar_wait_bounded(smem_u32(&c.drain), 0, kDrainNs, nullptr);
        }
        __syncwarp();
    } else if (warp >= kWarpsBeforeEpilogue) {
        // ---- epilogue -----------------------------------------------------------------
        // STEP threads own weight row i of the tile, i.e. one output feature: they take
        // the activation rows in turn (bf16: by twos).
        constexpr int NT = K::kEpilogue, STEP = NT / kTileM;
        const int tid = threadIdx.x - kWarpsBeforeEpilogue * 32;
        const int ew = tid >> 5, t_first = tid / kTileM;
        const int i = K::kTensor ? (warp & 3) * 32 + lane : tid & 127;
        const int64_t slot_floats = (int64_t)g.tokens * kTileM;
        T* hidden = (T*)g.hidden;
        const T* residual = (const T*)g.residual;
        T* y = (T*)g.y;
        int acc = 0, as = 0;
        uint32_t tp = 0, ap = 0;
        Ring ring;
        if (!K::kTensor) ring.set(c, g, b_ring, kFirst, g.tokens, BOX);
        bool second = false, ok = true;
        auto put_y = [&](int64_t o, float v) {
            if (residual) v += to_f32<T>(residual[o]);
            y[o] = from_f32<T>(v);
        };
        auto put_y4 = [&](int64_t o, float4 v) {   // four columns (o is a multiple of four)
            if constexpr (K::kTensor) {
                if (residual) {
                    const uint2 q = *reinterpret_cast<const uint2*>(residual + o);
                    v.x += __uint_as_float(q.x << 16);
                    v.y += __uint_as_float(q.x & 0xffff0000u);
                    v.z += __uint_as_float(q.y << 16);
                    v.w += __uint_as_float(q.y & 0xffff0000u);
                }
                const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
                *reinterpret_cast<uint2*>(y + o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                              *reinterpret_cast<const uint32_t*>(&b));
            } else {
                if (residual) {
                    const float4 q = *reinterpret_cast<const float4*>(residual + o);
                    v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
                }
                *reinterpret_cast<float4*>(y + o) = v;
            }
        };
        while (true) {
            ok = mbar_wait_warp(smem_u32(&c.q_full[q.slot]), q.parity, g.limit_ns, &c.abort_flag);
            if (!ok) few_abort(c, g.status);
            if (!epilogue_all<NT>(ok)) break;
            walk = c.queue[q.slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.q_empty[q.slot]));
            q.step();
            if (walk.phase == kEnd) break;
            const int me = walk.me;
            if (walk.phase == kSum) {
                // A slice of the tokens of an output tile that several shares have a part
                // of: once all parts are there, they are added in the shares' order.
                const int m = me / g.slices, sl = me - m * g.slices;
                const Walk& w = plan.second;
                const int d0 = w.holder(plan, 0, m, 0);
                const int d1 = w.holder(plan, plan.nact - 1, m, w.KB - 1);
                const int lo = g.tokens * sl / g.slices, hi = g.tokens * (sl + 1) / g.slices;
                if (d0 == d1 || lo == hi) continue;
                if (tid == 0) {
                    const uint64_t t0 = globaltimer_ns();
                    while (ok && load_acquire(&g.tiles_done[m]) < d1 - d0 + 1)
                        ok = !*(volatile int*)&c.abort_flag && globaltimer_ns() - t0 <= g.limit_ns;
                    if (!ok) few_abort(c, g.status);
                }
                if (!epilogue_all<NT>(ok)) break;
                // four columns a thread
                const int col = (tid & 31) * 4;
                if (m * kTileM + col >= g.d) continue;
                constexpr int PB = 8;   // parts at a time, so that their loads overlap
                #pragma unroll 1
                for (int t = lo + ew; t < hi; t += NT / 32) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    #pragma unroll 1
                    for (int b = d0; b <= d1; b += PB) {
                        float4 u[PB];
                        #pragma unroll
                        for (int j = 0; j < PB; ++j) {
                            u[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (b + j <= d1)
                                u[j] = __ldcg(reinterpret_cast<const float4*>(
                                    g.part2 + ((b + j) * 2 + (b + j == d0)) * slot_floats + t * kTileM + col));
                        }
                        #pragma unroll
                        for (int j = 0; j < PB; ++j) {
                            v.x += u[j].x; v.y += u[j].y; v.z += u[j].z; v.w += u[j].w;
                        }
                    }
                    put_y4((int64_t)t * g.d + m * kTileM + col, v);
                }
                continue;
            }
            if (walk.phase == kSecond && !second) {
                second = true;
                if (!K::kTensor) ring.set(c, g, b_ring, kSecond, plan.most_rows * RPS, BOX);
            }
            bool fresh = true;     // yacc holds nothing yet
            bool more = walk.next(plan, s);
            while (more) {
                const int e = plan.act[s.a];
                const int r0 = plan.off[e], rows = plan.off[e + 1] - r0;
                const int col = s.m * kTileM + i, width = second ? g.d : g.f;
                const bool whole = s.c0 == s.c1;   // no other share has a part of the unit
                const bool live = col < width;
                const T* bias = (const T*)(second ? g.b2 : g.b1);
                const float b = bias && live && s.kb0 == 0
                                    ? to_f32<T>(bias[(int64_t)e * width + col]) : 0.f;
                // unit of the first product cut over shares c0..c1
                const int c0 = s.c0, c1 = s.c1;
                float* mine = g.part1 + (me * 2 + (me == c0)) * slot_floats;
                if (second && fresh) {
                    epilogue_barrier<NT>();
                    for (int t = t_first; t < g.tokens; t += STEP) yacc[t * kTileM + i] = 0.f;
                    fresh = false;
                }
                // The share that a cut unit starts in comes to it last, and mostly finds the
                // others' parts written: then it adds them up (in yacc, which the first
                // product does not use) while the tensor core works on its own.
                bool rest = false;
                if (!second && !whole && me == c0) {
                    if (tid == 0) rest = load_acquire(&g.cnt->joined[c0]) == c1 - c0;
                    rest = epilogue_all<NT>(tid != 0 || rest);
                    if (rest) {
                        add_parts<NT>(g.part1, g.tokens, c0, c1, false, rows, tid, reinterpret_cast<float4*>(yacc));
                    }
                }
                // activation rows r and, with `two`, r + 1 of the expert
                auto put_hidden = [&](int r, bool two, float h0, float h1) {
                    if (!live) return;
                    if constexpr (K::kTensor) {
                        // GELU in two bf16 parts, 16 bits together
                        float v0, v1;
                        f2_unpack(gelu_two(h0, h1), v0, v1);
                        const __nv_bfloat162 hi = __floats2bfloat162_rn(v0, v1);
                        const float l0 = v0 - __low2float(hi), l1 = v1 - __high2float(hi);
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(isfinite(l0) ? l0 : 0.f,
                                                                        isfinite(l1) ? l1 : 0.f);
                        __nv_bfloat16* p = hidden + (int64_t)(r0 + r) * 2 * g.f + col;
                        p[0] = hi.x;
                        p[g.f] = lo.x;
                        if (two) {
                            p[2 * (int64_t)g.f] = hi.y;
                            p[3 * (int64_t)g.f] = lo.y;
                        }
                    } else {
                        hidden[(int64_t)(r0 + r) * g.f + col] = gelu_call(h0);
                    }
                };
                auto emit = [&](int r, bool two, float v0, float v1) {
                    v0 += b;
                    v1 += b;
                    if (second) {
                        float* p = yacc + plan.row_token[r0 + r] * kTileM + i;
                        *p = fmaf(plan.row_w[r0 + r], v0, *p);
                        if (two) {
                            p = yacc + plan.row_token[r0 + r + 1] * kTileM + i;
                            *p = fmaf(plan.row_w[r0 + r + 1], v1, *p);
                        }
                    } else if (whole || rest) {
                        if (rest) {
                            v0 += yacc[r * kTileM + i];
                            if (two) v1 += yacc[(r + 1) * kTileM + i];
                        }
                        put_hidden(r, two, v0, v1);
                    } else {
                        __stcg(mine + r * kTileM + i, v0);
                        if (two) __stcg(mine + (r + 1) * kTileM + i, v1);
                    }
                };
                if constexpr (K::kTensor) {
                    ok = mbar_wait_warp(smem_u32(&c.t_full[acc]), tp, g.limit_ns, &c.abort_flag);
                    if (!ok) few_abort(c, g.status);
                    if (!epilogue_all<NT>(ok)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc * kAccCols;
                    // Two rows a turn, not unrolled: instructions that run once cost more to
                    // fetch than these turns cost to wait for (7 us a unit of 16 rows against 2).
                    #pragma unroll 1
                    for (int r = 2 * t_first; r < rows; r += 2 * STEP) {
                        const bool two = r + 1 < rows;
                        float v[4];
                        if (second) {
                            tmem_ld4(base + 2 * r, v);   // high and low part of both rows
                            v[0] += v[1];
                            v[1] = v[2] + v[3];
                        } else {
                            tmem_ld_pair(base + plan.row_token[r0 + r],
                                         base + plan.row_token[r0 + (two ? r + 1 : r)], v[0], v[1]);
                        }
                        emit(r, two, v[0], v[1]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&c.t_empty[acc]));
                    if (++acc == 2) { acc = 0; tp ^= 1; }
                } else {
                    const int groups = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
                    const int nc = rows <= 4 ? 4 : 8;
                    const uint8_t* rt = plan.row_token + r0;
                    if (rows <= 4)
                        ok = products_f32<4, 1>(g, c, s, !second, rows, rt, smem_u32(a_ring), as, ap, ring, ew, lane, red);
                    else if (rows <= 8)
                        ok = products_f32<8, 1>(g, c, s, !second, rows, rt, smem_u32(a_ring), as, ap, ring, ew, lane, red);
                    else if (rows <= 16)
                        ok = products_f32<8, 2>(g, c, s, !second, rows, rt, smem_u32(a_ring), as, ap, ring, ew, lane, red);
                    else if (rows <= 32)
                        ok = products_f32<8, 4>(g, c, s, !second, rows, rt, smem_u32(a_ring), as, ap, ring, ew, lane, red);
                    else
                        ok = products_f32<8, 8>(g, c, s, !second, rows, rt, smem_u32(a_ring), as, ap, ring, ew, lane, red);
                    if (!ok) few_abort(c, g.status);
                    if (!epilogue_all<NT>(ok)) { ok = false; break; }
                    const int cols = groups * nc;
                    for (int r = t_first; r < rows; r += STEP) {
                        float v = 0.f;
                        for (int x = 0; x < 8 / groups; ++x) v += red[(x * cols + r) * kTileM + i];
                        emit(r, false, v, 0.f);
                    }
                    epilogue_barrier<NT>();
                }
                const int m = s.m;
                more = walk.next(plan, s);
                if (!second) {
                    bool finished = whole || rest;
                    if (!finished) {
                        // the last share to write its part adds the parts, in their order
                        epilogue_barrier<NT>();
                        if (tid == 0) c.last = add_acq_rel(&g.cnt->joined[c0], 1) == c1 - c0;
                        epilogue_barrier<NT>();
                        finished = c.last;
                        if (finished) {
                            add_parts<NT>(g.part1, g.tokens, c0, c1, true, rows, tid, reinterpret_cast<float4*>(yacc));
                            epilogue_barrier<NT>();
                            // one row (bf16: two) a turn, short code: it runs once
                            constexpr int W = K::kTensor ? 2 : 1;
                            #pragma unroll 1
                            for (int r = W * t_first; r < rows; r += W * STEP) {
                                const bool two = K::kTensor && r + 1 < rows;
                                put_hidden(r, two, yacc[r * kTileM + i], two ? yacc[(r + 1) * kTileM + i] : 0.f);
                            }
                        }
                    }
                    if (finished) {
                        epilogue_barrier<NT>();
                        if (tid == 0) {
                            fence_proxy_async_all();   // the rows are read by TMA
                            add_release(&g.cnt->done, 1);
                        }
                    }
                    continue;
                }
                // second product: the tile is left when the next segment is another's
                if (more && s.m == m) continue;
                fresh = true;
                const int d0 = walk.holder(plan, 0, m, 0);
                const int d1 = walk.holder(plan, plan.nact - 1, m, walk.KB - 1);
                epilogue_barrier<NT>();
                if (d0 == d1) {
                    for (int t = t_first; t < g.tokens && live; t += STEP)
                        put_y((int64_t)t * g.d + col, yacc[t * kTileM + i]);
                    continue;
                }
                float4* out = reinterpret_cast<float4*>(g.part2 + (me * 2 + (me == d0)) * slot_floats);
                for (int x = tid; x < g.tokens * (kTileM / 4); x += NT)
                    __stcg(out + x, reinterpret_cast<const float4*>(yacc)[x]);
                epilogue_barrier<NT>();
                if (tid == 0) add_release(&g.tiles_done[m], 1);
            }
            if (!ok) break;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (K::kTensor && warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kAccCols);
    }
}

// ---- host ---------------------------------------------------------------------------

size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

int few_blocks() {
    const int n = device_sm_count();
    return n < kMaxBlocks ? n : kMaxBlocks;
}

struct FewLayout {
    size_t logits, slots, counters, hidden, part1, part2, total;
};
FewLayout few_layout(const moe_shape& s) {
    FewLayout l;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t a = at; at += pad256(n); return a; };
    const size_t part = sizeof(float) * few_blocks() * 2 * s.T * kTileM;
    l.logits = take(sizeof(float) * s.T * s.E);
    l.slots = take(sizeof(float2) * s.T * s.k);
    l.counters = take(sizeof(Counters) + sizeof(int) * ((s.d + kTileM - 1) / kTileM));
    l.hidden = take((size_t)4 * s.T * s.k * s.f);   // fp32, or two bf16 parts
    l.part1 = take(part);
    l.part2 = take(part);
    l.total = at;
    return l;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// [n2][n1][n0] of T (n0 innermost), boxes of one K block x `rows` rows, 128-byte
// swizzle, zero outside
template <typename T>
bool few_map(CUtensorMap* m, const void* p, uint64_t n0, uint64_t n1, uint64_t n2, uint32_t rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const int rank = n2 ? 3 : 2;
    const cuuint64_t dims[3] = {n0, n1, n2};
    const cuuint64_t strides[2] = {n0 * sizeof(T), n0 * n1 * sizeof(T)};
    const cuuint32_t box[3] = {(cuuint32_t)Kind<T>::kBlock, rows, 1}, step[3] = {1, 1, 1};
    return fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
              rank, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// All that a block may have: with less it would still not share an SM with a block of the
// logits kernel, for want of registers.
constexpr int kFewSmem = 227 * 1024;

template <typename T> cudaError_t few_smem_limit(int* dynamic) {
    // what the static part leaves; set once for each device, as the limit is the device's
    static std::mutex lock;
    static int limit[64] = {0};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> hold(lock);
    if (limit[dev] == 0) {
        cudaFuncAttributes a;
        err = cudaFuncGetAttributes(&a, few_experts_kernel<T>);
        if (err != cudaSuccess) return err;
        const int most = (kFewSmem - (int)a.sharedSizeBytes) & ~127;
        err = cudaFuncSetAttribute(few_experts_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   most);
        if (err != cudaSuccess) return err;
        limit[dev] = most;
    }
    *dynamic = limit[dev];
    return cudaSuccess;
}

template <typename T, int TT, int RW, int U>
cudaError_t launch_direct(DirectArgs& g, cudaStream_t st) {
    constexpr int W = kDirectThreads / 32, step = 32 * Vec<T>::N;
    const int most = device_sm_count() * direct_blocks_per_sm<TT>();
    // Warps share a group of rows (each taking every n-th step along K) until there
    // are tasks for all blocks, then, while each keeps a full batch of loads, until
    // there are four a block: with fewer, blocks that take one more than the others
    // are what the rest waits for.
    auto split = [&](int64_t groups, int steps) {
        int n = 1;
        while (n < W) {
            const int64_t tasks = groups * n / W;
            if (tasks >= 4 * most || steps < (tasks < most ? 4 * n : 2 * n * U)) break;
            n *= 2;
        }
        return n;
    };
    const int experts = g.tokens * g.k < g.E ? g.tokens * g.k : g.E;
    const int64_t g1 = (g.f + RW - 1) / RW, g2 = (g.d + RW - 1) / RW;
    g.split1 = split(g1 * g.k, (g.d + step - 1) / step);
    g.split2 = split(g2, g.k * ((g.f + step - 1) / step));
    const int64_t tasks = experts * ((g1 * g.split1 + W - 1) / W) + (g2 * g.split2 + W - 1) / W;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(tasks < most ? tasks : most));
    cfg.blockDim = dim3(kDirectThreads);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few_direct_kernel<T, TT, RW, U>, g);
}

template <typename T>
cudaError_t run(const moe_shape& s, const moe_layer_params& p, const T* x, const T* residual, T* y,
                uint8_t* ws, int32_t* status, cudaStream_t st) {
    using K = Kind<T>;
    const FewLayout l = few_layout(s);
    const int t = (int)s.T;
    FewArgs g;
    g.tokens = t;
    g.d = s.d; g.f = s.f; g.E = s.E; g.k = s.k; g.renorm = s.renorm;
    const int KBlock = K::kBlock;
    g.tiles1 = (s.f + kTileM - 1) / kTileM;
    g.tiles2 = (s.d + kTileM - 1) / kTileM;
    g.KB1 = (s.d + KBlock - 1) / KBlock;
    g.KB2 = (s.f + KBlock - 1) / KBlock;
    g.logits = (float*)(ws + l.logits);
    g.slots = (float2*)(ws + l.slots);
    g.b1 = p.b1; g.b2 = p.b2; g.residual = residual; g.y = y;
    g.hidden = ws + l.hidden;
    g.part1 = (float*)(ws + l.part1);
    g.part2 = (float*)(ws + l.part2);
    g.cnt = (Counters*)(ws + l.counters);
    g.tiles_done = (int*)(g.cnt + 1);
    g.status = status;
    g.limit_ns = wait_limit_ns();

    const int words = (int)((sizeof(Counters) + sizeof(int) * ((s.d + kTileM - 1) / kTileM)) / 4);
    // Both launches may begin while the kernel before them in the stream ends; each
    // kernel waits for that one's end before it touches memory.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.stream = st;
    cfg.gridDim = t == 1 ? dim3((s.E + 1) / 2) : dim3((s.E + 3) / 4, (t + 3) / 4);
    cfg.blockDim = dim3(kLogitThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, t == 1 ? few_logits_kernel<T, 2, 1> : few_logits_kernel<T, 4, 4>,
                                       t, s.d, s.E, x, (const T*)p.Wg, p.logit_bias, (float*)g.logits,
                                       (int*)g.cnt, words);
    if (e != cudaSuccess) return e;
    if (t == 1 || (t <= kDirectTokens && (int64_t)t * s.k * 2 * s.d * s.f <= direct_weights<T>())) {
        DirectArgs q;
        q.d = s.d; q.f = s.f; q.E = s.E; q.k = s.k; q.renorm = s.renorm; q.tokens = t;
        q.logits = g.logits;
        q.x = x; q.W1 = p.W1; q.b1 = p.b1; q.W2 = p.W2; q.b2 = p.b2; q.residual = residual; q.y = y;
        q.hidden = (float*)g.hidden;
        q.ticket = &g.cnt->ticket;
        q.done = &g.cnt->done;
        q.status = status;
        q.limit_ns = g.limit_ns;
        return t == 1 ? launch_direct<T, 1, 4, 2>(q, st) : t == 2 ? launch_direct<T, 2, 2, 4>(q, st)
                                                                  : launch_direct<T, 4, 4, 2>(q, st);
    }

    int most = 0;
    e = few_smem_limit<T>(&most);
    if (e != cudaSuccess) return e;
    const int rows = t * K::kRowsPerSlot;     // activation rows a K block can have
    const int slot = (rows + K::kBox - 1) / K::kBox * K::kBox * kBlockBytes;   // at most
    const int nc = t <= 4 ? 4 : 8;
    int left = most - 1024 - t * kTileM * 4 - (K::kTensor ? 0 : 8 * nc * kTileM * 4);
    g.b_ring = slot * (slot <= 4096 ? kMaxBStages : slot <= 8192 ? 4 : 2);
    left -= g.b_ring;
    g.a_stages = left / kABytes < kMaxAStages ? left / kABytes : kMaxAStages;
    g.slices = few_blocks() / g.tiles2;
    g.slices = g.slices < 1 ? 1 : g.slices > t ? t : g.slices;
    if (g.a_stages < 2) return cudaErrorInvalidConfiguration;

    CUtensorMap w1, mx, w2, mh;
    if (!few_map<T>(&w1, p.W1, s.d, s.f, s.E, kTileM) || !few_map<T>(&mx, x, s.d, t, 0, K::kBox) ||
        !few_map<T>(&w2, p.W2, s.f, s.d, s.E, kTileM) ||
        !few_map<T>(&mh, g.hidden, s.f, (uint64_t)t * s.k * K::kRowsPerSlot, 0, K::kBox))
        return cudaErrorInvalidValue;

    cfg.gridDim = dim3((unsigned)few_blocks());
    cfg.blockDim = dim3(few_threads<T>());
    cfg.dynamicSmemBytes = (size_t)most;
    return cudaLaunchKernelEx(&cfg, few_experts_kernel<T>, w1, mx, w2, mh, g);
}

}  // namespace

bool few_supported(const moe_shape& s) {
    // points of a Walk's line fit 32 bits
    const int64_t block = s.dtype == MOE_BF16 ? Kind<__nv_bfloat16>::kBlock : Kind<float>::kBlock;
    const int64_t most = s.dtype == MOE_BF16 ? 1 : kMaxCost;
    const int64_t experts = s.T * s.k < s.E ? s.T * s.k : s.E;
    auto points = [&](int64_t out, int64_t in) {
        return experts * most * ((out + kTileM - 1) / kTileM) * ((in + block - 1) / block);
    };
    const int64_t limit = (int64_t(1) << 31) - 1;
    return points(s.f, s.d) <= limit && points(s.d, s.f) <= limit;
}

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
