// few.cu -- one whole MoE layer for a few tokens (T <= MOE_FEW_MAX_TOKENS):
// router, top-k gate, experts, combine and residual, for decode steps.
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

// ---- router logits -----------------------------------------------------------------
// L[t,e] = <x_t, Wg_e> + beta_e in fp32.  A block computes EE experts x TT tokens;
// its warps split d (16 bytes a lane and step), their sums are added in warp order.
// Small blocks, so that Wg streams to as many SMs as there are; it also clears the
// expert kernel's counters.
constexpr int kLogitThreads = 256;

template <typename T, int EE, int TT>
__global__ void __launch_bounds__(kLogitThreads)
    few_logits_kernel(int tokens, int d, int E, const T* __restrict__ x, const T* __restrict__ Wg,
                      const float* __restrict__ beta, float* __restrict__ logits,
                      int* __restrict__ counters, int words) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < words; i += kLogitThreads) counters[i] = 0;
    constexpr int N = Vec<T>::N, W = kLogitThreads / 32, V = EE * TT;
    __shared__ float part[W][V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.x * EE, t0 = blockIdx.y * TT;
    float acc[EE][TT] = {};
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
                for (int n = 0; n < N; ++n) acc[a][b] = fmaf(g[a][n], v[n], acc[a][b]);
        }
    }
    #pragma unroll
    for (int a = 0; a < EE; ++a)
        #pragma unroll
        for (int b = 0; b < TT; ++b) {
            float v = acc[a][b];
            #pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
            if (lane == 0) part[warp][a * TT + b] = v;
        }
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
// One warp, for NT tokens t0, t0 + step, ... in lockstep (their chains of reductions
// overlap): the k experts with the largest logits (equal ones by their index) and
// their softmax weights.  Lane l holds experts l, l + 32, ...
template <int EPL, int NT>
__device__ __forceinline__ void gate(const float* logits, int t0, int step, int tokens, int E, int k,
                                     int renorm, uint8_t* e_of, float* w, int32_t* status) {
    const int lane = threadIdx.x & 31;
    auto value = [](uint32_t x) { return __uint_as_float(x & 0x80000000u ? x & 0x7fffffffu : ~x); };
    uint32_t key[NT][EPL];   // ordered as the logits; 0: not an expert, or taken
    bool bad = false;
    #pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int t = t0 + i * step < tokens ? t0 + i * step : t0;   // past the end: the first again
        #pragma unroll
        for (int q = 0; q < EPL; ++q) {
            const int e = lane + 32 * q;
            key[i][q] = 0u;
            if (e < E) {
                float l = __ldcg(logits + t * E + e);
                if (!isfinite(l)) bad = true;
                if (isnan(l)) l = -INFINITY;                   // ranks below every number
                const uint32_t u = __float_as_uint(l + 0.f);   // one zero
                key[i][q] = u & 0x80000000u ? ~u : u | 0x80000000u;
            }
        }
    }
    if (__any_sync(kFull, bad) && lane == 0) report(status, MOE_ERR_NONFINITE);
    float m[NT], z[NT];
    #pragma unroll
    for (int i = 0; i < NT; ++i) {
        uint32_t high = key[i][0];
        #pragma unroll
        for (int q = 1; q < EPL; ++q) high = key[i][q] > high ? key[i][q] : high;
        m[i] = value(__reduce_max_sync(kFull, high));
    }
    #pragma unroll
    for (int i = 0; i < NT; ++i) {
        z[i] = 0.f;
        #pragma unroll
        for (int q = 0; q < EPL; ++q)
            if (lane + 32 * q < E) z[i] += expf(value(key[i][q]) - m[i]);
    }
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        #pragma unroll
        for (int i = 0; i < NT; ++i) z[i] += __shfl_xor_sync(kFull, z[i], o);
    int my_e[NT] = {};
    uint32_t my_key[NT] = {};
    for (int j = 0; j < k; ++j) {
        uint32_t best[NT], top[NT];
        int at[NT];
        #pragma unroll
        for (int i = 0; i < NT; ++i) {
            best[i] = key[i][0];
            at[i] = lane;
            #pragma unroll
            for (int q = 1; q < EPL; ++q)
                if (key[i][q] > best[i]) { best[i] = key[i][q]; at[i] = lane + 32 * q; }
        }
        #pragma unroll
        for (int i = 0; i < NT; ++i) top[i] = __reduce_max_sync(kFull, best[i]);
        #pragma unroll
        for (int i = 0; i < NT; ++i)
            at[i] = (int)__reduce_min_sync(kFull, best[i] == top[i] ? (unsigned)at[i] : 256u);
        #pragma unroll
        for (int i = 0; i < NT; ++i) {
            #pragma unroll
            for (int q = 0; q < EPL; ++q)
                if (at[i] == lane + 32 * q) key[i][q] = 0u;
            if (lane == j) { my_e[i] = at[i]; my_key[i] = top[i]; }
        }
    }
    float pr[NT], sum[NT];
    #pragma unroll
    for (int i = 0; i < NT; ++i) sum[i] = pr[i] = lane < k ? expf(value(my_key[i]) - m[i]) / z[i] : 0.f;
    if (renorm) {
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            #pragma unroll
            for (int i = 0; i < NT; ++i) sum[i] += __shfl_xor_sync(kFull, sum[i], o);
        #pragma unroll
        for (int i = 0; i < NT; ++i) pr[i] /= sum[i];
    }
    #pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int t = t0 + i * step;
        if (lane < k && t < tokens) {
            e_of[t * k + lane] = (uint8_t)my_e[i];
            w[t * k + lane] = pr[i];
        }
    }
}

template <int EPL>
__device__ __forceinline__ void gate_all(const float* logits, int tokens, int E, int k, int renorm,
                                         uint8_t* e_of, float* w, int32_t* status) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int t = warp;
    if (tokens <= warps) {
        if (t < tokens) gate<EPL, 1>(logits, t, warps, tokens, E, k, renorm, e_of, w, status);
        return;
    }
    for (; t < tokens; t += 3 * warps)
        gate<EPL, 3>(logits, t, warps, tokens, E, k, renorm, e_of, w, status);
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
__device__ __forceinline__ void add_release(int* p, int v) {
    asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// 16 bytes of T, streamed past L1
__device__ __forceinline__ uint4 stream16(const void* p) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
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
    if (warp < g.tokens) {
        int32_t* status = blockIdx.x == 0 ? g.status : nullptr;
        if (g.E <= 32) gate<1, 1>(g.logits, warp, W, g.tokens, g.E, g.k, g.renorm, e_of, w, status);
        else if (g.E <= 128) gate<4, 1>(g.logits, warp, W, g.tokens, g.E, g.k, g.renorm, e_of, w, status);
        else gate<8, 1>(g.logits, warp, W, g.tokens, g.E, g.k, g.renorm, e_of, w, status);
    }
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
        float acc[RW][TT] = {};
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
                        for (int n = 0; n < N; ++n) acc[r][t] = fmaf(wf[r][n], v[n], acc[r][t]);
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
                                if (q == t) acc[r][q] += v;
                        }
        #pragma unroll
        for (int r = 0; r < RW; ++r)
            #pragma unroll
            for (int t = 0; t < TT; ++t) {
                float v = acc[r][t];
                #pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
                if (lane == 0) part[warp][r * TT + t] = v;
            }
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
                        g.hidden[(int64_t)s * M + row] = w[s] * gelu_f(v);
                    }
                } else {
                    const int64_t o = (int64_t)t * M + row;
                    if (g.residual) v += to_f32<T>(((const T*)g.residual)[o]);
                    ((T*)g.y)[o] = from_f32<T>(v);
                }
            }
            if (one) __threadfence();
        }
        if (threadIdx.x == 0) next = claimed;
        __syncthreads();
        if (one && threadIdx.x == 0) add_release(g.done, 1);
    }
}

// ---- experts ----------------------------------------------------------------------
// See the file's header for the scheme.
constexpr int kTileM = 128;          // weight rows (output features) of a tile
constexpr int kBlockBytes = 128;     // one K block of a row: 64 bf16 or 32 fp32
constexpr int kABytes = kTileM * kBlockBytes;
constexpr int kMaxAStages = 12, kMaxBStages = 8;
constexpr int kWarpsBeforeEpilogue = 4;
// Times that decide whether the first product's units are cut: a K block of
// weights when all blocks stream, when few do, and adding the parts of cut units.
constexpr float kBlockNs = 366.f, kLoneBlockNs = 250.f, kJoinNs = 3000.f;

template <typename T> struct Kind;
template <> struct Kind<__nv_bfloat16> {
    static constexpr bool kTensor = true;
    static constexpr int kBox = 16;             // activation rows a TMA box takes
    static constexpr int kRowsPerSlot = 2;      // hidden rows of a slot: high and low part
    static constexpr int kBlock = 64;           // elements of a K block
    static constexpr int kEpilogue = 128;       // threads
};
template <> struct Kind<float> {
    static constexpr bool kTensor = false;
    static constexpr int kBox = 8;
    static constexpr int kRowsPerSlot = 1;
    static constexpr int kBlock = 32;
    static constexpr int kEpilogue = 256;
};
// bf16: the warps beyond the epilogue's only gate
template <typename T> constexpr int few_threads() {
    return Kind<T>::kTensor ? 384 : kWarpsBeforeEpilogue * 32 + Kind<T>::kEpilogue;
}

// counters in the workspace, zeroed by the logits kernel
struct Counters {
    int done;           // finished units (tasks) of the first product
    int ticket;         // tasks handed out
    int joined[512];    // per block: parts of the unit that starts in it and ends in another
    // then per output tile: parts written
};
constexpr int kMaxBlocks = 512;

struct FewArgs {
    int tokens, d, f, E, k, renorm;
    int tiles1, tiles2, KB1, KB2;         // of the two products: output tiles, K blocks
    int a_stages, b_stages, b_bytes;      // shared-memory rings
    const float* logits;
    const void *b1, *b2, *residual;
    void* y;
    void* hidden;          // [T k kRowsPerSlot][f]
    float *part1, *part2;  // [blocks][2][T][128] partial sums of the two products
    Counters* cnt;
    int* tiles_done;       // per output tile
    int32_t* status;
    uint64_t limit_ns;
};

struct FewCtrl {
    uint64_t a_full[kMaxAStages], a_empty[kMaxAStages];
    uint64_t b_full[kMaxBStages], b_empty[kMaxBStages];
    uint64_t t_full[2], t_empty[2], drain;
    uint32_t tmem;
    int abort_flag;
    int last;
};

// ---- dispatch -----------------------------------------------------------------------
// Every block of the expert kernel works out the gate for itself, a warp a token,
// and sorts the (token, slot) pairs (1024 of them at most): rows by expert, then by
// token.  That takes it less time than to wait for another block's result.
struct Sorted {
    unsigned long long tokens[256];   // bit t: token t goes to this expert
    int off[257];                     // first row of each expert
    int act[256];                     // experts with tokens, ascending
    int cost[257];                    // prefix sums over act of block_cost()
    int most;                         // largest block_cost()
    int nact;
    int warp_sum[8], warp_cost[8];
    float w[kMaxSlots];               // gate weight of slot (t, j)
    uint8_t e_of[kMaxSlots];          // its expert
    float row_w[kMaxSlots];           // gate weight of each row
    uint8_t row_token[kMaxSlots];     // token of each row
};

// Relative time of one K block with `rows` activation rows: the bytes of the
// weights, unless fp32 products take longer.
constexpr int kMaxCost = 10;
template <typename T> __device__ __forceinline__ int block_cost(int rows) {
    return sizeof(T) == 2 ? 1 : rows <= 16 ? 3 : rows <= 32 ? 5 : kMaxCost;
}

// One block's consecutive K blocks of one (expert, tile).
struct Seg {
    int phase;        // 0: first product, 1: second
    int a, m;         // active expert, tile
    int kb0, kb1;     // K blocks
    int c0, c1;       // blocks that hold the unit's first and last K block
};

// Walks a block's share of the first product, then of the second.  The K blocks
// of a product lie one after another on a line, each as long as its cost: in the
// first product an expert's tiles follow one another, in the second an output
// tile's experts.  The line is cut into equal shares, and a K block is the
// share's in which it begins; so every block works for the same time, and a
// share may begin and end inside a unit (an expert's tile).
struct Walk {
    const Sorted* p;
    const Walk* then;      // the share of the second product
    int phase;
    int tiles, KB;         // of the product
    int blocks, share, longer;   // the first `longer` shares are share + 1 long
    bool whole;            // first product: shares of whole units, counted in units
    int end;
    int a, m, kb;          // next K block

    __device__ int start(int block) const { return block * share + (block < longer ? block : longer); }
    __device__ int line(int a_, int m_, int kb_) const {   // where a K block begins
        const int c = p->cost[a_ + 1] - p->cost[a_];
        return phase == 0 ? p->cost[a_] * tiles * KB + (m_ * KB + kb_) * c
                          : (m_ * p->cost[p->nact] + p->cost[a_]) * KB + kb_ * c;
    }
    __device__ int holder(int a_, int m_, int kb_) const {   // the block whose share it is in
        const int x = line(a_, m_, kb_), cut = longer * (share + 1);
        return x < cut ? x / (share + 1) : longer + (x - cut) / share;
    }
    // needs the plan's act and cost
    __device__ void begin(const FewArgs& g, const Sorted* plan, int product, const Walk* then_) {
        p = plan;
        then = then_;
        phase = product;
        tiles = product == 0 ? g.tiles1 : g.tiles2;
        KB = product == 0 ? g.KB1 : g.KB2;
        const int grid = (int)gridDim.x, nact = p->nact, me = (int)blockIdx.x;
        const int units = nact * tiles;
        whole = false;
        if (product == 0) {
            const int rounds = (units + grid - 1) / grid;
            const float all = (float)units / (float)grid * kBlockNs;     // a K block of every unit
            const float each = units < grid ? fmaxf(all, kLoneBlockNs) : kBlockNs;
            whole = rounds * each * KB <= all * KB + kJoinNs;
        }
        const int total = whole ? units : p->cost[nact] * tiles * KB;
        // no share is shorter than a K block: each holds the beginning of one
        blocks = whole || p->most == 1 ? total : total / p->most;
        blocks = blocks < grid ? blocks : grid;
        share = total / blocks;
        longer = total - share * blocks;
        a = m = kb = 0;
        end = 0;
        if (me >= blocks) return;
        int x = start(me);
        end = start(me + 1);
        if (whole) {
            a = x / tiles;
            m = x - a * tiles;
            return;
        }
        // the first K block that begins at or after x
        const int per = product == 0 ? tiles * KB : KB;   // K blocks an expert
        if (product == 1) {
            m = x / (per * p->cost[nact]);
            x -= m * per * p->cost[nact];
        }
        int lo = 0, hi = nact;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p->cost[mid] * per <= x) lo = mid; else hi = mid;
        }
        a = lo;
        const int c = p->cost[a + 1] - p->cost[a];
        kb = x - p->cost[a] * per;
        if (c > 1) kb = (kb + c - 1) / c;
        if (product == 0) {
            m = kb / KB;
            kb -= m * KB;
        }
        wrap();
    }
    __device__ void wrap() {   // past the end of a unit, an expert, a tile
        if (kb >= KB) {
            kb = 0;
            if (phase == 0) ++m; else ++a;
        }
        if (phase == 0 && m >= tiles) { m = 0; ++a; }
        if (phase == 1 && a >= p->nact) { a = 0; ++m; }
    }
    __device__ bool left() const {
        if (whole) return a * tiles + m < end;
        return (phase == 0 ? a < p->nact : m < tiles) && line(a, m, kb) < end;
    }
    __device__ bool next(Seg& s) {
        if (!left()) {
            if (phase == 1) return false;
            *this = *then;
            if (!left()) return false;
        }
        s.phase = phase;
        s.a = a;
        s.m = m;
        s.kb0 = kb;
        s.kb1 = KB;
        s.c0 = s.c1 = (int)blockIdx.x;
        if (!whole) {
            const int c = p->cost[a + 1] - p->cost[a];
            int n = end - line(a, m, kb);
            if (c > 1) n = (n + c - 1) / c;
            if (kb + n < KB) s.kb1 = kb + n;
            if (kb > 0) s.c0 = holder(a, m, 0);
            if (s.kb1 < KB) s.c1 = holder(a, m, KB - 1);
        }
        kb = s.kb1;
        wrap();
        return true;
    }
};

// The sorted rows, and where this block's two shares begin.
struct Plan : Sorted {
    Walk first, second;
};

// Called by all threads of a block of at least 256.
template <typename T>
__device__ void make_plan(Plan& p, const FewArgs& g) {
    const int tokens = g.tokens, k = g.k;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < 256; e += blockDim.x) p.tokens[e] = 0ull;
    if (threadIdx.x == 0) p.most = 1;
    int32_t* status = blockIdx.x == 0 ? g.status : nullptr;
    if (g.E <= 32) gate_all<1>(g.logits, tokens, g.E, k, g.renorm, p.e_of, p.w, status);
    else if (g.E <= 128) gate_all<4>(g.logits, tokens, g.E, k, g.renorm, p.e_of, p.w, status);
    else gate_all<8>(g.logits, tokens, g.E, k, g.renorm, p.e_of, p.w, status);
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * k; i += blockDim.x)
        atomicOr(&p.tokens[p.e_of[i]], 1ull << (i / k));
    __syncthreads();
    // exclusive prefix sums over the experts: (rows, has rows) in one word, cost
    const int e = threadIdx.x;
    int n = 0, v = 0, c = 0;
    if (e < 256) {
        n = __popcll(p.tokens[e]);
        v = n | (n > 0 ? 1 << 16 : 0);
        c = n > 0 ? block_cost<T>(n) : 0;
        if (sizeof(T) == 4 && c > 1) atomicMax(&p.most, c);
        const int own = v, own_c = c;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, v, o), uc = __shfl_up_sync(kFull, c, o);
            if (lane >= o) { v += u; c += uc; }
        }
        if (lane == 31) { p.warp_sum[warp] = v; p.warp_cost[warp] = c; }
        v -= own;
        c -= own_c;
    }
    __syncthreads();
    if (e < 256) {
        for (int q = 0; q < warp; ++q) { v += p.warp_sum[q]; c += p.warp_cost[q]; }
        p.off[e] = v & 0xffff;
        if (n > 0) { p.act[v >> 16] = e; p.cost[v >> 16] = c; }
        if (e == 255) {
            const int na = (v >> 16) + (n > 0);
            p.off[256] = (v & 0xffff) + n;
            p.nact = na;
            p.cost[na] = c + (n > 0 ? block_cost<T>(n) : 0);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * k; i += blockDim.x) {
        const int ee = p.e_of[i], t = i / k;
        const int r = p.off[ee] + __popcll(p.tokens[ee] & ((1ull << t) - 1ull));
        p.row_token[r] = (uint8_t)t;
        p.row_w[r] = p.w[i];
    }
    if (lane == 0 && warp == 6) p.first.begin(g, &p, 0, &p.second);
    if (lane == 0 && warp == 7) p.second.begin(g, &p, 1, nullptr);
    __syncthreads();
}

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

// fp32 products on the CUDA cores: 8 warps, a lane holding 4 weight rows and NC
// activation rows.  With more than NC rows the warps split them into `groups`
// (1, 2, 4 or 8) and K into 8 / groups; sums run over even and odd k apart, as
// packed pairs.  The result goes to red[K slice][row][128].
template <int NC>
__device__ __forceinline__ bool products_f32(const FewArgs& g, FewCtrl& c, const Seg& s, int rows,
                                             const uint8_t* row_token, uint8_t* a_ring,
                                             uint8_t* b_ring, int& as, uint32_t& ap, int& bs,
                                             uint32_t& bp, int ew, int lane, int groups, float* red) {
    const int grp = ew % groups, slice = ew / groups;
    uint32_t brow[NC];
    #pragma unroll
    for (int j = 0; j < NC; ++j) {
        int r = grp * NC + j;
        r = r < rows ? r : rows - 1;
        brow[j] = s.phase == 0 ? row_token[r] : r;
    }
    uint64_t acc[4][NC];
    #pragma unroll
    for (int q = 0; q < 4; ++q)
        #pragma unroll
        for (int j = 0; j < NC; ++j) acc[q][j] = 0ull;
    for (int kb = s.kb0; kb < s.kb1; ++kb) {
        if (!mbar_wait_warp(smem_u32(&c.a_full[as]), ap, g.limit_ns, &c.abort_flag) ||
            !mbar_wait_warp(smem_u32(&c.b_full[bs]), bp, g.limit_ns, &c.abort_flag))
            return false;
        const uint8_t* A = a_ring + as * kABytes;
        const uint8_t* B = b_ring + bs * g.b_bytes;
        for (int i = 0; i < groups; ++i) {
            const int ch = slice * groups + i;   // 16-byte chunk of the K block
            ulonglong2 a[4];
            #pragma unroll
            for (int q = 0; q < 4; ++q)
                a[q] = *reinterpret_cast<const ulonglong2*>(A + (lane + 32 * q) * 128 +
                                                            ((ch ^ (lane & 7)) << 4));
            #pragma unroll
            for (int j = 0; j < NC; ++j) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(
                    B + brow[j] * 128 + ((ch ^ (brow[j] & 7)) << 4));
                #pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[q][j] = f2_fma(a[q].y, b.y, f2_fma(a[q].x, b.x, acc[q][j]));
            }
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&c.a_empty[as]));
            mbar_arrive(smem_u32(&c.b_empty[bs]));
        }
        if (++as == g.a_stages) { as = 0; ap ^= 1; }
        if (++bs == g.b_stages) { bs = 0; bp ^= 1; }
    }
    #pragma unroll
    for (int j = 0; j < NC; ++j)
        #pragma unroll
        for (int q = 0; q < 4; ++q) {
            float e, o;
            f2_unpack(acc[q][j], e, o);
            red[((slice * groups + grp) * NC + j) * kTileM + lane + 32 * q] = e + o;
        }
    return true;
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
    float* yacc = reinterpret_cast<float*>(b_ring + (size_t)g.b_stages * g.b_bytes);  // [T][128]
    float* red = yacc + g.tokens * kTileM;      // fp32 only
    __shared__ Plan plan;
    __shared__ FewCtrl c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        const int consumers = K::kTensor ? 1 : K::kEpilogue / 32;
        for (int i = 0; i < g.a_stages; ++i) {
            mbar_init(smem_u32(&c.a_full[i]), 1);
            mbar_init(smem_u32(&c.a_empty[i]), consumers);
        }
        for (int i = 0; i < g.b_stages; ++i) {
            mbar_init(smem_u32(&c.b_full[i]), 1);
            mbar_init(smem_u32(&c.b_empty[i]), consumers);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c.t_full[i]), 1);
            mbar_init(smem_u32(&c.t_empty[i]), K::kEpilogue / 32);
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
    make_plan<T>(plan, g);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = K::kTensor ? c.tmem : 0u;
    Walk walk = plan.first;
    Seg s;

    if (warp == 0) {
        // ---- weights: one box of 128 rows a K block, both products in one stream -----
        if (lane == 0) {
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(s)) {
                const int e = plan.act[s.a];
                const CUtensorMap* map = s.phase == 0 ? &mapW1 : &mapW2;
                for (int kb = s.kb0; kb < s.kb1; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&c.a_empty[st]), ph ^ 1, g.limit_ns, &c.abort_flag)) {
                        few_abort(c, g.status);
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(smem_u32(&c.a_full[st]), kABytes);
                    tma_load_3d(smem_u32(a_ring + st * kABytes), map, smem_u32(&c.a_full[st]),
                                kb * K::kBlock, s.m * kTileM, e);
                    if (issued < g.a_stages) ++issued;
                    if (++st == g.a_stages) { st = 0; ph ^= 1; }
                }
            }
            // copies in flight land before the block ends
            for (int i = 0; i < issued; ++i) {
                if (--st < 0) { st = g.a_stages - 1; ph ^= 1; }
                mbar_wait_bounded(smem_u32(&c.a_full[st]), ph, g.limit_ns, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- activations: all tokens' K block of x, or the expert's hidden rows -------
        if (lane == 0) {
            int st = 0, issued = 0;
            bool ready = false;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(s)) {
                const int e = plan.act[s.a];
                const int row0 = s.phase == 0 ? 0 : plan.off[e] * RPS;
                const int rows = s.phase == 0 ? g.tokens : (plan.off[e + 1] - plan.off[e]) * RPS;
                const int boxes = (rows + BOX - 1) / BOX;
                const CUtensorMap* map = s.phase == 0 ? &mapX : &mapH;
                if (s.phase == 1 && !ready) {
                    // All hidden rows are written.  (One counter for all experts: the
                    // shares are equal, so that waiting for some of them first gains nothing,
                    // and each further poll would cost a round trip to the L2.)
                    const uint64_t t0 = globaltimer_ns();
                    while (load_acquire(&g.cnt->done) < plan.nact * g.tiles1) {
                        if (*(volatile int*)&c.abort_flag || globaltimer_ns() - t0 > g.limit_ns) {
                            few_abort(c, g.status);
                            ok = false;
                            break;
                        }
                    }
                    if (!ok) break;
                    fence_proxy_async_all();
                    ready = true;
                }
                for (int kb = s.kb0; kb < s.kb1; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&c.b_empty[st]), ph ^ 1, g.limit_ns, &c.abort_flag)) {
                        few_abort(c, g.status);
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(smem_u32(&c.b_full[st]), boxes * BOX * kBlockBytes);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d(smem_u32(b_ring + st * g.b_bytes + i * BOX * kBlockBytes), map,
                                    smem_u32(&c.b_full[st]), kb * K::kBlock, row0 + i * BOX);
                    if (issued < g.b_stages) ++issued;
                    if (++st == g.b_stages) { st = 0; ph ^= 1; }
                }
            }
            // copies in flight land before the block ends
            for (int i = 0; i < issued; ++i) {
                if (--st < 0) { st = g.b_stages - 1; ph ^= 1; }
                mbar_wait_bounded(smem_u32(&c.b_full[st]), ph, g.limit_ns, nullptr);
            }
        }
        __syncwarp();
    } else if (K::kTensor && warp == 2) {
        // ---- tensor core: D[128 weight rows][activation rows], one accumulator a segment --
        if (lane == 0) {
            int as = 0, bs = 0, acc = 0;
            uint32_t ap = 0, bp = 0, tp = 0;
            bool ok = true;
            while (ok && walk.next(s)) {
                const int e = plan.act[s.a];
                const int rows = s.phase == 0 ? g.tokens : (plan.off[e + 1] - plan.off[e]) * RPS;
                const uint32_t idesc = idesc_bf16_f32(kTileM, (rows + 15) & ~15, false, false);
                if (!mbar_wait_bounded(smem_u32(&c.t_empty[acc]), tp ^ 1, g.limit_ns, &c.abort_flag)) {
                    few_abort(c, g.status);
                    break;
                }
                tc_fence_after();
                for (int kb = s.kb0; kb < s.kb1; ++kb) {
                    if (!mbar_wait_bounded(smem_u32(&c.a_full[as]), ap, g.limit_ns, &c.abort_flag) ||
                        !mbar_wait_bounded(smem_u32(&c.b_full[bs]), bp, g.limit_ns, &c.abort_flag)) {
                        few_abort(c, g.status);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc_sw128(smem_u32(a_ring + as * kABytes), 16, 1024);
                    const uint64_t bd = smem_desc_sw128(smem_u32(b_ring + bs * g.b_bytes), 16, 1024);
                    #pragma unroll
                    for (int kk = 0; kk < K::kBlock / 16; ++kk)
                        tc_mma_bf16(tmem + acc * kAccCols, ad + kk * 2, bd + kk * 2, idesc,
                                    kb > s.kb0 || kk > 0);
                    tc_commit(smem_u32(&c.a_empty[as]));
                    tc_commit(smem_u32(&c.b_empty[bs]));
                    if (++as == g.a_stages) { as = 0; ap ^= 1; }
                    if (++bs == g.b_stages) { bs = 0; bp ^= 1; }
                }
                if (!ok) break;
                tc_commit(smem_u32(&c.t_full[acc]));
                if (++acc == 2) { acc = 0; tp ^= 1; }
            }
            // every MMA issued has completed before TMEM is freed
            tc_commit(smem_u32(&c.drain));
            mbar_wait_bounded(smem_u32(&c.drain), 0, g.limit_ns, nullptr);
        }
        __syncwarp();
    } else if (warp >= kWarpsBeforeEpilogue && warp < kWarpsBeforeEpilogue + K::kEpilogue / 32) {
        // ---- epilogue -----------------------------------------------------------------
        // Thread i (of 128; fp32: two threads, alternate rows) owns weight row i of the
        // tile, i.e. one output feature, for all activation rows.
        constexpr int NT = K::kEpilogue;
        const int tid = threadIdx.x - kWarpsBeforeEpilogue * 32;
        const int ew = tid >> 5;
        const int i = K::kTensor ? (warp & 3) * 32 + lane : tid & 127;
        const int me = (int)blockIdx.x;
        const int64_t slot_floats = (int64_t)g.tokens * kTileM;
        T* hidden = (T*)g.hidden;
        int acc = 0, as = 0, bs = 0;
        uint32_t tp = 0, ap = 0, bp = 0;
        const T* residual = (const T*)g.residual;
        T* y = (T*)g.y;
        auto put_y = [&](int t, int m, float v) {
            const int col = m * kTileM + i;
            if (col >= g.d) return;
            const int64_t o = (int64_t)t * g.d + col;
            if (residual) v += to_f32<T>(residual[o]);
            y[o] = from_f32<T>(v);
        };
        bool more = walk.next(s);
        bool fresh = true;     // yacc holds nothing yet
        // tiles that other blocks add to as well: this block's first and last
        int m_a = 0, d_a = 0, n_a = 0, m_b = 0, d_b = 0, n_b = 0;
        bool gone = false;
        while (more) {
            const int e = plan.act[s.a];
            const int r0 = plan.off[e], rows = plan.off[e + 1] - r0;
            const int col = s.m * kTileM + i;
            const bool whole = s.c0 == s.c1;   // no other block has a part of the unit
            const bool live = col < (s.phase == 0 ? g.f : g.d);
            const T* bias = (const T*)(s.phase == 0 ? g.b1 : g.b2);
            const float b = bias && live && s.kb0 == 0
                                ? to_f32<T>(bias[(int64_t)e * (s.phase == 0 ? g.f : g.d) + col]) : 0.f;
            // unit of the first product cut over blocks c0..c1
            const int c0 = s.c0, c1 = s.c1;
            float* mine = g.part1 + (me * 2 + (me == c0)) * slot_floats;
            if (s.phase == 1 && fresh) {
                if (!K::kTensor) epilogue_barrier<NT>();
                for (int t = tid / kTileM; t < g.tokens; t += NT / kTileM) yacc[t * kTileM + i] = 0.f;
                if (!K::kTensor) epilogue_barrier<NT>();
                fresh = false;
            }
            auto put_hidden = [&](int r, float h) {
                if (!live) return;
                if constexpr (K::kTensor) {
                    // GELU in two bf16 parts, 16 bits together
                    const float a = gelu_fast(h);
                    const __nv_bfloat16 hi = __float2bfloat16_rn(a);
                    const float rest = a - __bfloat162float(hi);
                    __nv_bfloat16* p = hidden + (int64_t)(r0 + r) * 2 * g.f + col;
                    p[0] = hi;
                    p[g.f] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
                } else {
                    hidden[(int64_t)(r0 + r) * g.f + col] = gelu_f(h);
                }
            };
            auto emit = [&](int r, float v) {   // activation row r of the expert
                v += b;
                if (s.phase == 1) {
                    float* p = yacc + plan.row_token[r0 + r] * kTileM + i;
                    *p = fmaf(plan.row_w[r0 + r], v, *p);
                } else if (whole) {
                    put_hidden(r, v);
                } else {
                    __stcg(mine + r * kTileM + i, v);
                }
            };
            if constexpr (K::kTensor) {
                const bool ok = mbar_wait_warp(smem_u32(&c.t_full[acc]), tp, g.limit_ns, &c.abort_flag);
                if (!ok) few_abort(c, g.status);
                if (!epilogue_all<NT>(ok)) { gone = true; break; }
                tc_fence_after();
                const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc * kAccCols;
                if (s.phase == 0) {
                    unsigned long long left = plan.tokens[e];
                    int r = 0;
                    for (int q = 0; q * 16 < g.tokens; ++q, left >>= 16) {
                        if (!(left & 0xffffull)) continue;
                        float v[16];
                        tmem_ld16(base + q * 16, v);
                        #pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (left >> j & 1ull) emit(r++, v[j]);
                    }
                } else {
                    for (int q = 0; q * 8 < rows; ++q) {
                        float v[16];
                        tmem_ld16(base + q * 16, v);
                        #pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (q * 8 + j < rows) emit(q * 8 + j, v[2 * j] + v[2 * j + 1]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c.t_empty[acc]));
                if (++acc == 2) { acc = 0; tp ^= 1; }
            } else {
                const int groups = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
                const uint8_t* rt = plan.row_token + r0;
                bool ok;
                int nc;
                if (rows <= 2) {
                    nc = 2;
                    ok = products_f32<2>(g, c, s, rows, rt, a_ring, b_ring, as, ap, bs, bp, ew, lane, 1, red);
                } else if (rows <= 4) {
                    nc = 4;
                    ok = products_f32<4>(g, c, s, rows, rt, a_ring, b_ring, as, ap, bs, bp, ew, lane, 1, red);
                } else {
                    nc = 8;
                    ok = products_f32<8>(g, c, s, rows, rt, a_ring, b_ring, as, ap, bs, bp, ew, lane, groups, red);
                }
                if (!ok) few_abort(c, g.status);
                if (!epilogue_all<NT>(ok)) { gone = true; break; }
                const int cols = groups * nc;
                for (int r = tid / kTileM; r < rows; r += NT / kTileM) {
                    float v = 0.f;
                    for (int q = 0; q < 8 / groups; ++q) v += red[(q * cols + r) * kTileM + i];
                    emit(r, v);
                }
                epilogue_barrier<NT>();
            }
            if (s.phase == 0) {
                bool finished = whole;
                if (!whole) {
                    // the last block to write its part adds the parts, in block order
                    __threadfence();
                    epilogue_barrier<NT>();
                    if (tid == 0) c.last = atomicAdd(&g.cnt->joined[c0], 1) == c1 - c0;
                    epilogue_barrier<NT>();
                    finished = c.last;
                    if (finished) {
                        __threadfence();
                        // eight rows at a time, so that their loads overlap
                        for (int r = tid / kTileM; r < rows; r += 8 * (NT / kTileM)) {
                            float v[8];
                            #pragma unroll
                            for (int u = 0; u < 8; ++u) v[u] = 0.f;
                            for (int q = c0; q <= c1; ++q) {
                                const float* from = g.part1 + (q * 2 + (q == c0)) * slot_floats + i;
                                #pragma unroll
                                for (int u = 0; u < 8; ++u) {
                                    const int rr = r + u * (NT / kTileM);
                                    if (rr < rows) v[u] += __ldcg(from + rr * kTileM);
                                }
                            }
                            #pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                const int rr = r + u * (NT / kTileM);
                                if (rr < rows) put_hidden(rr, v[u]);
                            }
                        }
                    }
                }
                if (finished) {
                    __threadfence();
                    fence_proxy_async_all();
                    epilogue_barrier<NT>();
                    if (tid == 0) add_release(&g.cnt->done, 1);
                }
                more = walk.next(s);
                continue;
            }
            // second product: the tile is left when the next segment is another's
            const int m = s.m;
            more = walk.next(s);
            if (more && s.m == m) continue;
            fresh = true;
            const int last = walk.p->nact - 1;
            const int d0 = walk.holder(0, m, 0), d1 = walk.holder(last, m, walk.KB - 1);
            if (!K::kTensor) epilogue_barrier<NT>();
            if (d0 == d1) {
                for (int t = tid / kTileM; t < g.tokens; t += NT / kTileM)
                    put_y(t, m, yacc[t * kTileM + i]);
                continue;
            }
            float* out = g.part2 + (me * 2 + (me == d0)) * slot_floats;
            for (int t = tid / kTileM; t < g.tokens; t += NT / kTileM)
                __stcg(out + t * kTileM + i, yacc[t * kTileM + i]);
            __threadfence();
            epilogue_barrier<NT>();
            if (tid == 0) add_release(&g.tiles_done[m], 1);
            if (n_a == 0) { m_a = m; d_a = d0; n_a = d1 - d0 + 1; }
            else { m_b = m; d_b = d0; n_b = d1 - d0 + 1; }
        }
        // Tiles that several blocks have a part of: once all parts are there, each of
        // those blocks adds them, in block order, for its share of the tokens.
        for (int q = 0; q < 2 && !gone; ++q) {
            const int m = q ? m_b : m_a, d0 = q ? d_b : d_a, n = q ? n_b : n_a;
            if (n == 0) break;
            const int lo = g.tokens * (me - d0) / n, hi = g.tokens * (me - d0 + 1) / n;
            if (lo == hi) continue;
            bool ok = true;
            if (tid == 0) {
                const uint64_t t0 = globaltimer_ns();
                while (ok && load_acquire(&g.tiles_done[m]) < n)
                    ok = !*(volatile int*)&c.abort_flag && globaltimer_ns() - t0 <= g.limit_ns;
                if (!ok) few_abort(c, g.status);
            }
            if (!epilogue_all<NT>(ok)) break;
            for (int t = lo + tid / kTileM; t < hi; t += NT / kTileM) {
                const float* from = g.part2 + t * kTileM + i;
                float v = __ldcg(from + (d0 * 2 + 1) * slot_floats);
                #pragma unroll 8
                for (int b = d0 + 1; b < d0 + n; ++b) v += __ldcg(from + b * 2 * slot_floats);
                put_y(t, m, v);
            }
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
    size_t logits, counters, hidden, part1, part2, total;
};
FewLayout few_layout(const moe_shape& s) {
    FewLayout l;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t a = at; at += pad256(n); return a; };
    const size_t part = sizeof(float) * few_blocks() * 2 * s.T * kTileM;
    l.logits = take(sizeof(float) * s.T * s.E);
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

// Of the 227 KB a block may have; the rest lets blocks of the logits kernel share
// the SM, so that this kernel's blocks are set up while those run.
constexpr int kFewSmem = 222 * 1024;

template <typename T> cudaError_t few_smem_limit(int* dynamic) {
    // what the static part leaves; looked up once
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    static int most = 0;
    std::call_once(once, [] {
        cudaFuncAttributes a;
        err = cudaFuncGetAttributes(&a, few_experts_kernel<T>);
        if (err != cudaSuccess) return;
        most = (kFewSmem - (int)a.sharedSizeBytes) & ~127;
        err = cudaFuncSetAttribute(few_experts_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   most);
    });
    *dynamic = most;
    return err;
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
    g.b1 = p.b1; g.b2 = p.b2; g.residual = residual; g.y = y;
    g.hidden = ws + l.hidden;
    g.part1 = (float*)(ws + l.part1);
    g.part2 = (float*)(ws + l.part2);
    g.cnt = (Counters*)(ws + l.counters);
    g.tiles_done = (int*)(g.cnt + 1);
    g.status = status;
    g.limit_ns = wait_limit_ns();

    const int words = (int)((sizeof(Counters) + sizeof(int) * ((s.d + kTileM - 1) / kTileM)) / 4);
    if (t == 1)
        few_logits_kernel<T, 2, 1><<<(s.E + 1) / 2, kLogitThreads, 0, st>>>(
            t, s.d, s.E, x, (const T*)p.Wg, p.logit_bias, (float*)g.logits, (int*)g.cnt, words);
    else
        few_logits_kernel<T, 4, 8><<<dim3((s.E + 3) / 4, (t + 7) / 8), kLogitThreads, 0, st>>>(
            t, s.d, s.E, x, (const T*)p.Wg, p.logit_bias, (float*)g.logits, (int*)g.cnt, words);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (t <= kDirectTokens) {
        DirectArgs q;
        q.d = s.d; q.f = s.f; q.E = s.E; q.k = s.k; q.renorm = s.renorm; q.tokens = t;
        q.logits = g.logits;
        q.x = x; q.W1 = p.W1; q.b1 = p.b1; q.W2 = p.W2; q.b2 = p.b2; q.residual = residual; q.y = y;
        q.hidden = (float*)g.hidden;
        q.ticket = &g.cnt->ticket;
        q.done = &g.cnt->done;
        q.status = status;
        q.limit_ns = g.limit_ns;
        return t == 1 ? launch_direct<T, 1, 2, 4>(q, st) : t == 2 ? launch_direct<T, 2, 2, 4>(q, st)
                                                                  : launch_direct<T, 4, 4, 2>(q, st);
    }

    int most = 0;
    e = few_smem_limit<T>(&most);
    if (e != cudaSuccess) return e;
    const int rows = t * K::kRowsPerSlot;     // activation rows a K block can have
    g.b_bytes = (rows + K::kBox - 1) / K::kBox * K::kBox * kBlockBytes;
    const int nc = t <= 2 ? 2 : t <= 4 ? 4 : 8;
    int left = most - 1024 - t * kTileM * 4 - (K::kTensor ? 0 : 8 * nc * kTileM * 4);
    g.b_stages = g.b_bytes <= 4096 ? kMaxBStages : 4;
    left -= g.b_stages * g.b_bytes;
    g.a_stages = left / kABytes < kMaxAStages ? left / kABytes : kMaxAStages;
    if (g.a_stages < 2) return cudaErrorInvalidConfiguration;

    CUtensorMap w1, mx, w2, mh;
    if (!few_map<T>(&w1, p.W1, s.d, s.f, s.E, kTileM) || !few_map<T>(&mx, x, s.d, t, 0, K::kBox) ||
        !few_map<T>(&w2, p.W2, s.f, s.d, s.E, kTileM) ||
        !few_map<T>(&mh, g.hidden, s.f, (uint64_t)t * s.k * K::kRowsPerSlot, 0, K::kBox))
        return cudaErrorInvalidValue;

    // Blocks wait for one another's hidden rows: a cooperative launch, so that all
    // of them are resident.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)few_blocks());
    cfg.blockDim = dim3(few_threads<T>());
    cfg.dynamicSmemBytes = (size_t)most;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
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
