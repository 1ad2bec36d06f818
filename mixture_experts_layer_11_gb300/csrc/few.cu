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
                      const float* __restrict__ beta, float* __restrict__ logits,
                      int* __restrict__ counters, int words) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < words; i += kLogitThreads) counters[i] = 0;
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
    float row_w[kMaxSlots];           // gate weight of each row
    uint8_t row_token[kMaxSlots];     // token of each row
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
        const int r = p.off[ee] + __popcll(p.tokens[ee] & ((1ull << t) - 1ull));
        p.row_token[r] = (uint8_t)t;
        p.row_w[r] = p.w[i];
    }
    __syncthreads();
}

// ---- experts ----------------------------------------------------------------------
// See the file's header for the scheme.
constexpr int kTileM = 128;          // weight rows (output features) of a tile
constexpr int kBlockBytes = 128;     // one K block of a row: 64 bf16 or 32 fp32
constexpr int kABytes = kTileM * kBlockBytes;
constexpr int kMaxAStages = 12, kMaxBStages = 8;
constexpr int kWarpsBeforeEpilogue = 4;

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
template <typename T> constexpr int few_threads() {
    return kWarpsBeforeEpilogue * 32 + Kind<T>::kEpilogue;
}

// counters in the workspace, zeroed by the logits kernel
struct Counters {
    int done[256];      // per active expert: finished tiles of the first product
    int joined[512];    // per block: parts of the unit that starts in it and ends in another
    // then per output tile: parts written
};
constexpr int kMaxBlocks = 512;

struct FewArgs {
    int tokens, d, f, E, k, renorm;
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

// One block's consecutive K blocks of one (expert, tile).
struct Seg {
    int phase;        // 0: first product, 1: second
    int a, m;         // active expert, tile
    int kb0, kb1;     // K blocks
    int KB;           // of the whole unit
    long long unit;
};

// Walks a block's share of the first product, then of the second.  All K blocks
// of a product are numbered in one sequence and cut into equal shares, so that
// every block streams the same bytes; a share may begin and end inside a unit.
struct Walk {
    int nact, tiles[2], KB[2];
    long long total[2], at, end;
    int blocks[2];
    int phase, me;
    __device__ Walk(const FewArgs& g, int nact_, int block) {
        nact = nact_;
        me = (int)blockIdx.x;
        tiles[0] = (g.f + kTileM - 1) / kTileM;
        tiles[1] = (g.d + kTileM - 1) / kTileM;
        KB[0] = (g.d + block - 1) / block;
        KB[1] = (g.f + block - 1) / block;
        #pragma unroll
        for (int p = 0; p < 2; ++p) {
            total[p] = (long long)nact * tiles[p] * KB[p];
            blocks[p] = total[p] < (long long)gridDim.x ? (int)total[p] : (int)gridDim.x;
        }
        begin(0);
    }
    __device__ void begin(int p) {
        phase = p;
        at = end = 0;
        if (me < blocks[p]) {
            at = total[p] * me / blocks[p];
            end = total[p] * (me + 1) / blocks[p];
        }
    }
    __device__ bool next(Seg& s) {
        if (at >= end) {
            if (phase == 1) return false;
            begin(1);
            if (at >= end) return false;
        }
        const int KBp = KB[phase];
        s.phase = phase;
        s.KB = KBp;
        s.unit = at / KBp;
        if (phase == 0) {   // an expert's tiles one after another
            s.a = (int)(s.unit / tiles[0]);
            s.m = (int)(s.unit % tiles[0]);
        } else {            // an output tile's experts one after another
            s.m = (int)(s.unit / nact);
            s.a = (int)(s.unit % nact);
        }
        s.kb0 = (int)(at - s.unit * KBp);
        const long long stop = (s.unit + 1) * KBp;
        s.kb1 = (int)((end < stop ? end : stop) - s.unit * KBp);
        at += s.kb1 - s.kb0;
        return true;
    }
    // block that holds K block b of product p
    __device__ int holder(int p, long long b) const {
        return (int)(((b + 1) * blocks[p] - 1) / total[p]);
    }
};

__device__ __forceinline__ void few_abort(FewCtrl& c, int32_t* status) {
    *(volatile int*)&c.abort_flag = 1;
    report(status, MOE_ERR_TIMEOUT);
}

__device__ __forceinline__ int load_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void add_release(int* p, int v) {
    asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
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
// (1, 2 or 4) and K into 8 / groups; sums run over even and odd k apart, as
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
        tmem_alloc(smem_u32(&c.tmem), 256);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    make_plan(plan, g.logits, g.tokens, g.E, g.k, g.renorm, blockIdx.x == 0 ? g.status : nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = K::kTensor ? c.tmem : 0u;
    Walk walk(g, plan.nact, K::kBlock);
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
            int st = 0, issued = 0, ready = -1;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(s)) {
                const int e = plan.act[s.a];
                const int row0 = s.phase == 0 ? 0 : plan.off[e] * RPS;
                const int rows = s.phase == 0 ? g.tokens : (plan.off[e + 1] - plan.off[e]) * RPS;
                const int boxes = (rows + BOX - 1) / BOX;
                const CUtensorMap* map = s.phase == 0 ? &mapX : &mapH;
                if (s.phase == 1 && ready != s.a) {
                    // every tile of the expert's hidden rows is written
                    const uint64_t t0 = globaltimer_ns();
                    while (load_acquire(&g.cnt->done[s.a]) < walk.tiles[0]) {
                        if (*(volatile int*)&c.abort_flag || globaltimer_ns() - t0 > g.limit_ns) {
                            few_abort(c, g.status);
                            ok = false;
                            break;
                        }
                    }
                    if (!ok) break;
                    fence_proxy_async_all();
                    ready = s.a;
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
                        tc_mma_bf16(tmem + acc * 128, ad + kk * 2, bd + kk * 2, idesc,
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
    } else if (warp >= kWarpsBeforeEpilogue) {
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
        bool more = walk.next(s);
        bool fresh = true;     // yacc holds nothing yet
        while (more) {
            const int e = plan.act[s.a];
            const int r0 = plan.off[e], rows = plan.off[e + 1] - r0;
            const int col = s.m * kTileM + i;
            const bool whole = s.kb0 == 0 && s.kb1 == s.KB;
            const bool live = col < (s.phase == 0 ? g.f : g.d);
            const T* bias = (const T*)(s.phase == 0 ? g.b1 : g.b2);
            const float b = bias && live && s.kb0 == 0
                                ? to_f32<T>(bias[(int64_t)e * (s.phase == 0 ? g.f : g.d) + col]) : 0.f;
            // unit of the first product cut over blocks c0..c1
            int c0 = me, c1 = me;
            float* mine = nullptr;
            if (s.phase == 0 && !whole) {
                c0 = walk.holder(0, s.unit * s.KB);
                c1 = walk.holder(0, s.unit * s.KB + s.KB - 1);
                mine = g.part1 + (me * 2 + (me == c0)) * slot_floats;
            }
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
                if (!epilogue_all<NT>(ok)) break;
                tc_fence_after();
                const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc * 128;
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
                const int groups = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
                const uint8_t* rt = plan.row_token + r0;
                bool ok;
                int nc;
                if (rows <= 2) {
                    nc = 2;
                    ok = products_f32<2>(g, c, s, rows, rt, a_ring, b_ring, as, ap, bs, bp, ew, lane, 1, red);
                } else if (rows <= 4) {
                    nc = 4;
                    ok = products_f32<4>(g, c, s, rows, rt, a_ring, b_ring, as, ap, bs, bp, ew, lane, 1, red);
                } else if (rows <= 8) {
                    nc = 8;
                    ok = products_f32<8>(g, c, s, rows, rt, a_ring, b_ring, as, ap, bs, bp, ew, lane, 1, red);
                } else {
                    nc = 16;
                    ok = products_f32<16>(g, c, s, rows, rt, a_ring, b_ring, as, ap, bs, bp, ew, lane, groups, red);
                }
                if (!ok) few_abort(c, g.status);
                if (!epilogue_all<NT>(ok)) break;
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
                        const float* from = g.part1 + i;
                        for (int r = tid / kTileM; r < rows; r += NT / kTileM) {
                            float v = __ldcg(from + (c0 * 2 + 1) * slot_floats + r * kTileM);
                            #pragma unroll 4
                            for (int q = c0 + 1; q <= c1; ++q)
                                v += __ldcg(from + q * 2 * slot_floats + r * kTileM);
                            put_hidden(r, v);
                        }
                    }
                }
                if (finished) {
                    __threadfence();
                    fence_proxy_async_all();
                    epilogue_barrier<NT>();
                    if (tid == 0) add_release(&g.cnt->done[s.a], 1);
                }
                more = walk.next(s);
                continue;
            }
            // second product: the tile is left when the next segment is another's
            const int m = s.m;
            more = walk.next(s);
            if (more && s.m == m) continue;
            fresh = true;
            const long long per = (long long)walk.nact * walk.KB[1];
            const int d0 = walk.holder(1, m * per), d1 = walk.holder(1, (m + 1) * per - 1);
            if (!K::kTensor) epilogue_barrier<NT>();
            bool finished = d0 == d1;
            if (!finished) {
                float* out = g.part2 + (me * 2 + (me == d0)) * slot_floats;
                for (int t = tid / kTileM; t < g.tokens; t += NT / kTileM)
                    __stcg(out + t * kTileM + i, yacc[t * kTileM + i]);
                __threadfence();
                epilogue_barrier<NT>();
                if (tid == 0) c.last = atomicAdd(&g.tiles_done[m], 1) == d1 - d0;
                epilogue_barrier<NT>();
                finished = c.last;
                if (finished) __threadfence();
            }
            if (finished && m * kTileM + i < g.d) {
                const T* residual = (const T*)g.residual;
                T* y = (T*)g.y;
                for (int t = tid / kTileM; t < g.tokens; t += NT / kTileM) {
                    float v;
                    if (d0 == d1) {
                        v = yacc[t * kTileM + i];
                    } else {
                        const float* from = g.part2 + t * kTileM + i;
                        v = __ldcg(from + (d0 * 2 + 1) * slot_floats);
                        #pragma unroll 4
                        for (int q = d0 + 1; q <= d1; ++q) v += __ldcg(from + q * 2 * slot_floats);
                    }
                    const int64_t o = (int64_t)t * g.d + m * kTileM + i;
                    if (residual) v += to_f32<T>(residual[o]);
                    y[o] = from_f32<T>(v);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (K::kTensor && warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
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

constexpr int kFewSmem = 227 * 1024;

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

template <typename T>
cudaError_t run(const moe_shape& s, const moe_layer_params& p, const T* x, const T* residual, T* y,
                uint8_t* ws, int32_t* status, cudaStream_t st) {
    using K = Kind<T>;
    const FewLayout l = few_layout(s);
    const int t = (int)s.T;
    FewArgs g;
    g.tokens = t;
    g.d = s.d; g.f = s.f; g.E = s.E; g.k = s.k; g.renorm = s.renorm;
    g.logits = (float*)(ws + l.logits);
    g.b1 = p.b1; g.b2 = p.b2; g.residual = residual; g.y = y;
    g.hidden = ws + l.hidden;
    g.part1 = (float*)(ws + l.part1);
    g.part2 = (float*)(ws + l.part2);
    g.cnt = (Counters*)(ws + l.counters);
    g.tiles_done = (int*)(g.cnt + 1);
    g.status = status;
    g.limit_ns = wait_limit_ns();

    int most = 0;
    cudaError_t e = few_smem_limit<T>(&most);
    if (e != cudaSuccess) return e;
    const int rows = t * K::kRowsPerSlot;     // activation rows a K block can have
    g.b_bytes = (rows + K::kBox - 1) / K::kBox * K::kBox * kBlockBytes;
    const int nc = t <= 2 ? 2 : t <= 4 ? 4 : t <= 8 ? 8 : 16;
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

    const int words = (int)((sizeof(Counters) + sizeof(int) * ((s.d + kTileM - 1) / kTileM)) / 4);
    const unsigned ge = (unsigned)((s.E + kLogitE - 1) / kLogitE);
    if (t == 1)
        few_logits_kernel<T, 1><<<dim3(ge, 1), kLogitThreads, 0, st>>>(
            t, s.d, s.E, x, (const T*)p.Wg, p.logit_bias, (float*)g.logits, (int*)g.cnt, words);
    else
        few_logits_kernel<T, 8><<<dim3(ge, (unsigned)((t + 7) / 8)), kLogitThreads, 0, st>>>(
            t, s.d, s.E, x, (const T*)p.Wg, p.logit_bias, (float*)g.logits, (int*)g.cnt, words);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;

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
