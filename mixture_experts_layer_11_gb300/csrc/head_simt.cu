// head_simt.cu -- the three products of the losses over a vocabulary head in fp32,
// on the CUDA cores: fp32 is not split for the tensor cores.
//
// The FMA pipe bounds (152 SMs x 128 FMAs at about 1.9 GHz are 74 TFLOP/s), fed by
// fma.rn.f32x2 from shared memory that cp.async fills two or three steps ahead, in the
// order memory has them:
//   Z     both operands run along K: a pair is two neighbouring K values, whose sums
//         are added at the end.  64 x 128 tiles of 128 threads, 8 x 8 sums each;
//         16 x 128 where those would leave SMs idle; for the losses of few rows
//         8 TM x 64, so that there are blocks enough to stream W
//   DX    G runs along K, W across: pairs are neighbouring columns, G's value doubled
//   DW    both run across K.  Both 64 x 128 tiles of 128 threads, 8 x 8 sums each
// DX and DW are cut along their reduction as the tensor cores' are (split_tiles); shorter
// sums are the more exact ones, too (dx over 8009 entries 8e-7 off in place of 2e-6).
// 875 rows of 8009 entries, d = 768: Z 265 us (41 TFLOP/s, FMA pipe 61 % busy), DX and DW
// together 371 (58 TFLOP/s, 77 %), joining 14.  33 rows of 32000: 57 us, FMA pipe 55 %.
// 256 rows of 1000, d = 64: 8 and 14 us, latency.
#include "head.h"

namespace moe {
namespace {

constexpr int BM = 64, BN = 128, BK = 16, THREADS = 128;
constexpr int STAGES = 3;
constexpr int LDK = BK + 4;                 // a row of K values in shared memory
constexpr int KB = 64;                      // K values the reduction is cut in multiples of (SplitRule)
constexpr int kBlocksPerSm = 4;

enum Mode { Z = 0, ZKEEP = 1, DX = 2, DW = 3 };

__device__ __forceinline__ void copy16(float* dst, const float* src, bool on) {
    // off: 16 bytes of zeros (src is not read)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A step of an operand to shared memory.  KC: the reduction runs along memory
// ([M][K]), kept as [ROWS][LDK]; else across it ([K][M]), kept as [BK][ROWS + 4].
// Rows and columns past the edge are zero: only the vocabulary may end inside a group
// of four, and G is zero from there to its row's end.
template <bool KC, int ROWS, int NT, int BK = 16>
struct Loader {
    static constexpr int LD = KC ? (BK + 4) : ROWS + 4;
    static constexpr int SIZE = KC ? ROWS * (BK + 4) : BK * (ROWS + 4);
    static constexpr int G = KC ? BK / 4 : ROWS / 4;       // groups of four in a row of memory
    static constexpr int N = ROWS * BK / 4, COPIES = (N + NT - 1) / NT, SKIP = NT / G;
    static_assert(NT % G == 0, "a thread's groups lie under one another");
    const float* src;       // the thread's first group at K value 0
    int64_t ld, skip;       // values from one K step's or row's memory to the next
    int at, outer, edge, kl;   // place in shared memory; first row of memory, their end; K offset
    bool inner;
    __device__ __forceinline__ Loader(const float* p, int64_t ld_, int m0, int mmax, int tid) {
        const int in = tid % G * 4, out = tid / G;
        ld = ld_;
        skip = SKIP * ld_;
        at = out * LD + in;
        src = p + (KC ? (int64_t)(m0 + out) * ld_ + in : (int64_t)out * ld_ + m0 + in);
        outer = KC ? m0 + out : out;
        edge = mmax;
        kl = KC ? in : out;
        inner = KC || m0 + in < mmax;
    }
    __device__ __forceinline__ void copy(float* s, int k0, int kmax) const {
        const float* p = src + (KC ? k0 : k0 * ld);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            if (N % NT && i == COPIES - 1 && at / LD + i * SKIP >= (KC ? ROWS : BK)) break;
            const bool on = KC ? outer + i * SKIP < edge && k0 + kl < kmax : inner && k0 + kl + i * SKIP < kmax;
            copy16(s + at + i * SKIP * LD, on ? p + i * skip : src, on);
        }
    }
};

template <int W> __device__ __forceinline__ float lanes_max(float v) {   // over W lanes
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int W> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct SimtParams {
    HeadDev h;
    HeadOut dx, dW;          // out null: not wanted
    const float* xc;
    const float* W;
    float* part;             // [capx + capw][BM][BN] sums of cut tiles, DX's first
    int capx;
    int ux;                  // blocks of DX's (the first)
};

// ---- Z ---------------------------------------------------------------------------------
//
// TY x TX threads; thread (ty, tx) has rows ty + TY i and columns tx + TX j, so that
// its 16-byte loads (rows of 80 bytes) meet no bank conflict.
template <int TY, int TX, int TM, int TN, bool KEEP, int DEPTH, int BLOCKS, int BK = 16>
__global__ void __launch_bounds__(TY * TX, BLOCKS)
    head_simt_z_kernel(const __grid_constant__ SimtParams p) {
    constexpr int ROWS = TY * TM, COLS = TX * TN, NT = TY * TX;
    using LA = Loader<true, ROWS, NT, BK>;
    using LB = Loader<true, COLS, NT, BK>;
    __shared__ __align__(16) float smem[DEPTH][LA::SIZE + LB::SIZE];
    const HeadDev& h = p.h;
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    wait_front();
    const int n = head_rows(h);
    const int MT = (n + ROWS - 1) / ROWS;   // rows first: W's tile is shared
    const int mt = MT ? blockIdx.x % MT : 0, nt = MT ? blockIdx.x / MT : 0;
    const int m0 = mt * ROWS, n0 = nt * COLS;
    if (MT == 0 || n0 >= h.V) return;
    const LA la(p.xc, h.d, m0, n, tid);
    const LB lb(p.W, h.d, n0, h.V, tid);
    uint64_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = 0;
    const int steps = (h.d + BK - 1) / BK;
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) {
        if (s < steps) {
            la.copy(smem[s], s * BK, h.d);
            lb.copy(smem[s] + LA::SIZE, s * BK, h.d);
        }
        copies_commit();
    }
    for (int s = 0, cur = 0; s < steps; ++s) {
        copies_wait<DEPTH - 2>();
        __syncthreads();
        const int next = cur == 0 ? DEPTH - 1 : cur - 1;   // (s + DEPTH - 1) % DEPTH
        if (s + DEPTH - 1 < steps) {
            la.copy(smem[next], (s + DEPTH - 1) * BK, h.d);
            lb.copy(smem[next] + LA::SIZE, (s + DEPTH - 1) * BK, h.d);
        }
        copies_commit();
        const float* A = smem[cur] + ty * (BK + 4);
        const float* B = smem[cur] + LA::SIZE + tx * (BK + 4);
#pragma unroll
        for (int k = 0; k < BK; k += 4) {
            ulonglong2 a[TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(A + i * TY * (BK + 4) + k);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(B + j * TX * (BK + 4) + k);
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[i][j] = f2_fma(a[i].x, b.x, acc[i][j]);
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[i][j] = f2_fma(a[i].y, b.y, acc[i][j]);
            }
        }
        if (++cur == DEPTH) cur = 0;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = m0 + ty + TY * i;
        float v[TN], e[TN], m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            float a, b;
            f2_unpack(acc[i][j], a, b);
            v[j] = a + b;
            if (n0 + tx + TX * j < h.V) m = fmaxf(m, v[j]);
        }
        m = lanes_max<TX>(m);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            e[j] = n0 + tx + TX * j < h.V ? exp2f(fmaf(v[j] - m, h.c, kHeadShift)) : 0.f;
            sum += e[j];
        }
        sum = lanes_sum<TX>(sum);
        if (r >= n) continue;
        if (tx == 0) h.stats[(int64_t)nt * h.srows + r] = make_float2(m, sum);
        if (KEEP) {
            float* out = (float*)h.P + (int64_t)r * h.Vp + n0;
#pragma unroll
            for (int j = 0; j < TN; ++j)
                if (n0 + tx + TX * j < h.Vp) out[tx + TX * j] = e[j];
        }
        // the targets' logits
        const int t = head_token(h, r);
        int a = 0, b = 1;
        if (h.start) {
            const int blk = n0 / kHeadBlock;
            a = h.start[(int64_t)t * h.nblk + blk];
            b = blk + 1 < h.nblk ? h.start[(int64_t)t * h.nblk + blk + 1] : h.ent[t];
        }
        for (; a < b; ++a) {
            const int64_t rel = (h.target ? h.target[t] : h.sidx[(int64_t)t * h.K + a]) - n0;
            if (rel < 0 || rel >= COLS || rel % TX != tx) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j)
                if (tx + TX * j == (int)rel) h.lz[(int64_t)t * h.K + a] = v[j];
        }
    }
}

// ---- DX, DW ------------------------------------------------------------------------------

template <int MODE> struct Shape { int M, N, K, MT, NT; };
template <int MODE> __device__ __forceinline__ Shape<MODE> shape_of(const HeadDev& h) {
    const int n = head_rows(h);
    Shape<MODE> s;
    s.M = MODE == DW ? h.V : n;
    s.N = h.d;
    s.K = MODE == DX ? h.V : n;
    s.MT = (s.M + BM - 1) / BM;
    s.NT = (s.N + BN - 1) / BN;
    return s;
}
// Tiles that share the larger operand follow each other: W's columns over the rows
// (DX), G's columns over the width (DW).
template <int MODE> __device__ __forceinline__ void tile_at(const Shape<MODE>& s, int i, int& mt, int& nt) {
    if (MODE == DW) {
        mt = i / s.NT;
        nt = i % s.NT;
    } else {
        mt = i % s.MT;
        nt = i / s.MT;
    }
}

template <int MODE>
__device__ __forceinline__ void write4(const HeadOut& o, float* out, float4 v) {
    if (MODE == DW && o.accumulate) {
        const float4 b = *reinterpret_cast<const float4*>(out);
        v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
    }
    *reinterpret_cast<float4*>(out) = v;
}

template <int MODE> struct Loaders {
    using A = Loader<MODE == DX, BM, THREADS>;
    using B = Loader<false, BN, THREADS>;
    static constexpr int SIZE = A::SIZE + B::SIZE;
};

// The sums of a tile over K values k0 to k1: [row][pair of columns].
template <int MODE>
__device__ __forceinline__ void tile_sums(const SimtParams& p, const Shape<MODE>& sh, int m0, int n0, int k0, int k1,
                                          float* smem_raw, uint64_t (&acc)[8][4]) {
    using LA = typename Loaders<MODE>::A;
    using LB = typename Loaders<MODE>::B;
    float(*smem)[Loaders<MODE>::SIZE] = reinterpret_cast<float(*)[Loaders<MODE>::SIZE]>(smem_raw);
    const HeadDev& h = p.h;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const LA la((const float*)h.P, h.Vp, m0, sh.M, tid);
    const LB lb(MODE == DX ? p.W : p.xc, h.d, n0, sh.N, tid);

#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    const int steps = (k1 - k0 + BK - 1) / BK;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (s < steps) {
            la.copy(smem[s], k0 + s * BK, k1);
            lb.copy(smem[s] + LA::SIZE, k0 + s * BK, k1);
        }
        copies_commit();
    }
    for (int s = 0, cur = 0; s < steps; ++s) {
        copies_wait<STAGES - 2>();
        __syncthreads();
        const int next = cur == 0 ? STAGES - 1 : cur - 1;
        if (s + STAGES - 1 < steps) {
            la.copy(smem[next], k0 + (s + STAGES - 1) * BK, k1);
            lb.copy(smem[next] + LA::SIZE, k0 + (s + STAGES - 1) * BK, k1);
        }
        copies_commit();
        const float* A = smem[cur];
        const float* B = smem[cur] + LA::SIZE + tx * 4;
#pragma unroll
        for (int k4 = 0; k4 < BK; k4 += 4) {
            float4 ak[8];   // DX: the rows' four K values
            if (MODE == DX) {
#pragma unroll
                for (int i = 0; i < 8; ++i) ak[i] = *reinterpret_cast<const float4*>(A + (ty + 8 * i) * LDK + k4);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int k = k4 + kk;
                float a[8];
                if (MODE == DX) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = kk == 0 ? ak[i].x : kk == 1 ? ak[i].y : kk == 2 ? ak[i].z : ak[i].w;
                } else {
                    const float4 a0 = *reinterpret_cast<const float4*>(A + k * LA::LD + ty * 8);
                    const float4 a1 = *reinterpret_cast<const float4*>(A + k * LA::LD + ty * 8 + 4);
                    a[0] = a0.x, a[1] = a0.y, a[2] = a0.z, a[3] = a0.w;
                    a[4] = a1.x, a[5] = a1.y, a[6] = a1.z, a[7] = a1.w;
                }
                const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(B + k * LB::LD);
                const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(B + k * LB::LD + 64);
                const uint64_t b[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint64_t ai = f2_pack(a[i], a[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = f2_fma(ai, b[j], acc[i][j]);
                }
            }
        }
        if (++cur == STAGES) cur = 0;
    }
}

template <int MODE>
__device__ __forceinline__ void product(const SimtParams& p, int u, float* smem) {
    const HeadDev& h = p.h;
    const HeadOut& o = MODE == DX ? p.dx : p.dW;
    const Shape<MODE> sh = shape_of<MODE>(h);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const Split plan = h.splits[MODE == DW];
    const int rem = plan.tiles - plan.full;
    int tile = u, k0 = 0, k1 = sh.K, slot = -1;
    if (plan.parts > 1 && u >= plan.full) {
        const int v = u - plan.full, part = v / rem;
        if (part >= plan.parts) return;
        tile = plan.full + v % rem;
        k0 = part * plan.kbp * KB;
        k1 = min(k1, k0 + plan.kbp * KB);
        slot = (MODE == DX ? 0 : p.capx) + (tile - plan.full) * plan.parts + part;
    } else if (u >= plan.tiles) {
        return;
    }
    int mt, nt;
    tile_at<MODE>(sh, tile, mt, nt);
    const int m0 = mt * BM, n0 = nt * BN;
    uint64_t acc[8][4];
    tile_sums<MODE>(p, sh, m0, n0, k0, k1, smem, acc);

    const float scale = head_scale(h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int rl = MODE == DX ? ty + 8 * i : ty * 8 + i, r = m0 + rl;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f2_unpack(acc[i][j], v[2 * j], v[2 * j + 1]);
        if (r >= sh.M) continue;
        float* out = slot >= 0 ? p.part + ((int64_t)slot * BM + rl) * BN
                               : (float*)o.out + (int64_t)(MODE == DX ? head_token(h, r) : r) * h.d + n0;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const int c = jj * 64 + tx * 4;
            if (n0 + c >= sh.N) continue;
            const float4 w = make_float4(v[4 * jj], v[4 * jj + 1], v[4 * jj + 2], v[4 * jj + 3]);
            if (slot >= 0) *reinterpret_cast<float4*>(out + c) = w;
            else write4<MODE>(o, out + c, make_float4(w.x * scale, w.y * scale, w.z * scale, w.w * scale));
        }
    }
}

// DX's blocks, then DW's.
__global__ void __launch_bounds__(THREADS, kBlocksPerSm) head_simt_grad_kernel(const __grid_constant__ SimtParams p) {
    constexpr int SIZE = Loaders<DX>::SIZE > Loaders<DW>::SIZE ? Loaders<DX>::SIZE : Loaders<DW>::SIZE;
    __shared__ __align__(16) float smem[STAGES * SIZE];
    wait_front();
    if ((int)blockIdx.x < p.ux) product<DX>(p, blockIdx.x, smem);
    else product<DW>(p, blockIdx.x - p.ux, smem);
}

// Small products: a cluster of eight blocks a tile, each an eighth of the reduction.  The
// sums meet in shared memory, each block adds eight rows of them in order: no part goes
// to the workspace, and no launch joins (256 rows of 1000 entries, d = 64: 14 us in place
// of 16 and the join's launch; the call takes 36).
constexpr int kCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 load_from(uint32_t addr, int rank) {
    uint32_t there;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(there)
                 : "memory");
    return v;
}

template <int MODE>
__device__ __forceinline__ void cluster_product(const SimtParams& p, int tile, float* smem) {
    const HeadDev& h = p.h;
    const HeadOut& o = MODE == DX ? p.dx : p.dW;
    const Shape<MODE> sh = shape_of<MODE>(h);
    // (the same for all blocks of a cluster)
    if (tile >= sh.MT * sh.NT || (MODE == DW && sh.K == 0 && o.accumulate)) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, rank = (int)cluster_rank();
    int mt, nt;
    tile_at<MODE>(sh, tile, mt, nt);
    const int m0 = mt * BM, n0 = nt * BN;
    const int share = ((sh.K + BK - 1) / BK + kCluster - 1) / kCluster * BK;
    const int k0 = min(sh.K, rank * share), k1 = min(sh.K, k0 + share);
    uint64_t acc[8][4];
    tile_sums<MODE>(p, sh, m0, n0, k0, k1, smem, acc);
    copies_wait<0>();
    __syncthreads();   // the steps' memory is free
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float* row = smem + (MODE == DX ? ty + 8 * i : ty * 8 + i) * BN + tx * 4;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            float4 v;
            f2_unpack(acc[i][2 * jj], v.x, v.y);
            f2_unpack(acc[i][2 * jj + 1], v.z, v.w);
            *reinterpret_cast<float4*>(row + jj * 64) = v;
        }
    }
    cluster_sync();
    constexpr int ROWS = BM / kCluster;
    const float scale = head_scale(h);
#pragma unroll
    for (int i = 0; i < ROWS * BN / 4 / THREADS; ++i) {
        const int g = tid + i * THREADS, rl = rank * ROWS + g / (BN / 4), c = g % (BN / 4) * 4, r = m0 + rl;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < kCluster; ++q) {
            const float4 v = load_from(smem_u32(smem + rl * BN + c), q);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        if (r < sh.M && n0 + c < sh.N)
            write4<MODE>(o, (float*)o.out + (int64_t)(MODE == DX ? head_token(h, r) : r) * h.d + n0 + c,
                         make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale));
    }
    cluster_sync();   // no block ends while others read its sums
}

__global__ void __launch_bounds__(THREADS) head_simt_cluster_kernel(const __grid_constant__ SimtParams p) {
    constexpr int SIZE = Loaders<DX>::SIZE > Loaders<DW>::SIZE ? Loaders<DX>::SIZE : Loaders<DW>::SIZE;
    static_assert(STAGES * SIZE >= BM * BN, "a tile's sums fit the steps' memory");
    __shared__ __align__(16) float smem[STAGES * SIZE];
    wait_front();
    const int tile = blockIdx.x / kCluster;
    if (tile < p.ux) cluster_product<DX>(p, tile, smem);
    else cluster_product<DW>(p, tile - p.ux, smem);
}

// The parts of cut tiles, added in order.
template <int MODE>
__device__ __forceinline__ void join(const SimtParams& p, int i, float4 (*buf)[256]) {
    const HeadDev& h = p.h;
    const HeadOut& o = MODE == DX ? p.dx : p.dW;
    const Shape<MODE> sh = shape_of<MODE>(h);
    const Split plan = h.splits[MODE == DW];
    if (plan.parts <= 1 || plan.full + i >= plan.tiles) return;
    int mt, nt;
    tile_at<MODE>(sh, plan.full + i, mt, nt);
    const float scale = head_scale(h);
    const int rl = blockIdx.y * kJoinRows, r0 = mt * BM + rl, rows = sh.M - r0;
    if (rows <= 0) return;
    float4 s[kJoinRows];
    const int64_t slot = (MODE == DX ? 0 : p.capx) + (int64_t)i * plan.parts;
    const int c = join_rows<BN>(p.part + (slot * BM + rl) * BN, (int64_t)BM * BN, plan.parts, rows, buf, s);
    if (c < 0 || nt * BN + c >= sh.N) return;
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        if (r >= rows) break;
        float* out = (float*)o.out + (int64_t)(MODE == DX ? head_token(h, r0 + r) : r0 + r) * h.d + nt * BN + c;
        write4<MODE>(o, out, make_float4(s[r].x * scale, s[r].y * scale, s[r].z * scale, s[r].w * scale));
    }
}
__global__ void __launch_bounds__(256) head_simt_join_kernel(const __grid_constant__ SimtParams p, int nx) {
    __shared__ float4 buf[kJoinRows][256];
    wait_front();
    if ((int)blockIdx.x < nx) join<DX>(p, blockIdx.x, buf);
    else join<DW>(p, blockIdx.x - nx, buf);
}

int simt_units() { return kBlocksPerSm * device_sm_count(); }

template <int TM> cudaError_t launch_few(const SimtParams& p, cudaStream_t st) {
    return launch_early(head_simt_z_kernel<8, 16, TM, 4, false, 3, 1, 32>, dim3((unsigned)((p.h.V + 63) / 64)), 128, 0, 1, st, p);
}

int64_t tiles_of(int64_t m, int64_t n) { return (m + BM - 1) / BM * ((n + BN - 1) / BN); }
int64_t parts_dx(int64_t rows, int V, int d) {
    return (int64_t)split_bound(tiles_of(rows, d), (V + KB - 1) / KB, simt_units(), 1);
}
int64_t parts_dw(int64_t rows, int V, int d) {
    return (int64_t)split_bound(tiles_of(V, d), (rows + KB - 1) / KB, simt_units(), 1);
}

}  // namespace

// The most rows of a call without gradients that take narrow tiles (its statistics are
// over blocks of 64): 33 rows of 32000 entries, d = 768, 130 us in 64 x 128 tiles, 62
// in narrow ones.
int head_simt_few_rows() { return 64; }

size_t head_simt_part_bytes(int64_t rows, int V, int d) {
    return (size_t)(parts_dx(rows, V, d) + parts_dw(rows, V, d)) * BM * BN * 4;
}

SplitRule head_simt_rule(int64_t rows, int V, int d) {
    return SplitRule{BM, BN, simt_units(), (int)parts_dx(rows, V, d), (int)parts_dw(rows, V, d), 1, 1, 1, 1024, 0, 0, 0};
}

cudaError_t launch_head_simt(const HeadDev& h, const void* xc, const void* W, bool keep, cudaStream_t st) {
    SimtParams p{};
    p.h = h;
    p.xc = (const float*)xc;
    p.W = (const float*)W;
    if (h.nstat > h.nblk) {
        switch ((h.T + 7) / 8) {
            case 1: return launch_few<1>(p, st);
            case 2: return launch_few<2>(p, st);
            case 3: return launch_few<3>(p, st);
            case 4: return launch_few<4>(p, st);
            case 5: return launch_few<5>(p, st);
            case 6: return launch_few<6>(p, st);
            default: return launch_few<8>(p, st);
        }
    }
    const int64_t rows = h.T - h.p0 < h.rows ? h.T - h.p0 : h.rows, cols = (h.V + 127) / 128;
    // tiles of 16 rows where those of 64 would leave SMs idle
    if ((rows + 63) / 64 * cols < device_sm_count())
        return launch_early(keep ? head_simt_z_kernel<4, 32, 4, 4, true, 4, 1> : head_simt_z_kernel<4, 32, 4, 4, false, 4, 1>,
                            dim3((unsigned)((rows + 15) / 16 * cols)), 128, 0, 1, st, p);
    return launch_early(keep ? head_simt_z_kernel<8, 16, 8, 8, true, STAGES, 2> : head_simt_z_kernel<8, 16, 8, 8, false, STAGES, 2>,
                        dim3((unsigned)((rows + 63) / 64 * cols)), 128, 0, 1, st, p);
}

cudaError_t launch_head_simt_grad(const HeadDev& h, const void* xc, const void* W, const HeadOut& dx,
                                  const HeadOut& dW, float* part, const SplitRule& rule, cudaStream_t st) {
    SimtParams p{};
    p.h = h;
    p.dx = dx;
    p.dW = dW;
    p.xc = (const float*)xc;
    p.W = (const float*)W;
    p.part = part;
    p.capx = rule.capx;
    // (fewer live rows leave fewer tiles, but perhaps more parts: at most what the
    // workspace holds)
    const int64_t rows = h.T - h.p0 < h.rows ? h.T - h.p0 : h.rows;
    const int64_t tx = dx.out ? tiles_of(rows, h.d) : 0, tw = dW.out ? tiles_of(h.V, h.d) : 0;
    if ((tx + tw) * kCluster <= rule.units) {   // all clusters run at once
        p.ux = (int)tx;
        if (tx + tw == 0) return cudaSuccess;
        return launch_early(head_simt_cluster_kernel, dim3((unsigned)((tx + tw) * kCluster)), THREADS, 0, kCluster, st, p);
    }
    p.ux = (int)(tx ? tx + rule.capx : 0);
    const int64_t blocks = p.ux + (tw ? tw + rule.capw : 0);
    if (blocks == 0) return cudaSuccess;
    cudaError_t e = launch_early(head_simt_grad_kernel, dim3((unsigned)blocks), THREADS, 0, 1, st, p);
    if (e != cudaSuccess) return e;
    const int nx = rule.capx ? (int)(tx < rule.units ? tx : rule.units) : 0, nw = rule.capw ? (int)(tw % rule.units) : 0;
    if (nx + nw == 0) return cudaSuccess;
    const int most = nw || rows > BM ? BM : (int)rows;
    return launch_early(head_simt_join_kernel, dim3((unsigned)(nx + nw), (unsigned)((most + kJoinRows - 1) / kJoinRows)),
                        256, 0, 1, st, p, nx);
}

}  // namespace moe
