// head_simt.cu -- the three products of the losses over a vocabulary head in fp32,
// on the CUDA cores: fp32 is not split for the tensor cores.
//
// 64 x 128 tiles, 128 threads, 8 x 8 sums a thread held as packed pairs (64 FMAs a
// thread and K value for four 16-byte loads from shared memory), four blocks an SM.
// The FMA pipe bounds: 152 SMs x 128 FMAs at about 1.9 GHz are 74 TFLOP/s.  Half
// tiles of 128 x 128 cost half as many more loads from L2 and leave finer waves.
// DX and DW are cut along their reduction as the tensor cores' are (split_tiles).
#include "head.h"

namespace moe {
namespace {

constexpr int BM = 64, BN = 128, BK = 16, THREADS = 128;
constexpr int LDA = BM + 4, LDB = BN + 4;   // a K value's row in shared memory
constexpr int KB = 64;                      // K values the reduction is cut in multiples of
constexpr int kBlocksPerSm = 4;

enum Mode { Z = 0, ZKEEP = 1, DX = 2, DW = 3 };

// A ROWS x 16 step of an operand.  KC: the reduction runs along memory ([M][K]), else
// across it ([K][M]).  Rows and columns past the edge are zero: only the vocabulary
// may end inside a group of four, and G is zero from there to its row's end.
template <bool KC, int ROWS, int LD>
struct Loader {
    static constexpr int N = ROWS * BK / 4 / THREADS;
    const float* p;
    int64_t ld;
    int m0, mmax, kmax;
    float4 v[N];
    __device__ __forceinline__ void fetch(int k0, int tid) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int g = tid + i * THREADS;
            const int m = m0 + (KC ? g >> 2 : g % (ROWS / 4) * 4);
            const int k = k0 + (KC ? (g & 3) * 4 : g / (ROWS / 4));
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m < mmax && k < kmax)
                v[i] = *reinterpret_cast<const float4*>(p + (KC ? (int64_t)m * ld + k : (int64_t)k * ld + m));
        }
    }
    __device__ __forceinline__ void store(float (&s)[BK][LD], int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int g = tid + i * THREADS;
            if (KC) {
                const int m = g >> 2, k = (g & 3) * 4;
                s[k][m] = v[i].x;
                s[k + 1][m] = v[i].y;
                s[k + 2][m] = v[i].z;
                s[k + 3][m] = v[i].w;
            } else {
                *reinterpret_cast<float4*>(&s[g / (ROWS / 4)][g % (ROWS / 4) * 4]) = v[i];
            }
        }
    }
};

__device__ __forceinline__ float half_max(float v) {   // over 16 lanes
#pragma unroll
    for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct SimtParams {
    HeadDev h;
    HeadOut o;
    const float* A;
    const float* B;
    float* part;             // [cap][BM][BN] sums of cut tiles
    int cap;
    int units;               // blocks that run at once
};

template <int MODE> struct Shape { int M, N, K, MT, NT; };
template <int MODE> __device__ __forceinline__ Shape<MODE> shape_of(const HeadDev& h) {
    const int n = head_rows(h);
    Shape<MODE> s;
    s.M = MODE == DW ? h.V : n;
    s.N = MODE <= ZKEEP ? h.V : h.d;
    s.K = MODE <= ZKEEP ? h.d : MODE == DX ? h.V : n;
    s.MT = (s.M + BM - 1) / BM;
    s.NT = (s.N + BN - 1) / BN;
    return s;
}
template <int MODE> __device__ __forceinline__ Split plan_tiles(const SimtParams& p, const Shape<MODE>& s) {
    const int tiles = s.MT * s.NT, kb = (s.K + KB - 1) / KB;
    if (MODE <= ZKEEP) return Split{tiles, tiles, 1, kb};
    if (MODE == DW && s.K == 0) return Split{p.o.accumulate ? 0 : tiles, tiles, 1, 0};
    return split_tiles(tiles, kb, p.units, p.cap, 1, 1, 1, 1024);
}
// Tiles that share the larger operand follow each other: W's columns over the rows
// (Z, DX), G's columns over the width (DW).
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

template <int MODE>
__global__ void __launch_bounds__(THREADS, kBlocksPerSm) head_simt_kernel(const __grid_constant__ SimtParams p) {
    constexpr bool A_KC = MODE != DW, B_KC = MODE <= ZKEEP;
    __shared__ __align__(16) float As[2][BK][LDA], Bs[2][BK][LDB];
    __shared__ Split plan;
    const HeadDev& h = p.h;
    wait_front();
    const Shape<MODE> sh = shape_of<MODE>(h);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (tid < 32) {
        const Split s = plan_tiles<MODE>(p, sh);
        if (tid == 0) plan = s;
    }
    __syncthreads();
    const int u = blockIdx.x, rem = plan.tiles - min(plan.full, plan.tiles);
    int tile = u, k0 = 0, k1 = sh.K, slot = -1;
    if (plan.parts > 1 && u >= plan.full) {
        const int v = u - plan.full, part = v / rem;
        if (part >= plan.parts) return;
        tile = plan.full + v % rem;
        k0 = part * plan.kbp * KB;
        k1 = min(k1, k0 + plan.kbp * KB);
        slot = (tile - plan.full) * plan.parts + part;
    } else if (u >= plan.tiles) {
        return;
    }
    int mt, nt;
    tile_at<MODE>(sh, tile, mt, nt);
    const int m0 = mt * BM, n0 = nt * BN;
    Loader<A_KC, BM, LDA> la{p.A, MODE <= ZKEEP ? h.d : h.Vp, m0, sh.M, k1};
    Loader<B_KC, BN, LDB> lb{p.B, h.d, n0, sh.N, k1};

    uint64_t acc[8][4];   // [row][pair of columns]
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    const int steps = (k1 - k0 + BK - 1) / BK;
    if (steps > 0) {
        la.fetch(k0, tid);
        lb.fetch(k0, tid);
        la.store(As[0], tid);
        lb.store(Bs[0], tid);
    }
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        const int cur = s & 1;
        if (s + 1 < steps) {
            la.fetch(k0 + (s + 1) * BK, tid);
            lb.fetch(k0 + (s + 1) * BK, tid);
        }
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const float4 a0 = *reinterpret_cast<const float4*>(&As[cur][k][ty * 4]);
            const float4 a1 = *reinterpret_cast<const float4*>(&As[cur][k][32 + ty * 4]);
            const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&Bs[cur][k][tx * 4]);
            const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(&Bs[cur][k][64 + tx * 4]);
            const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            const uint64_t b[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t ai = f2_pack(a[i], a[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = f2_fma(ai, b[j], acc[i][j]);
            }
        }
        if (s + 1 < steps) {
            la.store(As[cur ^ 1], tid);
            lb.store(Bs[cur ^ 1], tid);
        }
        __syncthreads();
    }

    const float scale = MODE >= DX ? head_scale(h) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int rl = (i >> 2) * 32 + ty * 4 + (i & 3), r = m0 + rl;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) f2_unpack(acc[i][j], v[2 * j], v[2 * j + 1]);
        if (MODE <= ZKEEP) {
            // the row's 128 columns lie in 16 threads, eight each
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = n0 + (j >> 2) * 64 + tx * 4 + (j & 3);
                if (col < h.V) m = fmaxf(m, v[j]);
            }
            m = half_max(m) * h.c - kHeadShift;
            float sum = 0.f, e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = n0 + (j >> 2) * 64 + tx * 4 + (j & 3);
                e[j] = col < h.V ? exp2f(fmaf(v[j], h.c, -m)) : 0.f;
                sum += e[j];
            }
            sum = half_sum(sum);
            if (r >= sh.M) continue;
            if (tx == 0) h.stats[(int64_t)nt * h.srows + r] = make_float2(m, sum);
            if (MODE == ZKEEP) {
                float* out = (float*)h.P + (int64_t)r * h.Vp + n0;
#pragma unroll
                for (int jj = 0; jj < 2; ++jj)
                    if (n0 + jj * 64 < h.Vp)
                        *reinterpret_cast<float4*>(out + jj * 64 + tx * 4) =
                            make_float4(e[4 * jj], e[4 * jj + 1], e[4 * jj + 2], e[4 * jj + 3]);
            }
            const int t = head_token(h, r);
            int a = 0, b = 1;
            if (h.start) {
                a = h.start[(int64_t)t * h.nblk + nt];
                b = nt + 1 < h.nblk ? h.start[(int64_t)t * h.nblk + nt + 1] : h.ent[t];
            }
            for (; a < b; ++a) {
                const int64_t k = h.target ? h.target[t] : h.sidx[(int64_t)t * h.K + a];
                const int64_t rel = k - n0;
                if (rel < 0 || rel >= BN || ((rel & 63) >> 2) != tx) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if ((j >> 2) * 64 + tx * 4 + (j & 3) == (int)rel) h.lz[(int64_t)t * h.K + a] = v[j];
            }
        } else {
            if (r >= sh.M) continue;
            float* out = slot >= 0 ? p.part + ((int64_t)slot * BM + rl) * BN
                                   : (float*)p.o.out + (int64_t)(MODE == DX ? head_token(h, r) : r) * h.d + n0;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int c = jj * 64 + tx * 4;
                if (n0 + c >= sh.N) continue;
                const float4 w = make_float4(v[4 * jj], v[4 * jj + 1], v[4 * jj + 2], v[4 * jj + 3]);
                if (slot >= 0) *reinterpret_cast<float4*>(out + c) = w;
                else write4<MODE>(p.o, out + c, make_float4(w.x * scale, w.y * scale, w.z * scale, w.w * scale));
            }
        }
    }
}

// The parts of cut tiles, added in order.
template <int MODE>
__global__ void __launch_bounds__(256) head_simt_join_kernel(const __grid_constant__ SimtParams p) {
    __shared__ Split plan;
    __shared__ float4 buf[256];
    const HeadDev& h = p.h;
    wait_front();
    const Shape<MODE> sh = shape_of<MODE>(h);
    if (threadIdx.x < 32) {
        const Split s = plan_tiles<MODE>(p, sh);
        if (threadIdx.x == 0) plan = s;
    }
    __syncthreads();
    const int i = blockIdx.x;
    if (plan.parts <= 1 || plan.full + i >= plan.tiles) return;
    int mt, nt;
    tile_at<MODE>(sh, plan.full + i, mt, nt);
    const float scale = head_scale(h);
    for (int rl = blockIdx.y * kJoinRows; rl < (int)(blockIdx.y + 1) * kJoinRows; ++rl) {
        const int r = mt * BM + rl;
        if (r >= sh.M) return;
        float4 s;
        const int c = join_row<BN>(p.part + ((int64_t)i * plan.parts * BM + rl) * BN, (int64_t)BM * BN, plan.parts,
                                   buf, s);
        if (c < 0 || nt * BN + c >= sh.N) continue;
        float* out = (float*)p.o.out + (int64_t)(MODE == DX ? head_token(h, r) : r) * h.d + nt * BN + c;
        write4<MODE>(p.o, out, make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale));
    }
}

int simt_units() { return kBlocksPerSm * device_sm_count(); }

template <int MODE>
cudaError_t launch(SimtParams& p, int64_t M, int64_t N, int64_t K, size_t part_bytes, cudaStream_t st) {
    const int64_t tiles = (M + BM - 1) / BM * ((N + BN - 1) / BN);
    if (tiles == 0) return cudaSuccess;
    p.units = simt_units();
    p.cap = (int)(part_bytes / (BM * BN * 4));
    // (a device count below M or K leaves fewer tiles, but perhaps more parts: their
    // most is what the workspace holds)
    const int64_t units = MODE <= ZKEEP ? tiles : tiles + p.cap;
    cudaError_t e = launch_early(head_simt_kernel<MODE>, dim3((unsigned)units), THREADS, 0, 1, st, p);
    if constexpr (MODE >= DX) {
        if (e != cudaSuccess || p.cap == 0) return e;
        const int64_t rem = tiles < p.units ? tiles : p.units, rows = M < BM ? M : BM;
        e = launch_early(head_simt_join_kernel<MODE>,
                         dim3((unsigned)rem, (unsigned)((rows + kJoinRows - 1) / kJoinRows)), 256, 0, 1, st, p);
    }
    return e;
}

}  // namespace

size_t head_simt_part_bytes(int64_t rows, int V, int d) {
    const int64_t nt = (d + BN - 1) / BN;
    const size_t a = split_bound((rows + BM - 1) / BM * nt, (V + KB - 1) / KB, simt_units(), 1);
    const size_t b = split_bound((V + BM - 1) / BM * nt, (rows + KB - 1) / KB, simt_units(), 1);
    return (a > b ? a : b) * BM * BN * 4;
}

cudaError_t launch_head_simt(const HeadDev& h, const void* xc, const void* W, bool keep, cudaStream_t st) {
    SimtParams p{h, HeadOut{}, (const float*)xc, (const float*)W, nullptr, 0, 0};
    return keep ? launch<ZKEEP>(p, h.rows, h.V, h.d, 0, st) : launch<Z>(p, h.rows, h.V, h.d, 0, st);
}

cudaError_t launch_head_simt_dx(const HeadDev& h, const void* W, const HeadOut& o, float* part, size_t part_bytes,
                                cudaStream_t st) {
    SimtParams p{h, o, (const float*)h.P, (const float*)W, part, 0, 0};
    return launch<DX>(p, h.rows, h.d, h.V, part_bytes, st);
}

cudaError_t launch_head_simt_dw(const HeadDev& h, const void* xc, const HeadOut& o, float* part, size_t part_bytes,
                                cudaStream_t st) {
    SimtParams p{h, o, (const float*)h.P, (const float*)xc, part, 0, 0};
    return launch<DW>(p, h.V, h.d, h.rows, part_bytes, st);
}

}  // namespace moe
