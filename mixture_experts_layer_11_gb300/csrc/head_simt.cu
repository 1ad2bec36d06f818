// head_simt.cu -- the three products of the losses over a vocabulary head on the
// CUDA cores, in fp32: 128 x 128 tiles, 8 x 8 sums a thread held as packed pairs.
#include "head.h"

namespace moe {
namespace {

constexpr int BM = 128, BN = 128, BK = 16, THREADS = 256;
constexpr int LD = BM + 4;     // row of a K step in shared memory, 16-byte aligned

enum Mode { Z = 0, ZKEEP = 1, DX = 2, DW = 3 };

// A 128 x 16 step of an operand, as two groups of four values a thread.  KC: the
// reduction runs along memory (row-major [M][K]), else across it ([K][M]).  Rows
// and columns past the edge are zero; a group of four never straddles an edge
// but in the vocabulary (kmax or mmax not a multiple of 4), where it is masked.
template <bool KC>
struct Loader {
    const float* p;
    int64_t ld;
    int m0, mmax, kmax;
    float4 v[2];
    __device__ __forceinline__ void fetch(int k0, int tid) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = tid + i * THREADS;
            const int m = m0 + (KC ? g >> 2 : (g & 31) * 4), k = k0 + (KC ? (g & 3) * 4 : g >> 5);
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m < mmax && k < kmax) {
                v[i] = *reinterpret_cast<const float4*>(p + (KC ? (int64_t)m * ld + k : (int64_t)k * ld + m));
                const int left = KC ? kmax - k : mmax - m;
                if (left < 2) v[i].y = 0.f;
                if (left < 3) v[i].z = 0.f;
                if (left < 4) v[i].w = 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(float (&s)[BK][LD], int tid) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = tid + i * THREADS;
            if (KC) {
                const int m = g >> 2, k = (g & 3) * 4;
                s[k][m] = v[i].x;
                s[k + 1][m] = v[i].y;
                s[k + 2][m] = v[i].z;
                s[k + 3][m] = v[i].w;
            } else {
                *reinterpret_cast<float4*>(&s[g >> 5][(g & 31) * 4]) = v[i];
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

template <int MODE>
__global__ void __launch_bounds__(THREADS)
    head_simt_kernel(const HeadDev h, const float* A, const float* B, const HeadOut o) {
    constexpr bool A_KC = MODE != DW, B_KC = MODE <= ZKEEP;
    __shared__ __align__(16) float As[2][BK][LD], Bs[2][BK][LD];
    const int n = head_rows(h);
    const int M = MODE == DW ? h.V : n;
    const int N = MODE <= ZKEEP ? h.V : h.d;
    const int K = MODE <= ZKEEP ? h.d : MODE == DX ? h.V : n;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int m0 = blockIdx.x * BM, n0 = blockIdx.y * BN;
    if (m0 >= M) return;
    Loader<A_KC> la{A, MODE <= ZKEEP ? h.d : h.Vp, m0, M, K};
    Loader<B_KC> lb{B, h.d, n0, N, K};

    uint64_t acc[8][4];   // [row][pair of columns]
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    const int steps = (K + BK - 1) / BK;
    if (steps > 0) {
        la.fetch(0, tid);
        lb.fetch(0, tid);
        la.store(As[0], tid);
        lb.store(Bs[0], tid);
    }
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        const int cur = s & 1;
        if (s + 1 < steps) {
            la.fetch((s + 1) * BK, tid);
            lb.fetch((s + 1) * BK, tid);
        }
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const float4 a0 = *reinterpret_cast<const float4*>(&As[cur][k][ty * 4]);
            const float4 a1 = *reinterpret_cast<const float4*>(&As[cur][k][64 + ty * 4]);
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
        const int r = m0 + (i >> 2) * 64 + ty * 4 + (i & 3);
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
            if (r >= n) continue;
            if (tx == 0) h.stats[(int64_t)blockIdx.y * h.srows + r] = make_float2(m, sum);
            if (MODE == ZKEEP) {
                float* out = (float*)h.P + (int64_t)r * h.Vp;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int col = n0 + (j >> 2) * 64 + tx * 4 + (j & 3);
                    if (col < h.Vp) out[col] = e[j];
                }
            }
            const int t = head_token(h, r);
            int a = 0, b = 1;
            if (!h.target && h.K > 1) {
                a = h.start[(int64_t)t * h.nblk + blockIdx.y];
                b = (int)blockIdx.y + 1 < h.nblk ? h.start[(int64_t)t * h.nblk + blockIdx.y + 1] : h.ent[t];
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
            if (r >= M) continue;
            const int64_t row = MODE == DX ? head_token(h, r) : r;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = n0 + (j >> 2) * 64 + tx * 4 + (j & 3);
                if (col >= N) continue;
                const int64_t at = row * N + col;
                float* out = (float*)o.out;
                out[at] = o.accumulate ? fmaf(scale, v[j], out[at]) : scale * v[j];
            }
        }
    }
}

template <int MODE>
cudaError_t launch(const HeadDev& h, const void* A, const void* B, const HeadOut& o, int64_t M, int64_t N,
                   cudaStream_t st) {
    const dim3 grid((unsigned)((M + BM - 1) / BM), (unsigned)((N + BN - 1) / BN));
    if (grid.x == 0 || grid.y == 0) return cudaSuccess;
    head_simt_kernel<MODE><<<grid, THREADS, 0, st>>>(h, (const float*)A, (const float*)B, o);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head_simt(const HeadDev& h, const void* xc, const void* W, bool keep, cudaStream_t st) {
    const HeadOut o{};
    return keep ? launch<ZKEEP>(h, xc, W, o, h.rows, h.V, st) : launch<Z>(h, xc, W, o, h.rows, h.V, st);
}

cudaError_t launch_head_simt_dx(const HeadDev& h, const void* W, const HeadOut& o, cudaStream_t st) {
    return launch<DX>(h, h.P, W, o, h.rows, h.d, st);
}

cudaError_t launch_head_simt_dw(const HeadDev& h, const void* xc, const HeadOut& o, cudaStream_t st) {
    return launch<DW>(h, h.P, xc, o, h.V, h.d, st);
}

}  // namespace moe
