// head.h -- what the kernels of the losses over a vocabulary head share (internal
// to libmoe.so; the public interface is include/moe.h).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

// Softmax statistics are taken over blocks of this many vocabulary entries: each
// row's maximum and the sum of its exponentials.
constexpr int kHeadBlock = 128;
// Rows of the compacted hidden states and of the probabilities are padded to this.
constexpr int kHeadRows = 256;
// Exponentials are kept as 2^(c (z - m) + kHeadShift), z the logit, m the block's
// largest, c = log2(e) / temperature: at most 2^15, so that fp16 holds 11 bits of each
// down to 2^-29 of the block's largest, and 2^-39 of it before it falls to 0.  The
// differences come first, of logits and not of logits times c: what is between two logits
// of any size has the bits of the difference (from one fused c z - m, with lse as one
// number, p is 3e-4 of itself off where the logits reach 1e4 bits, and infinite from 2^24).
constexpr float kHeadShift = 15.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How the tiles of a reduction over kb blocks of 64 run on `units` CTAs (or pairs, or
// blocks at once): tiles before `full` whole, the uneven last wave behind them (or
// all, where there are few) in `parts` parts of kbp blocks, whose sums a second
// launch joins in order.  Costs, in a block's time: a part's blocks and `each` more
// (its start and end), and for cutting `once`, the joining launch, with a block for
// `bytes` parts written and read.  Parts have at least `least` blocks.  Called by a
// whole warp.
struct Split { int tiles, full, parts, kbp; };
constexpr int kMostParts = 64;
__device__ __forceinline__ Split split_tiles(int tiles, int kb, int units, int cap, int least, int each,
                                             int once, int bytes) {
    Split s{tiles, tiles, 1, kb};
    const int rem = tiles % units, lane = threadIdx.x & 31;
    if (rem == 0 || kb < 2 * least) return s;
    unsigned best = 0xffffffffu;
    for (int P = lane + 1; P <= kMostParts; P += 32) {
        if (P > 1 && (P * least > kb || rem * P > cap)) continue;
        const int kbp = (kb + P - 1) / P, parts = (kb + kbp - 1) / kbp;
        unsigned cost = (unsigned)((rem * parts + units - 1) / units * (kbp + each));
        if (parts > 1) cost += (unsigned)(once + rem * parts / bytes);
        const unsigned key = (cost < (1u << 24) ? cost : (1u << 24) - 1) << 8 | (unsigned)P;
        best = key < best ? key : best;
    }
    best = __reduce_min_sync(0xffffffffu, best);
    const int P = (int)(best & 255u);
    if (P > 1) {
        s.full = tiles - rem;
        s.kbp = (kb + P - 1) / P;
        s.parts = (kb + s.kbp - 1) / s.kbp;
    }
    return s;
}
// What the two products of a call need for that: tiles of tm x tn, reductions counted
// in blocks of 64.
struct SplitRule {
    int tm, tn, units, capx, capw, least, each, once, bytes;
    int dx, dw, accumulate;   // wanted; dW added to
};

// The kernels' view of one call, and of the piece of its rows that is being
// worked on.  Row r of a piece is row p0 + r of the live (not ignored) tokens, in
// their order; token live[p0 + r].
struct HeadDev {
    int T, V, d, K;
    int Vp;                  // row length of P (V rounded up to 64)
    int nblk;                // blocks of kHeadBlock entries
    int nstat;               // rows of stats: nblk, or for few rows two a CTA (fp32: tiles of 64)
    int p0, rows;            // first live row of the piece, its most rows
    int srows;               // row length of stats (rows, rounded up to kHeadRows)
    const int* n_live;       // null: rows are tokens, all T of them
    const int* live;
    const int64_t* target;   // targets [T], or null:
    const int* sidx;         // the teacher's indices, ascending [T][K] ...
    const float* q;          // ... their weights, and the logarithms of these
    const float* lq;
    const int* ent;          // entries present [T]
    const uint8_t* start;    // first entry of each block [T][nblk]
    float* lz;               // logits of the targets / entries [T][K]
    float2* stats;           // [nstat][srows]: largest logit, sum of exponentials (0: no entries)
    float4* row;             // [srows], with gradients: largest logit, weight over the sum of
                             // exponentials, and the target with its value of G (CE)
    Split* splits;           // DX's, DW's (head_gradient_kernel works them out)
    void* P;                 // [rows][Vp]: exponentials, then gradients by the logits
    const float* weight;
    float c;                 // log2(e) / temperature
    float per;               // 1 / temperature
    float loss_scale;        // temperature^2
    float grad_scale;        // scale * temperature
    int mean;
    float* loss;
    float* lse;
    int32_t* status;
};

__device__ __forceinline__ int head_live(const HeadDev& h) { return h.n_live ? *h.n_live : h.T; }
__device__ __forceinline__ int head_rows(const HeadDev& h) {
    const int n = head_live(h) - h.p0;
    return n < 0 ? 0 : n < h.rows ? n : h.rows;
}
__device__ __forceinline__ int head_token(const HeadDev& h, int r) {
    return h.live ? h.live[h.p0 + r] : h.p0 + r;
}
__device__ __forceinline__ float head_scale(const HeadDev& h) {
    if (!h.mean) return h.grad_scale;
    const int n = head_live(h);
    return h.grad_scale / (float)(n > 0 ? n : 1);
}

// The most parts that the workspace holds: four waves, and no more than split_tiles
// can ask for.  No less for more tiles or blocks.
inline size_t split_bound(int64_t tiles, int64_t kb, int units, int least) {
    if (kb < 2 * least) return 0;
    const int64_t rem = tiles < units ? tiles : units, most = kb / least < kMostParts ? kb / least : kMostParts;
    return (size_t)(rem * most < 4 * (int64_t)units ? rem * most : 4 * (int64_t)units);
}

// The sums of `parts` rows of N values, `stride` values apart, for kJoinRows
// neighbouring rows at once, by a block of 256 threads: in 1024 / N groups of threads,
// each every so manieth part, then the groups in order.  Returns the first column of
// the calling thread's four sums a row, or -1 in the threads that have none.  rows: of
// the kJoinRows that exist.
constexpr int kJoinRows = 4;
template <int N>
__device__ __forceinline__ int join_rows(const float* src, int64_t stride, int parts, int rows,
                                         float4 (*buf)[256], float4 (&s)[kJoinRows]) {
    constexpr int Q = N / 4, G = 256 / Q;
    const int q = threadIdx.x % Q, g = threadIdx.x / Q;
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = g; k < parts; k += G) {
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
            if (r >= rows) break;
            const float4 v = *reinterpret_cast<const float4*>(src + k * stride + r * N + q * 4);
            s[r].x += v.x;
            s[r].y += v.y;
            s[r].z += v.z;
            s[r].w += v.w;
        }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) buf[r][threadIdx.x] = s[r];
    __syncthreads();
    if (g) return -1;
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r)
#pragma unroll
        for (int i = 1; i < G; ++i) {
            const float4 v = buf[r][i * Q + q];
            s[r].x += v.x;
            s[r].y += v.y;
            s[r].z += v.z;
            s[r].w += v.w;
        }
    return q * 4;
}

// (a whole warp)
__device__ __forceinline__ void make_splits(const HeadDev& h, const SplitRule& p) {
    const int n = head_rows(h), NT = (h.d + p.tn - 1) / p.tn;
    const int kx = (h.V + 63) / 64, kw = (n + 63) / 64, tw = (h.V + p.tm - 1) / p.tm * NT;
    Split x{0, 0, 1, kx}, w{0, 0, 1, kw};
    if (p.dx) x = split_tiles((n + p.tm - 1) / p.tm * NT, kx, p.units, p.capx, p.least, p.each, p.once, p.bytes);
    if (p.dw && n > 0) w = split_tiles(tw, kw, p.units, p.capw, p.least, p.each, p.once, p.bytes);
    else if (p.dw && !p.accumulate) w = Split{tw, tw, 1, 0};   // no rows: zeros
    if ((threadIdx.x & 31) == 0) {
        h.splits[0] = x;
        h.splits[1] = w;
    }
}

// Kernels here begin while the one in front of them ends: nothing is touched before
// wait_front(), and nothing is read through the non-coherent path.
__device__ __forceinline__ void wait_front() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... A, typename... B>
cudaError_t launch_early(void (*kern)(A...), dim3 grid, int block, size_t smem, int cluster, cudaStream_t st,
                         const B&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The three products of a call:
//   Z   exponentials and statistics of xc W^T (KEEP: P is written too)
//   DX  dx = scale * G W
//   DW  dW (+)= scale * G^T xc
// part: room for the sums of cut tiles.
struct HeadOut {
    void* out;               // dx [T,d] or dW [V,d]; null: not wanted
    int f32;                 // fp32 (else bf16)
    int accumulate;
};
cudaError_t launch_head_simt(const HeadDev& h, const void* xc, const void* W, bool keep, cudaStream_t st);
cudaError_t launch_head_simt_grad(const HeadDev& h, const void* xc, const void* W, const HeadOut& dx,
                                  const HeadOut& dW, float* part, const SplitRule& rule, cudaStream_t st);
SplitRule head_simt_rule(int64_t rows, int V, int d);
size_t head_simt_part_bytes(int64_t rows, int V, int d);
int head_simt_few_rows();

// The same on the tensor cores, bf16 (single: up to 128 rows; xc may be x itself,
// where rows are tokens).  rows of a rule: those that head_part_bytes was asked for.
constexpr int kHeadFewRows = 128;
int head_few_tile(int V);
int head_few_stats(int V);   // rows of statistics of a few-row call
size_t head_part_bytes(int64_t rows, int V, int d);
cudaError_t launch_head_tc(const HeadDev& h, const void* xc, const void* W, bool keep, bool single,
                           cudaStream_t st);
cudaError_t launch_head_tc_grad(const HeadDev& h, const void* xc, const void* W, const HeadOut& dx,
                                const HeadOut& dW, float* part, const SplitRule& rule, cudaStream_t st);
cudaError_t head_tc_rule(int64_t rows, int V, int d, SplitRule* rule);

}  // namespace moe
