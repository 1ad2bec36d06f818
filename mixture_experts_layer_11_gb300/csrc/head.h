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
// Exponentials are kept as 2^(z2 - m2 + kHeadShift), z2 the logit in bits, m2 the
// block's largest: at most 2^15, so that fp16 holds 11 bits of each down to 2^-29
// of the block's largest, and 2^-39 of it before it falls to 0.
constexpr float kHeadShift = 15.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The kernels' view of one call, and of the piece of its rows that is being
// worked on.  Row r of a piece is row p0 + r of the live (not ignored) tokens, in
// their order; token live[p0 + r].
struct HeadDev {
    int T, V, d, K;
    int Vp;                  // row length of P (V rounded up to 64)
    int nblk;                // blocks of kHeadBlock entries
    int nstat;               // blocks the statistics are over (nblk, or of the few-row tiles)
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
    float2* stats;           // [nstat][srows]: largest exponent - kHeadShift, sum (0: no entries)
    float* lse2;             // [srows] log2 of the sum of exponentials
    void* P;                 // [rows][Vp]: exponentials, then gradients by the logits
    const float* weight;
    float c;                 // log2(e) / temperature
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

// The three products of a call:
//   Z   exponentials and statistics of xc W^T (KEEP: P is written too)
//   DX  dx = scale * G W
//   DW  dW (+)= scale * G^T xc
struct HeadOut {
    void* out;               // dx [T,d] or dW [V,d]
    int f32;                 // fp32 (else bf16)
    int accumulate;
};
cudaError_t launch_head_simt(const HeadDev& h, const void* xc, const void* W, bool keep, cudaStream_t st);
cudaError_t launch_head_simt_dx(const HeadDev& h, const void* W, const HeadOut& o, cudaStream_t st);
cudaError_t launch_head_simt_dw(const HeadDev& h, const void* xc, const HeadOut& o, cudaStream_t st);

// The same on the tensor cores, bf16 (single: up to 128 rows; xc may be x itself,
// where rows are tokens).  part: the cut tiles' sums.
constexpr int kHeadFewRows = 128;
int head_few_tile(int V);
size_t head_part_bytes(int64_t rows, int V, int d, bool single);
cudaError_t launch_head_tc(const HeadDev& h, const void* xc, const void* W, bool keep, bool single,
                           cudaStream_t st);
cudaError_t launch_head_tc_dx(const HeadDev& h, const void* W, const HeadOut& o, float* part,
                              size_t part_bytes, bool single, cudaStream_t st);
cudaError_t launch_head_tc_dw(const HeadDev& h, const void* xc, const HeadOut& o, float* part,
                              size_t part_bytes, cudaStream_t st);

}  // namespace moe
