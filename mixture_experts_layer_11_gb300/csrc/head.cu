// head.cu -- losses over a vocabulary head: cross entropy and distillation from a
// teacher's top logits, with the gradients of the hidden states and the head.
//
// With z the logits, c = log2(e) / temperature and blocks b of 128 vocabulary entries,
// the first product's epilogue leaves, a row,
//   m_b = max z,  s_b = sum E   and   E = 2^(c (z - m_b) + 15)
// so that, with m = max m_b and S = sum_b s_b 2^(c (m_b - m)),
//   lse = m / temperature + log(S / 2^15),  p = E 2^(c (m_b - m)) / S.  E has 16
// bits (fp16: 11 of precision, 2^-12 at most off), a piece of rows at a time; the
// logits are not kept.  head_gradient_kernel turns E into the gradients
//   G = w (p - q)
// in place, the only rounding to bf16 in front of the other two products, with the
// targets' own entries from their fp32 logits (p - 1 of a token that the model is
// sure of would have none of E's bits).  6 T V d operations; working out the logits
// a second time instead of keeping E would take 8 T V d; E costs 10 bytes of memory
// traffic a logit, of which the pass that turns it into G, 4, does not overlap products
// (5734 rows of 50257 entries: 168 us, against 290 for the logits again at d = 768, and
// 3 % of the call at d = 4096).
//
// Ignored tokens cost nothing: the live rows of x are gathered in front (their
// count stays on the device; grids are made for all tokens, tiles past the count
// end at once), which also keeps what ignored rows hold out of every product.
#include "head.h"

namespace moe {
namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kPieceBytes = int64_t(2) << 30;   // of E, where the caller sets no piece
constexpr int64_t kStatBytes = int64_t(256) << 20;  // of statistics, in a call without gradients
constexpr int64_t kPieceRows = 65536;               // ... and the most rows, for the gathered x
constexpr int64_t kMostPiece = 1 << 20;             // that a caller may ask for

inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

struct Plan {
    int64_t T, piece, pieces, Tp, Vp;
    int nblk, nstat, K, esize;
    // few: losses alone of up to kHeadFewRows rows, none gathered; single: as few rows in
    // bf16; wide: dW is summed in an fp32 buffer of the workspace
    bool few, single, backward, wide;
    size_t ctl, live, pos, xc, sidx, q, lq, ent, start, lz, stats, row, P, dW32, part, part_bytes, total;
};

Plan make_plan(const moe_head& h, const moe_head_grad* g, bool distill) {
    Plan p{};
    p.T = h.T;
    p.esize = h.dtype == MOE_BF16 ? 2 : 4;
    p.K = h.entries;
    p.backward = g != nullptr;
    p.few = !p.backward && h.T <= kHeadFewRows;
    p.single = h.dtype == MOE_BF16 && h.T <= kHeadFewRows;
    p.Vp = up(h.V, 64);
    p.nblk = (h.V + kHeadBlock - 1) / kHeadBlock;
    p.nstat = p.nblk;
    int most_stat = p.nblk;   // a call with more tokens needs no less workspace
    if (!p.backward) {
        const bool bf16 = h.dtype == MOE_BF16;
        const int few = bf16 ? head_few_stats(h.V) : (h.V + 63) / 64;
        if (p.few && (bf16 || h.T <= head_simt_few_rows())) p.nstat = few;
        if (few > most_stat) most_stat = few;
    }
    p.Tp = up(h.T > 0 ? h.T : 1, kHeadRows);
    int64_t most = p.backward ? kPieceBytes / (p.Vp * p.esize) : kStatBytes / (8 * (int64_t)p.nblk);
    if (most > kPieceRows) most = kPieceRows;
    if (p.backward && h.piece > 0) most = h.piece < kMostPiece ? h.piece : kMostPiece;
    // whole tiles: rounded up where asked for, down where the workspace is bounded
    most = p.backward && h.piece > 0 ? up(most, kHeadRows) : most / kHeadRows * kHeadRows;
    if (most < kHeadRows) most = kHeadRows;
    const int64_t piece = most < p.Tp ? most : p.Tp;
    p.piece = piece;
    p.pieces = h.T > 0 ? (h.T + piece - 1) / piece : 0;
    p.wide = p.backward && p.pieces > 1 && g->dW_dtype != MOE_F32;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t a = at;
        at += (bytes + kAlign - 1) / kAlign * kAlign;
        return a;
    };
    const size_t T = (size_t)(h.T > 0 ? h.T : 1), K = (size_t)p.K;
    p.ctl = take(256);
    p.lz = take(T * K * 4);
    p.stats = take((size_t)most_stat * piece * sizeof(float2));
    p.row = take((size_t)piece * sizeof(float4));
    if (distill) {
        p.sidx = take(T * K * 4);
        p.q = take(T * K * 4);
        p.lq = take(T * K * 4);
        p.ent = take(T * 4);
        if (p.K > 1) p.start = take(T * (size_t)p.nblk);
    }
    if (!p.few) {
        p.live = take((size_t)p.Tp * 4);
        p.pos = take((size_t)p.Tp * 4);
        p.xc = take((size_t)piece * h.d * p.esize);
    }
    if (p.backward) {
        p.P = take((size_t)piece * p.Vp * p.esize);
        p.part_bytes = h.dtype == MOE_BF16 ? head_part_bytes(piece, h.V, h.d)
                                           : head_simt_part_bytes(piece, h.V, h.d);
        p.part = take(p.part_bytes);
        if (p.wide) p.dW32 = take((size_t)h.V * h.d * 4);
    }
    p.total = at;
    return p;
}

// ---- a teacher's entries ---------------------------------------------------------
//
// A warp a token: the softmax of the logits that are present, the entries in
// ascending order of their index (absent ones behind), and the first entry of each
// vocabulary block, so that a product's epilogue finds a tile's entries with one
// load.  Bound by the comparisons that rank the entries, K of them each (4096 lists of 64
// over 50257 entries: 15 us).
__global__ void __launch_bounds__(128)
    head_entries_kernel(const HeadDev h, const int64_t* idx, const float* logits, float inv_temp,
                        int* sidx, float* q, float* lq, int* ent, uint8_t* start) {
    __shared__ int key[4][MOE_HEAD_MAX_ENTRIES], sorted[4][MOE_HEAD_MAX_ENTRIES];
    constexpr int N = MOE_HEAD_MAX_ENTRIES / 32;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * 4 + w;
    wait_front();
    if (t >= h.T) return;
    const int64_t at = (int64_t)t * h.K;
    float v[N], top = -INFINITY;
    int k[N];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = i * 32 + lane;
        k[i] = INT_MAX;
        v[i] = -INFINITY;
        if (j < h.K) {
            const int64_t g = idx[at + j];
            bad |= g >= h.V;
            if (g >= 0 && g < h.V && logits[at + j] != -INFINITY) {
                k[i] = (int)g;
                v[i] = logits[at + j];
                // NaN must not be lost in the maximum
                top = isnan(v[i]) || isnan(top) ? NAN : fmaxf(top, v[i]);
            }
        }
        key[w][j] = k[i];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, top, o);
        top = isnan(u) || isnan(top) ? NAN : fmaxf(top, u);
    }
    float sum = 0.f;
    int count = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool has = k[i] != INT_MAX;
        count += has;
        sum += has ? expf((v[i] - top) * inv_temp) : 0.f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
    }
    if (bad) report(h.status, MOE_ERR_INVALID);
    if (lane == 0) ent[t] = count;
    __syncwarp();
    const float lsum = logf(sum);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = i * 32 + lane;
        if (j >= h.K) continue;
        int rank = 0;
        for (int u = 0; u < h.K; ++u) rank += key[w][u] < k[i] || (key[w][u] == k[i] && u < j);
        const bool has = k[i] != INT_MAX;
        const float l = has ? (v[i] - top) * inv_temp - lsum : 0.f;
        sorted[w][rank] = k[i];
        sidx[at + rank] = k[i];
        const float e = has ? expf(l) : 0.f;
        q[at + rank] = e;
        lq[at + rank] = e == 0.f ? 0.f : l;   // l may be -infinity there; NaN stays
    }
    __syncwarp();
    if (h.K == 1) return;
    for (int b = lane; b < h.nblk; b += 32) {
        const int first = b * kHeadBlock;
        int lo = 0, hi = count;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sorted[w][mid] < first) lo = mid + 1;
            else hi = mid;
        }
        start[(int64_t)t * h.nblk + b] = (uint8_t)lo;
    }
}

// ---- live rows ---------------------------------------------------------------------

__device__ __forceinline__ bool token_live(const HeadDev& h, int t) {
    if (!h.target) return h.ent[t] > 0;
    const int64_t y = h.target[t];
    return y >= 0 && y < h.V;
}

// The live tokens' rows.  Up to kScanTokens tokens each block of head_gather_kernel
// counts them all for itself (64 KB of targets from L2 for 8192 tokens: 2 us, against
// a launch of one block that takes 5 us and its gap); more are counted once, by this
// block.
constexpr int kScanTokens = 16384;

__global__ void __launch_bounds__(1024) head_scan_kernel(const HeadDev h, int* pos, int* n_live) {
    __shared__ int part[2][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int base = 0;
    wait_front();
    for (int t0 = 0, it = 0; t0 < h.T; t0 += 1024, ++it) {
        const int t = t0 + threadIdx.x;
        const bool on = t < h.T && token_live(h, t);
        const unsigned mask = __ballot_sync(0xffffffffu, on);
        if (lane == 0) part[it & 1][w] = __popc(mask);
        __syncthreads();
        const int v = part[it & 1][lane];
        const int before = __reduce_add_sync(0xffffffffu, lane < w ? v : 0);
        if (t < h.T) pos[t] = on ? base + before + __popc(mask & ((1u << lane) - 1)) : -1;
        base += __reduce_add_sync(0xffffffffu, v);
    }
    if (threadIdx.x == 0) *n_live = base;
}

// A warp a token: the x of one that is live in this piece goes to its row of xc, an
// ignored one's outputs are zeros (written with the first piece); and row i of xc behind
// the live ones, up to the end of a K block of 64 (of the tensor cores' products, where
// it meets zeros of G), is zeros.  A copy at most (8192 tokens, 5734 live, d = 768: 10 us);
// short calls wait for the counting (256 tokens: 4 us).
template <bool COUNT>
__global__ void __launch_bounds__(1024)
    head_gather_kernel(const HeadDev h, const uint4* x, uint4* xc, uint4* dx, int vecs, int* live, const int* pos,
                       int* n_live) {
    __shared__ int part[2][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = blockIdx.x * 32, t = first + w;
    wait_front();
    const bool on = t < h.T && token_live(h, t);
    int row = -1, n;
    if (COUNT) {
        int before = 0, all = 0;
        for (int i = threadIdx.x; i < h.T; i += 1024) {
            const int v = token_live(h, i);
            all += v;
            before += i < first ? v : 0;
        }
        all = __reduce_add_sync(0xffffffffu, all);
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            part[0][w] = all;
            part[1][w] = before;
        }
        __syncthreads();
        n = __reduce_add_sync(0xffffffffu, part[0][lane]);
        before = __reduce_add_sync(0xffffffffu, part[1][lane]);
        const int i = first + lane;
        const unsigned mask = __ballot_sync(0xffffffffu, i < h.T && token_live(h, i));
        if (on) row = before + __popc(mask & ((1u << w) - 1));
        if (blockIdx.x == 0 && threadIdx.x == 0) *n_live = n;
    } else {
        n = *n_live;
        if (on) row = pos[t];
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (on) {
        const uint4* src = x + (int64_t)t * vecs;
        const int to = row - h.p0;
        uint4* dst = xc + (int64_t)to * vecs;
        int v = to >= 0 && to < h.rows ? lane : vecs;
        for (; v + 96 < vecs; v += 128) {
            const uint4 a = src[v], b = src[v + 32], c = src[v + 64], d = src[v + 96];
            dst[v] = a;
            dst[v + 32] = b;
            dst[v + 64] = c;
            dst[v + 96] = d;
        }
        for (; v < vecs; v += 32) dst[v] = src[v];
        if (lane == 0) live[row] = t;
    } else if (t < h.T && h.p0 == 0) {
        if (lane == 0) {
            if (h.target && h.target[t] >= h.V) report(h.status, MOE_ERR_INVALID);
            h.loss[t] = 0.f;
            if (h.lse) h.lse[t] = 0.f;
        }
        if (dx)
            for (int v = lane; v < vecs; v += 32) dx[(int64_t)t * vecs + v] = zero;
    }
    if (t >= n && t < (n + 63) / 64 * 64 && t >= h.p0 && t < h.p0 + h.rows)
        for (int v = lane; v < vecs; v += 32) xc[(int64_t)(t - h.p0) * vecs + v] = zero;
}

// ---- statistics to losses ----------------------------------------------------------
//
// A block takes 32 rows; lane = row, a warp every 32nd vocabulary block: the loads are
// whole lines, eight of them in flight a warp (5734 rows, 393 blocks: 18 MB in 12 us; one
// row of 304 shares: 4 us, latency).  Then a warp a row joins the shares.
constexpr int kLossLoads = 8;   // in flight a thread
__global__ void __launch_bounds__(1024) head_loss_kernel(const HeadDev h) {
    __shared__ float ms[32][33], ss[32][33];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_front();
    const int n = head_rows(h), r0 = blockIdx.x * 32;
    if (r0 >= n) return;
    float m = -INFINITY, s = 0.f;
    if (r0 + lane < n) {
        const float2* src = h.stats + r0 + lane;
        for (int b = w; b < h.nstat; b += 32 * kLossLoads) {
            float2 v[kLossLoads];
#pragma unroll
            for (int i = 0; i < kLossLoads; ++i)
                v[i] = b + 32 * i < h.nstat ? src[(int64_t)(b + 32 * i) * h.srows] : make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kLossLoads; ++i) {
                if (v[i].y == 0.f) continue;   // no entries
                // (NaN: the comparison fails, and the sum takes it on)
                if (v[i].x > m) {
                    s = s * exp2f((m - v[i].x) * h.c) + v[i].y;
                    m = v[i].x;
                } else {
                    s += v[i].y * exp2f((v[i].x - m) * h.c);
                }
            }
        }
    }
    ms[w][lane] = m;
    ss[w][lane] = s;
    __syncthreads();
    // now lane = warp's share, warp = row
    const int r = r0 + w;
    if (r >= n) return;
    m = ms[lane][w];
    s = ss[lane][w];
    float top = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // (a share without blocks has m = -inf and s = 0)
    s = s == 0.f ? 0.f : s * exp2f((m - top) * h.c);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float sum = s * 0x1p-15f;
    static_assert(kHeadShift == 15.f, "the sums' scale");
    const float lse = fmaf(top, h.per, logf(sum));
    // log2 of the sum over a target's exponential: small where the model is sure of it,
    // and not the difference of two numbers of the logits' size
    auto above = [&](float z) {
        const float d = (z - top) * h.c;
        return fabsf(d) <= 64.f ? log2f(sum * exp2f(-d)) : log2f(sum) - d;
    };
    const int t = head_token(h, r);
    if (!h.n_live && !token_live(h, t)) {
        if (lane == 0) {
            if (h.target && h.target[t] >= h.V) report(h.status, MOE_ERR_INVALID);
            h.loss[t] = 0.f;
            if (h.lse) h.lse[t] = 0.f;
        }
        return;
    }
    const int64_t at = (int64_t)t * h.K;
    const float weight = h.row && h.weight ? h.weight[t] : 1.f;
    float loss = 0.f, g = 0.f;
    int k = -1;
    if (h.target) {
        loss = above(h.lz[at]) * kLn2;
        if (loss < 0.f) loss = 0.f;   // of a certain token, by the sum's rounding; NaN stays
        k = (int)h.target[t];
        g = weight * expm1f(-loss);
    } else {
        const int e = h.ent[t];
        float gs[MOE_HEAD_MAX_ENTRIES / 32];
#pragma unroll
        for (int i = 0; i < MOE_HEAD_MAX_ENTRIES / 32; ++i) {
            const int j = i * 32 + lane;
            if (j >= e) break;
            const float gap = above(h.lz[at + j]);
            float q = h.q[at + j];
            loss += q * (h.lq[at + j] + gap * kLn2);
            if (h.row) {   // an index that is there more than once: its first entry has the sum of all
                const int me = h.sidx[at + j];
                for (int u = j + 1; u < e && h.sidx[at + u] == me; ++u) q += h.q[at + u];
                gs[i] = weight * (exp2f(-gap) - q);
            }
        }
        if (h.row) {   // the entries' values of G, in place of their logits
#pragma unroll
            for (int i = 0; i < MOE_HEAD_MAX_ENTRIES / 32; ++i)
                if (i * 32 + lane < e) h.lz[at + i * 32 + lane] = gs[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
        loss *= h.loss_scale;
    }
    if (lane == 0) {
        if (!isfinite(loss) || !isfinite(lse)) report(h.status, MOE_ERR_NONFINITE);
        h.loss[t] = loss;
        if (h.lse) h.lse[t] = lse;
        if (h.row) h.row[r] = make_float4(top, weight / s, __int_as_float(k), g);
    }
}

// ---- exponentials to gradients, in place ------------------------------------------------

template <typename T> struct Pair;   // T: the gradients' type
template <> struct Pair<__nv_bfloat16> {
    static constexpr int N = 8;      // values of 16 bytes
    static __device__ __forceinline__ uint4 scale(uint4 u, float f, int left) {
        __half2* e = reinterpret_cast<__half2*>(&u);
        uint4 out;
        __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(&out);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(e[i]);
            o[i] = __floats2bfloat162_rn(2 * i < left ? v.x * f : 0.f, 2 * i + 1 < left ? v.y * f : 0.f);
        }
        return out;
    }
};
template <> struct Pair<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ uint4 scale(uint4 u, float f, int left) {
        return make_uint4(left > 0 ? __float_as_uint(__uint_as_float(u.x) * f) : 0u,
                          left > 1 ? __float_as_uint(__uint_as_float(u.y) * f) : 0u,
                          left > 2 ? __float_as_uint(__uint_as_float(u.z) * f) : 0u,
                          left > 3 ? __float_as_uint(__uint_as_float(u.w) * f) : 0u);
    }
};

// A warp takes kGradCols columns of a row, eight loads of 16 bytes a lane in flight.
// HBM bounds: 1.15 GB moved in 168 us (5734 rows of 50257 entries), 2.15 GB in 305 us
// (4096 of 131072), 7 TB/s with what L2 still holds; 256 rows of 1000 entries 5 us.
constexpr int kGradWarps = 8, kGradCols = 2048;

template <typename T>
__global__ void __launch_bounds__(32 * kGradWarps)
    head_gradient_kernel(const __grid_constant__ HeadDev h, const __grid_constant__ SplitRule rule) {
    constexpr int N = Pair<T>::N, LOADS = 8, PART = 32 * N * LOADS;   // columns of 8 loads
    wait_front();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x < 32) make_splits(h, rule);   // for the products that come next
    const int n = head_rows(h), nck = (h.Vp + kGradCols - 1) / kGradCols;
    const int64_t it = (int64_t)blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    // the last rows first: L2 still holds some of them
    const int r = (n + 63) / 64 * 64 - 1 - (int)(it / nck), c0 = (int)(it % nck) * kGradCols;
    if (r < 0) return;
    const bool on = r < n;   // else a row of the last K block, behind the live ones: zeros
    T* row = (T*)h.P + (int64_t)r * h.Vp;
    float4 info = make_float4(0.f, 0.f, 0.f, 0.f);
    int a = 0, b = 0;
    int64_t at = 0;
    if (on) info = h.row[r];
    if (on && !h.target) {   // the entries in these columns
        const int t = head_token(h, r);
        at = (int64_t)t * h.K;
        b = h.ent[t];
        if (h.start) {
            const uint8_t* st = h.start + (int64_t)t * h.nblk;
            a = st[c0 / kHeadBlock];
            if (c0 + kGradCols < h.V) b = st[(c0 + kGradCols) / kHeadBlock];
        }
    }
#pragma unroll 1
    for (int c1 = c0; c1 < c0 + kGradCols; c1 += PART) {
        uint4 v[LOADS];
        float m[LOADS];
        const int c = c1 + lane * N;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            m[i] = 0.f;
            if (on && c + i * 32 * N < h.Vp) {
                v[i] = *reinterpret_cast<const uint4*>(row + c + i * 32 * N);
                m[i] = h.stats[(int64_t)((c + i * 32 * N) / kHeadBlock) * h.srows + r].x;
            }
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (c + i * 32 * N < h.Vp)
                *reinterpret_cast<uint4*>(row + c + i * 32 * N) =
                    Pair<T>::scale(v[i], info.y * exp2f((m[i] - info.x) * h.c), h.V - c - i * 32 * N);
    }
    __syncwarp();
    // the targets' own values
    if (h.target) {
        const int k = __float_as_int(info.z);
        if (on && lane == 0 && k >= c0 && k < c0 + kGradCols) row[k] = from_f32<T>(info.w);
    } else {
        for (int j = a + lane; j < b; j += 32) {
            const int k = h.sidx[at + j];
            const bool first = j == 0 || h.sidx[at + j - 1] != k;   // of the same index
            if (first && k >= c0 && k < c0 + kGradCols) row[k] = from_f32<T>(h.lz[at + j]);
        }
    }
}

// dW of several rounds, summed in fp32, to bf16: a copy.
__global__ void __launch_bounds__(256) head_round_kernel(const float4* in, uint2* out, int64_t n4) {
    wait_front();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
        const float4 v = in[i];
        __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        out[i] = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
    }
}

}  // namespace

// What is made for a call with gradients is used by ones without them too (an object's
// scores): these take other rounds, and gather up to kPieceRows rows whatever the piece.
size_t head_workspace(const moe_head& h, const moe_head_grad* g) {
    const size_t with = make_plan(h, g, true).total, alone = make_plan(h, nullptr, true).total;
    return with > alone ? with : alone;
}

cudaError_t launch_head(const HeadCall& c, cudaStream_t st) {
    const moe_head& s = c.h;
    const bool bf16 = s.dtype == MOE_BF16;
    const bool distill = c.teacher != nullptr;
    const moe_head_grad* g = c.g;
    const bool want_dx = g && g->dx, want_dW = g && g->dW;
    if (s.T == 0) {
        if (want_dW && !g->accumulate)
            return cudaMemsetAsync(g->dW, 0, (size_t)s.V * s.d * (g->dW_dtype == MOE_F32 ? 4 : 2), st);
        return cudaSuccess;
    }
    const Plan p = make_plan(s, g, distill);
    uint8_t* ws = (uint8_t*)c.ws;
    HeadDev h{};
    h.T = (int)s.T;
    h.V = s.V;
    h.d = s.d;
    h.K = s.entries;
    h.Vp = (int)p.Vp;
    h.nblk = p.nblk;
    h.nstat = p.nstat;
    h.rows = (int)p.piece;
    h.srows = (int)p.piece;
    if (!p.few) {
        h.n_live = (const int*)(ws + p.ctl);
        h.live = (const int*)(ws + p.live);
    }
    if (distill) {
        h.sidx = (const int*)(ws + p.sidx);
        h.q = (const float*)(ws + p.q);
        h.lq = (const float*)(ws + p.lq);
        h.ent = (const int*)(ws + p.ent);
        h.start = p.K > 1 ? ws + p.start : nullptr;
    } else {
        h.target = c.idx;
    }
    h.lz = (float*)(ws + p.lz);
    h.stats = (float2*)(ws + p.stats);
    if (g) h.row = (float4*)(ws + p.row);
    h.P = ws + p.P;
    h.splits = (Split*)(ws + p.ctl + 64);
    h.c = kLog2e / c.temperature;
    h.per = 1.f / c.temperature;
    h.loss_scale = c.temperature * c.temperature;
    if (g) {
        h.weight = g->weight;
        h.grad_scale = g->scale * c.temperature;
        h.mean = g->mean;
    }
    h.loss = c.loss;
    h.lse = c.lse;
    h.status = c.status;

    cudaError_t e = cudaSuccess;
    if (distill)
        e = launch_early(head_entries_kernel, dim3((unsigned)((s.T + 3) / 4)), 128, 0, 1, st, h, c.idx, c.teacher,
                         1.f / c.temperature, (int*)(ws + p.sidx), (float*)(ws + p.q), (float*)(ws + p.lq),
                         (int*)(ws + p.ent), ws + p.start);
    const void* xc = p.few ? c.x : ws + p.xc;
    float* part = (float*)(ws + p.part);
    int *live = (int*)(ws + p.live), *pos = (int*)(ws + p.pos), *n_live = (int*)(ws + p.ctl);
    const bool count = s.T <= kScanTokens;
    if (e == cudaSuccess && !p.few && !count)
        e = launch_early(head_scan_kernel, dim3(1), 1024, 0, 1, st, h, pos, n_live);
    for (int64_t i = 0; i < p.pieces && e == cudaSuccess; ++i) {
        h.p0 = (int)(i * p.piece);
        const int64_t left = p.Tp - h.p0;
        h.rows = (int)(left < p.piece ? left : p.piece);
        if (!p.few)
            e = launch_early(count ? head_gather_kernel<true> : head_gather_kernel<false>, dim3((unsigned)(p.Tp / 32)),
                             1024, 0, 1, st, h, (const uint4*)c.x, (uint4*)(ws + p.xc),
                             want_dx ? (uint4*)g->dx : (uint4*)nullptr, s.d * p.esize / 16, live, (const int*)pos,
                             n_live);
        if (e != cudaSuccess) break;
        e = bf16 ? launch_head_tc(h, xc, c.W, p.backward, p.single, st)
                 : launch_head_simt(h, xc, c.W, p.backward, st);
        if (e != cudaSuccess) break;
        // rows that there may be: no more than tokens
        const int64_t rows = s.T - h.p0 < h.rows ? s.T - h.p0 : h.rows;
        e = launch_early(head_loss_kernel, dim3((unsigned)((rows + 31) / 32)), 1024, 0, 1, st, h);
        if (!p.backward || e != cudaSuccess) continue;
        if (!want_dx && !want_dW) continue;
        const HeadOut dx{want_dx ? g->dx : nullptr, !bf16, 0};
        const HeadOut dW{want_dW ? p.wide ? (void*)(ws + p.dW32) : g->dW : nullptr,
                         p.wide || g->dW_dtype == MOE_F32, g->accumulate || i > 0};
        SplitRule rule;
        if (bf16) e = head_tc_rule(p.piece, s.V, s.d, &rule);
        else rule = head_simt_rule(p.piece, s.V, s.d);
        if (e != cudaSuccess) break;
        rule.dx = want_dx;
        rule.dw = want_dW;
        rule.accumulate = dW.accumulate;
        const int64_t items = up(rows, 64) * (up(p.Vp, kGradCols) / kGradCols);
        e = launch_early(bf16 ? head_gradient_kernel<__nv_bfloat16> : head_gradient_kernel<float>,
                         dim3((unsigned)((items + kGradWarps - 1) / kGradWarps)), 32 * kGradWarps, 0, 1, st, h, rule);
        if (e != cudaSuccess) break;
        e = bf16 ? launch_head_tc_grad(h, xc, c.W, dx, dW, part, rule, st)
                 : launch_head_simt_grad(h, xc, c.W, dx, dW, part, rule, st);
    }
    if (e == cudaSuccess && want_dW && p.wide) {
        const int64_t n4 = (int64_t)s.V * s.d / 4;
        const int64_t blocks = (n4 + 255) / 256;
        e = launch_early(head_round_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), 256, 0, 1, st,
                         (const float4*)(ws + p.dW32), (uint2*)g->dW, n4);
    }
    return e;
}

}  // namespace moe
