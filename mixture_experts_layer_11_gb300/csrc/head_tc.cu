// head_tc.cu -- the three products of the losses over a vocabulary head in bf16 on
// the tensor cores (tcgen05.mma, fp32 accumulators in TMEM, operands by TMA).
//
//   Z, ZKEEP  tiles of xc W^T whose epilogue leaves a row's largest logit and sum of
//             exponentials a 128 columns, its targets' logits and (ZKEEP) the
//             exponentials as fp16
//   GRAD      dx = scale G W (DX: a reduction over the vocabulary) and
//             dW (+)= scale G^T xc (DW: over the live rows), one launch for both
//
// CTA = 10 warps: warp 0 issues the TMA loads into a ring of stages of 64 K values,
// one thread of warp 1 the MMAs into one of two TMEM accumulators of 256 columns,
// eight warps drain the other one: warp w the lanes of quarter w % 4 and 128
// columns.  PAIR: clusters of two CTAs, tiles of 256 x 256 (cta_group::2, each CTA
// holds its 128 rows of A and 128 columns of B, 32 KB a stage, six stages); else
// one CTA, 128 rows (48 KB, four stages), for Z of calls of up to 128 tokens, where
// W's bytes bound and half a pair's rows would be empty.
//
// A persistent grid walks the tiles.  What is left of a product's last, uneven wave
// (or everything, with few tiles) is cut along the reduction into parts whose sums go
// to the workspace in fp32 and are added in order by head_join_kernel.  The number
// of live tokens, and with it tiles and parts, is read on the device.
//
// What bounds, and times: the tensor pipe in DX and DW (94 and 90 % busy; 5734 rows of
// 50257 entries, d = 768: 241 and 251 us, 1800 TFLOP/s) and in Z with long rows (8191
// rows, d = 2048, no exponentials kept: 1230 us, 1790 TFLOP/s; the power cap sets the
// clock).  ZKEEP at d = 768 takes 287 us, about 71 % busy: the exponentials' way out through
// shared memory meets the MMAs' operands there (without it 248), and taking a block's
// largest logit off before the temperature costs 6 of the 287.  Up to 128 tokens W's
// bytes bound: 13 tokens of 131072 entries, d = 4096, 164 us, 6.5 TB/s; one token of
// 50257, d = 768, 17 us, half of it before the first and after the last load.
//
// Every wait is bounded; on expiry the CTA records MOE_ERR_TIMEOUT, waits for its
// copies and MMAs in flight, frees TMEM and exits.
#include <cudaTypedefs.h>
#include <stdio.h>
#include <stdlib.h>

#include <mutex>

#include "head.h"

namespace moe {
namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int SLAB = 64 * BK * 2;            // 64 columns of BK rows, MN-major
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (2 + EPI_WARPS);
constexpr int BOX = 32 * 128;                // an epilogue warp's staged box: 32 rows of 128 bytes
constexpr int TMEM_COLS = 512;
// Z's sums leave TMEM in chunks of K blocks and are added in registers, rounded to
// nearest.  The tensor cores drop what is below the accumulator's last bit, which in one
// chain over d = 4096 moves a logit by 4e-6 of itself towards zero.
//   up to 128 rows  every kChunk blocks (256 products): the loss of a lone token that the
//             model is sure of shows it (1.2e-6 of a loss of 0.36 in place of 4e-5), and
//             W's bytes bound (13 tokens of 131072 entries, d = 4096: 167 -> 171 us)
//   more      rows longer than kWhole blocks in about equal chunks of 13 to 20: losses
//             are off by 5e-7 of their norm in place of 2e-6 at d = 4096 and 1.1e-6 at
//             2048 (8191 rows of 65536 entries, d = 2048: 1237 -> 1248 us; 16384 of
//             32768, d = 4096: 2551 -> 2601).  Chunks of 8 blocks took 5 to 10 % longer:
//             the MMAs of two have to cover an epilogue.  Shorter rows stay whole (8.5e-7
//             at d = 1536).
constexpr int kChunk = 4, kWhole = 24;
__device__ __forceinline__ int z_chunk(int kb) {
    const int n = kb <= kWhole ? 1 : (kb + 7) / 16;
    return (kb + n - 1) / n;
}
// Row tiles that follow each other on one column tile's operand, as a power of two: DX's 8;
// Z's as many as keep their rows of x, 512 d bytes a tile, within 32 MB of the second-level
// cache.  Losses of 8191 rows of 65536 entries, d = 2048: 1234 us by 32, 1253 by 16; of
// 16384 rows of 32768 entries, d = 4096: 2645 us by 32, 2523 by 16, 2657 by 8; of 16384
// entries, d = 8192: 2834 us by 16, 2783 by 8.
constexpr int DX_SHIFT = 3;
__device__ __forceinline__ int z_shift(int d) { return d <= 2048 ? 5 : d <= 4096 ? 4 : 3; }

enum Mode { Z = 0, ZKEEP = 1, GRAD = 2, DX = 3, DW = 4 };   // GRAD: both of the others

template <bool PAIR> struct Shape {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TILE_M = BM * CTAS;
    static constexpr int BN_CTA = BN / CTAS;
    static constexpr int A_BYTES = BM * BK * 2;
    static constexpr int B_BYTES = BN_CTA * BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = PAIR ? 6 : 4;
};

// Quotients by one divisor, without the hundreds of cycles of a division: they are
// worked out by one thread or warp between two tiles.
struct Quotient {
    unsigned d, m;   // divisor, floor(2^32 / d) (2^32 - 1 for 1)
    __device__ __forceinline__ void set(int by) {
        d = (unsigned)(by > 0 ? by : 1);
        m = d == 1 ? 0xffffffffu : (unsigned)(0x100000000ull / d);
    }
    __device__ __forceinline__ int of(int n, int& rest) const {
        unsigned q = __umulhi((unsigned)n, m), r = (unsigned)n - q * d;
        // at most two too small
        if (r >= d) ++q, r -= d;
        if (r >= d) ++q, r -= d;
        rest = (int)r;
        return (int)q;
    }
};

// A product's tiles, their split, K blocks and units.
struct Product {
    Split s;
    int MT, NT, kb, shift, chunk;
    Quotient group, rest;   // of tiles; of cut ones
    __device__ __forceinline__ int units() const { return s.full + (s.tiles - s.full) * s.parts; }
};
struct Plan { Product x, w; };   // Z's or DX's; DW's

template <bool B> struct Flag { static constexpr bool value = B; };

template <int STAGES> struct Ctrl {
    uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    Plan plan;
};

template <bool PAIR> constexpr size_t smem_bytes() {
    using S = Shape<PAIR>;
    return 1024 + (size_t)S::STAGES * S::STAGE + EPI_WARPS * BOX + sizeof(Ctrl<S::STAGES>);
}

struct TcParams {
    HeadDev h;
    int tile_n;              // columns of a tile (Z, single CTAs: any multiple of 16; else 256)
    int a_rows;              // rows of A's box
    int few;                 // losses alone of up to 128 rows: running statistics a CTA
    HeadOut dx, dW;          // out null: not wanted
    float* part;             // [capx + capw][256][BN] sums of cut tiles, DX's first
    int capx;
    int units;               // pairs of GRAD's launches
    uint64_t limit_ns;
    int withhold_unit, withhold_kb;   // test hook: see launch_tc
};

template <int MODE, bool PAIR> __device__ __forceinline__ Plan make_plan(const TcParams& p) {
    constexpr int TM = Shape<PAIR>::TILE_M;
    const HeadDev& h = p.h;
    const int n = head_rows(h);
    Plan q{};
    q.x.MT = (n + TM - 1) / TM;
    if (MODE <= ZKEEP) {
        q.x.NT = (h.V + p.tile_n - 1) / p.tile_n;
        q.x.kb = (h.d + BK - 1) / BK;
        q.x.s = Split{q.x.MT * q.x.NT, q.x.MT * q.x.NT, 1, q.x.kb};
        q.x.shift = z_shift(h.d);
        q.x.chunk = PAIR ? z_chunk(q.x.kb) : kChunk;
        q.x.group.set(q.x.NT << q.x.shift);
        return q;
    }
    q.x.NT = q.w.NT = (h.d + BN - 1) / BN;
    q.x.kb = (h.V + BK - 1) / BK;
    q.w.MT = (h.V + TM - 1) / TM;
    q.w.kb = (n + BK - 1) / BK;
    q.x.s = q.w.s = Split{0, 0, 1, 0};
    if (p.dx.out) q.x.s = h.splits[0];
    if (p.dW.out) q.w.s = h.splits[1];
    q.x.shift = DX_SHIFT;
    q.x.group.set(q.x.NT << DX_SHIFT);
    q.w.group.set(q.w.NT);
    q.x.rest.set(q.x.s.tiles - q.x.s.full);
    q.w.rest.set(q.w.s.tiles - q.w.s.full);
    return q;
}

struct Tile { int mt, nt, kb0, nkb, slot; bool dw; };   // slot: of a part, else -1

// Where tile i of a product lies: 2^shift row tiles share a column tile's operand; DW's
// columns follow each other (they share G's).
template <bool DWS> __device__ __forceinline__ void place(const Product& a, int i, Tile& t) {
    if (DWS) {
        t.mt = a.group.of(i, t.nt);
        return;
    }
    int l;
    const int g = a.group.of(i, l), first = g << a.shift, gm = min(1 << a.shift, a.MT - first);
    if (gm == 1 << a.shift) {
        t.mt = first + (l & (gm - 1));
        t.nt = l >> a.shift;
    } else {
        t.mt = first + l % gm;
        t.nt = l / gm;
    }
}

template <bool DWS> __device__ __forceinline__ Tile product_tile(const Product& a, int u, int slot0) {
    Tile t;
    t.kb0 = 0;
    t.nkb = a.kb;
    t.slot = -1;
    int i = u;
    if (u >= a.s.full && a.s.parts > 1) {
        // part after part: the parts of the same K range run at the same time
        int left;
        const int part = a.rest.of(u - a.s.full, left);
        i = a.s.full + left;
        t.kb0 = part * a.s.kbp;
        t.nkb = min(a.s.kbp, a.kb - t.kb0);
        t.slot = slot0 + left * a.s.parts + part;
    }
    place<DWS>(a, i, t);
    return t;
}
template <int MODE> __device__ __forceinline__ Tile get_tile(const Plan& q, const TcParams& p, int u) {
    Tile t;
    if (MODE <= ZKEEP) {
        t = product_tile<false>(q.x, u, 0);
        t.dw = false;
        return t;
    }
    const int ux = MODE == DW ? 0 : q.x.units();
    t.dw = MODE == DW || (MODE == GRAD && u >= ux);
    const bool dw = t.dw;
    t = dw ? product_tile<true>(q.w, u - ux, p.capx) : product_tile<false>(q.x, u, 0);
    t.dw = dw;
    return t;
}

template <typename C> __device__ __forceinline__ void raise_abort(C& c, const TcParams& p) {
    *(volatile int*)&c.abort_flag = 1;
    report(p.h.status, MOE_ERR_TIMEOUT);
}

// ---- pairs of CTAs ---------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t mapa(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_cluster(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// a load that completes on the even CTA's barrier
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                              int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(map), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
template <bool PAIR> __device__ __forceinline__ void tm_alloc(uint32_t dst) {
    if (!PAIR) {
        tmem_alloc(dst, TMEM_COLS);
        tmem_relinquish();
        return;
    }
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <bool PAIR> __device__ __forceinline__ void tm_free(uint32_t base) {
    if (!PAIR) tmem_dealloc(base, TMEM_COLS);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(TMEM_COLS)
                     : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (!PAIR) {
        tc_mma_bf16(d, a, b, idesc, accumulate);
        return;
    }
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
// arrive, in both CTAs of a pair, when every MMA issued so far is done
template <bool PAIR> __device__ __forceinline__ void commit(uint32_t bar) {
    if (!PAIR) {
        tc_commit(bar);
        return;
    }
    const uint16_t both = 3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(both)
        : "memory");
}
template <bool PAIR> __device__ __forceinline__ void commit_local(uint32_t bar) {
    if (!PAIR) tc_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void add_box(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Loads 32 columns of the thread's TMEM lane; the values are there after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// (the values go through, so that none is used before)
__device__ __forceinline__ void tmem_ld_wait(float (&v)[4][32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 32; ++j) asm volatile("" : "+f"(v[i][j]));
}

// 16-byte chunk j of row r of a staged box (the TMA's 128-byte swizzle)
__device__ __forceinline__ uint32_t box_at(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t bf2_bits(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// CUT (Z, ZKEEP): a tile's sums leave TMEM every plan.x.chunk K blocks
template <int MODE, bool PAIR, bool CUT>
__global__ void __launch_bounds__(THREADS, 1)
    head_tc_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                   const __grid_constant__ CUtensorMap mapC, const __grid_constant__ CUtensorMap mapD,
                   const __grid_constant__ CUtensorMap mapO, const __grid_constant__ TcParams p) {
    // Z: A xc, B W, O P.  GRAD: A G, B W (DX); C G, D xc, O dW (DW).
    using S = Shape<PAIR>;
    constexpr int STAGES = S::STAGES;
    auto is_dw = [](const Tile& t) { return MODE == DW || (MODE == GRAD && t.dw); };
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* boxes = base + STAGES * S::STAGE;
    Ctrl<STAGES>& c = *reinterpret_cast<Ctrl<STAGES>*>(boxes + EPI_WARPS * BOX);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    const bool leader = rank == 0;
    const int unit0 = blockIdx.x / S::CTAS, nunits = gridDim.x / S::CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&c.full[s]), S::CTAS);   // each CTA's producer (used in the even one)
            mbar_init(smem_u32(&c.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&c.tfull[b]), 1);
            mbar_init(smem_u32(&c.tempty[b]), EPI_WARPS * S::CTAS);
        }
        mbar_init(smem_u32(&c.drain), 1);
        c.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tm_alloc<PAIR>(smem_u32(&c.tmem_base));
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&mapA);
        tma_prefetch_map(&mapB);
    }
    wait_front();
    if (threadIdx.x == 64) c.plan = make_plan<MODE, PAIR>(p);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = c.tmem_base;
    const Plan& plan = c.plan;
    const int units = plan.x.units() + plan.w.units(), chunk = plan.x.chunk;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued[STAGES];
            uint32_t phase = 0;
            bool ok = true;
            for (int s = 0; s < STAGES; ++s) issued[s] = -1;
            // the stages' bytes: whole boxes, also where they lie past an edge
            const uint32_t bytes = MODE >= GRAD || PAIR ? (uint32_t)S::STAGE
                                                        : (uint32_t)((p.a_rows + p.tile_n) * BK * 2);
            for (int u = unit0; u < units && ok; u += nunits) {
                const Tile t = get_tile<MODE>(plan, p, u);
                const int m0 = t.mt * S::TILE_M + rank * BM;
                const int n0 = t.nt * p.tile_n + rank * S::BN_CTA;
                auto fill = [&](auto dw) {
                    constexpr bool DWT = decltype(dw)::value;
                    for (int k = 0; k < t.nkb; ++k) {
                        const int k0 = (t.kb0 + k) * BK;
                        if (leader && u == p.withhold_unit && k == p.withhold_kb) return false;
                        if (!mbar_wait_bounded(smem_u32(&c.empty[stage]), phase ^ 1, p.limit_ns, &c.abort_flag)) {
                            raise_abort(c, p);
                            return false;
                        }
                        const uint32_t sA = smem_u32(base + stage * S::STAGE), sB = sA + S::A_BYTES;
                        const uint32_t fb = smem_u32(&c.full[stage]);
                        const uint32_t bar = PAIR ? mapa(fb, 0) : fb;
                        if (PAIR && !leader) arrive_expect_cluster(bar, bytes);
                        else mbar_arrive_expect_tx(fb, bytes);
                        auto load = [&](uint32_t dst, const CUtensorMap* m, int c0, int c1) {
                            if (PAIR) tma_load_pair(dst, m, bar, c0, c1);
                            else tma_load_2d(dst, m, fb, c0, c1);
                        };
                        if (MODE < GRAD) {
                            load(sA, &mapA, k0, m0);
                            load(sB, &mapB, k0, n0);
                        } else if (!DWT) {
                            load(sA, &mapA, k0, m0);
#pragma unroll
                            for (int i = 0; i < S::BN_CTA / 64; ++i) load(sB + i * SLAB, &mapB, n0 + i * 64, k0);
                        } else {
#pragma unroll
                            for (int i = 0; i < BM / 64; ++i) load(sA + i * SLAB, &mapC, m0 + i * 64, k0);
#pragma unroll
                            for (int i = 0; i < S::BN_CTA / 64; ++i) load(sB + i * SLAB, &mapD, n0 + i * 64, k0);
                        }
                        issued[stage] = (int)phase;
                        if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    }
                    return true;
                };
                ok = is_dw(t) ? fill(Flag<true>{}) : fill(Flag<false>{});
            }
            if (!ok && leader)   // the copies that this CTA's barriers still count
                for (int s = 0; s < STAGES; ++s)
                    if (issued[s] >= 0)
                        mbar_wait_bounded(smem_u32(&c.full[s]), (uint32_t)issued[s], p.limit_ns, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            if (lane == 0) {
                // a stage or a K step moves only the start address (16-byte units);
                // operands along K ("k") or across it ("n")
                const uint32_t s0 = smem_u32(base), width = (uint32_t)(p.tile_n >> 3) << 17;
                const uint64_t ak = smem_desc_sw128(s0, 16, 1024), an = smem_desc_sw128(s0, SLAB, 1024);
                const uint64_t bk = smem_desc_sw128(s0 + S::A_BYTES, 16, 1024);
                const uint64_t bn = smem_desc_sw128(s0 + S::A_BYTES, SLAB, 1024);
                constexpr uint32_t STEP_K = 32 >> 4, STEP_N = 2048 >> 4;
                int stage = 0, acc = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool ok = true;
                for (int u = unit0; u < units && ok; u += nunits) {
                    const Tile t = get_tile<MODE>(plan, p, u);
                    if (t.nkb == 0) continue;
                    auto acquire = [&]() {
                        if (!mbar_wait_bounded(smem_u32(&c.tempty[acc]), acc_phase ^ 1, p.limit_ns, &c.abort_flag)) {
                            raise_abort(c, p);
                            return false;
                        }
                        tc_fence_after();
                        return true;
                    };
                    auto hand_over = [&]() {
                        commit<PAIR>(smem_u32(&c.tfull[acc]));
                        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                    };
                    // (a loop for each product: what is issued a stage is constant)
                    auto issue = [&](auto dw, int nkb) {
                        constexpr bool a_n = decltype(dw)::value, b_n = MODE >= GRAD;
                        const uint32_t idesc = idesc_bf16_f32(S::TILE_M, 0, a_n, b_n) | width;
                        const uint64_t ad0 = a_n ? an : ak, bd0 = b_n ? bn : bk;
                        for (int k = 0; k < nkb; ++k) {
                            if (!mbar_wait_bounded(smem_u32(&c.full[stage]), phase, p.limit_ns, &c.abort_flag)) {
                                raise_abort(c, p);
                                return false;
                            }
                            tc_fence_after();
                            const uint64_t so = (uint64_t)(stage * (S::STAGE >> 4));
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                mma<PAIR>(tmem + acc * BN, ad0 + so + kk * (a_n ? STEP_N : STEP_K),
                                          bd0 + so + kk * (b_n ? STEP_N : STEP_K), idesc, (k | kk) != 0);
                            commit<PAIR>(smem_u32(&c.empty[stage]));
                            if (++stage == STAGES) { stage = 0; phase ^= 1; }
                        }
                        return true;
                    };
                    const int most = CUT ? chunk : t.nkb;
                    for (int k = 0; k < t.nkb && ok; k += most) {
                        const int nkb = min(most, t.nkb - k);
                        ok = acquire() && (is_dw(t) ? issue(Flag<true>{}, nkb) : issue(Flag<false>{}, nkb));
                        if (ok) hand_over();
                    }
                }
                // every MMA issued has completed before TMEM is freed
                commit_local<PAIR>(smem_u32(&c.drain));
                mbar_wait_bounded(smem_u32(&c.drain), 0, p.limit_ns, nullptr);
            }
            __syncwarp();
        }
    } else {
        const HeadDev& h = p.h;
        const int ew = warp - 2, q = warp & 3, half = ew >> 2;
        uint8_t* box = boxes + ew * BOX;
        const int n = head_rows(h);
        const float scale = MODE >= GRAD ? head_scale(h) : 1.f;
        // a few-row call's tiles all have the same rows: their statistics run on
        float few_m = -INFINITY, few_s = 0.f;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int u = unit0; u < units; u += nunits) {
            const Tile t = get_tile<MODE>(plan, p, u);
            const bool dw = is_dw(t);
            const int r0 = t.mt * S::TILE_M + rank * BM + q * 32, r = r0 + lane;
            const int col0 = t.nt * p.tile_n + half * 128;   // of the warp's columns
            const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN + half * 128);
            // what the epilogue reads of the row, in front of the wait
            int tok = 0, e0 = 0, e1 = 0, tgt = -1;
            if (!dw && r < n) tok = head_token(h, r);
            if (MODE <= ZKEEP && r < n) {
                if (h.target) {
                    const int64_t y = h.target[tok];
                    tgt = y >= 0 && y < h.V ? (int)y : -1;
                } else if (h.start && !(p.tile_n & 127)) {
                    const int b = col0 / kHeadBlock;
                    const uint8_t* s = h.start + (int64_t)tok * h.nblk;
                    if (b < h.nblk) {
                        e0 = s[b];
                        e1 = b + 1 < h.nblk ? s[b + 1] : h.ent[tok];
                    }
                } else {   // tiles that are no whole blocks, or one entry: first entry of the columns
                    e1 = h.ent[tok];
                    const int* s = h.sidx + (int64_t)tok * h.K;
                    int hi = e1;
                    while (e0 < hi) {
                        const int mid = (e0 + hi) >> 1;
                        if (s[mid] < col0) e0 = mid + 1;
                        else hi = mid;
                    }
                }
                if (!h.target && e0 < e1) tgt = h.sidx[(int64_t)tok * h.K + e0];
            }
            if (t.nkb > 0) {
                if (!mbar_wait_warp(smem_u32(&c.tfull[acc]), acc_phase, p.limit_ns, &c.abort_flag)) {
                    raise_abort(c, p);
                    break;
                }
                tc_fence_after();
            }
            auto release = [&]() {
                if (t.nkb == 0) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t tb = smem_u32(&c.tempty[acc]);
                    if (PAIR && !leader) arrive_cluster(mapa(tb, 0));
                    else mbar_arrive(tb);
                }
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            };
            if (MODE <= ZKEEP) {
                const int width = min(p.tile_n - half * 128, 128);
                const int left = min(width, h.V - col0);   // the warp's columns (maybe none)
                if (left <= 0) {
                    release();
                    bool ok = true;
                    for (int k = chunk; CUT && k < t.nkb && ok; k += chunk) {
                        ok = mbar_wait_warp(smem_u32(&c.tfull[acc]), acc_phase, p.limit_ns, &c.abort_flag);
                        if (ok) release();
                    }
                    if (!ok) {
                        raise_abort(c, p);
                        break;
                    }
                    continue;
                }
                float v[4][32];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    if (ch * 32 < left) tmem_ld32_start(trow + ch * 32, v[ch]);
                tmem_ld_wait(v);
                release();
                if (CUT) {
                    bool ok = true;
                    for (int k = chunk; k < t.nkb && ok; k += chunk) {
                        ok = mbar_wait_warp(smem_u32(&c.tfull[acc]), acc_phase, p.limit_ns, &c.abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t more = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN + half * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (i * 16 >= left) break;
                            float w[16];
                            tmem_ld16(more + i * 16, w);
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[i >> 1][(i & 1) * 16 + j] += w[j];
                        }
                        release();
                    }
                    if (!ok) {
                        raise_abort(c, p);
                        break;
                    }
                }
                if (left < 128) {
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (ch * 32 + j >= left) v[ch][j] = -INFINITY;
                }
                // the targets' logits
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    while (true) {
                        const int rel = tgt - (col0 + ch * 32);
                        const bool hit = tgt >= 0 && rel >= 0 && rel < 32 && ch * 32 + rel < left;
                        if (!__any_sync(0xffffffffu, hit)) break;
                        float w = v[ch][0];
#pragma unroll
                        for (int j = 1; j < 32; ++j) w = rel == j ? v[ch][j] : w;
                        if (hit) {
                            const int64_t at = (int64_t)tok * h.K + e0;
                            h.lz[at] = w;
                            ++e0;
                            tgt = !h.target && e0 < e1 ? h.sidx[at + 1] : -1;
                        }
                    }
                }
                float m4[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], v[ch][j]);
                const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                uint64_t sum[2] = {0, 0};
                const uint64_t c2 = f2_pack(h.c, h.c), m2 = f2_pack(-m, -m), s2 = f2_pack(kHeadShift, kHeadShift);
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float a, b;
                        f2_unpack(f2_fma(f2_add(f2_pack(v[ch][j], v[ch][j + 1]), m2), c2, s2), a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        sum[(j >> 1) & 1] = f2_add(sum[(j >> 1) & 1], f2_pack(a, b));
                        v[ch][j] = a;
                        v[ch][j + 1] = b;
                    }
                float sa, sb;
                f2_unpack(f2_add(sum[0], sum[1]), sa, sb);
                sa += sb;
                if (p.few) {
                    // (NaN: the comparison fails, and the sum takes it on)
                    if (m > few_m) {
                        few_s = few_s == 0.f ? sa : few_s * ex2_approx((few_m - m) * h.c) + sa;
                        few_m = m;
                    } else {
                        few_s += sa * ex2_approx((m - few_m) * h.c);
                    }
                } else if (r < n) {
                    h.stats[(int64_t)(col0 / kHeadBlock) * h.srows + r] = make_float2(m, sa);
                }
                if (MODE == ZKEEP) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        if (col0 + hh * 64 >= h.Vp) break;
                        if (lane == 0) bulk_wait_read();   // the box's last store has read it
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float* s = &v[hh * 2 + (j >> 2)][(j & 3) * 8];
                            *reinterpret_cast<uint4*>(box + box_at(lane, j)) =
                                make_uint4(half2_bits(s[0], s[1]), half2_bits(s[2], s[3]),
                                           half2_bits(s[4], s[5]), half2_bits(s[6], s[7]));
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            store_box(&mapO, smem_u32(box), col0 + hh * 64, r0);
                            bulk_commit();
                        }
                    }
                }
            } else {
                const int rows = (dw ? h.V : n) - r0;      // valid rows of the warp's 32
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    const int col = col0 + ch * 32;
                    if (col >= h.d) break;
                    float v[32];
                    if (t.nkb > 0) {
                        tmem_ld32(trow + ch * 32, v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0.f;
                    }
                    if (t.slot >= 0) {
                        if (lane < rows) {
                            float4* o = reinterpret_cast<float4*>(
                                p.part + ((int64_t)t.slot * S::TILE_M + rank * BM + q * 32 + lane) * BN + half * 128 +
                                ch * 32);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        }
                        continue;
                    }
                    if (rows <= 0) break;
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= scale;
                    if (dw && p.dW.f32) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4*>(box + box_at(lane, j)) =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (p.dW.accumulate) add_box(&mapO, smem_u32(box), col, r0);
                            else store_box(&mapO, smem_u32(box), col, r0);
                            bulk_commit();
                        }
                        continue;
                    }
                    // bf16: 64 columns make a box
                    const int part = (ch & 1) * 4;
                    if (part == 0) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(box + box_at(lane, part + j)) =
                            make_uint4(bf2_bits(v[8 * j], v[8 * j + 1]), bf2_bits(v[8 * j + 2], v[8 * j + 3]),
                                       bf2_bits(v[8 * j + 4], v[8 * j + 5]), bf2_bits(v[8 * j + 6], v[8 * j + 7]));
                    if (part == 0 && col + 32 < h.d) continue;
                    const int cb = col - part * 8;   // first column of the box
                    if (dw) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            store_box(&mapO, smem_u32(box), cb, r0);
                            bulk_commit();
                        }
                    } else {
                        // rows go to their tokens: eight lanes a row, four rows at a time
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int rr = i * 4 + (lane >> 3), j = lane & 7;
                            const int to = __shfl_sync(0xffffffffu, tok, rr);
                            if (rr < rows && cb + j * 8 < h.d)
                                *reinterpret_cast<uint4*>((__nv_bfloat16*)p.dx.out + (int64_t)to * h.d + cb + j * 8) =
                                    *reinterpret_cast<const uint4*>(box + box_at(rr, j));
                        }
                        __syncwarp();
                    }
                }
                release();
            }
        }
        if (MODE == Z && p.few && q * 32 + lane < n)
            h.stats[(int64_t)(blockIdx.x * 2 + half) * h.srows + q * 32 + lane] = make_float2(few_m, few_s);
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tm_free<PAIR>(tmem);
    }
}

// The parts of cut tiles, added in order: blocks of kJoinRows rows of a tile; the
// first `nx` tiles are DX's.
__global__ void __launch_bounds__(256) head_join_kernel(const __grid_constant__ TcParams p, int nx) {
    constexpr int TM = 2 * BM;
    __shared__ float4 buf[kJoinRows][256];
    wait_front();
    const HeadDev& h = p.h;
    const bool dw = (int)blockIdx.x >= nx;
    const int i = dw ? blockIdx.x - nx : blockIdx.x;   // tile behind the whole ones
    Product a;
    a.s = h.splits[dw];
    if (a.s.parts <= 1 || a.s.full + i >= a.s.tiles) return;
    const int M = dw ? h.V : head_rows(h);
    a.MT = (M + TM - 1) / TM;
    a.NT = (h.d + BN - 1) / BN;
    a.shift = DX_SHIFT;
    a.group.set(dw ? a.NT : a.NT << DX_SHIFT);
    Tile t;
    if (dw) place<true>(a, a.s.full + i, t);
    else place<false>(a, a.s.full + i, t);
    const float scale = head_scale(h);
    const int rl = blockIdx.y * kJoinRows, r0 = t.mt * TM + rl, rows = M - r0;
    if (rows <= 0) return;
    float4 sums[kJoinRows];
    const int64_t slot = (dw ? p.capx : 0) + (int64_t)i * a.s.parts;
    const int cl = join_rows<BN>(p.part + (slot * TM + rl) * BN, (int64_t)TM * BN, a.s.parts, rows, buf, sums);
    const int col = t.nt * BN + cl;
    if (cl < 0 || col >= h.d) return;
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
        if (r >= rows) break;
        float4 s = sums[r];
        s.x *= scale;
        s.y *= scale;
        s.z *= scale;
        s.w *= scale;
        const int64_t at = (int64_t)(dw ? r0 + r : head_token(h, r0 + r)) * h.d + col;
        if (dw && p.dW.f32) {
            float4* o = reinterpret_cast<float4*>((float*)p.dW.out + at);
            if (p.dW.accumulate) {
                const float4 b = *o;
                s = make_float4(s.x + b.x, s.y + b.y, s.z + b.z, s.w + b.w);
            }
            *o = s;
        } else {
            *reinterpret_cast<uint2*>((__nv_bfloat16*)(dw ? p.dW.out : p.dx.out) + at) =
                make_uint2(bf2_bits(s.x, s.y), bf2_bits(s.z, s.w));
        }
    }
}

// ---- host side -------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// [rows][cols] of 16-bit (or fp32) values, rows `ld` values apart, in boxes of 128
// bytes by box_rows.
bool make_map(CUtensorMap* m, const void* ptr, int64_t cols, int64_t rows, int64_t ld, int box_rows,
              CUtensorMapDataType dt) {
    auto fn = encode_fn();
    if (!fn) return false;
    const int size = dt == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)(ld * size)};
    cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows}, es[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void*>(ptr), dims, stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

// CTAs or pairs that run at once on the current device.
template <int MODE, bool PAIR, bool CUT> cudaError_t resident(int* units) {
    static std::mutex mu;
    static int of[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (of[dev] == 0) {
        auto kern = head_tc_kernel<MODE, PAIR, CUT>;
        constexpr size_t SMEM = smem_bytes<PAIR>();
        static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
        if (e != cudaSuccess) return e;
        int n = device_sm_count();
        if (PAIR) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim = {2, 1, 1};
            cfg.gridDim = dim3(2 * n);
            cfg.blockDim = dim3(THREADS);
            cfg.dynamicSmemBytes = SMEM;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int k = 0;
            e = cudaOccupancyMaxActiveClusters(&k, kern, &cfg);
            if (e != cudaSuccess) return e;
            n = k > 0 ? k : n / 2;
        }
        of[dev] = n;
    }
    *units = of[dev];
    return cudaSuccess;
}

// Test hook MOE_DEBUG_HEAD_WITHHOLD=mode:unit:kb (0 Z, 2 DX or DW): that unit's
// producer issues nothing from K block kb on, so that the waits on it run out.
void withhold_hook(int mode, TcParams& p) {
    p.withhold_unit = p.withhold_kb = -1;
    const char* s = getenv("MOE_DEBUG_HEAD_WITHHOLD");
    int m, u, k;
    if (!s || sscanf(s, "%d:%d:%d", &m, &u, &k) != 3 || m != mode || u < 0 || k < 0) return;
    p.withhold_unit = u;
    p.withhold_kb = k;
}

template <int MODE, bool PAIR, bool CUT>
cudaError_t launch_tc(const CUtensorMap (&m)[5], TcParams& p, int64_t tiles, cudaStream_t st) {
    int units = 0;
    const cudaError_t e = resident<MODE, PAIR, CUT>(&units);
    if (e != cudaSuccess) return e;
    if (MODE <= ZKEEP && tiles < units) units = (int)(tiles > 0 ? tiles : 1);
    // (the tiles are cut for so many; all products' CTAs are alike, so that is all of them)
    if (MODE >= GRAD && p.units < units) units = p.units;
    p.limit_ns = wait_limit_ns();
    withhold_hook(MODE <= ZKEEP ? Z : GRAD, p);
    return launch_early(head_tc_kernel<MODE, PAIR, CUT>, dim3((unsigned)(units * Shape<PAIR>::CTAS)), THREADS,
                        smem_bytes<PAIR>(), Shape<PAIR>::CTAS, st, m[0], m[1], m[2], m[3], m[4], p);
}

inline int64_t tiles_of(int64_t m, int tm, int64_t n, int tn) { return (m + tm - 1) / tm * ((n + tn - 1) / tn); }

constexpr size_t kTileBytes = (size_t)2 * BM * BN * 4;

int64_t parts_dx(int64_t rows, int V, int d) {
    return (int64_t)split_bound(tiles_of(rows, 2 * BM, d, BN), (V + BK - 1) / BK, device_sm_count() / 2, 4);
}
int64_t parts_dw(int64_t rows, int V, int d) {
    return (int64_t)split_bound(tiles_of(V, 2 * BM, d, BN), (rows + BK - 1) / BK, device_sm_count() / 2, 4);
}

}  // namespace

size_t head_part_bytes(int64_t rows, int V, int d) {
    return (size_t)(parts_dx(rows, V, d) + parts_dw(rows, V, d)) * kTileBytes;
}

cudaError_t head_tc_rule(int64_t rows, int V, int d, SplitRule* r) {
    *r = SplitRule{2 * BM, BN, 0, (int)parts_dx(rows, V, d), (int)parts_dw(rows, V, d), 4, 4, 12, 8, 0, 0, 0};
    return resident<GRAD, true, false>(&r->units);
}

// Columns of a tile where W's bytes bound: about equal tiles for whole waves of CTAs.
int head_few_tile(int V) {
    const int sms = device_sm_count();
    const int waves = (V + sms * BN - 1) / (sms * BN);
    const int n = (V + sms * waves - 1) / (sms * waves);
    return n <= 32 ? 32 : (n + 15) / 16 * 16;
}

int head_few_stats(int V) {
    const int n = head_few_tile(V), tiles = (V + n - 1) / n, sms = device_sm_count();
    return 2 * (tiles < sms ? tiles : sms);
}

cudaError_t launch_head_tc(const HeadDev& h, const void* xc, const void* W, bool keep, bool single,
                           cudaStream_t st) {
    TcParams p{};
    p.h = h;
    CUtensorMap m[5];
    const int64_t xrows = single && !h.n_live ? h.T : h.rows;
    p.few = single && !keep;
    p.tile_n = p.few ? head_few_tile(h.V) : BN;
    p.a_rows = single ? (int)((xrows < BM ? xrows : BM) + 7) / 8 * 8 : BM;
    if (!make_map(&m[0], xc, h.d, xrows, h.d, p.a_rows, kBf16) ||
        !make_map(&m[1], W, h.d, h.V, h.d, single ? p.tile_n : BM, kBf16))
        return cudaErrorInvalidValue;
    m[2] = m[3] = m[4] = m[0];
    if (keep && !make_map(&m[4], h.P, h.Vp, h.srows, h.Vp, 32, CU_TENSOR_MAP_DATA_TYPE_FLOAT16))
        return cudaErrorInvalidValue;
    const int64_t tiles = tiles_of(single ? BM : h.rows, single ? BM : 2 * BM, h.V, p.tile_n);
    if (single) return keep ? launch_tc<ZKEEP, false, true>(m, p, tiles, st) : launch_tc<Z, false, true>(m, p, tiles, st);
    if (h.d > kWhole * BK)
        return keep ? launch_tc<ZKEEP, true, true>(m, p, tiles, st) : launch_tc<Z, true, true>(m, p, tiles, st);
    return keep ? launch_tc<ZKEEP, true, false>(m, p, tiles, st) : launch_tc<Z, true, false>(m, p, tiles, st);
}

cudaError_t launch_head_tc_grad(const HeadDev& h, const void* xc, const void* W, const HeadOut& dx,
                                const HeadOut& dW, float* part, const SplitRule& rule, cudaStream_t st) {
    TcParams p{};
    p.h = h;
    p.dx = dx;
    p.dW = dW;
    p.tile_n = BN;
    p.a_rows = BM;
    p.part = part;
    p.capx = rule.capx;
    p.units = rule.units;
    // rows that are never made need not be read
    const int64_t made = ((h.T - h.p0 < h.rows ? h.T - h.p0 : h.rows) + 63) / 64 * 64;
    CUtensorMap m[5];
    if (!make_map(&m[0], h.P, h.V, made, h.Vp, BM, kBf16) || !make_map(&m[1], W, h.d, h.V, h.d, 64, kBf16) ||
        !make_map(&m[2], h.P, h.V, made, h.Vp, 64, kBf16) || !make_map(&m[3], xc, h.d, made, h.d, 64, kBf16))
        return cudaErrorInvalidValue;
    m[4] = m[0];
    if (dW.out && !make_map(&m[4], dW.out, h.d, h.V, h.d, 32, dW.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : kBf16))
        return cudaErrorInvalidValue;
    // at most: DX's tiles of all rows, where that is less than a wave; DW's are known
    const int64_t tx = dx.out ? tiles_of(made, 2 * BM, h.d, BN) : 0, tw = dW.out ? tiles_of(h.V, 2 * BM, h.d, BN) : 0;
    // Short products in one launch (33 tokens of 32000 entries, d = 2048: 3 us less);
    // long ones in two, each of which begins with all pairs in step, so that tiles that
    // share an operand find it in L2 (4096 tokens of 131072 entries, d = 4096: 3% less)
    const bool apart = tx * ((h.V + BK - 1) / BK) + tw * (made / BK) > 512 * (int64_t)(device_sm_count() / 2);
    cudaError_t e;
    if (apart && tx && tw) {
        p.dW.out = nullptr;
        e = launch_tc<DX, true, false>(m, p, 0, st);
        if (e != cudaSuccess) return e;
        p.dW = dW;
        p.dx.out = nullptr;
        e = launch_tc<DW, true, false>(m, p, 0, st);
        p.dx = dx;
    } else {
        e = launch_tc<GRAD, true, false>(m, p, 0, st);
    }
    if (e != cudaSuccess) return e;
    const int nx = rule.capx ? (int)(tx < p.units ? tx : p.units) : 0, nw = rule.capw ? (int)(tw % p.units) : 0;
    if (nx + nw == 0) return cudaSuccess;
    const int64_t most = nw || made > 2 * BM ? 2 * BM : made;
    return launch_early(head_join_kernel, dim3((unsigned)(nx + nw), (unsigned)((most + kJoinRows - 1) / kJoinRows)),
                        256, 0, 1, st, p, nx);
}

}  // namespace moe
