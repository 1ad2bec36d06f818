// head_tc.cu -- the three products of the losses over a vocabulary head in bf16 on
// the tensor cores (tcgen05.mma, fp32 accumulators in TMEM, operands by TMA).
//
//   Z, ZKEEP  tiles of xc W^T whose epilogue leaves a row's largest logit and sum of
//             exponentials a 128 columns, its targets' logits and (ZKEEP) the
//             exponentials as fp16
//   DX        dx = scale G W       reduction over the vocabulary
//   DW        dW (+)= scale G^T xc reduction over the live tokens
//
// CTA = 10 warps: warp 0 issues the TMA loads into a ring of stages of 64 K values,
// one thread of warp 1 the MMAs into one of two TMEM accumulators of 256 columns,
// eight warps drain the other one: warp w the lanes of quarter w % 4 and 128
// columns.  PAIR: clusters of two CTAs, tiles of 256 x 256 (cta_group::2, each CTA
// holds its 128 rows of A and 128 columns of B, 32 KB a stage, six stages); else
// one CTA, 128 rows (48 KB, four stages), for calls of up to 128 tokens, where W's
// bytes bound and half a pair's rows would be empty.
//
// A persistent grid walks the tiles.  What is left of the last, uneven wave (or
// everything, with few tiles) is cut along the reduction into parts whose sums go
// to the workspace in fp32 and are added in order by head_join_kernel.  The number
// of live tokens, and with it tiles and parts, is read on the device.
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
constexpr int GROUP_Z = 16, GROUP_DX = 8;    // row tiles that share a column tile's operand

enum Mode { Z = 0, ZKEEP = 1, DX = 2, DW = 3 };

template <bool PAIR> struct Shape {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TILE_M = BM * CTAS;
    static constexpr int BN_CTA = BN / CTAS;
    static constexpr int A_BYTES = BM * BK * 2;
    static constexpr int B_BYTES = BN_CTA * BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = PAIR ? 6 : 4;
};

template <int STAGES> struct Ctrl {
    uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    int tiles, full_tiles, parts, kbp, kb;
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
    HeadOut o;
    float* part;             // [cap][TILE_M][BN] sums of cut tiles
    int cap;
    int units;               // CTAs or pairs of the launch
    uint64_t limit_ns;
    int withhold_unit, withhold_kb;   // test hook: see launch_tc
};

// Tiles and K blocks of a mode's product.
template <int MODE, bool PAIR>
__device__ __forceinline__ Split plan_tiles(const TcParams& p, int& kb) {
    constexpr int TM = Shape<PAIR>::TILE_M;
    const HeadDev& h = p.h;
    const int n = head_rows(h);
    const int MT = ((MODE == DW ? h.V : n) + TM - 1) / TM;
    const int NT = ((MODE <= ZKEEP ? h.V : h.d) + p.tile_n - 1) / p.tile_n;
    kb = ((MODE <= ZKEEP ? h.d : MODE == DX ? h.V : n) + BK - 1) / BK;
    if (MODE <= ZKEEP) return Split{MT * NT, MT * NT, 1, kb};
    // nothing to add: no tiles; without accumulation dW's zeros are written
    if (MODE == DW && n == 0) return Split{p.o.accumulate ? 0 : MT * NT, MT * NT, 1, 0};
    return split_tiles(MT * NT, kb, p.units, p.cap, 4, 4, 12, PAIR ? 8 : 16);
}

struct Tile { int mt, nt, kb0, nkb, slot; };   // slot: of a part, else -1

template <int MODE, bool PAIR, typename C>
__device__ __forceinline__ Tile get_tile(const C& c, const TcParams& p, int u) {
    constexpr int TM = Shape<PAIR>::TILE_M;
    Tile t;
    int i = u;
    t.kb0 = 0;
    t.nkb = c.kb;
    t.slot = -1;
    if (MODE >= DX && u >= c.full_tiles && c.parts > 1) {
        // part after part: the parts of the same K range run at the same time
        const int rem = c.tiles - c.full_tiles, v = u - c.full_tiles;
        const int part = v / rem;
        i = c.full_tiles + v % rem;
        t.kb0 = part * c.kbp;
        t.nkb = min(c.kbp, c.kb - t.kb0);
        t.slot = (i - c.full_tiles) * c.parts + part;
    }
    const int n = head_rows(p.h);
    const int NT = ((MODE <= ZKEEP ? p.h.V : p.h.d) + p.tile_n - 1) / p.tile_n;
    if (MODE == DW) {
        t.mt = i / NT;
        t.nt = i % NT;
    } else {
        constexpr int G = MODE == DX ? GROUP_DX : GROUP_Z;
        const int MT = (n + TM - 1) / TM;
        const int g = i / (G * NT), l = i - g * G * NT;
        const int gm = min(G, MT - g * G);
        t.mt = g * G + l % gm;
        t.nt = l / gm;
    }
    return t;
}
template <int MODE, typename C>
__device__ __forceinline__ int unit_count(const C& c) {
    return c.full_tiles + (c.tiles - c.full_tiles) * c.parts;
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

template <int MODE, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    head_tc_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                   const __grid_constant__ CUtensorMap mapO, const __grid_constant__ TcParams p) {
    using S = Shape<PAIR>;
    constexpr int STAGES = S::STAGES;
    constexpr bool A_MN = MODE == DW, B_MN = MODE >= DX;
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
    if (warp == 2) {
        int kb;
        const Split s = plan_tiles<MODE, PAIR>(p, kb);
        if (lane == 0) {
            c.tiles = s.tiles;
            c.full_tiles = s.full < s.tiles ? s.full : s.tiles;
            c.parts = s.parts;
            c.kbp = s.kbp;
            c.kb = kb;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = c.tmem_base;
    const int units = unit_count<MODE>(c);

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued[STAGES];
            uint32_t phase = 0;
            bool ok = true;
            for (int s = 0; s < STAGES; ++s) issued[s] = -1;
            const uint32_t bytes =
                (uint32_t)(A_MN ? S::A_BYTES : p.a_rows * BK * 2) +
                (uint32_t)(B_MN || PAIR ? S::B_BYTES : p.tile_n * BK * 2);
            for (int u = unit0; u < units && ok; u += nunits) {
                const Tile t = get_tile<MODE, PAIR>(c, p, u);
                const int m0 = t.mt * S::TILE_M + rank * BM;
                const int n0 = t.nt * p.tile_n + rank * S::BN_CTA;
                for (int k = 0; k < t.nkb; ++k) {
                    if (leader && u == p.withhold_unit && k == p.withhold_kb) {
                        ok = false;
                        break;
                    }
                    if (!mbar_wait_bounded(smem_u32(&c.empty[stage]), phase ^ 1, p.limit_ns, &c.abort_flag)) {
                        raise_abort(c, p);
                        ok = false;
                        break;
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
                    const int k0 = (t.kb0 + k) * BK;
                    if (!A_MN) {
                        load(sA, &mapA, k0, m0);
                    } else {
#pragma unroll
                        for (int i = 0; i < BM / 64; ++i) load(sA + i * SLAB, &mapA, m0 + i * 64, k0);
                    }
                    if (!B_MN) {
                        load(sB, &mapB, k0, n0);
                    } else {
#pragma unroll
                        for (int i = 0; i < S::BN_CTA / 64; ++i) load(sB + i * SLAB, &mapB, n0 + i * 64, k0);
                    }
                    issued[stage] = (int)phase;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
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
                const uint32_t idesc = idesc_bf16_f32(S::TILE_M, 0, A_MN, B_MN) | (uint32_t)(p.tile_n >> 3) << 17;
                const uint32_t s0 = smem_u32(base);
                // a stage or a K step moves only the start address (16-byte units)
                const uint64_t ad0 = smem_desc_sw128(s0, A_MN ? SLAB : 16, 1024);
                const uint64_t bd0 = smem_desc_sw128(s0 + S::A_BYTES, B_MN ? SLAB : 16, 1024);
                constexpr uint32_t A_STEP = (A_MN ? 2048 : 32) >> 4, B_STEP = (B_MN ? 2048 : 32) >> 4;
                int stage = 0, acc = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool ok = true;
                for (int u = unit0; u < units && ok; u += nunits) {
                    const Tile t = get_tile<MODE, PAIR>(c, p, u);
                    if (t.nkb == 0) continue;
                    if (!mbar_wait_bounded(smem_u32(&c.tempty[acc]), acc_phase ^ 1, p.limit_ns, &c.abort_flag)) {
                        raise_abort(c, p);
                        break;
                    }
                    tc_fence_after();
                    for (int k = 0; k < t.nkb; ++k) {
                        if (!mbar_wait_bounded(smem_u32(&c.full[stage]), phase, p.limit_ns, &c.abort_flag)) {
                            raise_abort(c, p);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t so = (uint64_t)(stage * (S::STAGE >> 4));
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma<PAIR>(tmem + acc * BN, ad0 + so + kk * A_STEP, bd0 + so + kk * B_STEP, idesc,
                                      (k | kk) != 0);
                        commit<PAIR>(smem_u32(&c.empty[stage]));
                        if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    }
                    if (!ok) break;
                    commit<PAIR>(smem_u32(&c.tfull[acc]));
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
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
        const float scale = MODE >= DX ? head_scale(h) : 1.f;
        // a few-row call's tiles all have the same rows: their statistics run on
        float few_m = -INFINITY, few_s = 0.f;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int u = unit0; u < units; u += nunits) {
            const Tile t = get_tile<MODE, PAIR>(c, p, u);
            const int r0 = t.mt * S::TILE_M + rank * BM + q * 32, r = r0 + lane;
            const int col0 = t.nt * p.tile_n + half * 128;   // of the warp's columns
            const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN + half * 128);
            // what the epilogue reads of the row, in front of the wait
            int tok = 0, e0 = 0, e1 = 0, tgt = -1;
            if (MODE != DW && r < n) tok = head_token(h, r);
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
                    continue;
                }
                float v[4][32];
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    if (ch * 32 < left) tmem_ld32(trow + ch * 32, v[ch]);
                release();
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
                const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * h.c - kHeadShift;
                uint64_t sum[2] = {0, 0};
                const uint64_t c2 = f2_pack(h.c, h.c), m2 = f2_pack(-m, -m);
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float a, b;
                        f2_unpack(f2_fma(f2_pack(v[ch][j], v[ch][j + 1]), c2, m2), a, b);
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
                        few_s = few_s == 0.f ? sa : few_s * ex2_approx(few_m - m) + sa;
                        few_m = m;
                    } else {
                        few_s += sa * ex2_approx(m - few_m);
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
                const int rows = (MODE == DW ? h.V : n) - r0;      // valid rows of the warp's 32
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
                    if (MODE == DW && p.o.f32) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4*>(box + box_at(lane, j)) =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (p.o.accumulate) add_box(&mapO, smem_u32(box), col, r0);
                            else store_box(&mapO, smem_u32(box), col, r0);
                            bulk_commit();
                        }
                        continue;
                    }
                    // bf16: 64 columns make a box
                    const int part = (ch & 1) * 4;
                    if (part == 0) {
                        if (MODE == DW && lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(box + box_at(lane, part + j)) =
                            make_uint4(bf2_bits(v[8 * j], v[8 * j + 1]), bf2_bits(v[8 * j + 2], v[8 * j + 3]),
                                       bf2_bits(v[8 * j + 4], v[8 * j + 5]), bf2_bits(v[8 * j + 6], v[8 * j + 7]));
                    if (part == 0 && col + 32 < h.d) continue;
                    const int cb = col - part * 8;   // first column of the box
                    if (MODE == DW) {
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
                                *reinterpret_cast<uint4*>((__nv_bfloat16*)p.o.out + (int64_t)to * h.d + cb + j * 8) =
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

// The parts of cut tiles, added in order.
template <int MODE, bool PAIR>
__global__ void __launch_bounds__(256) head_join_kernel(const __grid_constant__ TcParams p) {
    constexpr int TM = Shape<PAIR>::TILE_M;
    __shared__ Split ss;
    __shared__ float4 buf[kJoinRows][256];
    wait_front();
    if (threadIdx.x < 32) {
        int kb;
        const Split s = plan_tiles<MODE, PAIR>(p, kb);
        if (threadIdx.x == 0) ss = s;
    }
    __syncthreads();
    const HeadDev& h = p.h;
    const int i = blockIdx.x;                       // tile behind the whole ones
    if (ss.parts <= 1 || ss.full + i >= ss.tiles) return;
    struct { int tiles, full_tiles, parts, kbp, kb; } c{ss.tiles, ss.full, ss.parts, ss.kbp, 1};
    const Tile t = get_tile<MODE, PAIR>(c, p, ss.full + i);
    const int M = MODE == DW ? h.V : head_rows(h);
    const float scale = head_scale(h);
    const int rl = blockIdx.y * kJoinRows, r0 = t.mt * TM + rl, rows = M - r0;
    if (rows <= 0) return;
    float4 sums[kJoinRows];
    const int cl = join_rows<BN>(p.part + ((int64_t)i * ss.parts * TM + rl) * BN, (int64_t)TM * BN, ss.parts, rows, buf,
                                 sums);
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
        const int64_t at = (int64_t)(MODE == DX ? head_token(h, r0 + r) : r0 + r) * h.d + col;
        if (MODE == DW && p.o.f32) {
            float4* o = reinterpret_cast<float4*>((float*)p.o.out + at);
            if (p.o.accumulate) {
                const float4 b = *o;
                s = make_float4(s.x + b.x, s.y + b.y, s.z + b.z, s.w + b.w);
            }
            *o = s;
        } else {
            *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o.out + at) = make_uint2(bf2_bits(s.x, s.y), bf2_bits(s.z, s.w));
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
template <int MODE, bool PAIR> cudaError_t resident(int* units) {
    static std::mutex mu;
    static int of[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (of[dev] == 0) {
        auto kern = head_tc_kernel<MODE, PAIR>;
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

// Test hook MOE_DEBUG_HEAD_WITHHOLD=mode:unit:kb (0 Z, 2 DX, 3 DW): that unit's
// producer issues nothing from K block kb on, so that the waits on it run out.
void withhold_hook(int mode, TcParams& p) {
    p.withhold_unit = p.withhold_kb = -1;
    const char* s = getenv("MOE_DEBUG_HEAD_WITHHOLD");
    int m, u, k;
    if (!s || sscanf(s, "%d:%d:%d", &m, &u, &k) != 3 || m != mode || u < 0 || k < 0) return;
    p.withhold_unit = u;
    p.withhold_kb = k;
}

template <int MODE, bool PAIR>
cudaError_t launch_tc(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o, TcParams& p,
                      int64_t tiles, cudaStream_t st) {
    auto kern = head_tc_kernel<MODE, PAIR>;
    int units = 0;
    cudaError_t e = resident<MODE, PAIR>(&units);
    if (e != cudaSuccess) return e;
    // (tiles that are cut need every unit)
    if (MODE <= ZKEEP && tiles < units) units = (int)(tiles > 0 ? tiles : 1);
    p.units = units;
    p.limit_ns = wait_limit_ns();
    withhold_hook(MODE == ZKEEP ? Z : MODE, p);
    e = launch_early(kern, dim3((unsigned)(units * Shape<PAIR>::CTAS)), THREADS, smem_bytes<PAIR>(),
                     Shape<PAIR>::CTAS, st, a, b, o, p);
    if constexpr (MODE >= DX) {
        if (e != cudaSuccess || p.cap == 0) return e;
        // tiles: of all rows, where that is known to be less than a wave
        const int64_t rem = tiles < units ? tiles : units;
        const int64_t M = MODE == DW ? p.h.V : p.h.n_live ? p.h.rows : p.h.T;
        const int rows = M < Shape<PAIR>::TILE_M ? (int)M : Shape<PAIR>::TILE_M;
        e = launch_early(head_join_kernel<MODE, PAIR>, dim3((unsigned)rem, (rows + kJoinRows - 1) / kJoinRows), 256, 0,
                         1, st, p);
    }
    return e;
}

inline int64_t tiles_of(int64_t m, int tm, int64_t n, int tn) { return (m + tm - 1) / tm * ((n + tn - 1) / tn); }

inline size_t tile_bytes(bool single) { return (size_t)(single ? BM : 2 * BM) * BN * 4; }

}  // namespace

size_t head_part_bytes(int64_t rows, int V, int d, bool single) {
    const int sms = device_sm_count();
    const size_t a = split_bound(tiles_of(rows, single ? BM : 2 * BM, d, BN), (V + BK - 1) / BK,
                                 sms / (single ? 1 : 2), 4) * tile_bytes(single);
    const size_t b = split_bound(tiles_of(V, 2 * BM, d, BN), (rows + BK - 1) / BK, sms / 2, 4) * tile_bytes(false);
    return a > b ? a : b;
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
    CUtensorMap a, b, o;
    const int64_t xrows = single && !h.n_live ? h.T : h.rows;
    p.few = single && !keep;
    p.tile_n = p.few ? head_few_tile(h.V) : BN;
    p.a_rows = single ? (int)((xrows < BM ? xrows : BM) + 7) / 8 * 8 : BM;
    if (!make_map(&a, xc, h.d, xrows, h.d, p.a_rows, kBf16) ||
        !make_map(&b, W, h.d, h.V, h.d, single ? p.tile_n : BM, kBf16))
        return cudaErrorInvalidValue;
    o = a;
    if (keep && !make_map(&o, h.P, h.Vp, h.srows, h.Vp, 32, CU_TENSOR_MAP_DATA_TYPE_FLOAT16))
        return cudaErrorInvalidValue;
    const int64_t tiles = tiles_of(single ? BM : h.rows, single ? BM : 2 * BM, h.V, p.tile_n);
    if (single) return keep ? launch_tc<ZKEEP, false>(a, b, o, p, tiles, st) : launch_tc<Z, false>(a, b, o, p, tiles, st);
    return keep ? launch_tc<ZKEEP, true>(a, b, o, p, tiles, st) : launch_tc<Z, true>(a, b, o, p, tiles, st);
}

cudaError_t launch_head_tc_dx(const HeadDev& h, const void* W, const HeadOut& out, float* part, size_t part_bytes,
                              bool single, cudaStream_t st) {
    TcParams p{};
    p.h = h;
    p.o = out;
    p.tile_n = BN;
    p.a_rows = BM;
    p.part = part;
    p.cap = (int)(part_bytes / tile_bytes(single));
    CUtensorMap a, b;
    if (!make_map(&a, h.P, h.V, h.srows, h.Vp, BM, kBf16) || !make_map(&b, W, h.d, h.V, h.d, 64, kBf16))
        return cudaErrorInvalidValue;
    const int64_t tiles = tiles_of(h.rows, single ? BM : 2 * BM, h.d, BN);
    return single ? launch_tc<DX, false>(a, b, a, p, tiles, st) : launch_tc<DX, true>(a, b, a, p, tiles, st);
}

cudaError_t launch_head_tc_dw(const HeadDev& h, const void* xc, const HeadOut& out, float* part, size_t part_bytes,
                              cudaStream_t st) {
    TcParams p{};
    p.h = h;
    p.o = out;
    p.tile_n = BN;
    p.a_rows = BM;
    p.part = part;
    p.cap = (int)(part_bytes / tile_bytes(false));
    CUtensorMap a, b, o;
    if (!make_map(&a, h.P, h.V, h.srows, h.Vp, 64, kBf16) || !make_map(&b, xc, h.d, h.rows, h.d, 64, kBf16) ||
        !make_map(&o, out.out, h.d, h.V, h.d, 32, out.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : kBf16))
        return cudaErrorInvalidValue;
    return launch_tc<DW, true>(a, b, o, p, tiles_of(h.V, 2 * BM, h.d, BN), st);
}

}  // namespace moe
