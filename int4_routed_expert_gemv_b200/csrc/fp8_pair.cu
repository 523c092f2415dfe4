// Block-scaled e4m3 products for more than 16 tokens: pairs of CTAs (cta_group::2) on tiles
// of 256 tokens by 256 weight rows.
//
// Each CTA of a pair loads 128 tokens (the MMA's M side) and 128 weight rows (half of the N
// side, which the pair's MMA reads from both), so a K step of 128 costs a CTA 32 KB for
// 128 x 256 outputs; one CTA alone would move 48 KB, which shared memory cannot feed at the
// tensor rate.  A K step is one scale block: it gets an accumulator buffer of its own in
// tensor memory, and the two warpgroups add it, times xs * ws, to sums in registers (a
// thread: one token, 128 columns) while the next K step runs.  The tokens are on the M side
// because a thread's scale is then one number per K step and 128-row block; with the
// weights there, the scales of all columns come from shared memory, and those reads, beside
// the MMA's own, took 3 times as long as everything else.
//
// The tokens of an expert lie one after another: GATE_UP reads a copy of rows and scales in list
// order, made by a launch before.  (Gathering tensor copies, four rows each, took 77 cycles a copy, 2500 a
// K step; cp.async by two warps 2000, as each hand-over to the MMA waits for the copies
// behind it.)
//
// The two row blocks of a tile: DENSE and DOWN neighbours, GATE_UP the gate and the up rows of
// the same 128 intermediate columns, which are one scale block of h.  Warpgroup g has columns
// 64 g .. of both.
//
// CTA, 12 warps:
//   warps 0-7   two warpgroups: scaled accumulation, outputs
//   warp 8      TMA producer of this CTA's tokens and weight rows
//   warp 9      tensor memory; in rank 0, with warp 11, the pair's single-thread tcgen05.mma
//               issuers, a K step each in turn
//   warp 10     briefs: looks the next tiles up for the accumulating warps, whose time it would
//               take (2500 cycles a tile)
// A part of a split tile goes to the workspace; the last one to arrive adds the parts up in
// K order (Schedule).
//
// Measured in graphs of 30 calls: 4096 x 4096 x 6144 to bf16 117 us (1.8 PFLOP/s), 16384 x 6144 x 2048 onto an fp32
// residual 310 to 340 us, GLM-shaped gate/up of 2048 tokens over 32 uneven lists 620 us (1.5 PFLOP/s of the tokens'
// products); in loops of seconds, where the power limit holds the clock down, 139, 355 and 720 us.  No one resource is
// used up (gate/up: the tensor pipe runs 42 % of the cycles, 39 % of the issue slots are taken, L2 is at 27 %).
// Left out one at a time, in us of 117 / 310 / 620: the weights' copies 112 / 295 / 577, the tokens' 113 / 285 / 589,
// the arithmetic of the accumulation 103 / 280 / 550, that and three quarters of its loads 101 / 280 / 519; for
// the second also the copies out 271, the residual 264, both of bf16 and no residual 225.  So what bounds a K step is
// the hand-over from MMA to accumulation and back, through two buffers that fill tensor memory, and where the
// outputs are wide their copies add to it.  (GATE_UP with 3 / 4 / 5 / 6 stages: 625 / 607 / 613 / 620 us.)
#include <string.h>

#include <type_traits>

#include "fp8_tiles.cuh"

namespace coli {
namespace {

using namespace fp8;

constexpr uint32_t kSite = 80;
constexpr int NT = 256;                           // tokens of a tile
constexpr int C = 128;                            // columns of a thread
constexpr uint32_t kTile = kM * 128;              // bytes of a CTA's tokens or weights per K step
constexpr uint32_t kStage = 2 * kTile;
constexpr int kBufs = 2;
constexpr uint32_t kTmem = kBufs * 256;
constexpr int kLeast = 6;                         // K steps of a run at least
constexpr int kJoin = 12;                         // what joining the parts of a tile costs, in K steps
constexpr uint32_t kOutBox = 32 * 128;            // a warp's 32 rows of 128 bytes of output

// DENSE and DOWN stage a tile's outputs, which leaves room for three stages; GATE_UP, which does not, has the four
// that took least time (above).
template <int MODE>
struct Shape {
    static constexpr int kStages = MODE == FP8_GATE_UP ? 4 : 3;
    static constexpr int kBoxes = MODE == FP8_DENSE ? 4 : MODE == FP8_DOWN ? 3 : 0;      // output boxes of a warp
    static constexpr int kGroups = MODE == FP8_DENSE ? 1 : kMaxGroups;
};

// What the accumulating warps need to know of an item, looked up by a warp of its own.
struct Brief {
    Item it;                 // it.tile < 0: no more
    int rb, expert, t0, n;   // row block, expert, first token of the group, tokens
    int base;                // first row of the group
};
constexpr int kBriefs = 4;

template <int MODE>
struct Smem {
    using S = Shape<MODE>;
    uint8_t stage[S::kStages][kStage];
    uint8_t box[kEpi / 32][S::kBoxes > 0 ? S::kBoxes : 1][S::kBoxes > 0 ? kOutBox : 16];
    uint32_t top[2][kM];                 // maxima of the SwiGLU rows, by warpgroup
    Groups<S::kGroups> groups;
    int first[S::kGroups];
    int n_groups, tiles, last;
    uint32_t tmem;
    uint64_t full[S::kStages];           // rank 0: both CTAs' tiles landed
    uint64_t empty[S::kStages];          // MMAs done with the stage
    uint64_t acc_full[kBufs];            // MMA commit
    uint64_t acc_empty[kBufs];           // rank 0: read by every accumulating warp of the pair
    uint64_t mma_done[2];
    uint64_t res[kEpi / 32];             // a warp's part of the residual landed
    uint64_t brief_full[kBriefs], brief_empty[kBriefs];
    Brief brief[kBriefs];
};
template <int MODE>
constexpr size_t kSmem = sizeof(Smem<MODE>) + 1024;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_id()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t n_clusters()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t map_to(const void* p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrival on a barrier of either CTA (a shared::cluster address).  What these barriers hand
// over is tensor memory and tiles that TMA and the MMAs touch, ordered by their own
// completion and the tcgen05 fences, so the arrival carries no cluster-wide release (a
// release there costs a fence of the thread's global accesses, 1500 cycles a K step).
__device__ __forceinline__ void arrive_pair(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Loads into this CTA that complete on a barrier of rank 0 (a shared::cluster address).
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on the barrier at this offset in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// acc[16] += v[16] * s.  Single FFMAs: packed pairs cost more in moves, since the values that
// tcgen05.ld leaves are not where pairs have to be.
__device__ __forceinline__ void scaled_add(float* acc, const uint32_t (&v)[16], float s)
{
#pragma unroll
    for (int j = 0; j < 16; j++) acc[j] = fmaf(__uint_as_float(v[j]), s, acc[j]);
}

__device__ __forceinline__ void store_box(const CUtensorMap* map, int x, int y, int z, const void* src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
                 "r"(z), "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Until at most N of this thread's stores have still to read their boxes.
template <int N = 0>
__device__ __forceinline__ void boxes_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// The columns of a warp's output: two runs of 64, at c0 and c0 + 128, in boxes of 128 bytes a row.
template <class Y>
struct Boxes {
    static constexpr int W = 128 / (int)sizeof(Y), N = C / W;
    __device__ static __forceinline__ int column(int c0, int j) { return c0 + j / (N / 2) * kM + j % (N / 2) * W; }
};

// One lane: the warp's part of the residual (rows from y0) into its boxes, once the stores before
// have read them.
template <class Y>
__device__ __forceinline__ void ask_residual(const Params& p, int c0, int y0, uint8_t* box, uint64_t* bar)
{
    boxes_read();
    uint32_t bytes = 0;
#pragma unroll
    for (int j = 0; j < Boxes<Y>::N; j++) bytes += Boxes<Y>::column(c0, j) < p.rows ? kOutBox : 0;
    mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int j = 0; j < Boxes<Y>::N; j++)
        if (Boxes<Y>::column(c0, j) < p.rows) tma_load_3d(box + j * kOutBox, &p.res, Boxes<Y>::column(c0, j), y0, 0, bar);
}

// A warp's 32 rows of outputs, one per thread, to rows from y0 of the map (rows and columns
// beyond its end are left out), plus the residual that its boxes hold, rounded once.  The copies
// out run while the next tile's sums are formed.  With `ragged`, the first `left` rows only, by
// the warp itself: the rows behind them are another tile's.
template <class Y, bool RES, int NB>
__device__ __forceinline__ void store_boxes(const CUtensorMap* map, int c0, int y0, int z, int rows, const float (&acc)[C],
                                            uint8_t* box, int lane, Y* ragged = nullptr, int left = 32)
{
    constexpr int ES = (int)sizeof(Y), W = Boxes<Y>::W, N = Boxes<Y>::N;
    if (!RES) {
        if (lane == 0) boxes_read<0>();
        __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < N; j++) {
        if (Boxes<Y>::column(c0, j) >= rows) break;       // and all later ones
        if (j >= NB) {
            if (lane == 0) boxes_read<NB - 1>();
            __syncwarp();
        }
        uint8_t* mine = box + (j % NB) * kOutBox + lane * 128;
#pragma unroll
        for (int c = 0; c < 8; c++) {
            uint4* at = reinterpret_cast<uint4*>(mine + ((c ^ (lane & 7)) << 4));      // 128-byte swizzle
            const uint4 u = RES ? *at : make_uint4(0, 0, 0, 0);
            const uint32_t r[4] = {u.x, u.y, u.z, u.w};
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (ES == 4) {
                    const float f = acc[j * W + 4 * c + e];
                    w[e] = __float_as_uint(RES ? f + __uint_as_float(r[e]) : f);
                } else {
                    float lo = acc[j * W + 8 * c + 2 * e], hi = acc[j * W + 8 * c + 2 * e + 1];
                    if (RES) {
                        lo += __uint_as_float(r[e] << 16);
                        hi += __uint_as_float(r[e] & 0xFFFF0000u);
                    }
                    w[e] = bf16x2_bits(lo, hi);
                }
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (ragged) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int r = i * 4 + (lane >> 3), piece = lane & 7;
                const uint4 v = *reinterpret_cast<const uint4*>(box + (j % NB) * kOutBox + r * 128 + ((piece ^ (r & 7)) << 4));
                if (r < left)
                    *reinterpret_cast<uint4*>(ragged + (size_t)(y0 + r) * rows + Boxes<Y>::column(c0, j) + piece * (16 / ES)) = v;
            }
            __syncwarp();
            continue;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) store_box(map, Boxes<Y>::column(c0, j), y0, z, box + (j % NB) * kOutBox);
    }
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ Params p)
{
    using S = Shape<MODE>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the same offset in both CTAs of the pair: dynamic shared memory starts at one address in
    // every CTA of a launch
    Smem<MODE>& sm =
        *reinterpret_cast<Smem<MODE>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();
    if (tid == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < kBufs; b++) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], 2 * kEpi / 32);
        }
        mbar_init(&sm.mma_done[0], 1);
        mbar_init(&sm.mma_done[1], 1);
        for (int w = 0; w < kEpi / 32; w++) mbar_init(&sm.res[w], 1);
        for (int b = 0; b < kBriefs; b++) {
            mbar_init(&sm.brief_full[b], 1);
            mbar_init(&sm.brief_empty[b], kEpi / 32);
        }
        fence_barrier_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_launch_dependents();
    pdl_wait();
    if (warp == 8) {
        const int ng = read_groups<MODE>(p, lane, sm.groups);
        const int tiles = plan_tiles(p, sm.groups, ng, NT, lane, sm.first);
        if (lane == 0) {
            sm.n_groups = ng;
            sm.tiles = tiles;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int n_groups = sm.n_groups;
    Schedule sch;
    sch.init(sm.tiles, p.kb, (int)n_clusters(), (int)cluster_id(), kLeast, kJoin, p.slices);
    bool dead = false;
    Item it;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 8) {
            // ----------------------------- TMA producer ---------------------------------
            uint32_t n = 0, sent = 0;
            while (sch.next(it)) {
                const Tile tl = tile_of(p, sm.groups, sm.first, n_groups, NT, it.tile);
                const int shared = tl.g.expert < 0 ? 1 : 0;
                const CUtensorMap* wm = &p.w[shared];
                const CUtensorMap* xm = &p.x[MODE == FP8_GATE_UP ? shared : 0];
                const int z = shared ? 0 : tl.g.expert;
                const int r0 = MODE == FP8_GATE_UP ? tl.rb * kM + rank * p.I : (tl.rb * 2 + rank) * kM;
                const int n1 = max(tl.n - kM, 0);      // token rows of rank 1
                const bool tokens = rank == 0 || n1 > 0;
                const uint32_t bytes = (n1 > 0 ? 4 : 3) * kTile;
                const int base = MODE == FP8_DENSE || (MODE == FP8_GATE_UP && shared) ? 0 : tl.g.base;
                const int row0 = base + tl.t0 + rank * kM;
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int s = n % kStages;
                    warp_wait(dead, &sm.empty[s], ((n / kStages) & 1) ^ 1, p.status, kSite + 1);
                    if (dead) continue;
                    sent = n + 1;
                    if (lane == 0) {
                        uint8_t* st = sm.stage[s];
                        const uint32_t bar = map_to(&sm.full[s], 0);
                        if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], bytes);
                        pair_load_3d(st + kTile, wm, kb * 128, r0, z, bar);
                        if (tokens) pair_load_2d(st, xm, kb * 128, row0, bar);
                    }
                    __syncwarp();
                }
            }
            // no copy of the pair is in flight when it ends
            if (lane == 0 && rank == 0) drain(sm.full, kStages, sent, p.status, kSite + 2);
        } else if (warp == 9 || warp == 11) {
            // ----------------------------- MMA issuers -----------------------------------
            // K steps alternate between the two: an issuer is held up until its MMAs have nearly
            // run, and the other waits for the next step's barriers meanwhile.  (256 columns an
            // MMA: two of 128, with buffers of their own, took as long each.)
            if (lane == 0 && rank == 0) {
                const uint32_t idesc = idesc_e4m3(2 * kM, 2 * kM), odd = warp == 11;
                uint32_t n = 0;
                while (sch.next(it)) {
                    for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                        if ((n & 1) != odd) continue;
                        const int s = n % kStages, b = n % kBufs;
                        const uint8_t* st = sm.stage[s];
                        const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + kTile);
                        // In this order: with three stages an issuer sees every other phase of full[s] only, and a
                        // parity alone cannot tell step n from step n - 6.  The buffer's hand-back says
                        // that step n - 2 has been added up, hence that step n - 3, the stage's last, had landed.
                        lane_wait(dead, &sm.acc_empty[b], ((n / kBufs) & 1) ^ 1, p.status, kSite + 3);
                        lane_wait(dead, &sm.full[s], (n / kStages) & 1, p.status, kSite + 4);
                        tc_fence_after();
                        if (!dead) {
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)      // 32 e4m3 values = 32 bytes per MMA
                                umma_pair(tmem + (uint32_t)(b * 256), ad + 2 * kk, bd + 2 * kk, idesc, kk != 0);
                        }
                        commit_pair(&sm.acc_full[b]);
                        commit_pair(&sm.empty[s]);
                    }
                }
                commit_pair(&sm.mma_done[odd]);
                mbar_wait(&sm.mma_done[odd], 0, p.status, kSite + 5);
            }
        } else if (warp == 10) {
            // ------------------------------- briefs -----------------------------------------
            uint32_t m = 0;
            for (bool more = true; more; m++) {
                const int slot = m % kBriefs;
                more = sch.next(it);
                Tile tl{};
                if (more) tl = tile_of(p, sm.groups, sm.first, n_groups, NT, it.tile);
                warp_wait(dead, &sm.brief_empty[slot], ((m / kBriefs) & 1) ^ 1, p.status, kSite + 11);
                if (lane == 0 && !dead) {      // (a slot that was not handed back may still be read)
                    if (!more) it.tile = -1;
                    sm.brief[slot] = Brief{it, tl.rb, tl.g.expert, tl.t0, tl.n, tl.g.base};
                    mbar_arrive(&sm.brief_full[slot]);
                }
                __syncwarp();
                if (MODE == FP8_DOWN && more && tl.rb == 0 && it.kb0 == 0 && tl.g.expert >= 0)
                    for (int j = rank * kM + lane; j < min(tl.n, (rank + 1) * kM); j += 32) place_row(p, tl.g.base + tl.t0 + j);
            }
        }
    } else {
        // ------------------------- scaled accumulation, outputs -------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int wg = warp >> 2, q = warp & 3;     // warpgroup, tensor memory lane quarter
        const int row = q * 32 + lane;              // token within the CTA's 128
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
        float acc[C];
        uint32_t asked = 0, briefs = 0;             // residual parts asked for, briefs read
        uint32_t n = 0;
        const uint32_t ae = map_to(&sm.acc_empty[0], 0);
        const int nb = fp8_blocks(p.rows);
        // What a tile needs besides its sums.  The next tile's brief is taken, and its first scales
        // are on their way, before this one's outputs are written.
        struct Work {
            Item it;
            int rb, expert, left;        // row block, expert, tokens of this warp
            int xrow, orow;              // row of the token's scales, row of y / h / z (-1: none)
            int y0;                      // the warp's first row of y / z
        };
        float xn[4], an[4], bn[4];       // scales of four K steps: token, both row blocks
        auto fetch = [&](const Work& w, int kb) {      // kb: a multiple of 4
            const float* xs = (MODE == FP8_GATE_UP && w.expert < 0 ? p.xs_shared : p.xs) + (size_t)w.xrow * p.kb;
            const float* wa = w.expert < 0 ? p.ws[1]
                                           : reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(p.ws[0]) +
                                                                            (uint64_t)w.expert * p.ws_stride);
            wa += (size_t)(MODE == FP8_GATE_UP ? w.rb : 2 * w.rb) * p.kb;
            const float* wb = MODE == FP8_GATE_UP ? wa + (size_t)nb * p.kb : 2 * w.rb + 1 < nb ? wa + p.kb : wa;
            if (p.kb % 4 == 0) {
                // a row's four in one load: 32 rows a warp are 32 accesses either way
                const float4 x = *reinterpret_cast<const float4*>(xs + kb);
                const float4 a = __ldg(reinterpret_cast<const float4*>(wa + kb));
                const float4 b = __ldg(reinterpret_cast<const float4*>(wb + kb));
                xn[0] = x.x, xn[1] = x.y, xn[2] = x.z, xn[3] = x.w;
                an[0] = a.x, an[1] = a.y, an[2] = a.z, an[3] = a.w;
                bn[0] = b.x, bn[1] = b.y, bn[2] = b.z, bn[3] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int k = min(kb + i, p.kb - 1);
                    xn[i] = xs[k];
                    an[i] = __ldg(wa + k);
                    bn[i] = __ldg(wb + k);
                }
            }
        };
        auto look_up = [&](Work& w) {
            const int slot = briefs % kBriefs;
            warp_wait(dead, &sm.brief_full[slot], (briefs / kBriefs) & 1, p.status, kSite + 12);
            const Brief tl = sm.brief[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.brief_empty[slot]);
            briefs++;
            if (dead) {
                // no brief any more: the same items, without tokens, since the other warps wait for this one
                // at named barriers
                w.left = 0;
                w.orow = -1;         // (the rest goes unread)
                Schedule again;      // (made here: registers are dear)
                again.init(sm.tiles, p.kb, (int)n_clusters(), (int)cluster_id(), kLeast, kJoin, p.slices);
                return again.at((int)briefs - 1, w.it);
            }
            if (tl.it.tile < 0) return false;
            w.it = tl.it;
            w.rb = tl.rb;
            w.expert = tl.expert;
            w.left = tl.n - rank * kM - q * 32;
            const int tok = tl.t0 + rank * kM + row;            // token of the group
            w.xrow = 0;
            w.orow = -1;
            w.y0 = (MODE == FP8_DENSE ? 0 : tl.base) + tok - lane;
            if (lane < w.left) {
                if (MODE == FP8_DENSE) {
                    w.xrow = w.orow = tok;
                } else if (tl.expert < 0) {
                    w.xrow = MODE == FP8_DOWN ? tl.base + tok : tok;
                    w.orow = tl.base + tok;
                } else {
                    w.xrow = w.orow = tl.base + tok;      // GATE_UP's scales are in list order too
                }
            }
            if (w.left > 0) fetch(w, w.it.kb0 & ~3);
            return true;
        };
        // (DENSE has more to write, and the registers are dear: there it is taken when due.)
        constexpr bool kAhead = MODE != FP8_DENSE;
        Work next;
        bool more = kAhead ? look_up(next) : true;
        while (more) {
            if (!kAhead && !look_up(next)) break;
            const Work w = next;
            const int left = w.left;
            it = w.it;
#pragma unroll
            for (int j = 0; j < C; j++) acc[j] = 0.0f;
            // the residual of a whole tile is asked for a few steps into it, when the stores of
            // the tile before have read the boxes
            const int c0 = 2 * w.rb * kM + wg * 64;       // output columns: two runs of 64
            bool ask = MODE == FP8_DENSE && p.residual && p.slices == 1 && left > 0;
            auto ask_now = [&]() {
                if (lane == 0) {
                    if (p.y_bf16) ask_residual<__nv_bfloat16>(p, c0, w.y0, sm.box[warp][0], &sm.res[warp]);
                    else ask_residual<float>(p, c0, w.y0, sm.box[warp][0], &sm.res[warp]);
                }
                __syncwarp();
                ask = false;
                asked++;
            };
            const bool whole = it.kb1 - it.kb0 == p.kb;
            if (left > 0) {
                // scales of four K steps at a time, fetched four steps ahead
                for (int kb = it.kb0 & ~3; kb < it.kb1; kb += 4) {
                    float sa[4], sb[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        sa[i] = xn[i] * an[i];
                        sb[i] = xn[i] * bn[i];
                    }
                    if (kb + 4 < it.kb1) fetch(w, kb + 4);
                    if constexpr (MODE == FP8_DENSE)
                        if (ask && whole && kb > it.kb0) ask_now();
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (kb + i < it.kb0 || kb + i >= it.kb1) continue;
                        const int b = n % kBufs;
                        warp_wait(dead, &sm.acc_full[b], (n / kBufs) & 1, p.status, kSite + 7);
                        tc_fence_after();
                        const uint32_t ta = lane_addr + (uint32_t)(b * 256 + wg * 64);
                        // loads run one chunk of 16 columns ahead of the arithmetic
                        uint32_t v[2][16];
                        tmem_ld16(ta, v[0]);
#pragma unroll
                        for (int c = 0; c < 8; c++) {
                            tmem_wait_ld(v[c & 1]);
                            if (c < 7) tmem_ld16(ta + (c + 1) * 16 + (c >= 3 ? 64 : 0), v[(c + 1) & 1]);
                            else {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) arrive_pair(ae + b * 8);
                            }
                            scaled_add(acc + c * 16, v[c & 1], c < 4 ? sa[i] : sb[i]);
                        }
                        n++;
                    }
                }
            } else {
                // no token in this warp: only hand the buffers on
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int b = n % kBufs;
                    warp_wait(dead, &sm.acc_full[b], (n / kBufs) & 1, p.status, kSite + 7);
                    __syncwarp();
                    if (lane == 0) arrive_pair(ae + b * 8);
                }
            }
            if (kAhead) more = look_up(next);
            if (!whole && p.slices == 1) {
                // store the sums; the last part to arrive adds all of them up
                const int o0 = sch.owner(it.tile * p.kb), o1 = sch.owner(it.tile * p.kb + p.kb - 1);
                float4* dst = reinterpret_cast<float4*>(p.partial) +
                              ((size_t)(2 * sch.c + (it.kb0 == 0 ? 1 : 0)) * 2 + rank) * (C / 4) * kEpi + tid;
                if (left > 0) {
#pragma unroll
                    for (int j = 0; j < C / 4; j++) {
                        __stcg(dst + j * kEpi, make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]));
                    }
                }
                named_bar(1, kEpi);
                if (tid == 0) sm.last = arrive_last(&p.tickets[2 * o0 + rank], (uint32_t)(o1 - o0 + 1));
                named_bar(1, kEpi);
                if (!sm.last) continue;
                if (left > 0) {
#pragma unroll
                    for (int j = 0; j < C; j++) acc[j] = 0.0f;
                    for (int o = o0; o <= o1; o++) {
                        const float4* src = reinterpret_cast<const float4*>(p.partial) +
                                            ((size_t)(2 * o + (o == o0 ? 1 : 0)) * 2 + rank) * (C / 4) * kEpi + tid;
#pragma unroll
                        for (int j = 0; j < C / 4; j++) {
                            const float4 f = __ldcg(src + (size_t)j * kEpi);
                            acc[4 * j] += f.x;
                            acc[4 * j + 1] += f.y;
                            acc[4 * j + 2] += f.z;
                            acc[4 * j + 3] += f.w;
                        }
                    }
                }
            }
            if (MODE != FP8_GATE_UP) {
                if (left <= 0) continue;
                constexpr int NB = S::kBoxes > 0 ? S::kBoxes : 1;
                if (MODE == FP8_DOWN) {
                    // (H is a multiple of 64: a box has all of its columns)
                    store_boxes<float, false, NB>(&p.out, c0, w.y0, 0, p.rows, acc, sm.box[warp][0], lane,
                                                  left < 32 ? p.z : nullptr, left);
                } else if (p.slices > 1) {
                    store_boxes<float, false, NB>(&p.out, c0, w.y0, it.slice, p.pitch, acc, sm.box[warp][0], lane);
                } else if (p.residual) {
                    if (ask && !dead) ask_now();
                    warp_wait(dead, &sm.res[warp], (asked - 1) & 1, p.status, kSite + 9);
                    if (dead) continue;       // the boxes may still be written to
                    if (p.y_bf16) store_boxes<__nv_bfloat16, true, NB>(&p.out, c0, w.y0, 0, p.rows, acc, sm.box[warp][0], lane);
                    else store_boxes<float, true, NB>(&p.out, c0, w.y0, 0, p.rows, acc, sm.box[warp][0], lane);
                } else {
                    if (p.y_bf16) store_boxes<__nv_bfloat16, false, NB>(&p.out, c0, w.y0, 0, p.rows, acc, sm.box[warp][0], lane);
                    else store_boxes<float, false, NB>(&p.out, c0, w.y0, 0, p.rows, acc, sm.box[warp][0], lane);
                }
            } else {
                // SwiGLU of 64 columns; the scale block is this and the other warpgroup's
                uint32_t top = 0;
                if (left > 0 && w.rb * kM + wg * 64 < p.I) {            // I is a multiple of 64
#pragma unroll
                    for (int j = 0; j < 64; j++) {
                        acc[j] = swiglu(acc[j], acc[64 + j]);
                        top = max(top, __float_as_uint(acc[j]) & 0x7FFFFFFFu);
                    }
                }
                sm.top[wg][row] = top;
                named_bar(1, kEpi);
                top = max(top, sm.top[wg ^ 1][row]);
                named_bar(1, kEpi);      // read before the next tile's
                const Quantizer qz(top);
                const int i0 = w.rb * kM + wg * 64;
                if (w.orow >= 0 && i0 < p.I) {
                    uint4* to = reinterpret_cast<uint4*>(p.hq + (size_t)w.orow * p.I + i0);
#pragma unroll
                    for (int j = 0; j < 64; j += 16) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const float* f = acc + j + 4 * e;
                            w[e] = qz.codes(f[0], f[1]) | qz.codes(f[2], f[3]) << 16;
                        }
                        to[j / 16] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (wg == 0) p.hs[(size_t)w.orow * nb + w.rb] = qz.scale;
                }
            }
        }
        // this warp's copies, in and out, are complete
        if (lane == 0) {
            if (asked) mbar_wait(&sm.res[warp], (asked - 1) & 1, p.status, kSite + 10);
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    // The commits' arrivals in rank 1 have all come before it ends.  (Its sums are formed by now, so the last MMAs
    // are done; from the start on this wait would give up in a launch that takes longer than its limit.)
    if (rank == 1 && tid < 2) mbar_wait(&sm.mma_done[tid], 0, p.status, kSite + 6);
    __syncwarp();
    cluster_sync();        // the other CTA's barriers and tiles stay in use until here
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

template <int MODE>
cudaError_t launch(const Params& p, int grid, cudaStream_t s)
{
    const cudaError_t e = allow_smem<fp8_pair_kernel<MODE>>(kSmem<MODE>);
    if (e != cudaSuccess) return e;
    return launch_early<fp8_pair_kernel<MODE>>(grid, kThreads, kSmem<MODE>, s, p);
}

}  // namespace

cudaError_t fp8_pair_launch(int mode, const fp8::Params& p, int num_sms, cudaStream_t s)
{
    const int grid = (num_sms < kFp8Ctas ? num_sms : kFp8Ctas) / 2 * 2;
    return mode == FP8_DENSE     ? launch<FP8_DENSE>(p, grid, s)
           : mode == FP8_GATE_UP ? launch<FP8_GATE_UP>(p, grid, s)
                                 : launch<FP8_DOWN>(p, grid, s);
}

}  // namespace coli
