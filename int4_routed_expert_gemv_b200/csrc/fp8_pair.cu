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
// The two row blocks of a tile: DENSE and DOWN neighbours (warpgroup g has block g), GATE_UP
// the gate and the up rows of the same 128 intermediate columns, which are one scale block of
// h (warpgroup g has columns 64 g .. of both).
//
// CTA, 10 warps of use in 12:
//   warps 0-7   two warpgroups: scaled accumulation, outputs
//   warp 8      TMA producer of this CTA's tokens (rows one after another, or gathered by the
//               union lists) and weight rows
//   warp 9      tensor memory; in rank 0 the pair's single-thread tcgen05.mma issuer
// A part of a split tile goes to the workspace; the last one to arrive adds the parts up in
// K order (Schedule).
#include <string.h>

#include "fp8_tiles.cuh"

namespace coli {
namespace {

using namespace fp8;

constexpr uint32_t kSite = 80;
constexpr int NT = 256;                           // tokens of a tile
constexpr int C = 128;                            // columns of a thread
constexpr uint32_t kTile = kM * 128;              // bytes of a CTA's tokens or weights per K step
constexpr uint32_t kStage = 2 * kTile;
constexpr int kStages = 6;
constexpr int kBufs = 2;
constexpr uint32_t kTmem = kBufs * 256;
constexpr int kBox = 64;                          // rows of a token box
constexpr int kLeast = 6;                         // K steps of a run at least
constexpr int kPad = 20;                          // floats of a staged row: 16 and a gap
constexpr size_t kOut = (size_t)(kEpi / 32) * 32 * kPad * 4;
constexpr size_t kSmem = 1024 + kStages * (size_t)kStage + kOut + 2 * kM * 4 + (kMaxGroups + 3) / 4 * 4 * 4 + 16 + 256;

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

// Four rows of a 2-D map (box one row high) into four consecutive 128-byte rows.
__device__ __forceinline__ void pair_gather4(void* dst, const CUtensorMap* map, int x, int4 y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar)
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

__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}

// acc[16 pairs] += v[32] * s
__device__ __forceinline__ void scaled_add(uint64_t* acc, const uint32_t (&v)[32], uint64_t s)
{
#pragma unroll
    for (int j = 0; j < 32; j += 2) acc[j / 2] = ffma2(pk2(v[j], v[j + 1]), s, acc[j / 2]);
}

// 16 columns of a warp's 32 rows, from a thread's own row to rows written side by side: calls
// put(row, column, float4) with 4 consecutive columns.
template <class Put>
__device__ __forceinline__ void through_smem(float* stage, const float* v, int lane, Put put)
{
#pragma unroll
    for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4*>(stage + lane * kPad + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = i * 8 + (lane >> 2), c = (lane & 3) * 4;
        put(i, r, c, *reinterpret_cast<const float4*>(stage + r * kPad + c));
    }
    __syncwarp();
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ Params p)
{
    constexpr bool kGather = MODE == FP8_GATE_UP;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the same offset in both CTAs of the pair: dynamic shared memory starts at one address in
    // every CTA of a launch
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* out_stage = reinterpret_cast<float*>(smem + kStages * (size_t)kStage);
    uint32_t* tops = reinterpret_cast<uint32_t*>(out_stage + kOut / 4);      // [2][kM] maxima of the SwiGLU rows
    int* first = reinterpret_cast<int*>(tops + 2 * kM);
    int* flags = first + (kMaxGroups + 3) / 4 * 4;         // [0] groups [1] tiles [2] last part [3] tensor memory
    uint64_t* bars = reinterpret_cast<uint64_t*>(flags + 4);
    uint64_t* full = bars;                       // [kStages] rank 0: both CTAs' tiles landed
    uint64_t* empty = full + kStages;            // [kStages] MMAs done with the stage
    uint64_t* acc_full = empty + kStages;        // [kBufs] MMA commit
    uint64_t* acc_empty = acc_full + kBufs;      // [kBufs] rank 0: read by every accumulating warp of the pair
    uint64_t* mma_done = acc_empty + kBufs;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();
    if (tid == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kBufs; b++) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEpi / 32);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&flags[3])),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == 8) plan_tiles<MODE>(p, NT, lane, first, &flags[0], &flags[1]);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];
    const int n_groups = flags[0];
    Schedule sch;
    sch.init(flags[1], p.kb, (int)n_clusters(), (int)cluster_id(), kLeast);
    bool dead = false;
    Item it;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            // ----------------------------- TMA producer ---------------------------------
            uint32_t n = 0;
            while (sch.next(it)) {
                const Tile tl = tile_of<MODE>(p, first, n_groups, NT, it.tile);
                const int shared = tl.g.expert < 0 ? 1 : 0;
                const CUtensorMap* wm = &p.w[shared];
                const int z = shared ? 0 : tl.g.expert;
                const int r0 = MODE == FP8_GATE_UP ? tl.rb * kM + rank * p.I : (tl.rb * 2 + rank) * kM;
                // token rows of each CTA; copies come in boxes or in gathered fours
                const int n0 = min(tl.n, kM), n1 = tl.n - n0, mine = rank ? n1 : n0;
                const int unit = kGather ? 4 : kBox;
                const int copies = (mine + unit - 1) / unit;
                const uint32_t bytes = 2 * kTile + (uint32_t)((n0 + unit - 1) / unit + (n1 + unit - 1) / unit) * unit * 128;
                int4 rows = make_int4(0, 0, 0, 0);
                if (kGather && lane < copies) {
                    int* rr = reinterpret_cast<int*>(&rows);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int i = tl.t0 + rank * kM + min(4 * lane + j, mine - 1);
                        const int a = shared ? i * p.k : position_of(p, tl.g.base + i);
                        if (a < 0) set_flag(p.status, DEV_BAD_INDEX);
                        rr[j] = max(a, 0) / p.k;
                    }
                }
                const int row0 = (MODE == FP8_DENSE ? tl.t0 : tl.g.base + tl.t0) + rank * kM;
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int s = n % kStages;
                    if (!dead && !mbar_wait(&empty[s], ((n / kStages) & 1) ^ 1, p.status, kSite + 1)) dead = true;
                    if (dead) continue;
                    uint8_t* st = smem + (size_t)s * kStage;
                    const uint32_t bar = map_to(&full[s], 0);
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                        pair_load_3d(st + kTile, wm, kb * 128, r0, z, bar);
                        if (!kGather)
                            for (int b = 0; b < copies; b++)
                                pair_load_2d(st + b * kBox * 128, &p.x, kb * 128, row0 + b * kBox, bar);
                    }
                    __syncwarp();
                    if (kGather && lane < copies) pair_gather4(st + lane * 512, &p.x, kb * 128, rows, bar);
                }
            }
            // no copy of the pair is in flight when it ends
            if (lane == 0 && rank == 0) {
                const uint32_t last = n < (uint32_t)kStages ? n : (uint32_t)kStages;
                for (uint32_t i = 0; i < last; i++) {
                    const uint32_t m = n - 1 - i;
                    mbar_wait(&full[m % kStages], (m / kStages) & 1, p.status, kSite + 2);
                }
            }
        } else if (warp == 9) {
            // ----------------------------- MMA issuer -----------------------------------
            if (lane == 0 && rank == 0) {
                const uint32_t idesc = idesc_e4m3(2 * kM, 2 * kM);
                uint32_t n = 0;
                while (sch.next(it)) {
                    for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                        const int s = n % kStages, b = n % kBufs;
                        if (!dead && !mbar_wait(&acc_empty[b], ((n / kBufs) & 1) ^ 1, p.status, kSite + 3)) dead = true;
                        if (!dead && !mbar_wait(&full[s], (n / kStages) & 1, p.status, kSite + 4)) dead = true;
                        tc_fence_after();
                        if (!dead) {
                            const uint8_t* st = smem + (size_t)s * kStage;
                            const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + kTile);
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)      // 32 e4m3 values = 32 bytes per MMA
                                umma_pair(tmem + (uint32_t)(b * 256), ad + 2 * kk, bd + 2 * kk, idesc, kk != 0);
                        }
                        commit_pair(&empty[s]);
                        commit_pair(&acc_full[b]);
                    }
                }
                commit_pair(mma_done);
                mbar_wait(mma_done, 0, p.status, kSite + 5);
            }
        }
    } else {
        // ------------------------- scaled accumulation, outputs -------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int wg = warp >> 2, q = warp & 3;     // warpgroup, tensor memory lane quarter
        const int row = q * 32 + lane;              // token within the CTA's 128
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
        // columns of the thread: two runs of 64
        const uint32_t ca = (uint32_t)(MODE == FP8_GATE_UP ? wg * 64 : wg * 128);
        const uint32_t cb = (uint32_t)(MODE == FP8_GATE_UP ? 128 + wg * 64 : wg * 128 + 64);
        uint64_t acc[C / 2];
        float* accf = reinterpret_cast<float*>(acc);
        float* stage = out_stage + warp * 32 * kPad;
        uint32_t n = 0;
        const uint32_t ae = map_to(&acc_empty[0], 0);
        const int nb = fp8_blocks(p.rows);
        while (sch.next(it)) {
            const Tile tl = tile_of<MODE>(p, first, n_groups, NT, it.tile);
            const int left = tl.n - rank * kM - q * 32;         // tokens of this warp
            const int tok = tl.t0 + rank * kM + row;            // token of the group
            const bool valid = lane < left;
            // row of x, and where the outputs go: row of y / h, or of z (-1: nowhere)
            int xrow = MODE == FP8_DENSE || tl.g.expert < 0 ? tok : 0, orow = valid ? tok : -1;
            if (MODE != FP8_DENSE && valid) {
                const int a = tl.g.expert < 0 ? 0 : position_of(p, tl.g.base + tok);
                if (MODE == FP8_DOWN) {
                    xrow = tl.g.base + tok;
                    orow = tl.g.expert < 0 ? xrow : a;
                    if (a < 0) set_flag(p.status, DEV_BAD_INDEX);
                    else if (tl.g.expert >= 0 && tl.rb == 0 && wg == 0) p.present[a] = 1;
                } else {
                    if (tl.g.expert >= 0) xrow = max(a, 0) / p.k;
                    orow = tl.g.base + tok;
                }
            }
            const float* xs = p.xs + (size_t)(valid ? xrow : 0) * p.kb;
            const float* wbase = tl.g.expert < 0
                                     ? p.ws[1]
                                     : reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(p.ws[0]) +
                                                                      (uint64_t)tl.g.expert * p.ws_stride);
            const int blk = MODE == FP8_GATE_UP ? tl.rb : min(2 * tl.rb + wg, nb - 1);
            const float* wa = wbase + (size_t)blk * p.kb;
            const float* wb = MODE == FP8_GATE_UP ? wa + (size_t)nb * p.kb : wa;
#pragma unroll
            for (int j = 0; j < C / 2; j++) acc[j] = 0;
            if (left > 0) {
                float x1 = __ldg(xs + it.kb0), a1 = __ldg(wa + it.kb0), b1 = MODE == FP8_GATE_UP ? __ldg(wb + it.kb0) : 0.0f;
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int b = n % kBufs;
                    const float sa = x1 * a1, sb = MODE == FP8_GATE_UP ? x1 * b1 : sa;
                    if (kb + 1 < it.kb1) {       // the next step's scales
                        x1 = __ldg(xs + kb + 1);
                        a1 = __ldg(wa + kb + 1);
                        if (MODE == FP8_GATE_UP) b1 = __ldg(wb + kb + 1);
                    }
                    if (!dead && !mbar_wait(&acc_full[b], (n / kBufs) & 1, p.status, kSite + 7)) dead = true;
                    tc_fence_after();
                    const uint32_t ta = lane_addr + (uint32_t)(b * 256);
                    // loads run one chunk of 32 columns ahead of the arithmetic
                    uint32_t v0[32], v1[32];
                    tmem_ld32(ta + ca, v0);
                    tmem_wait_ld();
                    tmem_ld32(ta + ca + 32, v1);
                    scaled_add(acc, v0, pk2f(sa, sa));
                    tmem_wait_ld();
                    tmem_ld32(ta + cb, v0);
                    scaled_add(acc + 16, v1, pk2f(sa, sa));
                    tmem_wait_ld();
                    tmem_ld32(ta + cb + 32, v1);
                    scaled_add(acc + 32, v0, pk2f(sb, sb));
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_pair(ae + b * 8);
                    scaled_add(acc + 48, v1, pk2f(sb, sb));
                }
            } else {
                // no token in this warp: only hand the buffers on
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int b = n % kBufs;
                    if (!dead && !mbar_wait(&acc_full[b], (n / kBufs) & 1, p.status, kSite + 7)) dead = true;
                    __syncwarp();
                    if (lane == 0) arrive_pair(ae + b * 8);
                }
            }
            if (it.kb1 - it.kb0 < p.kb) {
                // store the sums; the last part to arrive adds all of them up
                const int o0 = sch.owner(it.tile * p.kb), o1 = sch.owner(it.tile * p.kb + p.kb - 1);
                float4* dst = reinterpret_cast<float4*>(p.partial) +
                              ((size_t)(2 * sch.c + (it.kb0 == 0 ? 1 : 0)) * 2 + rank) * (C / 4) * kEpi + tid;
                if (left > 0) {
#pragma unroll
                    for (int j = 0; j < C / 4; j++) {
                        const float2 a = unpk2(acc[2 * j]), b2 = unpk2(acc[2 * j + 1]);
                        __stcg(dst + j * kEpi, make_float4(a.x, a.y, b2.x, b2.y));
                    }
                }
                __threadfence();
                named_bar(1, kEpi);
                if (tid == 0) {
                    uint32_t* t = &p.tickets[2 * o0 + rank];
                    const bool last = atomicAdd(t, 1u) == (uint32_t)(o1 - o0);
                    if (last) *t = 0;
                    flags[2] = last;
                }
                named_bar(1, kEpi);
                if (!flags[2]) continue;
                __threadfence();
                if (left > 0) {
#pragma unroll
                    for (int j = 0; j < C / 2; j++) acc[j] = 0;
                    for (int o = o0; o <= o1; o++) {
                        const float4* src = reinterpret_cast<const float4*>(p.partial) +
                                            ((size_t)(2 * o + (o == o0 ? 1 : 0)) * 2 + rank) * (C / 4) * kEpi + tid;
#pragma unroll
                        for (int j = 0; j < C / 4; j++) {
                            const float4 f = __ldcg(src + (size_t)j * kEpi);
                            acc[2 * j] = fadd2(acc[2 * j], pk2f(f.x, f.y));
                            acc[2 * j + 1] = fadd2(acc[2 * j + 1], pk2f(f.z, f.w));
                        }
                    }
                }
            }
            if (MODE != FP8_GATE_UP) {
                if (left <= 0) continue;
                const int c0 = (2 * tl.rb + wg) * kM;            // first output column
                const bool vec = p.rows % 4 == 0;
#pragma unroll
                for (int j0 = 0; j0 < C; j0 += 16) {
                    through_smem(stage, accf + j0, lane, [&](int, int r, int c, float4 v) {
                        const int to = __shfl_sync(0xffffffffu, orow, r);
                        const int col = c0 + j0 + c;
                        if (to < 0 || col >= p.rows) return;
                        const size_t o = (size_t)to * p.rows + col;
                        float f[4] = {v.x, v.y, v.z, v.w};
                        if (MODE == FP8_DOWN) {
                            *reinterpret_cast<float4*>(p.z + o) = v;
                        } else if (p.y_bf16) {
                            __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(p.y) + o;
                            const __nv_bfloat16* res = reinterpret_cast<const __nv_bfloat16*>(p.residual) + o;
                            if (vec) {
                                if (p.residual) {
                                    const uint2 u = *reinterpret_cast<const uint2*>(res);
                                    f[0] += __uint_as_float(u.x << 16);
                                    f[1] += __uint_as_float(u.x & 0xFFFF0000u);
                                    f[2] += __uint_as_float(u.y << 16);
                                    f[3] += __uint_as_float(u.y & 0xFFFF0000u);
                                }
                                *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]));
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    if (col + e < p.rows)
                                        y[e] = __float2bfloat16_rn(f[e] + (p.residual ? __bfloat162float(res[e]) : 0.0f));
                            }
                        } else {
                            float* y = reinterpret_cast<float*>(p.y) + o;
                            const float* res = reinterpret_cast<const float*>(p.residual) + o;
                            if (vec) {
                                if (p.residual) {
                                    const float4 u = *reinterpret_cast<const float4*>(res);
                                    v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                                }
                                *reinterpret_cast<float4*>(y) = v;
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    if (col + e < p.rows) y[e] = f[e] + (p.residual ? res[e] : 0.0f);
                            }
                        }
                    });
                }
            } else {
                // SwiGLU of 64 columns; the scale block is this and the other warpgroup's
                uint32_t top = 0;
                if (left > 0 && tl.rb * kM + wg * 64 < p.I) {            // I is a multiple of 64
#pragma unroll
                    for (int j = 0; j < 64; j++) {
                        accf[j] = swiglu(accf[j], accf[64 + j]);
                        top = max(top, __float_as_uint(accf[j]) & 0x7FFFFFFFu);
                    }
                }
                tops[wg * kM + row] = top;
                named_bar(1, kEpi);
                top = max(top, tops[(wg ^ 1) * kM + row]);
                named_bar(1, kEpi);      // read before the next tile's
                const float scale = __fdiv_rn(__uint_as_float(top), kFp8Max);
                const int i0 = tl.rb * kM + wg * 64;
                if (orow >= 0 && i0 < p.I) {
                    uint4* to = reinterpret_cast<uint4*>(p.hq + (size_t)orow * p.I + i0);
#pragma unroll
                    for (int j = 0; j < 64; j += 16) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const float* f = accf + j + 4 * e;
                            w[e] = (uint32_t)code_of(f[0], scale) | (uint32_t)code_of(f[1], scale) << 8 |
                                   (uint32_t)code_of(f[2], scale) << 16 | (uint32_t)code_of(f[3], scale) << 24;
                        }
                        to[j / 16] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (wg == 0) p.hs[(size_t)orow * nb + tl.rb] = scale;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();        // the other CTA's barriers and tiles stay in use until here
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

template <int MODE>
cudaError_t launch(const Params& p, int grid, cudaStream_t s)
{
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_pair_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    fp8_pair_kernel<MODE><<<grid, kThreads, kSmem, s>>>(p);
    return cudaGetLastError();
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
