// Block-scaled e4m3 products for batches in between: more than 16 tokens, but so few per expert
// (or in all, for a dense product) that reading the weights still counts most.
//
// As for 16 tokens (fp8_decode.cu) the weights sit on the MMA's M side, two 128-row blocks a
// tile, and the tokens, 64 columns, on its N side: a K step of 128 brings a CTA 32 KB of weights
// and takes it less time than those take to arrive.  The pairs of fp8_pair.cu bring a CTA 16 KB a
// step, and their step, 1000 cycles, is what 64 experts of 8 rows each waited for (GLM-shaped
// gate/up of 64 tokens: 392 us, against 250 for reading the weights).  Here, bounded by those
// reads: gate/up of 17 tokens 236 us (6.0 TB/s) and of 64 tokens 272 us (6.0 TB/s), dense 12288 x 6144 for
// 64 tokens 24 us (3.1 TB/s: 48 tiles of 48 K steps, joined once each).
//
// The columns of a tile are rows of one group, one after another: tokens (DENSE), or an expert's
// rows in list order (GATE_UP reads a copy of x in that order, made by a launch before; DOWN writes
// z in that order for the combine).  The scales of the columns come from shared memory.
//
// CTA (one per SM), 12 warps:
//   warps 0-7   two warpgroups: scaled accumulation of each K step, and the tile's outputs;
//               warpgroup g has columns 32 g .. 32 g + 31 of both row blocks
//   warp 8      TMA producer: weight tiles (3-D map over all experts) and token rows
//   warp 9      TMEM allocator and single-thread tcgen05.mma issuer
//   warp 10     products of token and weight scales of each K step, into a ring
//   warp 11     DOWN: where the combine finds the rows of z
// Work is cut into (tile, K step) units (Schedule); the last part of a split tile to arrive adds
// the parts up in K order.
#include <string.h>

#include "fp8_tiles.cuh"

namespace coli {
namespace {

using namespace fp8;

constexpr int NT = 64;                  // tokens of a tile
constexpr int C = NT / 2;               // columns of a thread, per row block
constexpr int kStages = 5;
constexpr uint32_t kStage = 2 * kM * 128 + NT * 128;
constexpr int kBox = 16;                // rows of a token box
constexpr int kBufs = 4;                // accumulator buffers in tensor memory
constexpr uint32_t kTmem = kBufs * 2 * NT;
constexpr int kLeast = 4;               // K steps of a run at least
constexpr int kJoin = 14;               // what joining the parts of a tile costs, in K steps
constexpr uint32_t kSite = 100;

template <int MODE>
struct Smem {
    static constexpr int kGroups = MODE == FP8_DENSE ? 1 : kMaxGroups;
    uint8_t stage[kStages][kStage];
    float scale[kSlots][2][NT];
    uint32_t top[2][4][C];              // maxima of the SwiGLU rows, by warp
    Quantizer quantizer[2][C];          // of each column
    Groups<kGroups> groups;
    int first[kGroups];
    uint32_t tmem;
    int n_groups, tiles, last;
    uint64_t full[kStages];             // tiles landed
    uint64_t empty[kStages];            // MMAs done with the stage
    uint64_t acc_full[kBufs];           // MMA commit
    uint64_t acc_empty[kBufs];          // read by every accumulating warp
    uint64_t sc_full[kSlots], sc_empty[kSlots];
    uint64_t mma_done;
};
template <int MODE>
constexpr size_t kSmem = sizeof(Smem<MODE>) + 1024;

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) fp8_mid_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<MODE>& sm =
        *reinterpret_cast<Smem<MODE>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < kBufs; b++) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], kEpi / 32);
        }
        for (int s = 0; s < kSlots; s++) {
            mbar_init(&sm.sc_full[s], 1);
            mbar_init(&sm.sc_empty[s], kEpi / 32);
        }
        mbar_init(&sm.mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(&sm.tmem, kTmem);
    if (warp == 8 && lane == 0) {
        prefetch_map(&p.w[0]);
        prefetch_map(&p.x[0]);
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
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    Schedule sch;
    sch.init(sm.tiles, p.kb, (int)gridDim.x, (int)blockIdx.x, kLeast, kJoin, p.slices);
    bool dead = false;
    Item it;
    auto look_up = [&](int tile) { return tile_of(p, sm.groups, sm.first, sm.n_groups, NT, tile); };

    if (warp == 8) {
        // ------------------------------- TMA producer -----------------------------------
        uint32_t n = 0, sent = 0;
        while (sch.next(it)) {
            const Tile tl = look_up(it.tile);
            const int shared = tl.g.expert < 0 ? 1 : 0;
            const CUtensorMap* wm = &p.w[shared];
            const CUtensorMap* xm = &p.x[MODE == FP8_GATE_UP ? shared : 0];
            const int z = max(tl.g.expert, 0);
            const int r0 = MODE == FP8_GATE_UP ? tl.rb * kM : tl.rb * 2 * kM;
            const int r1 = MODE == FP8_GATE_UP ? r0 + p.I : r0 + kM;
            const int row0 = (MODE == FP8_DENSE || (MODE == FP8_GATE_UP && shared) ? 0 : tl.g.base) + tl.t0;
            const int boxes = (tl.n + kBox - 1) / kBox;
            for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                const int s = n % kStages;
                warp_wait(dead, &sm.empty[s], ((n / kStages) & 1) ^ 1, p.status, kSite + 1);
                if (dead) continue;
                sent = n + 1;
                uint8_t* st = sm.stage[s];
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm.full[s], 2 * kM * 128 + (uint32_t)boxes * kBox * 128);
                    tma_load_3d(st, wm, kb * 128, r0, z, &sm.full[s]);
                    tma_load_3d(st + kM * 128, wm, kb * 128, r1, z, &sm.full[s]);
                    for (int b = 0; b < boxes; b++)
                        tma_load_2d(st + 2 * kM * 128 + b * kBox * 128, xm, kb * 128, row0 + b * kBox, &sm.full[s]);
                }
                __syncwarp();
            }
        }
        // no copy is in flight when the CTA ends
        if (lane == 0) drain(sm.full, kStages, sent, p.status, kSite + 2);
    } else if (warp == 9) {
        // ------------------------------- MMA issuer -------------------------------------
        if (lane == 0) {
            uint32_t n = 0;
            while (sch.next(it)) {
                const Tile tl = look_up(it.tile);
                const uint32_t idesc = idesc_e4m3(kM, (tl.n + 15) / 16 * 16);
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int s = n % kStages, b = n % kBufs;
                    lane_wait(dead, &sm.acc_empty[b], ((n / kBufs) & 1) ^ 1, p.status, kSite + 3);
                    lane_wait(dead, &sm.full[s], (n / kStages) & 1, p.status, kSite + 4);
                    tc_fence_after();
                    if (!dead) {
                        const uint8_t* st = sm.stage[s];
                        const uint64_t bd = sw128_desc(st + 2 * kM * 128);
#pragma unroll
                        for (int m = 0; m < 2; m++) {
                            const uint64_t ad = sw128_desc(st + m * kM * 128);
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)      // 32 e4m3 values = 32 bytes per MMA
                                umma_e4m3(tmem + (uint32_t)(b * 2 * NT + m * NT), ad + 2 * kk, bd + 2 * kk, idesc, kk != 0);
                        }
                    }
                    umma_commit(&sm.empty[s]);
                    umma_commit(&sm.acc_full[b]);
                }
            }
            umma_commit(&sm.mma_done);
            mbar_wait(&sm.mma_done, 0, p.status, kSite + 5);
        }
    } else if (warp == 10) {
        // ------------------------------- scale products ---------------------------------
        // lane: columns lane and lane + 32; K steps are fetched B at a time, a batch ahead
        constexpr int B = 4;
        const int nb = fp8_blocks(p.rows);     // row blocks of a matrix
        uint32_t n = 0;
        while (sch.next(it)) {
            const Tile tl = look_up(it.tile);
            const bool shared = tl.g.expert < 0;
            const float* xs0 = MODE == FP8_GATE_UP && shared ? p.xs_shared : p.xs;
            const int row0 = (MODE == FP8_DENSE || (MODE == FP8_GATE_UP && shared) ? 0 : tl.g.base) + tl.t0;
            const float* xs[2];
#pragma unroll
            for (int l = 0; l < 2; l++)
                xs[l] = xs0 + (size_t)(row0 + min(lane + 32 * l, tl.n - 1)) * p.kb;
            const float* w0 = shared ? p.ws[1]
                                     : reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(p.ws[0]) +
                                                                      (uint64_t)tl.g.expert * p.ws_stride);
            w0 += (size_t)(MODE == FP8_GATE_UP ? tl.rb : 2 * tl.rb) * p.kb;
            const float* w1 = MODE == FP8_GATE_UP ? w0 + (size_t)nb * p.kb : 2 * tl.rb + 1 < nb ? w0 + p.kb : w0;
            float xv[B][2], av[B], bv[B];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < B; i++) {
                    const int k = min(kb + i, it.kb1 - 1);
                    xv[i][0] = xs[0][k];
                    xv[i][1] = xs[1][k];
                    av[i] = __ldg(w0 + k);
                    bv[i] = __ldg(w1 + k);
                }
            };
            fetch(it.kb0);
            for (int kb = it.kb0; kb < it.kb1; kb += B) {
                float s[B][2][2];
#pragma unroll
                for (int i = 0; i < B; i++)
#pragma unroll
                    for (int l = 0; l < 2; l++) {
                        s[i][0][l] = xv[i][l] * av[i];
                        s[i][1][l] = xv[i][l] * bv[i];
                    }
                if (kb + B < it.kb1) fetch(kb + B);
#pragma unroll
                for (int i = 0; i < B; i++) {
                    if (kb + i >= it.kb1) break;
                    const int slot = n % kSlots;
                    warp_wait(dead, &sm.sc_empty[slot], ((n / kSlots) & 1) ^ 1, p.status, kSite + 6);
#pragma unroll
                    for (int m = 0; m < 2; m++)
#pragma unroll
                        for (int l = 0; l < 2; l++) sm.scale[slot][m][lane + 32 * l] = s[i][m][l];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.sc_full[slot]);
                    n++;
                }
            }
        }
    } else if (warp == 11) {
        if (MODE == FP8_DOWN)
            while (sch.next(it)) {
                const Tile tl = look_up(it.tile);
                if (tl.rb != 0 || it.kb0 != 0 || tl.g.expert < 0) continue;
                for (int j = lane; j < tl.n; j += 32) place_row(p, tl.g.base + tl.t0 + j);
            }
    } else {
        // ------------------------- scaled accumulation, outputs -------------------------
        const int wg = warp >> 2, q = warp & 3;     // warpgroup, TMEM lane quarter
        const int row = q * 32 + lane;              // weight row within a 128-row block
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(wg * C);
        float acc[2][C];
        uint32_t n = 0;
        while (sch.next(it)) {
            const Tile tl = look_up(it.tile);
            const int mine = min(max(tl.n - wg * C, 0), C);   // columns of this warpgroup in use
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int j = 0; j < C; j++) acc[m][j] = 0.0f;
            for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                const int b = n % kBufs, s = n % kSlots;
                warp_wait(dead, &sm.sc_full[s], (n / kSlots) & 1, p.status, kSite + 8);
                warp_wait(dead, &sm.acc_full[b], (n / kBufs) & 1, p.status, kSite + 7);
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < C; c0 += 16) {
                    if (c0 >= mine) break;
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        uint32_t v[16];
                        tmem_ld16(lane_addr + (uint32_t)(b * 2 * NT + m * NT + c0), v);
                        float4 f[4];
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            f[j] = *reinterpret_cast<const float4*>(&sm.scale[s][m][wg * C + c0 + 4 * j]);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            float* a = &acc[m][c0 + 4 * j];
                            a[0] = fmaf(__uint_as_float(v[4 * j]), f[j].x, a[0]);
                            a[1] = fmaf(__uint_as_float(v[4 * j + 1]), f[j].y, a[1]);
                            a[2] = fmaf(__uint_as_float(v[4 * j + 2]), f[j].z, a[2]);
                            a[3] = fmaf(__uint_as_float(v[4 * j + 3]), f[j].w, a[3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.acc_empty[b]);
                    mbar_arrive(&sm.sc_empty[s]);
                }
            }
            if (it.kb1 - it.kb0 < p.kb && p.slices == 1) {
                // part of a tile: store the sums; the last part to arrive adds all of them up
                const int o0 = sch.owner(it.tile * p.kb), o1 = sch.owner(it.tile * p.kb + p.kb - 1);
                float* dst = p.partial + (size_t)(2 * blockIdx.x + (it.kb0 == 0 ? 1 : 0)) * 2 * C * kEpi + tid;
#pragma unroll
                for (int m = 0; m < 2; m++)
#pragma unroll
                    for (int j = 0; j < C; j++)
                        if (j < mine) __stcg(dst + (m * C + j) * kEpi, acc[m][j]);
                named_bar(1, kEpi);
                if (tid == 0) sm.last = arrive_last(&p.tickets[o0], (uint32_t)(o1 - o0 + 1));
                named_bar(1, kEpi);
                if (!sm.last) continue;
#pragma unroll
                for (int m = 0; m < 2; m++)
#pragma unroll
                    for (int j = 0; j < C; j++) acc[m][j] = 0.0f;
                for (int o = o0; o <= o1; o++) {
                    const float* src = p.partial + (size_t)(2 * o + (o == o0 ? 1 : 0)) * 2 * C * kEpi + tid;
#pragma unroll
                    for (int m = 0; m < 2; m++)
#pragma unroll
                        for (int j = 0; j < C; j++)
                            if (j < mine) acc[m][j] += __ldcg(src + (m * C + j) * kEpi);
                }
            }
            const int col0 = tl.t0 + wg * C;          // first row of the group of this warpgroup
            if (MODE != FP8_GATE_UP) {
                // rows of y (or of a slice), or of z in list order
                const bool sums = MODE == FP8_DOWN || p.slices > 1;
                const int width = MODE == FP8_DENSE && p.slices > 1 ? p.pitch : p.rows;
                float* plain = MODE == FP8_DOWN ? p.z + (size_t)tl.g.base * p.rows
                                                : p.slices > 1 ? p.partial + (size_t)it.slice * p.T * p.pitch
                                                               : reinterpret_cast<float*>(p.y);
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    const int r = (2 * tl.rb + m) * kM + row;
                    if (r >= p.rows) continue;
                    const size_t o = (size_t)col0 * width + r;
#pragma unroll
                    for (int j0 = 0; j0 < C; j0 += 16) {
                        if (j0 >= mine) break;
                        if (!sums && p.residual) {
                            float res[16];      // loads under way together: the stores may alias them
#pragma unroll
                            for (int j = 0; j < 16; j++)
                                res[j] = j0 + j >= mine ? 0.0f
                                         : p.y_bf16
                                             ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(
                                                   p.residual)[o + (size_t)(j0 + j) * width])
                                             : reinterpret_cast<const float*>(p.residual)[o + (size_t)(j0 + j) * width];
#pragma unroll
                            for (int j = 0; j < 16; j++) acc[m][j0 + j] += res[j];
                        }
#pragma unroll
                        for (int j = 0; j < 16; j++) {
                            if (j0 + j >= mine) break;
                            if (!sums && p.y_bf16)
                                reinterpret_cast<__nv_bfloat16*>(p.y)[o + (size_t)(j0 + j) * width] =
                                    __float2bfloat16_rn(acc[m][j0 + j]);
                            else
                                plain[o + (size_t)(j0 + j) * width] = acc[m][j0 + j];
                        }
                    }
                }
            } else {
                // SwiGLU; its 128 rows are one scale block of h
                const int i = tl.rb * kM + row;
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    acc[0][j] = i < p.I ? swiglu(acc[0][j], acc[1][j]) : 0.0f;
                    const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(acc[0][j]) & 0x7FFFFFFFu);
                    if (lane == 0) sm.top[wg][q][j] = t;
                }
                named_bar(2 + wg, 128);
                // a column's quantiser is made by one lane: with its divisions in every thread, GLM-shaped gate/up of 64
                // tokens took 290 us, so 266
                const int ib = fp8_blocks(p.I);
                if (q == 0 && lane < mine) {
                    const Quantizer qz(
                        max(max(sm.top[wg][0][lane], sm.top[wg][1][lane]), max(sm.top[wg][2][lane], sm.top[wg][3][lane])));
                    sm.quantizer[wg][lane] = qz;
                    p.hs[(size_t)(tl.g.base + col0 + lane) * ib + tl.rb] = qz.scale;
                }
                named_bar(2 + wg, 128);
                uint8_t* to = p.hq + (size_t)(tl.g.base + col0) * p.I + i;
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    const Quantizer qz = sm.quantizer[wg][j];
                    if (i < p.I) to[(size_t)j * p.I] = (uint8_t)qz.codes(acc[0][j], 0.0f);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

template <int MODE>
cudaError_t launch(const Params& p, int grid, cudaStream_t s)
{
    const cudaError_t e = allow_smem<fp8_mid_kernel<MODE>>(kSmem<MODE>);
    if (e != cudaSuccess) return e;
    return launch_early<fp8_mid_kernel<MODE>>(grid, kThreads, kSmem<MODE>, s, p);
}

}  // namespace

cudaError_t fp8_mid_launch(int mode, const fp8::Params& p, int num_sms, cudaStream_t s)
{
    const int grid = num_sms < kFp8Ctas ? num_sms : kFp8Ctas;
    return mode == FP8_DENSE     ? launch<FP8_DENSE>(p, grid, s)
           : mode == FP8_GATE_UP ? launch<FP8_GATE_UP>(p, grid, s)
                                 : launch<FP8_DOWN>(p, grid, s);
}

}  // namespace coli
