// Block-scaled e4m3 products for at most 16 tokens, where reading the weights is all that
// counts.
//
// A tile is two 128-row blocks of weights (for gate/up: the gate rows and the up rows of the
// same 128 intermediate columns, which are one scale block of h) by all tokens of the batch:
// the weights sit on the MMA's M side and the tokens, 16 columns, on its N side, so a
// thread's accumulators belong to one weight row and 32 neighbouring lanes write 32
// neighbouring outputs.  Column j is token j in every mode:
//   DENSE    every tile has the K steps of one product;
//   GATE_UP  a tile belongs to an expert; it takes the rows of all tokens and keeps the
//            columns that chose the expert;
//   DOWN     the K steps of a tile are those of every expert of the union, one expert after
//            another, shared first: the combine is the accumulation, with the routing weight
//            as one more factor of a column's scale, and the columns that did not choose an
//            expert masked.  So y is written once, in one launch, in one fixed order.
//
// CTA (one per SM), 12 warps:
//   warps 0-7   two warpgroups: scaled accumulation of each K step of 128, and the tile's
//               outputs; warpgroup g has columns 8g .. 8g + 7 of both row blocks
//   warp 8      TMA producer: weight tiles (3-D map over all experts) and token rows
//   warp 9      TMEM allocator and single-thread tcgen05.mma issuer
//   warp 10     products of token and weight scales of each K step, into a ring
//   warp 11     checks of the lists
//
// Work is cut into (tile, K step) units (Schedule).  A CTA with a part of a tile writes its
// sums to the workspace and the last one to arrive adds the parts up in K order, so nothing
// waits and results do not depend on the order of arrival.
//
// Bounded by reading the weights from HBM, and below some 100 MB by what a launch takes before the
// first tile lands and after the last (lists, barriers, the first copies: 4 us; joining parts: 3 us).  Measured
// back to back: GLM-shaped gate/up of one token 40 us (5.7 TB/s; no tile is split), of 16 tokens 135 us
// (6.3 TB/s); down of one token 29 us (3.9 TB/s, every tile in 6 to 8 parts), of 16 82 us (5.1 TB/s); dense
// 1 x 12288 x 6144 19 us (4.0 TB/s).
#include <string.h>

#include "fp8_tiles.cuh"

namespace coli {
namespace {

using namespace fp8;

constexpr int NT = 16;                  // columns: tokens
constexpr int C = NT / 2;               // columns of a thread, per row block
constexpr int kStages = 6;
constexpr uint32_t kStage = 2 * kM * 128 + NT * 128;
constexpr int kBufs = 4;                // accumulator buffers in tensor memory
constexpr uint32_t kTmem = kBufs * 2 * NT;
// K steps of a run at least: 2 / 4 took, in us, dense 16 x 2048 x 6144 12.2 / 10.3, down of 16 tokens at hidden 1024
// 16.2 / 13.8 (of one token 8.4 / 8.9), gate/up of one and four tokens there 7.4 / 8.3 and 9.0 / 9.6.
constexpr int least(int mode) { return mode == FP8_GATE_UP ? 2 : 4; }
constexpr int kJoin = 3;                // what joining the parts of a tile costs, in K steps
constexpr int kMaxPos = NT * 32;        // positions of the union lists: 16 tokens, top-32
constexpr uint32_t kSite = 60;

struct Tables {
    Groups<kMaxGroups> g;
    int pos[kMaxPos];                   // t * k + slot of each list position (-1: not of this batch)
    float wt[kMaxPos];                  // routing weights [t * k + slot]
    uint32_t named[kMaxPos / 32];       // positions that the lists have named (bits)
};

struct Smem {
    uint8_t stage[kStages][kStage];
    float scale[kSlots][2][NT];
    uint32_t mask[kSlots];              // DOWN: columns of the step's expert
    uint32_t top[2][4][C];              // maxima of the SwiGLU rows, by warp
    Quantizer quantizer[2][C];          // of each column
    int col_pos[NT];
    uint32_t tmem;
    int n_groups, last;
    uint64_t full[kStages];             // tiles landed
    uint64_t empty[kStages];            // MMAs done with the stage
    uint64_t acc_full[kBufs];           // MMA commit
    uint64_t acc_empty[kBufs];          // read by every accumulating warp
    uint64_t sc_full[kSlots], sc_empty[kSlots];
    uint64_t mma_done;
    Tables t;
};
constexpr size_t kSmem = sizeof(Smem) + 1024;

// Four rows of a 2-D map (box one row high) into four consecutive 128-byte rows.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int x, int4 y, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(smem_u32(bar))
        : "memory");
}

// A run of K steps of one expert's matrix within an item.
struct Segment {
    int g, rb;         // group, row block
    int k0, k1;        // K steps
};

// The segments of an item, in order.
template <int MODE>
struct Segments {
    int rb, g, u, u1, kb;
    __device__ Segments(const Params& p, const Item& it)
    {
        kb = p.kb;
        u = it.kb0;
        u1 = it.kb1;
        rb = MODE == FP8_GATE_UP ? it.tile % p.rb : it.tile;
        g = MODE == FP8_GATE_UP ? it.tile / p.rb : 0;
    }
    __device__ bool next(Segment& s)
    {
        if (u >= u1) return false;
        const int skip = MODE == FP8_DOWN ? u / kb : 0;
        s.g = g + skip;
        s.rb = rb;
        s.k0 = u - skip * kb;
        s.k1 = min(kb, s.k0 + u1 - u);
        u += s.k1 - s.k0;
        return true;
    }
};

// List position of token j in group g (its row of h), -1 if the group has none.
__device__ __forceinline__ int row_of(const Params& p, const Tables& t, int g, int j)
{
    if (j >= p.T) return -1;
    if (t.g.expert[g] < 0) return t.g.base[g] + j;
    int r = -1;
    for (int l = 0; l < t.g.count[g]; l++) {
        const int a = t.pos[t.g.base[g] + l];
        if (a >= 0 && a / p.k == j) r = t.g.base[g] + l;
    }
    return r;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) fp8_decode_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
    if (MODE == FP8_DENSE && warp == 8 && lane == 0) {
        // the first weights, while the kernel before ends
        Schedule first;
        Item f;
        first.init(p.rb, p.kb, (int)gridDim.x, (int)blockIdx.x, least(MODE), kJoin);
        if (first.next(f))
            for (int kb = f.kb0; kb < min(f.kb1, f.kb0 + kStages); kb++) {
                prefetch_box(&p.w[0], kb * 128, f.tile * 2 * kM, 0);
                prefetch_box(&p.w[0], kb * 128, f.tile * 2 * kM + kM, 0);
            }
    }
    pdl_wait();
    if (warp == 8) {
        const int ng = read_groups<MODE>(p, lane, sm.t.g);
        if (lane == 0) sm.n_groups = ng;
    } else if (MODE != FP8_DENSE && warp < 8) {
        for (int i = tid; i < p.T * p.k; i += kEpi) {
            sm.t.pos[i] = position_of(p, i);
            if (MODE == FP8_DOWN) sm.t.wt[i] = p.wts[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    Schedule sch;
    const int ng = sm.n_groups, steps = MODE == FP8_DOWN ? max(ng, 1) * p.kb : p.kb;
    sch.init(MODE == FP8_GATE_UP ? ng * p.rb : p.rb, steps, (int)gridDim.x, (int)blockIdx.x, least(MODE), kJoin);
    bool dead = false;
    Item it;
    Segment sg;

    if (warp == 8) {
        // ------------------------------- TMA producer -----------------------------------
        uint32_t n = 0, sent = 0;
        while (sch.next(it)) {
            Segments<MODE> segs(p, it);
            while (segs.next(sg)) {
                const int expert = sm.t.g.expert[sg.g];
                const CUtensorMap* wm = &p.w[expert < 0 ? 1 : 0];
                const int z = max(expert, 0);
                const int r0 = MODE == FP8_GATE_UP ? sg.rb * kM : sg.rb * 2 * kM;
                const int r1 = MODE == FP8_GATE_UP ? r0 + p.I : r0 + kM;
                int4 rows = make_int4(0, 0, 0, 0);
                if (MODE == FP8_DOWN) {
                    // any row (0) for the columns that are masked
                    const int r = lane < NT ? max(row_of(p, sm.t, sg.g, lane), 0) : 0;
                    rows.x = __shfl_sync(0xffffffffu, r, (lane & 3) * 4);
                    rows.y = __shfl_sync(0xffffffffu, r, (lane & 3) * 4 + 1);
                    rows.z = __shfl_sync(0xffffffffu, r, (lane & 3) * 4 + 2);
                    rows.w = __shfl_sync(0xffffffffu, r, (lane & 3) * 4 + 3);
                }
                for (int kb = sg.k0; kb < sg.k1; kb++, n++) {
                    const int s = n % kStages;
                    warp_wait(dead, &sm.empty[s], ((n / kStages) & 1) ^ 1, p.status, kSite + 1);
                    if (dead) continue;
                    sent = n + 1;
                    uint8_t* st = sm.stage[s];
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sm.full[s], kStage);
                        tma_load_3d(st, wm, kb * 128, r0, z, &sm.full[s]);
                        tma_load_3d(st + kM * 128, wm, kb * 128, r1, z, &sm.full[s]);
                        if (MODE != FP8_DOWN) tma_load_2d(st + 2 * kM * 128, &p.x[0], kb * 128, 0, &sm.full[s]);
                    }
                    __syncwarp();
                    if (MODE == FP8_DOWN && lane < NT / 4)
                        tma_gather4(st + 2 * kM * 128 + lane * 512, &p.x[0], kb * 128, rows, &sm.full[s]);
                }
            }
        }
        // no copy is in flight when the CTA ends
        if (lane == 0) drain(sm.full, kStages, sent, p.status, kSite + 2);
    } else if (warp == 9) {
        // ------------------------------- MMA issuer -------------------------------------
        if (lane == 0) {
            const uint32_t idesc = idesc_e4m3(kM, NT);
            uint32_t n = 0;
            while (sch.next(it)) {
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
        // lane m * 16 + j: row block m, column j; K steps are fetched B at a time, a batch ahead
        constexpr int B = 4;
        const int m = lane >> 4, j = lane & 15;
        const int nb = fp8_blocks(p.rows);     // row blocks of a matrix
        uint32_t n = 0;
        while (sch.next(it)) {
            Segments<MODE> segs(p, it);
            while (segs.next(sg)) {
                const int expert = sm.t.g.expert[sg.g];
                const int row = MODE == FP8_DOWN ? row_of(p, sm.t, sg.g, j) : j < p.T ? j : -1;
                const float wt = MODE != FP8_DOWN || expert < 0 || row < 0 ? 1.0f : sm.t.wt[sm.t.pos[row]];
                const uint32_t mask = __ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu;
                const float* xs = p.xs + (size_t)max(row, 0) * p.kb;
                const float* wb = expert < 0 ? p.ws[1]
                                             : reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(p.ws[0]) +
                                                                              (uint64_t)expert * p.ws_stride);
                const int blk = MODE == FP8_GATE_UP ? sg.rb + m * nb : min(2 * sg.rb + m, nb - 1);
                const float* ws = wb + (size_t)blk * p.kb;
                float xv[B], wv[B];
                auto fetch = [&](int kb) {
#pragma unroll
                    for (int i = 0; i < B; i++) {
                        const int k = min(kb + i, sg.k1 - 1);
                        xv[i] = xs[k];
                        wv[i] = __ldg(ws + k);
                    }
                };
                fetch(sg.k0);
                for (int kb = sg.k0; kb < sg.k1; kb += B) {
                    float s[B];
#pragma unroll
                    for (int i = 0; i < B; i++) s[i] = row < 0 ? 0.0f : xv[i] * wv[i] * wt;
                    if (kb + B < sg.k1) fetch(kb + B);
#pragma unroll
                    for (int i = 0; i < B; i++) {
                        if (kb + i >= sg.k1) break;
                        const int slot = n % kSlots;
                        warp_wait(dead, &sm.sc_empty[slot], ((n / kSlots) & 1) ^ 1, p.status, kSite + 6);
                        sm.scale[slot][m][j] = s[i];
                        if (MODE == FP8_DOWN && lane == 0) sm.mask[slot] = mask;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.sc_full[slot]);
                        n++;
                    }
                }
            }
        }
    } else if (warp < 8) {
        // ------------------------- scaled accumulation, outputs -------------------------
        const int wg = warp >> 2, q = warp & 3;     // warpgroup, TMEM lane quarter
        const int row = q * 32 + lane;              // weight row within a 128-row block
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(wg * C);
        const int mine = min(max(p.T - wg * C, 0), C);   // columns of this warpgroup in use
        float acc[2][C];
        uint32_t n = 0;
        while (sch.next(it)) {
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int j = 0; j < C; j++) acc[m][j] = 0.0f;
            for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                const int b = n % kBufs, s = n % kSlots;
                warp_wait(dead, &sm.sc_full[s], (n / kSlots) & 1, p.status, kSite + 8);
                warp_wait(dead, &sm.acc_full[b], (n / kBufs) & 1, p.status, kSite + 7);
                tc_fence_after();
                if (mine > 0) {
                    uint32_t v[2][C];
#pragma unroll
                    for (int m = 0; m < 2; m++) tmem_ld8(lane_addr + (uint32_t)(b * 2 * NT + m * NT), v[m]);
                    float sc[2][C];
#pragma unroll
                    for (int m = 0; m < 2; m++)
#pragma unroll
                        for (int j = 0; j < C; j += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(&sm.scale[s][m][wg * C + j]);
                            sc[m][j] = f.x;
                            sc[m][j + 1] = f.y;
                            sc[m][j + 2] = f.z;
                            sc[m][j + 3] = f.w;
                        }
                    const uint32_t mask = MODE == FP8_DOWN ? sm.mask[s] >> (wg * C) : 0xFFu;
                    tmem_wait_ld(v[0], v[1]);
#pragma unroll
                    for (int m = 0; m < 2; m++)
#pragma unroll
                        for (int j = 0; j < C; j++)
                            if (MODE != FP8_DOWN || (mask >> j & 1))
                                acc[m][j] = fmaf(__uint_as_float(v[m][j]), sc[m][j], acc[m][j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.acc_empty[b]);
                    mbar_arrive(&sm.sc_empty[s]);
                }
            }
            if (it.kb1 - it.kb0 < steps) {
                // part of a tile: store the sums; the last part to arrive adds all of them up
                const int o0 = sch.owner(it.tile * steps), o1 = sch.owner(it.tile * steps + steps - 1);
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
                // four parts' loads are under way together
                for (int o = o0; o <= o1; o += 4) {
                    float v[4][2][C];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float* src = p.partial + (size_t)(2 * (o + e) + (o + e == o0 ? 1 : 0)) * 2 * C * kEpi + tid;
#pragma unroll
                        for (int m = 0; m < 2; m++)
#pragma unroll
                            for (int j = 0; j < C; j++)
                                v[e][m][j] = j < mine && o + e <= o1 ? __ldcg(src + (m * C + j) * kEpi) : 0.0f;
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++)
#pragma unroll
                        for (int m = 0; m < 2; m++)
#pragma unroll
                            for (int j = 0; j < C; j++) acc[m][j] += v[e][m][j];
                }
            }
            if (MODE != FP8_GATE_UP) {
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    const int r = it.tile * 2 * kM + m * kM + row;
                    if (r >= p.rows) continue;
                    const size_t o = (size_t)(wg * C) * p.rows + r;
                    if (p.residual) {
                        float res[C];      // loads under way together: the stores may alias them
#pragma unroll
                        for (int j = 0; j < C; j++)
                            res[j] = j >= mine    ? 0.0f
                                     : p.y_bf16 ? __bfloat162float(
                                                      reinterpret_cast<const __nv_bfloat16*>(p.residual)[o + (size_t)j * p.rows])
                                                : reinterpret_cast<const float*>(p.residual)[o + (size_t)j * p.rows];
#pragma unroll
                        for (int j = 0; j < C; j++) acc[m][j] += res[j];
                    }
#pragma unroll
                    for (int j = 0; j < C; j++) {
                        if (j >= mine) break;
                        if (p.y_bf16)
                            reinterpret_cast<__nv_bfloat16*>(p.y)[o + (size_t)j * p.rows] = __float2bfloat16_rn(acc[m][j]);
                        else
                            reinterpret_cast<float*>(p.y)[o + (size_t)j * p.rows] = acc[m][j];
                    }
                }
            } else {
                // SwiGLU; its 128 rows are one scale block of h
                const int g = it.tile / p.rb, rb = it.tile - g * p.rb, i = rb * kM + row;
                if (row < C) sm.col_pos[wg * C + row] = row_of(p, sm.t, g, wg * C + row);
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    acc[0][j] = i < p.I ? swiglu(acc[0][j], acc[1][j]) : 0.0f;
                    const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(acc[0][j]) & 0x7FFFFFFFu);
                    if (lane == 0) sm.top[wg][q][j] = t;
                }
                named_bar(2 + wg, 128);
                // a column's quantiser, with its divisions, is made by one lane
                int pos[C];
#pragma unroll
                for (int j = 0; j < C; j++) pos[j] = sm.col_pos[wg * C + j];
                if (q == 0 && lane < mine && sm.col_pos[wg * C + lane] >= 0) {
                    const Quantizer qz(
                        max(max(sm.top[wg][0][lane], sm.top[wg][1][lane]), max(sm.top[wg][2][lane], sm.top[wg][3][lane])));
                    sm.quantizer[wg][lane] = qz;
                    p.hs[(size_t)sm.col_pos[wg * C + lane] * fp8_blocks(p.I) + rb] = qz.scale;
                }
                named_bar(2 + wg, 128);
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    if (pos[j] < 0 || i >= p.I) continue;
                    const Quantizer qz = sm.quantizer[wg][j];
                    p.hq[(size_t)pos[j] * p.I + i] = (uint8_t)qz.codes(acc[0][j], 0.0f);
                }
            }
        }
    } else if (MODE != FP8_DENSE && blockIdx.x == 0) {
        // warp 11: list positions that are none of the batch's or are named again, or whose token the list names again
        bool bad = false;
        if (lane < kMaxPos / 32) sm.t.named[lane] = 0;
        __syncwarp();
        for (int g = p.n_shared + lane; g < ng; g += 32) {
            const int count = sm.t.g.count[g], base = sm.t.g.base[g];
            bad |= count > p.T;
            for (int l = 0; l < min(count, p.T); l++) {
                const int a = sm.t.pos[base + l];
                if (a < 0) bad = true;
                else bad |= atomicOr(&sm.t.named[a / 32], 1u << a % 32) >> a % 32 & 1;
                for (int i = l + 1; i < min(count, p.T); i++) bad |= a / p.k == sm.t.pos[base + i] / p.k;
            }
        }
        if (bad) set_flag(p.status, DEV_BAD_INDEX);
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
    const cudaError_t e = allow_smem<fp8_decode_kernel<MODE>>(kSmem);
    if (e != cudaSuccess) return e;
    return launch_early<fp8_decode_kernel<MODE>>(grid, kThreads, kSmem, s, p);
}

}  // namespace

cudaError_t fp8_decode_launch(int mode, const fp8::Params& p, int num_sms, cudaStream_t s)
{
    const int grid = num_sms < kFp8Ctas ? num_sms : kFp8Ctas;
    return mode == FP8_DENSE     ? launch<FP8_DENSE>(p, grid, s)
           : mode == FP8_GATE_UP ? launch<FP8_GATE_UP>(p, grid, s)
                                 : launch<FP8_DOWN>(p, grid, s);
}

}  // namespace coli
