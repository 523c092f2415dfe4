// Block-scaled e4m3 products for at most 16 tokens (and 16 rows a tile), where reading the
// weights is all that counts.
//
// A tile is two 128-row blocks of weights (for gate/up: the gate rows and the up rows of the
// same 128 intermediate columns, which are one scale block of h) by 16 tokens: the weights sit
// on the MMA's M side, so one token costs a 16-column tile, a thread's accumulators belong to
// one weight row, and 32 neighbouring lanes write 32 neighbouring outputs.
//
// CTA (one per SM), 12 warps:
//   warps 0-7   two warpgroups: scaled accumulation of each K step of 128, and the tile's
//               outputs; warpgroup g has columns 8g .. 8g + 7 of both row blocks
//   warp 8      TMA producer: weight tiles (3-D map over all experts) and token rows
//   warp 9      TMEM allocator and single-thread tcgen05.mma issuer
//   warp 10     products of token and weight scales of each K step, into a ring
//   warp 11     idle
//
// Work is cut into (tile, K step) units (Schedule).  A CTA with a part of a tile writes its
// sums to the workspace and the last one to arrive adds the parts up in K order, so nothing
// waits and results do not depend on the order of arrival.
#include <string.h>

#include "fp8_tiles.cuh"

namespace coli {
namespace {

using namespace fp8;

constexpr int NT = 16;                  // tokens of a tile
constexpr int kStages = 6;
constexpr uint32_t kStage = 2 * kM * 128 + NT * 128;
constexpr int kBufs = 4;                // accumulator buffers in tensor memory
constexpr uint32_t kTmem = kBufs * 2 * NT;
constexpr int kLeast = 2;               // K steps of a run at least
constexpr uint32_t kSite = 60;
constexpr size_t kSmem = 1024 + kStages * (size_t)kStage + (size_t)kSlots * 2 * NT * 4 + 2 * 4 * (NT / 2) * 4 +
                         (kMaxGroups + 3) / 4 * 4 * 4 + 16 + 64 + 512;

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) fp8_decode_kernel(const __grid_constant__ Params p)
{
    constexpr int C = NT / 2;      // columns of a thread, per row block
    // The experts' first product takes all tokens' rows for every expert and keeps the
    // columns that chose it.
    constexpr bool kAllTokens = MODE == FP8_GATE_UP;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scale_ring = reinterpret_cast<float*>(smem + kStages * (size_t)kStage);
    uint32_t* tops = reinterpret_cast<uint32_t*>(scale_ring + kSlots * 2 * NT);
    int* first = reinterpret_cast<int*>(tops + 2 * 4 * C);              // token tiles before each group
    int* flags = first + (kMaxGroups + 3) / 4 * 4;                      // [0] groups [1] tiles [2] last [3] tmem
    int* col_pos = flags + 4;                                           // [16]
    uint64_t* bars = reinterpret_cast<uint64_t*>(col_pos + 16);
    uint64_t* full = bars;                       // [kStages] tiles landed
    uint64_t* empty = full + kStages;         // [kStages] MMAs done with the stage
    uint64_t* acc_full = empty + kStages;     // [kBufs] MMA commit
    uint64_t* acc_empty = acc_full + kBufs;   // [kBufs] read by every accumulating warp
    uint64_t* sc_full = acc_empty + kBufs;    // [kSlots]
    uint64_t* sc_empty = sc_full + kSlots;       // [kSlots]
    uint64_t* mma_done = sc_empty + kSlots;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kBufs; b++) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kEpi / 32);
        }
        for (int s = 0; s < kSlots; s++) {
            mbar_init(&sc_full[s], 1);
            mbar_init(&sc_empty[s], kEpi / 32);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(reinterpret_cast<uint32_t*>(&flags[3]), kTmem);
    if (warp == 8) plan_tiles<MODE>(p, NT, lane, first, &flags[0], &flags[1]);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];
    const int n_groups = flags[0];
    Schedule sch;
    sch.init(flags[1], p.kb, (int)gridDim.x, (int)blockIdx.x, kLeast);
    bool dead = false;
    Item it;

    if (warp == 8) {
        // ------------------------------- TMA producer -----------------------------------
        uint32_t n = 0;
        while (sch.next(it)) {
            const Tile tl = tile_of<MODE>(p, first, n_groups, NT, it.tile);
            const int shared = tl.g.expert < 0 ? 1 : 0;
            const CUtensorMap* wm = &p.w[shared];
            const int z = shared ? 0 : tl.g.expert;
            const int r0 = p.row_off + (MODE == FP8_GATE_UP ? tl.rb * kM : tl.rb * 2 * kM);
            const int r1 = MODE == FP8_GATE_UP ? r0 + p.I : r0 + kM;
            const int row0 = MODE == FP8_DENSE ? tl.t0 : kAllTokens ? 0 : tl.g.base + tl.t0;
            for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                const int s = n % kStages;
                if (!dead && !mbar_wait(&empty[s], ((n / kStages) & 1) ^ 1, p.status, kSite + 1)) dead = true;
                if (dead) continue;
                uint8_t* st = smem + (size_t)s * kStage;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], kStage);
                    tma_load_3d(st, wm, kb * 128, r0, z, &full[s]);
                    tma_load_3d(st + kM * 128, wm, kb * 128, r1, z, &full[s]);
                    tma_load_2d(st + 2 * kM * 128, &p.x[0], kb * 128, row0, &full[s]);
                }
            }
        }
        // no copy is in flight when the CTA ends
        if (lane == 0) {
            const uint32_t last = n < (uint32_t)kStages ? n : (uint32_t)kStages;
            for (uint32_t i = 0; i < last; i++) {
                const uint32_t m = n - 1 - i;
                mbar_wait(&full[m % kStages], (m / kStages) & 1, p.status, kSite + 2);
            }
        }
    } else if (warp == 9) {
        // ------------------------------- MMA issuer -------------------------------------
        if (lane == 0) {
            uint32_t n = 0;
            while (sch.next(it)) {
                const Tile tl = tile_of<MODE>(p, first, n_groups, NT, it.tile);
                const uint32_t idesc = idesc_e4m3(kM, NT);
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int s = n % kStages, b = n % kBufs;
                    if (!dead && !mbar_wait(&acc_empty[b], ((n / kBufs) & 1) ^ 1, p.status, kSite + 3)) dead = true;
                    if (!dead && !mbar_wait(&full[s], (n / kStages) & 1, p.status, kSite + 4)) dead = true;
                    tc_fence_after();
                    if (!dead) {
                        const uint8_t* st = smem + (size_t)s * kStage;
                        const uint64_t bd = sw128_desc(st + 2 * kM * 128);
#pragma unroll
                        for (int m = 0; m < 2; m++) {
                            const uint64_t ad = sw128_desc(st + m * kM * 128);
#pragma unroll
                            for (int kk = 0; kk < 4; kk++)      // 32 e4m3 values = 32 bytes per MMA
                                umma_e4m3(tmem + (uint32_t)(b * 2 * NT + m * NT), ad + 2 * kk, bd + 2 * kk, idesc,
                                          kk != 0);
                        }
                    }
                    umma_commit(&empty[s]);
                    umma_commit(&acc_full[b]);
                }
            }
            umma_commit(mma_done);
            mbar_wait(mma_done, 0, p.status, kSite + 5);
        }
    } else if (warp == 10) {
        // ------------------------------- scale products ---------------------------------
        uint32_t n = 0;
        ScaleWarp<NT, 2, 4> sw;
        while (sch.next(it)) {
            const Tile tl = tile_of<MODE>(p, first, n_groups, NT, it.tile);
            const int row = lane >= (kAllTokens ? p.T : tl.n) ? -1
                            : MODE == FP8_DENSE               ? tl.t0 + lane
                            : kAllTokens                      ? lane
                                                              : tl.g.base + tl.t0 + lane;
            sw.xrow[0] = row < 0 || lane >= NT ? nullptr : p.xs + (size_t)row * p.kb;
            const float* wbase = tl.g.expert < 0 ? p.ws[1]
                                                 : reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(p.ws[0]) +
                                                                                  (uint64_t)tl.g.expert * p.ws_stride);
            const int nb = fp8_blocks(p.rows);     // row blocks of the matrix
            const int b0 = MODE == FP8_GATE_UP ? tl.rb : 2 * tl.rb;
            sw.w[0] = wbase + (size_t)b0 * p.kb;
            sw.w[1] = MODE == FP8_GATE_UP ? sw.w[0] + (size_t)nb * p.kb : b0 + 1 < nb ? sw.w[0] + p.kb : nullptr;
            sw.run(it, lane, scale_ring, sc_full, sc_empty, n, dead, p.status, kSite + 6);
        }
    } else if (warp < 8) {
        // ------------------------- scaled accumulation, outputs -------------------------
        const int wg = warp >> 2, q = warp & 3;     // warpgroup, TMEM lane quarter
        const int row = q * 32 + lane;              // weight row within a 128-row block
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(wg * C);
        uint64_t acc[2][C / 2];
        float* accf = reinterpret_cast<float*>(acc);
        uint32_t n = 0;
        while (sch.next(it)) {
            const Tile tl = tile_of<MODE>(p, first, n_groups, NT, it.tile);
            const int ncol = kAllTokens ? p.T : tl.n;         // columns of the tile in use
            const int mine = min(max(ncol - wg * C, 0), C);   // this warpgroup's
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int j = 0; j < C / 2; j++) acc[m][j] = 0;
            for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                const int b = n % kBufs, s = n % kSlots;
                if (!dead && !mbar_wait(&acc_full[b], (n / kBufs) & 1, p.status, kSite + 7)) dead = true;
                if (!dead && !mbar_wait(&sc_full[s], (n / kSlots) & 1, p.status, kSite + 8)) dead = true;
                tc_fence_after();
                const float* sc = scale_ring + s * 2 * NT + wg * C;
                if (mine > 0) {
                    uint32_t v[2][C];
#pragma unroll
                    for (int m = 0; m < 2; m++) tmem_ld8(lane_addr + (uint32_t)(b * 2 * NT + m * NT), v[m]);
                    tmem_wait_ld();
#pragma unroll
                    for (int m = 0; m < 2; m++)
#pragma unroll
                        for (int j = 0; j < C; j += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(sc + m * NT + j);
                            acc[m][j / 2] = ffma2(pk2(v[m][j], v[m][j + 1]), pk2f(f.x, f.y), acc[m][j / 2]);
                            acc[m][j / 2 + 1] = ffma2(pk2(v[m][j + 2], v[m][j + 3]), pk2f(f.z, f.w), acc[m][j / 2 + 1]);
                        }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&acc_empty[b]);
                    mbar_arrive(&sc_empty[s]);
                }
            }
            if (it.kb1 - it.kb0 < p.kb) {
                // part of a tile: store the sums; the last part to arrive adds all of them up
                const int o0 = sch.owner(it.tile * p.kb), o1 = sch.owner(it.tile * p.kb + p.kb - 1);
                const size_t slot = (size_t)(2 * blockIdx.x + (it.kb0 == 0 ? 1 : 0)) * 2 * C * kEpi;
                float4* dst = reinterpret_cast<float4*>(p.partial + slot);
#pragma unroll
                for (int m = 0; m < 2; m++)
#pragma unroll
                    for (int j = 0; j < C / 2; j += 2) {
                        const float2 a = unpk2(acc[m][j]), b2 = unpk2(acc[m][j + 1]);
                        if (2 * j < mine)
                            __stcg(dst + (m * (C / 4) + j / 2) * kEpi + tid, make_float4(a.x, a.y, b2.x, b2.y));
                    }
                __threadfence();
                named_bar(1, kEpi);
                if (tid == 0) {
                    const uint32_t old = atomicAdd(&p.tickets[o0], 1u);
                    const bool last = old == (uint32_t)(o1 - o0);
                    if (last) p.tickets[o0] = 0;
                    flags[2] = last;
                }
                named_bar(1, kEpi);
                if (!flags[2]) continue;
                __threadfence();
#pragma unroll
                for (int m = 0; m < 2; m++)
#pragma unroll
                    for (int j = 0; j < C / 2; j++) acc[m][j] = 0;
                for (int o = o0; o <= o1; o++) {
                    const size_t from = (size_t)(2 * o + (o == o0 ? 1 : 0)) * 2 * C * kEpi;
                    const float4* src = reinterpret_cast<const float4*>(p.partial + from);
#pragma unroll
                    for (int m = 0; m < 2; m++)
#pragma unroll
                        for (int j = 0; j < C / 2; j += 2)
                            if (2 * j < mine) {
                                const float4 f = __ldcg(src + (m * (C / 4) + j / 2) * kEpi + tid);
                                acc[m][j] = fadd2(acc[m][j], pk2f(f.x, f.y));
                                acc[m][j + 1] = fadd2(acc[m][j + 1], pk2f(f.z, f.w));
                            }
                }
            }
            if (MODE == FP8_DENSE) {
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    const int r = tl.rb * 2 * kM + m * kM + row;
                    if (r >= p.rows) continue;
#pragma unroll
                    for (int j = 0; j < C; j++) {
                        if (j >= mine) break;
                        const size_t o = (size_t)(tl.t0 + wg * C + j) * p.rows + r;
                        float v = accf[m * C + j];
                        if (p.y_bf16) {
                            if (p.residual) v += __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.residual)[o]);
                            reinterpret_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
                        } else {
                            if (p.residual) v += reinterpret_cast<const float*>(p.residual)[o];
                            reinterpret_cast<float*>(p.y)[o] = v;
                        }
                    }
                }
            } else if (MODE == FP8_DOWN) {
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    const int pos = tl.g.base + tl.t0 + wg * C + j;
                    const int a = tl.g.expert < 0 ? pos : position_of(p, pos);
                    if (a < 0) {
                        if (tid == 0) set_flag(p.status, DEV_BAD_INDEX);
                        continue;
                    }
                    if (tl.rb == 0 && row == 0 && tl.g.expert >= 0) p.present[a] = 1;
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        const int r = tl.rb * 2 * kM + m * kM + row;
                        if (r < p.rows) p.z[(size_t)a * p.rows + r] = accf[m * C + j];
                    }
                }
            } else {
                // SwiGLU; its 128 rows are one scale block of h
                const int i = tl.rb * kM + row;
                uint32_t* top = tops + (wg * 4 + q) * C;
                int* cp = col_pos + wg * C;       // rows of h of this warpgroup's columns
                if (row < C) cp[row] = -1;
                named_bar(2 + wg, 128);
                for (int l = row; l < tl.g.count; l += 128) {
                    const int a = tl.g.expert < 0 ? l * p.k : position_of(p, tl.g.base + l);
                    if (a < 0) set_flag(p.status, DEV_BAD_INDEX);
                    const int t = a < 0 ? -1 : a / p.k;
                    if (t >= wg * C && t < wg * C + C) cp[t - wg * C] = tl.g.base + l;
                }
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    const float gv = accf[j], uv = accf[C + j];
                    const float h = i < p.I ? swiglu(gv, uv) : 0.0f;
                    accf[j] = h;
                    const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu);
                    if (lane == 0) top[j] = t;
                }
                named_bar(2 + wg, 128);
                const int ib = fp8_blocks(p.I);
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    const uint32_t* t4 = tops + wg * 4 * C + j;
                    const uint32_t t = max(max(t4[0], t4[C]), max(t4[2 * C], t4[3 * C]));
                    const Quantizer qz(t);
                    const int pos = cp[j];
                    if (pos < 0 || i >= p.I) continue;
                    p.hq[(size_t)pos * p.I + i] = (uint8_t)qz.codes(accf[j], 0.0f);
                    if (row == 0) p.hs[(size_t)pos * ib + tl.rb] = qz.scale;
                }
                named_bar(2 + wg, 128);      // the maxima are read before the next tile's
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
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_decode_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    fp8_decode_kernel<MODE><<<grid, kThreads, kSmem, s>>>(p);
    return cudaGetLastError();
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
