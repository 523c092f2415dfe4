// Products of e4m3 operands with fp32 scales per block of 128, on the 5th-generation tensor
// cores: a dense matrix product, and the two products of the experts over a batch union.
//
//   out[t][n] = sum_b xs[t][b] * ws[n / 128][b] * sum_{c in block b} xq[t][c] * wq[n][c]
//
// A scale block is one K step of 128: its inner sum runs on the tensor cores (kind::f8f6f4,
// fp32 accumulation in tensor memory), and the scaled sums are added up in fp32 registers.
// The weights sit on the MMA's M side (128 rows) and the tokens on its N side, so one token
// costs a 16-column tile, a thread's accumulators belong to one weight row, and 32
// neighbouring lanes write 32 neighbouring outputs.  A tile is two 128-row blocks (for
// gate/up: the gate rows and the up rows of the same 128 intermediate columns, which are one
// scale block of h) by NT tokens.
//
//   DENSE    y = round(residual + out)
//   GATE_UP  row p of the union lists: h = silu(g) * u, then codes and scales of h
//   DOWN     z[t * k + slot] = out (fp32); a second launch adds residual, the shared row and
//            the routing-weighted rows of each token in a fixed order
//
// CTA (one per SM), 12 warps:
//   warps 0-7   two warpgroups: scaled accumulation of each K step, and the tile's outputs;
//               warpgroup g has columns g * NT / 2 .. of both row blocks
//   warp 8      TMA producer: weight tiles (3-D map over all experts) and token tiles (rows
//               one after another, or gathered by the union lists)
//   warp 9      TMEM allocator and single-thread tcgen05.mma issuer
//   warp 10     products xs * ws of each K step, into a ring in shared memory
//   warp 11     idle
//
// Work: (tile, K step) units.  Whole tiles go round the CTAs; the tiles of the last
// incomplete waves (or all, when there are few) are cut into equal runs of K steps, one per
// CTA.  A CTA with a part of a tile writes its sums to the workspace and the last one to
// arrive adds the parts up in K order, so nothing waits and results do not depend on order.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <string.h>

#include "common.cuh"
#include "fp8.cuh"
#include "tcgen05.cuh"

namespace coli {
namespace {

constexpr int kM = 128;                 // weight rows of one MMA
constexpr int kThreads = 384;
constexpr int kEpi = 256;               // threads of the two accumulating warpgroups
constexpr int kSlots = 8;               // ring of scale products
constexpr uint32_t kSite = 60;
constexpr int kMaxGroups = 1024 + 1;    // experts and the shared one

template <int NT>
struct Shape {
    static constexpr int kCols = NT / 2;                               // columns of a thread, per row block
    static constexpr uint32_t kTok = NT * 128;                         // token tile bytes
    static constexpr uint32_t kStage = 2 * kM * 128 + kTok;
    static constexpr int kStages = NT == 128 ? 4 : 6;
    static constexpr int kBufs = NT == 128 ? 2 : 4;                    // accumulator buffers in TMEM
    static constexpr uint32_t kTmem = kBufs * 2 * NT;
    static constexpr int kBox = NT == 16 ? 16 : 32;                    // rows of a token box
    static constexpr size_t kScaleBytes = (size_t)kSlots * 2 * NT * 4;
    static constexpr size_t kTopBytes = (size_t)2 * 4 * kCols * 4;     // maxima of the SwiGLU rows
    static constexpr size_t kSmem = 1024 + kStages * (size_t)kStage + kScaleBytes + kTopBytes +
                                    (kMaxGroups + 3) / 4 * 4 * 4 + 16 + 64 + 512;
};

struct Params {
    CUtensorMap w[2];             // dense or routed experts, shared expert
    CUtensorMap x;
    int K, kb;                    // contraction length and its scale blocks
    int rows, rb;                 // output rows of a matrix, 256-row (or gate/up pair) blocks
    int T, k, E, n_shared, I;
    int row_off;                  // rows before the wanted matrix inside a blob's map
    const float* ws[2];           // dense: scales; experts: first blob's scales, shared's
    uint64_t ws_stride;           // bytes between experts' scales
    const float* xs;
    const int32_t* union_ids;
    const int32_t* n_union;
    const int32_t* offsets;
    const int32_t* assign;
    const void* residual;
    void* y;
    int y_bf16;
    uint8_t* hq;
    float* hs;
    float* z;                     // DOWN: [T*k + T*n_shared][rows]
    uint8_t* present;             // DOWN: [T*k] 1 where z has the row
    float* partial;               // [2 * grid][2][NT / 2][kEpi] sums of split tiles
    uint32_t* tickets;
    uint32_t* status;
};

// kind::f8f6f4 instruction descriptor: e4m3 A and B, fp32 D, both K-major, M x N.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Four rows of a 2-D map (box one row high) into four consecutive 128-byte rows.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int x, int4 y, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[N])
{
    if constexpr (N == 8) tmem_ld8(a, r);
    else tmem_ld16(a, r);
}

// Group g of a product: the shared expert first (the longest), then the union.
struct Group {
    int expert;   // -1: shared
    int base;     // first row (position in the union lists; T*k + t for the shared expert)
    int count;    // 0 where the lists are not a batch union's: nothing of them is read or written
    bool bad;
};

template <int MODE>
__device__ __forceinline__ Group group_of(const Params& p, int g)
{
    Group v;
    v.bad = false;
    if (MODE == FP8_DENSE) {
        v.expert = 0;
        v.base = 0;
        v.count = p.T;
    } else if (g < p.n_shared) {
        v.expert = -1;
        v.base = p.T * p.k;
        v.count = p.T;
    } else {
        const int u = g - p.n_shared;
        v.expert = p.union_ids[u];
        v.base = p.offsets[u];
        v.count = p.offsets[u + 1] - v.base;
        v.bad = v.expert < 0 || v.expert >= p.E || v.base < 0 || v.count < 0 || v.base > p.T * p.k - v.count;
        if (v.bad) {
            v.expert = 0;
            v.base = 0;
            v.count = 0;
        }
    }
    return v;
}

// Token of row `pos` of the union lists (-1: not a position of this batch).
__device__ __forceinline__ int position_of(const Params& p, int pos)
{
    const int a = p.assign[pos];
    return a < 0 || a >= p.T * p.k ? -1 : a;
}

struct Item {
    int tile, kb0, kb1;
};

// The items of CTA c of G: a run of K steps over the first `split` tiles, then whole tiles.
struct Schedule {
    int tiles, split, kb, G, c;
    int per, more, n_run;         // units per CTA, CTAs with one more, CTAs with a run
    int u, u1, t;

    __device__ void init(int tiles_, int kb_, int G_, int c_)
    {
        tiles = tiles_;
        kb = kb_;
        G = G_;
        c = c_;
        const int rest = tiles % G;
        split = rest == 0 ? 0 : tiles < G ? tiles : rest + G;
        n_run = G;
        const int units = split * kb;
        per = units / n_run;
        more = units - per * n_run;
        u = start(c);
        u1 = start(c + 1);
        t = split + c;
    }
    __device__ int start(int cc) const { return cc >= n_run ? split * kb : cc * per + min(cc, more); }
    __device__ int owner(int unit) const
    {
        const int big = more * (per + 1);
        return unit < big ? unit / (per + 1) : more + (unit - big) / max(per, 1);
    }
    __device__ bool next(Item& it)
    {
        if (u < u1) {
            it.tile = u / kb;
            it.kb0 = u - it.tile * kb;
            it.kb1 = min(kb, it.kb0 + u1 - u);
            u += it.kb1 - it.kb0;
            return true;
        }
        if (t < tiles) {
            it.tile = t;
            it.kb0 = 0;
            it.kb1 = kb;
            t += G;
            return true;
        }
        return false;
    }
};

// Where a tile lies: its group, first token of the group, tokens, row block.
struct Tile {
    Group g;
    int t0, n, rb;
};

template <int MODE, int NT>
__device__ __forceinline__ Tile tile_of(const Params& p, const int* first, int n_groups, int tile)
{
    Tile v;
    const int q = tile / p.rb;
    v.rb = tile - q * p.rb;
    int lo = 0, hi = n_groups;                 // last group with first[g] <= q
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= q) lo = mid;
        else hi = mid;
    }
    v.g = group_of<MODE>(p, lo);
    v.t0 = (q - first[lo]) * NT;
    v.n = min(NT, v.g.count - v.t0);
    return v;
}

template <int MODE, int NT>
__global__ void __launch_bounds__(kThreads, 1) fp8_product_kernel(const __grid_constant__ Params p)
{
    using S = Shape<NT>;
    constexpr int C = S::kCols;
    // With 16 tokens at most, the experts' first product takes all tokens' rows for every
    // expert and keeps the columns that chose it; otherwise rows are gathered.
    constexpr bool kAllTokens = MODE == FP8_GATE_UP && NT == 16;
    constexpr bool kGather = MODE == FP8_GATE_UP && !kAllTokens;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scale_ring = reinterpret_cast<float*>(smem + S::kStages * (size_t)S::kStage);
    uint32_t* tops = reinterpret_cast<uint32_t*>(scale_ring + kSlots * 2 * NT);
    int* first = reinterpret_cast<int*>(tops + 2 * 4 * C);              // token tiles before each group
    int* flags = first + (kMaxGroups + 3) / 4 * 4;                      // [0] groups [1] tiles [2] last [3] tmem
    int* col_pos = flags + 4;                                           // [16]
    uint64_t* bars = reinterpret_cast<uint64_t*>(col_pos + 16);
    uint64_t* full = bars;                       // [kStages] tiles landed
    uint64_t* empty = full + S::kStages;         // [kStages] MMAs done with the stage
    uint64_t* acc_full = empty + S::kStages;     // [kBufs] MMA commit
    uint64_t* acc_empty = acc_full + S::kBufs;   // [kBufs] read by every accumulating warp
    uint64_t* sc_full = acc_empty + S::kBufs;    // [kSlots]
    uint64_t* sc_empty = sc_full + kSlots;       // [kSlots]
    uint64_t* mma_done = sc_empty + kSlots;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < S::kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < S::kBufs; b++) {
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
    if (warp == 9) tmem_alloc(reinterpret_cast<uint32_t*>(&flags[3]), S::kTmem);
    if (warp == 8) {
        // token tiles before each group, by one warp
        int ng = 1;
        if (MODE != FP8_DENSE) {
            const int nu = *p.n_union;
            if ((nu < 0 || nu > p.E) && lane == 0) set_flag(p.status, DEV_BAD_INDEX);
            ng = p.n_shared + min(max(nu, 0), p.E);
        }
        int base = 0;
        for (int g0 = 0; g0 < ng; g0 += 32) {
            const int g = g0 + lane;
            int n = 0;
            if (g < ng) {
                const Group v = group_of<MODE>(p, g);
                if (v.bad) set_flag(p.status, DEV_BAD_INDEX);
                n = (v.count + NT - 1) / NT;
            }
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += v;
            }
            if (g < ng) first[g] = base + x - n;
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) {
            flags[0] = ng;
            flags[1] = base * p.rb;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];
    const int n_groups = flags[0];
    Schedule sch;
    sch.init(flags[1], p.kb, (int)gridDim.x, (int)blockIdx.x);
    bool dead = false;
    Item it;

    if (warp == 8) {
        // ------------------------------- TMA producer -----------------------------------
        uint32_t n = 0;
        while (sch.next(it)) {
            const Tile tl = tile_of<MODE, NT>(p, first, n_groups, it.tile);
            const int shared = tl.g.expert < 0 ? 1 : 0;
            const CUtensorMap* wm = &p.w[shared];
            const int z = shared ? 0 : tl.g.expert;
            const int r0 = p.row_off + (MODE == FP8_GATE_UP ? tl.rb * kM : tl.rb * 2 * kM);
            const int r1 = MODE == FP8_GATE_UP ? r0 + p.I : r0 + kM;
            int4 rows = make_int4(0, 0, 0, 0);
            const int quads = (tl.n + 3) / 4, boxes = (tl.n + S::kBox - 1) / S::kBox;
            if (kGather && lane < quads) {
                int* rr = reinterpret_cast<int*>(&rows);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int i = min(4 * lane + j, tl.n - 1) + tl.t0;
                    const int a = shared ? i * p.k : position_of(p, tl.g.base + i);
                    if (a < 0) set_flag(p.status, DEV_BAD_INDEX);
                    rr[j] = max(a, 0) / p.k;
                }
            }
            const int row0 = MODE == FP8_DENSE ? tl.t0 : kAllTokens ? 0 : tl.g.base + tl.t0;
            for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                const int s = n % S::kStages;
                if (!dead && !mbar_wait(&empty[s], ((n / S::kStages) & 1) ^ 1, p.status, kSite + 1)) dead = true;
                if (dead) continue;
                uint8_t* st = smem + (size_t)s * S::kStage;
                uint8_t* tok = st + 2 * kM * 128;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], 2 * kM * 128 + (kGather ? quads * 512 : boxes * S::kBox * 128));
                    tma_load_3d(st, wm, kb * 128, r0, z, &full[s]);
                    tma_load_3d(st + kM * 128, wm, kb * 128, r1, z, &full[s]);
                    if (!kGather)
                        for (int b = 0; b < boxes; b++)
                            tma_load_2d(tok + b * S::kBox * 128, &p.x, kb * 128, row0 + b * S::kBox, &full[s]);
                }
                __syncwarp();
                if (kGather && lane < quads) tma_gather4(tok + lane * 512, &p.x, kb * 128, rows, &full[s]);
            }
        }
        // no copy is in flight when the CTA ends
        if (lane == 0) {
            const uint32_t last = n < (uint32_t)S::kStages ? n : (uint32_t)S::kStages;
            for (uint32_t i = 0; i < last; i++) {
                const uint32_t m = n - 1 - i;
                mbar_wait(&full[m % S::kStages], (m / S::kStages) & 1, p.status, kSite + 2);
            }
        }
    } else if (warp == 9) {
        // ------------------------------- MMA issuer -------------------------------------
        if (lane == 0) {
            uint32_t n = 0;
            while (sch.next(it)) {
                const Tile tl = tile_of<MODE, NT>(p, first, n_groups, it.tile);
                const uint32_t idesc = idesc_e4m3(kM, kAllTokens ? 16 : (tl.n + 15) / 16 * 16);
                for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                    const int s = n % S::kStages, b = n % S::kBufs;
                    if (!dead && !mbar_wait(&acc_empty[b], ((n / S::kBufs) & 1) ^ 1, p.status, kSite + 3)) dead = true;
                    if (!dead && !mbar_wait(&full[s], (n / S::kStages) & 1, p.status, kSite + 4)) dead = true;
                    tc_fence_after();
                    if (!dead) {
                        const uint8_t* st = smem + (size_t)s * S::kStage;
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
        constexpr int L = (NT + 31) / 32;          // columns of a lane
        constexpr int B = 4;                       // K steps fetched ahead
        uint32_t n = 0;
        while (sch.next(it)) {
            const Tile tl = tile_of<MODE, NT>(p, first, n_groups, it.tile);
            const float* xrow[L];
#pragma unroll
            for (int l = 0; l < L; l++) {
                const int j = lane + 32 * l;
                int row = -1;
                if (kAllTokens) row = j < p.T ? j : -1;
                else if (j < tl.n) {
                    const int i = tl.t0 + j;
                    if (MODE == FP8_DENSE) row = i;
                    else if (MODE == FP8_DOWN) row = tl.g.base + i;
                    else row = tl.g.expert < 0 ? i : max(position_of(p, tl.g.base + i), 0) / p.k;
                }
                xrow[l] = row < 0 ? nullptr : p.xs + (size_t)row * p.kb;
            }
            const float* wbase = tl.g.expert < 0 ? p.ws[1]
                                                 : reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(p.ws[0]) +
                                                                                  (uint64_t)tl.g.expert * p.ws_stride);
            const int nb = fp8_blocks(p.rows);     // row blocks of the matrix
            const int b0 = MODE == FP8_GATE_UP ? tl.rb : 2 * tl.rb;
            const float* w0 = wbase + (size_t)b0 * p.kb;
            const float* w1 = MODE == FP8_GATE_UP ? w0 + (size_t)nb * p.kb : b0 + 1 < nb ? w0 + p.kb : nullptr;
            float xv[B][L], wv[B][2];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < B; i++) {
                    const bool in = kb + i < it.kb1;
#pragma unroll
                    for (int l = 0; l < L; l++) xv[i][l] = in && xrow[l] ? __ldg(xrow[l] + kb + i) : 0.0f;
                    wv[i][0] = in ? __ldg(w0 + kb + i) : 0.0f;
                    wv[i][1] = in && w1 ? __ldg(w1 + kb + i) : 0.0f;
                }
            };
            fetch(it.kb0);
            for (int kb = it.kb0; kb < it.kb1; kb += B) {
                float s0[B][L], s1[B][L];
#pragma unroll
                for (int i = 0; i < B; i++)
#pragma unroll
                    for (int l = 0; l < L; l++) {
                        s0[i][l] = xv[i][l] * wv[i][0];
                        s1[i][l] = xv[i][l] * wv[i][1];
                    }
                if (kb + B < it.kb1) fetch(kb + B);
#pragma unroll
                for (int i = 0; i < B; i++) {
                    if (kb + i >= it.kb1) break;
                    const int s = n % kSlots;
                    if (!dead && !mbar_wait(&sc_empty[s], ((n / kSlots) & 1) ^ 1, p.status, kSite + 6)) dead = true;
                    float* d = scale_ring + s * 2 * NT;
#pragma unroll
                    for (int l = 0; l < L; l++) {
                        const int j = lane + 32 * l;
                        if (j < NT) {
                            d[j] = s0[i][l];
                            d[NT + j] = s1[i][l];
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_full[s]);
                    n++;
                }
            }
        }
    } else if (warp < 8) {
        // ------------------------- scaled accumulation, outputs -------------------------
        constexpr int LD = C < 16 ? 8 : 16;         // columns of one TMEM load
        const int wg = warp >> 2, q = warp & 3;     // warpgroup, TMEM lane quarter
        const int row = q * 32 + lane;              // weight row within a 128-row block
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(wg * C);
        uint64_t acc[2][C / 2];
        float* accf = reinterpret_cast<float*>(acc);
        uint32_t n = 0;
        while (sch.next(it)) {
            const Tile tl = tile_of<MODE, NT>(p, first, n_groups, it.tile);
            const int ncol = kAllTokens ? p.T : tl.n;         // columns of the tile in use
            const int mine = min(max(ncol - wg * C, 0), C);   // this warpgroup's
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int j = 0; j < C / 2; j++) acc[m][j] = 0;
            for (int kb = it.kb0; kb < it.kb1; kb++, n++) {
                const int b = n % S::kBufs, s = n % kSlots;
                if (!dead && !mbar_wait(&acc_full[b], (n / S::kBufs) & 1, p.status, kSite + 7)) dead = true;
                if (!dead && !mbar_wait(&sc_full[s], (n / kSlots) & 1, p.status, kSite + 8)) dead = true;
                tc_fence_after();
                const float* sc = scale_ring + s * 2 * NT + wg * C;
#pragma unroll
                for (int c0 = 0; c0 < C; c0 += LD) {
                    if (c0 >= mine) break;
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        uint32_t v[LD];
                        tmem_ld<LD>(lane_addr + (uint32_t)(b * 2 * NT + m * NT + c0), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < LD; j += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(sc + m * NT + c0 + j);
                            acc[m][(c0 + j) / 2] = ffma2(pk2(v[j], v[j + 1]), pk2f(f.x, f.y), acc[m][(c0 + j) / 2]);
                            acc[m][(c0 + j) / 2 + 1] =
                                ffma2(pk2(v[j + 2], v[j + 3]), pk2f(f.z, f.w), acc[m][(c0 + j) / 2 + 1]);
                        }
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
                const int* cp = nullptr;
                if (kAllTokens) {
                    named_bar(2 + wg, 128);
                    if (tid - wg * 128 < 8) col_pos[wg * 8 + tid - wg * 128] = -1;
                    named_bar(2 + wg, 128);
                    for (int l = tid - wg * 128; l < tl.g.count; l += 128) {
                        const int a = tl.g.expert < 0 ? l * p.k : position_of(p, tl.g.base + l);
                        if (a < 0) set_flag(p.status, DEV_BAD_INDEX);
                        const int t = a < 0 ? -1 : a / p.k;
                        if (t >= wg * 8 && t < wg * 8 + 8) col_pos[t] = tl.g.base + l;
                    }
                    cp = col_pos + wg * 8;
                }
#pragma unroll
                for (int j = 0; j < C; j++) {
                    if (j >= mine) break;
                    const float gv = accf[j], uv = accf[C + j];
                    const float h = i < p.I ? gv / (1.0f + expf(-gv)) * uv : 0.0f;
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
                    const float scale = __fdiv_rn(__uint_as_float(t), kFp8Max);
                    const int pos = kAllTokens ? cp[j] : tl.g.base + tl.t0 + wg * C + j;
                    if (pos < 0 || i >= p.I) continue;
                    const float v = scale != 0.0f ? __fdiv_rn(accf[j], scale) : 0.0f;
                    p.hq[(size_t)pos * p.I + i] = (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
                    if (row == 0) p.hs[(size_t)pos * ib + tl.rb] = scale;
                }
                named_bar(2 + wg, 128);      // the maxima are read before the next tile's
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmem);
    }
}

// y[t] = residual[t] + z[T*k + t] (shared) + sum over slots of w[t][s] * z[t*k + s], in slot
// order; slots that the lists leave out add nothing.
__global__ void __launch_bounds__(256) fp8_combine_kernel(int T, int k, int H, int n_shared, const float* z,
                                                          const uint8_t* present, const float* w,
                                                          const float* residual, float* y)
{
    const int h4 = H / 4;
    const int64_t total = (int64_t)T * h4;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int t = (int)(i / h4), c = (int)(i - (int64_t)t * h4);
        float4 v = residual ? reinterpret_cast<const float4*>(residual)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        if (n_shared) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(z) + ((size_t)T * k + t) * h4 + c);
            v.x += a.x;
            v.y += a.y;
            v.z += a.z;
            v.w += a.w;
        }
        for (int s = 0; s < k; s++) {
            const size_t r = (size_t)t * k + s;
            if (!present[r]) continue;
            const float ws = w[r];
            const float4 a = __ldcs(reinterpret_cast<const float4*>(z) + r * h4 + c);
            v.x = fmaf(ws, a.x, v.x);
            v.y = fmaf(ws, a.y, v.y);
            v.z = fmaf(ws, a.z, v.z);
            v.w = fmaf(ws, a.w, v.w);
        }
        reinterpret_cast<float4*>(y)[i] = v;
    }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
bool weight_map(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint64_t n, uint64_t stride)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {K, rows, n};
    cuuint64_t strides[2] = {K, stride};
    cuuint32_t box[3] = {128, (cuuint32_t)kM, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool token_map(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, int box_rows)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {K, rows};
    cuuint64_t strides[1] = {K};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int NT>
cudaError_t launch(const Params& p, int grid, cudaStream_t s)
{
    const int smem = (int)Shape<NT>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(fp8_product_kernel<MODE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    fp8_product_kernel<MODE, NT><<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

inline size_t up(size_t v) { return (v + 255) / 256 * 256; }

inline int token_tile(int64_t T) { return T <= 16 ? 16 : 128; }

inline size_t partial_bytes(int64_t T) { return up((size_t)2 * kFp8Ctas * token_tile(T) * kEpi * sizeof(float)); }

}  // namespace

size_t fp8_scratch_bytes(int mode, int64_t T, int H, int k, int n_shared)
{
    size_t n = partial_bytes(T);
    if (mode == FP8_DOWN) n += up((size_t)T * k) + up((size_t)T * (k + n_shared) * H * sizeof(float));
    return n;
}

cudaError_t fp8_product_launch(const Fp8ProductArgs& a, cudaStream_t s)
{
    Params p;
    memset(&p, 0, sizeof(p));
    const int nt = token_tile(a.T);
    const bool gather = a.mode == FP8_GATE_UP && nt > 16;
    const int box = gather ? 1 : nt == 16 ? 16 : 32;
    bool ok = true;
    if (a.mode == FP8_DENSE) {
        p.K = a.K;
        p.rows = a.N;
        ok &= weight_map(&p.w[0], a.w, a.K, a.N, 1, (uint64_t)a.K * a.N);
        p.ws[0] = a.wscale;
        ok &= token_map(&p.x, a.x, a.K, a.T, box);
    } else {
        const bool gu = a.mode == FP8_GATE_UP;
        const uint64_t IH = (uint64_t)a.I * a.H;
        const uint64_t off = gu ? 0 : 2 * IH;
        const uint64_t sc = 3 * IH + (gu ? 0 : (uint64_t)8 * fp8_blocks(a.H) * fp8_blocks(a.I));
        p.K = gu ? a.H : a.I;
        p.rows = gu ? a.I : a.H;
        const uint64_t map_rows = gu ? 2 * (uint64_t)a.I : a.H;
        const uint8_t* sh = a.n_shared ? a.shared : a.experts;
        ok &= weight_map(&p.w[0], a.experts + off, p.K, map_rows, a.E, a.stride);
        ok &= weight_map(&p.w[1], sh + off, p.K, map_rows, 1, a.stride);
        p.ws[0] = reinterpret_cast<const float*>(a.experts + sc);
        p.ws[1] = reinterpret_cast<const float*>(sh + sc);
        p.ws_stride = a.stride;
        ok &= token_map(&p.x, a.x, p.K, gu ? a.T : (uint64_t)a.T * (a.k + a.n_shared), box);
    }
    if (!ok) return cudaErrorInvalidValue;
    p.kb = fp8_blocks(p.K);
    p.rb = a.mode == FP8_GATE_UP ? fp8_blocks(p.rows) : (p.rows + 255) / 256;
    p.T = a.T;
    p.k = a.k;
    p.E = a.E;
    p.n_shared = a.n_shared;
    p.I = a.I;
    p.xs = a.xs;
    p.union_ids = a.union_ids;
    p.n_union = a.n_union;
    p.offsets = a.offsets;
    p.assign = a.assign;
    p.residual = a.residual;
    p.y = a.y;
    p.y_bf16 = a.y_bf16;
    p.hq = a.hq;
    p.hs = a.hs;
    p.status = a.status;
    p.tickets = a.tickets;
    p.partial = reinterpret_cast<float*>(a.scratch);
    const int grid = a.num_sms < kFp8Ctas ? a.num_sms : kFp8Ctas;
    if (a.mode == FP8_DENSE)
        return nt == 16 ? launch<FP8_DENSE, 16>(p, grid, s) : launch<FP8_DENSE, 128>(p, grid, s);
    if (a.mode == FP8_GATE_UP)
        return nt == 16 ? launch<FP8_GATE_UP, 16>(p, grid, s) : launch<FP8_GATE_UP, 128>(p, grid, s);
    uint8_t* at = a.scratch + partial_bytes(a.T);
    p.present = at;
    p.z = reinterpret_cast<float*>(at + up((size_t)a.T * a.k));
    cudaError_t e = cudaMemsetAsync(p.present, 0, (size_t)a.T * a.k, s);
    if (e != cudaSuccess) return e;
    e = nt == 16 ? launch<FP8_DOWN, 16>(p, grid, s) : launch<FP8_DOWN, 128>(p, grid, s);
    if (e != cudaSuccess) return e;
    const int64_t work = (int64_t)a.T * (a.H / 4);
    const int blocks = (int)(work + 255 < (int64_t)256 * a.num_sms * 8 ? (work + 255) / 256 : (int64_t)a.num_sms * 8);
    fp8_combine_kernel<<<blocks, 256, 0, s>>>(a.T, a.k, a.H, a.n_shared, p.z, p.present, a.wts,
                                              reinterpret_cast<const float*>(a.residual), reinterpret_cast<float*>(a.y));
    return cudaGetLastError();
}

}  // namespace coli
