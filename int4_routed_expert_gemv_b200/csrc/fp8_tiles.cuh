// Pieces shared by the three kernels of the e4m3 products (fp8_decode.cu, fp8_mid.cu, fp8_pair.cu): the
// launch's parameters, waits, groups of tokens, the schedule of tiles, tensor-core wrappers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fp8.cuh"
#include "tcgen05.cuh"

namespace coli {
namespace fp8 {

constexpr int kM = 128;                 // weight rows of a CTA's MMA operand
constexpr int kThreads = 384;
constexpr int kEpi = 256;               // threads of the two accumulating warpgroups
constexpr int kSlots = 8;               // ring of scale products
constexpr int kMaxGroups = 1024 + 1;    // experts and the shared one

// Parameters of a launch.
struct Params {
    CUtensorMap w[2];             // dense or routed experts, shared expert
    CUtensorMap out, res;         // above 16 tokens: y, slices or z, and the residual, 32 rows of 128 bytes
    CUtensorMap x[2];             // tokens; GATE_UP above 16 tokens: in list order, and as given
    int K, kb;                    // contraction length and its scale blocks
    int rows, rb;                 // output rows of a matrix, 256-row (or gate/up pair) blocks
    int T, k, E, n_shared, I;
    const float* ws[2];           // dense: scales; experts: first blob's scales, shared's
    uint64_t ws_stride;           // bytes between experts' scales
    const float* xs;              // scales of the token codes (GATE_UP above 16 tokens: in list order)
    const float* xs_shared;       // GATE_UP above 16 tokens: as given
    const float* wts;             // DOWN: routing weights
    const int32_t* union_ids;
    const int32_t* n_union;
    const int32_t* offsets;
    const int32_t* assign;
    const void* residual;
    void* y;
    int y_bf16;
    uint8_t* hq;
    float* hs;
    float* z;                     // DOWN above 16 tokens: [T*k + T*n_shared][rows], in list order
    int32_t* z_row;               // [T*k] 1 + row of z of t * k + slot, 0 where the lists leave it out
    float* partial;               // sums of the parts of split tiles, or slices [slices][T][pitch]
    int slices, pitch;
    uint32_t* tickets;            // parts that have arrived, by the first part's worker
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

// One thread: until the last copies that it sent into a ring of stages have landed.
__device__ __forceinline__ void drain(uint64_t* full, uint32_t stages, uint32_t sent, uint32_t* status, uint32_t site)
{
    for (uint32_t m = sent - min(sent, stages); m < sent; m++) mbar_wait(&full[m % stages], (m / stages) & 1, status, site);
}

__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
}

// A group of tokens: all of them (DENSE), the shared expert's, or those of one expert of the
// union.  The shared expert, the longest, comes first.
struct Group {
    int expert;   // -1: shared
    int base;     // first row (position in the union lists; T*k + t for the shared expert)
    int count;    // 0 where the lists are not a batch union's: nothing of them is read or written
};

template <int N>
struct Groups {
    int expert[N], base[N], count[N];
    __device__ __forceinline__ Group at(int g) const { return Group{expert[g], base[g], count[g]}; }
};

// One warp: the groups of a launch into shared memory (loads that do not wait for one
// another); returns how many there are.
template <int MODE, int N>
__device__ __forceinline__ int read_groups(const Params& p, int lane, Groups<N>& t)
{
    int ng = 1;
    if (MODE != FP8_DENSE) {
        const int nu = *p.n_union;
        for (int u = lane; u < p.E; u += 32) {
            const int id = p.union_ids[u], b = p.offsets[u], e = p.offsets[u + 1];
            const bool bad = id < 0 || id >= p.E || b < 0 || e < b || e > p.T * p.k;
            const int g = p.n_shared + u;
            t.expert[g] = bad ? 0 : id;
            t.base[g] = bad ? 0 : b;
            t.count[g] = bad ? 0 : e - b;
            if (u >= nu) break;
            if (bad) set_flag(p.status, DEV_BAD_INDEX);
        }
        if ((nu < 0 || nu > p.E) && lane == 0) set_flag(p.status, DEV_BAD_INDEX);
        ng = p.n_shared + min(max(nu, 0), p.E);
    }
    if (lane == 0) {
        if (MODE != FP8_DENSE && p.n_shared) {
            t.expert[0] = -1;
            t.base[0] = p.T * p.k;
            t.count[0] = p.T;
        } else if (MODE == FP8_DENSE || ng == 0) {
            t.expert[0] = t.base[0] = 0;
            t.count[0] = MODE == FP8_DENSE ? p.T : 0;
        }
    }
    __syncwarp();
    return ng;
}

// Token of row `pos` of the union lists (-1: not a position of this batch).
__device__ __forceinline__ int position_of(const Params& p, int pos)
{
    const int a = p.assign[pos];
    return a < 0 || a >= p.T * p.k ? -1 : a;
}

// DOWN above 16 tokens: where the combine finds row `pos` of z.  A position that the lists name again is flagged, and
// the last one counts, whatever the order.
__device__ __forceinline__ void place_row(const Params& p, int pos)
{
    const int a = position_of(p, pos);
    if (a < 0 || atomicMax(&p.z_row[a], pos + 1) != 0) set_flag(p.status, DEV_BAD_INDEX);
}

struct Item {
    int tile, kb0, kb1, slice;
};

// The items of worker c of G (a CTA or a pair): a run of K steps over the first `split` tiles,
// then whole tiles.  `least`: K steps of a run at least, so that the parts of a tile, which
// one worker adds up, stay few.
// Or, with slices > 1, every tile in so many equal runs of K steps, whose sums another launch
// adds up.
struct Schedule {
    int tiles, split, kb, G, c, slices;
    int per, more, n_run;         // units per run, runs with one more, runs
    int u, u1, t;

    // join: what joining the parts of a tile costs, in K steps.  Splitting has to save more;
    // a worker alone streams a quarter faster than all of them together.
    __host__ __device__ void init(int tiles_, int kb_, int G_, int c_, int least, int join, int slices_ = 1)
    {
        slices = slices_;
        tiles = tiles_;
        kb = kb_;
        G = G_;
        c = c_;
        const int rest = tiles % G;
        const int waves = (tiles + G - 1) / G;
        const int whole = waves == 1 ? kb * max(tiles, 4 * G / 5) / G : waves * kb;
        split = slices > 1 || rest == 0 || whole <= (int)((int64_t)tiles * kb / G) + join ? 0 : tiles < G ? tiles : rest + G;
        const int units = split * kb;
        n_run = min(G, max(1, units / least));
        per = units / n_run;
        more = units - per * n_run;
        u = start(min(c, n_run));
        u1 = start(min(c + 1, n_run));
        t = split + c;
    }
    __host__ __device__ int start(int cc) const { return cc >= n_run ? split * kb : cc * per + min(cc, more); }
    __host__ __device__ int owner(int unit) const
    {
        const int big = more * (per + 1);
        return unit < big ? unit / (per + 1) : more + (unit - big) / max(per, 1);
    }
    __host__ __device__ bool next(Item& it)
    {
        if (u < u1) {
            it.tile = u / kb;
            it.kb0 = u - it.tile * kb;
            it.kb1 = min(kb, it.kb0 + u1 - u);
            it.slice = 0;
            u += it.kb1 - it.kb0;
            return true;
        }
        if (t < tiles * slices) {
            whole(t, it);
            t += G;
            return true;
        }
        return false;
    }
    // Item i, as the (i + 1)-th next() gives it.
    __host__ __device__ bool at(int i, Item& it) const
    {
        const int a = start(min(c, n_run)), b = start(min(c + 1, n_run));
        const int parts = b > a ? (b - 1) / kb - a / kb + 1 : 0;
        if (i < parts) {
            it.tile = a / kb + i;
            it.kb0 = max(a - it.tile * kb, 0);
            it.kb1 = min(b - it.tile * kb, kb);
            it.slice = 0;
            return true;
        }
        const int64_t n = split + c + (int64_t)(i - parts) * G;
        if (n >= (int64_t)tiles * slices) return false;
        whole((int)n, it);
        return true;
    }
    __host__ __device__ void whole(int n, Item& it) const
    {
        it.tile = n / slices;
        it.slice = n - it.tile * slices;
        it.kb0 = (int)((int64_t)kb * it.slice / slices);
        it.kb1 = (int)((int64_t)kb * (it.slice + 1) / slices);
    }
};

// Where a tile lies: its group, first token of the group, tokens, row block.
struct Tile {
    Group g;
    int t0, n, rb;
};

// first[g]: tiles of nt tokens before group g.
template <int N>
__device__ __forceinline__ Tile tile_of(const Params& p, const Groups<N>& t, const int* first, int n_groups, int nt, int tile)
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
    v.g = t.at(lo);
    v.t0 = (q - first[lo]) * nt;
    v.n = min(nt, v.g.count - v.t0);
    return v;
}

// One warp: first[] of every group; returns the tiles.
template <int N>
__device__ __forceinline__ int plan_tiles(const Params& p, const Groups<N>& t, int ng, int nt, int lane, int* first)
{
    int base = 0;
    for (int g0 = 0; g0 < ng; g0 += 32) {
        const int g = g0 + lane;
        const int n = g < ng ? (t.count[g] + nt - 1) / nt : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += v;
        }
        if (g < ng) first[g] = base + x - n;
        base += __shfl_sync(0xffffffffu, x, 31);
    }
    return base * p.rb;
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// silu(g) * u = g * u / (1 + e^-g).  e^-g is 2^t, t = -g / ln 2 rounded, times 1 + c, where
// c = -g - t ln 2 is what the rounding of t left out (one FMA, nearly exact, as its terms nearly cancel; c^2 is
// far below a rounding).  The quotient is an approximate reciprocal's with one correction by its
// remainder, as Quantizer's.  With g held to -88 the denominator stays finite, and from 2^126 on its
// reciprocal is flushed to 0, which the quotient is to within 2^-119.  An infinite g is its own quotient, whose
// remainder, inf - inf, has to stay out of it: fminf passes the NaN over.
__device__ __forceinline__ float swiglu(float g, float u)
{
    const float x = fminf(fmaxf(g, -88.0f), 200.0f);
    const float t = x * -1.44269504f, c = fmaf(t, -0.693147181f, -x);
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    const float d = 1.0f + fmaf(e, c, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float q = g * r;
    return fmaf(fminf(fmaf(-q, d, g), 3.4028235e38f), r, q) * u;
}

// One thread, after its CTA's barrier: counts a part of a tile whose sums the CTA has stored.
// True for the last of `parts`, which then sees the others' sums; the counter is 0 again.
__device__ __forceinline__ bool arrive_last(uint32_t* ticket, uint32_t parts)
{
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(ticket) : "memory");
    const bool last = old == parts - 1;
    if (last) *ticket = 0;
    return last;
}

// A box of a 3-D map into L2.  Open before pdl_wait: L2 is where every SM's writes meet, so a line
// fetched early is not stale later, as a copy into shared memory could be.
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int x, int y, int z)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Dynamic shared memory of a kernel, allowed once per kernel and device.
template <auto Kernel>
inline cudaError_t allow_smem(size_t bytes)
{
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

// Launch that may begin while the kernel before it in the stream ends: its set-up then costs
// no time of its own.  Kernels launched so wait (pdl_wait) before they touch memory, and read what a call
// is given with ordinary loads: the read-only path (__ldg) is for memory that nothing writes while
// the kernel runs, which these already do while the kernel before writes.  Only weights, laid out
// long before, go through it.
template <auto Kernel, class... A>
inline cudaError_t launch_early(int grid, int threads, size_t smem, cudaStream_t s, const A&... args)
{
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, Kernel, args...);
}

}  // namespace fp8

// One launch of a product: for at most 16 tokens, for few more (or few per expert), for many.
cudaError_t fp8_decode_launch(int mode, const fp8::Params& p, int num_sms, cudaStream_t s);
cudaError_t fp8_mid_launch(int mode, const fp8::Params& p, int num_sms, cudaStream_t s);
cudaError_t fp8_pair_launch(int mode, const fp8::Params& p, int num_sms, cudaStream_t s);

}  // namespace coli
