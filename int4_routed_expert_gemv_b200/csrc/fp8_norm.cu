// Residual addition, RMSNorm and quantisation to e4m3 with one scale per row and 128
// columns, in one pass over the row.
//
//   sum = x + residual (one rounding to the stream's type; the norm sees the rounded sum),
//   n   = float(sum * gamma / sqrt(mean(sum^2) + eps))   (sum of squares and root in double
//         and one rounding at the end, like coli_rmsnorm: n feeds the router, whose top-k is
//         decided on floats),
//   scale[b] = max |n| of the block / 448,  q = e4m3(n / scale) (fp32 quotient, to nearest
//         even; 0 where the scale is 0).
//
// Memory-bound: a row is read once into registers (8 consecutive columns a thread and step),
// reduced across the CTA, and written out as sum, n, codes and scales.  16 neighbouring lanes
// hold one scale block, so its maximum is four shuffles.  The scaling is done in pairs of
// floats rather than doubles, whose conversions (16 a cycle and SM) cost more than the loads.
// Measured: 8192 x 6144 with residual and out, bf16 91 us (6.1 TB/s), fp32 133 us (6.4 TB/s); codes alone, from
// bf16, 71 us, where instructions bound (10 us of them the quantiser's); 4 rows 4 us, a launch's length.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8_tiles.cuh"

namespace coli {
namespace {

using fp8::bf16x2_bits;

// 8 columns as they are kept: fp32, or bf16 pairs.
template <bool BF16>
struct Piece {
    uint32_t w[BF16 ? 4 : 8];

    __device__ __forceinline__ void load(const void* base, size_t elem)
    {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(base) + elem * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); i++) {
            const uint4 u = p[i];
            w[4 * i] = u.x;
            w[4 * i + 1] = u.y;
            w[4 * i + 2] = u.z;
            w[4 * i + 3] = u.w;
        }
    }
    __device__ __forceinline__ void store(void* base, size_t elem) const
    {
        uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(base) + elem * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); i++) p[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < (BF16 ? 4 : 8); i++) w[i] = 0;
    }
    __device__ __forceinline__ float at(int j) const
    {
        if (!BF16) return __uint_as_float(w[j]);
        return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    }
    // this + a, rounded to the type
    __device__ __forceinline__ void add(const Piece& a)
    {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float lo = at(j) + a.at(j), hi = at(j + 1) + a.at(j + 1);
            if (BF16) w[j / 2] = bf16x2_bits(lo, hi);
            else {
                w[j] = __float_as_uint(lo);
                w[j + 1] = __float_as_uint(hi);
            }
        }
    }
};

// n = v * g * r of 8 columns, each rounded once, r = rh + rl: the product as a sum of two floats
// (FMA gives the products' remainders), which is off by less than 2^-44 before the rounding;
// where something could underflow or is not finite, in double.  One test for all 8: a branch per
// column took 8192 x 6144 in bf16 from 94 to 105 us, where instructions are what bounds.
__device__ __forceinline__ void scaled(float (&n)[8], const float (&v)[8], const float (&g)[8], double r, float rh, float rl)
{
    float least = 1.0f, most = 1.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float p = v[j] * g[j], e = fmaf(v[j], g[j], -p);
        const float hi = p * rh;
        n[j] = hi + fmaf(e, rh, fmaf(p, rl, fmaf(p, rh, -hi)));
        least = fminf(least, fminf(fabsf(p), fabsf(hi)));
        most = fmaxf(most, fabsf(hi));
    }
    // (NaN, which the comparisons pass over, is NaN either way)
    if (least > 0x1p-90f && most < 0x1p90f && rh < 0x1p90f && rh > 0x1p-60f) return;
#pragma unroll
    for (int j = 0; j < 8; j++) n[j] = (float)((double)v[j] * (double)g[j] * r);
}

// One CTA per row, blockDim.x a multiple of 32, STEPS * blockDim.x * 8 >= H.  x may alias
// sum, and so may the residual: each element is read and written by the same thread.
template <bool BF16, int STEPS, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) fp8_norm_kernel(Fp8NormParams p)
{
    __shared__ double part[32];
    pdl_launch_dependents();      // a product that follows may fetch its first weights now
    const int nthr = blockDim.x, tid = threadIdx.x;
    const size_t row = (size_t)blockIdx.x * p.H;
    Piece<BF16> x[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; i++) {
        const int c = (i * nthr + tid) * 8;
        x[i].clear();
        if (c < p.H) x[i].load(p.x, row + c);
    }
    if (p.residual) {
        Piece<BF16> a[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; i++) {
            const int c = (i * nthr + tid) * 8;
            a[i].clear();
            if (c < p.H) a[i].load(p.residual, row + c);
        }
#pragma unroll
        for (int i = 0; i < STEPS; i++) x[i].add(a[i]);
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < STEPS; i++) {
        const int c = (i * nthr + tid) * 8;
        if (p.sum && c < p.H) x[i].store(p.sum, row + c);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const double d = x[i].at(j);
            ss = fma(d, d, ss);
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 31) == 0) part[tid >> 5] = ss;
    __syncthreads();
    double tot = 0.0;
    for (int w = 0; w < nthr / 32; w++) tot += part[w];
    const double r = 1.0 / sqrt(tot / (double)p.H + p.eps);
    const float rh = (float)r, rl = (float)(r - (double)rh);
    const int nb = fp8_blocks(p.H);
#pragma unroll
    for (int i = 0; i < STEPS; i++) {
        const int c = (i * nthr + tid) * 8;
        const bool in = c < p.H;
        Piece<false> g;
        if (p.gamma && in) g.load(p.gamma, c);
        float n[8], v[8], gs[8];
        uint32_t top = 0;      // bits of the largest |n|; a NaN's bits are above every number's
#pragma unroll
        for (int j = 0; j < 8; j++) {
            v[j] = x[i].at(j);
            gs[j] = p.gamma ? g.at(j) : 1.0f;
        }
        if (in) {
            scaled(n, v, gs, r, rh, rl);
#pragma unroll
            for (int j = 0; j < 8; j++) top = max(top, __float_as_uint(n[j]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!in) continue;
        if (p.out) {
            float4* f = reinterpret_cast<float4*>(p.out + row + c);
            f[0] = make_float4(n[0], n[1], n[2], n[3]);
            f[1] = make_float4(n[4], n[5], n[6], n[7]);
        }
        const Quantizer qz(top);
        const uint32_t lo = qz.codes(n[0], n[1]) | qz.codes(n[2], n[3]) << 16;
        const uint32_t hi = qz.codes(n[4], n[5]) | qz.codes(n[6], n[7]) << 16;
        *reinterpret_cast<uint2*>(p.q + row + c) = make_uint2(lo, hi);
        if ((tid & 15) == 0) p.scales[(size_t)blockIdx.x * nb + c / kFp8Block] = qz.scale;
    }
}

template <bool BF16>
cudaError_t launch(const Fp8NormParams& p, int num_sms, cudaStream_t s)
{
    const int chunks = (p.H + 7) / 8;                 // 8-column pieces of a row
    // With few rows a piece a thread, for the shortest way through a row.  With many, up to
    // four pieces a thread and about 256 threads, so that four or five rows are on an SM and one's
    // loads run beside another's reduction.  8192 x 6144 with residual and out, three pieces: four rows
    // an SM 91 us in bf16 (6.1 TB/s), 132 in fp32 (6.5 TB/s); five, which spill, 94 and 142.  4096 x 8192,
    // four pieces, bf16 residual: four rows 56 us, three 60, five 58.
    auto threads = [&](int steps) { return ((chunks + steps - 1) / steps + 31) / 32 * 32; };
    const int many = p.T > 2 * num_sms ? (chunks + 255) / 256 : 0;
    if (many == 2) fp8_norm_kernel<BF16, 2, 256, 5><<<p.T, threads(2), 0, s>>>(p);
    else if (many == 3) fp8_norm_kernel<BF16, 3, 256, 4><<<p.T, threads(3), 0, s>>>(p);
    else if (many == 4) fp8_norm_kernel<BF16, 4, 256, 4><<<p.T, threads(4), 0, s>>>(p);
    else if (chunks <= 768) fp8_norm_kernel<BF16, 1, 768, 1><<<p.T, threads(1), 0, s>>>(p);
    else if (chunks <= 1536) fp8_norm_kernel<BF16, 2, 768, 1><<<p.T, threads(2), 0, s>>>(p);
    else fp8_norm_kernel<BF16, 4, 1024, 1><<<p.T, threads(4), 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t fp8_norm_launch(const Fp8NormParams& p, int num_sms, cudaStream_t s)
{
    return p.bf16 ? launch<true>(p, num_sms, s) : launch<false>(p, num_sms, s);
}

}  // namespace coli
