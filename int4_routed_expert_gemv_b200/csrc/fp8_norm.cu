// Residual addition, RMSNorm and quantisation to e4m3 with one scale per row and 128
// columns, in one pass over the row.
//
//   sum = x + residual (one rounding to the stream's type; the norm sees the rounded sum),
//   n   = float(sum * gamma / sqrt(mean(sum^2) + eps))   (sum of squares and scaling in
//         double and rounded once, like coli_rmsnorm: n feeds the router, whose top-k is
//         decided on floats),
//   scale[b] = max |n| of the block / 448,  q = e4m3(n / scale) (fp32 quotient, to nearest
//         even; 0 where the scale is 0).
//
// Memory-bound: a row is read once into registers (8 consecutive columns a thread and step),
// reduced across the CTA, and written out as sum, n, codes and scales.  16 neighbouring lanes
// hold one scale block, so its maximum is four shuffles.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8_tiles.cuh"

namespace coli {
namespace {

using fp8::bf16x2_bits;

struct Row8 {
    float v[8];
};

template <bool BF16>
__device__ __forceinline__ Row8 load8(const void* base, size_t elem)
{
    Row8 r;
    if (BF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + elem);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            r.v[2 * j] = __uint_as_float(w[j] << 16);
            r.v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
        const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + elem);
        const float4 a = f[0], b = f[1];
        r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
        r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, size_t elem, const Row8& r)
{
    if (BF16) {
        uint4 u;
        u.x = bf16x2_bits(r.v[0], r.v[1]);
        u.y = bf16x2_bits(r.v[2], r.v[3]);
        u.z = bf16x2_bits(r.v[4], r.v[5]);
        u.w = bf16x2_bits(r.v[6], r.v[7]);
        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + elem) = u;
    } else {
        float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + elem);
        f[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
        f[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
    }
}

// One CTA per row, blockDim.x a multiple of 32, STEPS * blockDim.x * 8 >= H.  x may alias
// sum, and so may the residual: each element is read and written by the same thread.
template <bool BF16, int STEPS>
__global__ void __launch_bounds__(STEPS == 4 ? 1024 : 768) fp8_norm_kernel(Fp8NormParams p)
{
    __shared__ double part[32];
    const int nthr = blockDim.x, tid = threadIdx.x;
    const size_t row = (size_t)blockIdx.x * p.H;
    Row8 r[STEPS];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < STEPS; i++) {
        const int c = (i * nthr + tid) * 8;
        if (c < p.H) {
            r[i] = load8<BF16>(p.x, row + c);
            if (p.residual) {
                const Row8 a = load8<BF16>(p.residual, row + c);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float s = r[i].v[j] + a.v[j];
                    r[i].v[j] = BF16 ? __bfloat162float(__float2bfloat16_rn(s)) : s;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) r[i].v[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const double d = r[i].v[j];
            ss = fma(d, d, ss);
        }
    }
    if (p.sum) {
#pragma unroll
        for (int i = 0; i < STEPS; i++) {
            const int c = (i * nthr + tid) * 8;
            if (c < p.H) store8<BF16>(p.sum, row + c, r[i]);
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 31) == 0) part[tid >> 5] = ss;
    __syncthreads();
    double tot = 0.0;
    for (int w = 0; w < nthr / 32; w++) tot += part[w];
    const double rinv = 1.0 / sqrt(tot / (double)p.H + p.eps);
    const int nb = fp8_blocks(p.H);
#pragma unroll
    for (int i = 0; i < STEPS; i++) {
        const int c = (i * nthr + tid) * 8;
        const bool in = c < p.H;
        float g[8];
        if (p.gamma && in) {
            const Row8 gr = load8<false>(p.gamma, c);
#pragma unroll
            for (int j = 0; j < 8; j++) g[j] = gr.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) g[j] = 1.0f;
        }
        uint32_t top = 0;      // bits of the largest |n|; a NaN's bits are above every number's
#pragma unroll
        for (int j = 0; j < 8; j++) {
            r[i].v[j] = in ? (float)((double)r[i].v[j] * rinv * (double)g[j]) : 0.0f;
            top = max(top, __float_as_uint(r[i].v[j]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!in) continue;
        if (p.out) store8<false>(p.out, row + c, r[i]);
        const Quantizer qz(top);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const float* f = r[i].v + 4 * h;
            w[h] = qz.codes(f[0], f[1]) | qz.codes(f[2], f[3]) << 16;
        }
        *reinterpret_cast<uint2*>(p.q + row + c) = make_uint2(w[0], w[1]);
        if ((tid & 15) == 0) p.scales[(size_t)blockIdx.x * nb + c / kFp8Block] = qz.scale;
    }
}

template <bool BF16>
cudaError_t launch(const Fp8NormParams& p, int num_sms, cudaStream_t s)
{
    const int chunks = (p.H + 7) / 8;                 // 8-column pieces of a row
    // With few rows a piece a thread, for the shortest way through a row; with many, four, so
    // that more rows are on an SM and one's loads run beside another's reduction.
    auto threads = [&](int steps) { return ((chunks + steps - 1) / steps + 31) / 32 * 32; };
    if (p.T > 2 * num_sms && chunks >= 128) fp8_norm_kernel<BF16, 4><<<p.T, threads(4), 0, s>>>(p);
    else if (chunks <= 768) fp8_norm_kernel<BF16, 1><<<p.T, threads(1), 0, s>>>(p);
    else if (chunks <= 1536) fp8_norm_kernel<BF16, 2><<<p.T, threads(2), 0, s>>>(p);
    else fp8_norm_kernel<BF16, 4><<<p.T, threads(4), 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t fp8_norm_launch(const Fp8NormParams& p, int num_sms, cudaStream_t s)
{
    return p.bf16 ? launch<true>(p, num_sms, s) : launch<false>(p, num_sms, s);
}

}  // namespace coli
