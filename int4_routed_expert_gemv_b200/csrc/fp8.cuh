// 8-bit floating point path (e4m3 codes, fp32 scales per block of 128): host-visible
// descriptions of the norm that quantises and of the block-scaled products.
//
// Scales: an activation row has one per 128 columns ([rows][ceil(cols / 128)]), a weight
// matrix one per 128 rows and 128 columns ([ceil(rows / 128)][ceil(cols / 128)]).
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace coli {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;     // largest e4m3 value
constexpr int kFp8Ctas = 148;         // CTAs of a product launch at most (one per SM)

__host__ __device__ inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

#ifdef __CUDACC__
// Codes of one scale block: scale = max / 448, code = e4m3(v / scale), 0 at scale 0.  The fp32
// quotient is formed as P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor" (1990), does: a correctly rounded reciprocal, the product, its exact
// remainder and one correction give the correctly rounded quotient, as long as nothing
// underflows.  The remainder's last bit is 2^-48 of v, so with a scale of 2^-90 or more every v
// that is not far below the smallest code is safe.  Scales outside 2^-90 .. 2^90 come into that
// range, with v, by a power of two.  (A branch to a division per pair of codes took 2.4 us a tile of
// 128 rows by 128 columns, as long as the SwiGLU.)
struct alignas(16) Quantizer {
    float scale, r, by, s;      // s: scale * by, 0 for an infinite scale (finite values get code 0)

    Quantizer() = default;
    // max_bits: bits of the largest |v| (a NaN's are above every number's)
    __device__ __forceinline__ explicit Quantizer(uint32_t max_bits)
    {
        scale = __fdiv_rn(__uint_as_float(max_bits), kFp8Max);
        by = scale < 0x1p-90f ? 0x1p100f : scale > 0x1p90f ? 0x1p-100f : 1.0f;
        s = scale * by;
        r = __frcp_rn(s);
        if (s == 0.0f || s == __uint_as_float(0x7F800000u)) r = s = 0.0f;
    }
    __device__ __forceinline__ float quotient(float v) const
    {
        v *= by;
        const float q = __fmul_rn(v, r);
        return __fmaf_rn(__fmaf_rn(-q, s, v), r, q);
    }
    // codes of a (low byte) and b
    __device__ __forceinline__ uint32_t codes(float a, float b) const
    {
        return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(quotient(a), quotient(b)), __NV_SATFINITE, __NV_E4M3);
    }
};
#endif

// Bytes of one expert blob: Gq | Uq | Dq (one byte per weight) | Gs | Us | Ds (fp32).
inline size_t fp8_blob_bytes(int H, int I)
{
    return 3 * (size_t)H * I + 3 * sizeof(float) * (size_t)fp8_blocks(H) * fp8_blocks(I);
}

constexpr int kFp8NormMaxHidden = 32768;

struct Fp8NormParams {
    int H, T, bf16;
    const void* x;          // [T][H] fp32 or bf16
    const void* residual;   // [T][H] same type, or null
    const float* gamma;     // [H], or null for ones
    double eps;
    void* sum;              // [T][H] same type, or null
    float* out;             // [T][H], or null
    uint8_t* q;             // [T][H]
    float* scales;          // [T][blocks]
};
cudaError_t fp8_norm_launch(const Fp8NormParams& p, int num_sms, cudaStream_t s);

enum Fp8Mode : int { FP8_DENSE = 0, FP8_GATE_UP = 1, FP8_DOWN = 2 };

// One block-scaled product.  DENSE: y [T][N] from x [T][K] and w [N][K].  GATE_UP / DOWN:
// over the union lists and the shared expert, K = H or I.
struct Fp8ProductArgs {
    int mode;
    int T, N, K;                 // DENSE
    const uint8_t* w;            // DENSE
    const float* wscale;         // DENSE
    int H, I, E, k, n_shared;    // experts
    const uint8_t* experts;
    uint64_t stride;
    const uint8_t* shared;
    const uint8_t* x;            // codes: [T][K], or h [T*k + T*n_shared][I] for DOWN
    const float* xs;             // their scales
    const int32_t* union_ids;
    const int32_t* n_union;
    const int32_t* offsets;
    const int32_t* assign;
    const float* wts;            // DOWN: routing weights [T][k]
    const void* residual;        // DENSE (y's type) / DOWN (fp32), or null
    void* y;                     // DENSE: [T][N] fp32 or bf16; DOWN: [T][H] fp32
    int y_bf16;                  // DENSE
    uint8_t* hq;                 // GATE_UP: [rows][I]
    float* hs;                   // GATE_UP: [rows][blocks of I]
    uint32_t* status;            // workspace header
    uint32_t* tickets;           // kFp8Ctas counters, zero between launches
    uint8_t* scratch;            // fp8_scratch_bytes()
    int num_sms;
};
// Scratch of one product: partial tiles, and for DOWN the rows before the combine.
size_t fp8_scratch_bytes(int mode, int64_t T, int H, int k, int n_shared);
cudaError_t fp8_product_launch(const Fp8ProductArgs& a, cudaStream_t s);

}  // namespace coli
