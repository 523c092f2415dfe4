// The e4m3 products of the fp8 path: which kernel a call takes, its tensor maps, and the
// combine of the experts' second product.
//
//   out[t][n] = sum_b xs[t][b] * ws[n / 128][b] * sum_{c in block b} xq[t][c] * wq[n][c]
//
// xs * ws is formed first, in fp32, so that a term costs one FMA.  Where it is below 2^-126 it is off by up to
// 2^-150 and a block's sum of codes, at most 128 * 448^2 < 2^25, times that: outputs are off by less than 2^-125 a
// block, far below what a layer's values hold.
//
//   DENSE    y = round(residual + out)
//   GATE_UP  row p of the union lists: h = silu(g) * u, then codes and scales of h
//   DOWN     up to 16 tokens the combine is part of the product (fp8_decode.cu); above,
//            z = out (fp32, one row per position of the lists), and a second launch adds residual,
//            the shared row and the routing-weighted rows of each token in a fixed order
#include <string.h>

#include "fp8_tiles.cuh"

namespace coli {
namespace {

using namespace fp8;

// y = residual + the slices' sums, in K order.  One thread 4 columns of a row.
template <class Y>
__global__ void __launch_bounds__(256) fp8_join_kernel(int T, int N, int pitch, int slices, const float* part,
                                                       const Y* residual, Y* y)
{
    pdl_launch_dependents();
    pdl_wait();
    const int n4 = pitch / 4;
    const int64_t total = (int64_t)T * n4;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int t = (int)(i / n4), c = (int)(i - (int64_t)t * n4) * 4;
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // 16 slices' loads under way together: 4 at a time took 2.5 us longer over 12 slices
        for (int s0 = 0; s0 < slices; s0 += 16) {
            float4 a[16];
#pragma unroll
            for (int j = 0; j < 16; j++)
                a[j] = s0 + j < slices ? __ldcs(reinterpret_cast<const float4*>(part) + (size_t)(s0 + j) * total + i)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 16; j++) {
                f[0] += a[j].x;
                f[1] += a[j].y;
                f[2] += a[j].z;
                f[3] += a[j].w;
            }
        }
        const size_t o = (size_t)t * N + c;
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (c + e < N) y[o + e] = (Y)(f[e] + (residual ? (float)residual[o + e] : 0.0f));
    }
}

// y[t] = residual[t] + z[T*k + t] (shared) + sum over slots of w[t][s] * its row of z, in slot
// order; slots that the lists leave out add nothing.
__global__ void __launch_bounds__(256) fp8_combine_kernel(int T, int k, int H, int n_shared, const float* z,
                                                          const int32_t* z_row, const float* w,
                                                          const float* residual, float* y)
{
    pdl_launch_dependents();
    pdl_wait();
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
        // 4 slots' loads under way together
        for (int s0 = 0; s0 < k; s0 += 4) {
            float4 a[4];
            float ws[4];
            int r[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                r[j] = s0 + j < k ? z_row[(size_t)t * k + s0 + j] - 1 : -1;
                ws[j] = s0 + j < k ? w[(size_t)t * k + s0 + j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (r[j] >= 0) a[j] = __ldcs(reinterpret_cast<const float4*>(z) + (size_t)r[j] * h4 + c);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (r[j] < 0) continue;
                v.x = fmaf(ws[j], a[j].x, v.x);
                v.y = fmaf(ws[j], a[j].y, v.y);
                v.z = fmaf(ws[j], a[j].z, v.z);
                v.w = fmaf(ws[j], a[j].w, v.w);
            }
        }
        reinterpret_cast<float4*>(y)[i] = v;
    }
}

__global__ void __launch_bounds__(256) fp8_clear_kernel(size_t n, uint4* p)
{
    pdl_launch_dependents();
    pdl_wait();
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = make_uint4(0, 0, 0, 0);
}

// Rows of x and their scales in list order: row p is token assign[p] / k.  Positions that are none
// of the batch's are flagged and get zeros.  Copied are the rows up to the largest end of a list that the product takes
// (read_groups), whatever the lists behind it say: it may read no row that an earlier call left here.
__global__ void __launch_bounds__(256) fp8_gather_kernel(int positions, int k, int E, int pieces, int kb,
                                                         const int32_t* n_union, const int32_t* offsets,
                                                         const int32_t* assign, const uint4* x, const float* xs, uint4* to,
                                                         float* to_s, uint32_t* status)
{
    __shared__ int end;
    const int warps = gridDim.x * 8, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) end = 0;
    pdl_launch_dependents();
    pdl_wait();
    const int nu = *n_union;
    int most = 0;
    for (int u = threadIdx.x; u < E; u += 256) {
        const int b = offsets[u], e = offsets[u + 1];
        if (u < nu && b >= 0 && e >= b && e <= positions) most = max(most, e);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    __syncthreads();
    if (lane == 0) atomicMax(&end, most);
    __syncthreads();
    const int rows = end;
    // a warp a row
    for (int p = blockIdx.x * 8 + (threadIdx.x >> 5); p < rows; p += warps) {
        const int a = assign[p];
        const bool in = a >= 0 && a < positions;
        const int t = in ? a / k : 0;
        if (!in && lane == 0) set_flag(status, DEV_BAD_INDEX);
        for (int c = lane; c < pieces; c += 32)
            to[(size_t)p * pieces + c] = in ? x[(size_t)t * pieces + c] : make_uint4(0, 0, 0, 0);
        for (int c = lane; c < kb; c += 32) to_s[(size_t)p * kb + c] = in ? xs[(size_t)t * kb + c] : 0.0f;
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

// Outputs [n][rows][cols] of es bytes a value, in boxes of 32 rows by 128 bytes.
bool out_map(CUtensorMap* m, const void* base, int es, uint64_t cols, uint64_t rows, uint64_t n)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {cols, rows, n};
    cuuint64_t strides[2] = {cols * es, cols * es * rows};
    cuuint32_t box[3] = {(cuuint32_t)(128 / es), 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

inline size_t up(size_t v) { return (v + 255) / 256 * 256; }

constexpr int kDecodeTokens = 16;       // at most: the kernel that reads weights for 16 tokens

// Two parts of a CTA, 256 threads: both row blocks of 16 tokens, or 128 tokens by 256 rows.
inline size_t partial_bytes(int64_t T)
{
    return up((size_t)2 * kFp8Ctas * (T <= kDecodeTokens ? 16 : 128) * kEpi * sizeof(float));
}

// Batches above 16 tokens for which reading the weights counts more than the tensor rate: up to
// so many tokens in all (DENSE), or rows of an expert on the average; for gate/up fewer where there are
// few K steps to a tile, since its 64 tokens' SwiGLU and codes then take longer than the weights.  fp8_mid.cu /
// fp8_pair.cu, us: dense 12288 x 6144, 64 tokens 24 / 34, 128 tokens 41 / 35; gate/up at hidden 6144 and
// intermediate 2048 over even lists, 32 rows 296 / 416, 48 rows 313 / 430, 96 rows 566 / 455; over uneven
// ones at 4096 and 1024, 16 rows 86 / 107, 32 rows 133 / 130, 48 rows 157 / 148; at 2048 and 768, 32 rows 92 / 105, 48
// rows 121 / 117; at 1024 and 512, 16 rows 26 / 31, 32 rows 35 / 34; at 512 and 256, 4 rows 13.7 / 12.3, 32 rows 15.4 / 13.3;
// down over even lists at 6144, 64 rows 229 / 291, 96 rows 307 / 316, 128 rows 391 / 356.
constexpr int kMidTokens = 64, kMidGateUp = 48, kMidDown = 80;

bool mid_batch(int mode, int64_t T, int k, int E, int K)
{
    if (mode == FP8_DENSE) return T <= kMidTokens;
    int rows = kMidDown;
    if (mode == FP8_GATE_UP) {
        rows = 6 * (fp8_blocks(K) - 4);
        if (rows > kMidGateUp) rows = kMidGateUp;
    }
    return T * k <= (int64_t)rows * E;
}

}  // namespace

size_t fp8_scratch_bytes(int mode, int64_t T, int H, int k, int n_shared)
{
    size_t n = partial_bytes(T);
    if (mode == FP8_GATE_UP && T > kDecodeTokens) n += up((size_t)T * k * H) + up((size_t)T * k * fp8_blocks(H) * 4);
    if (mode == FP8_DOWN && T > kDecodeTokens) n += up((size_t)T * k * 4) + up((size_t)T * (k + n_shared) * H * sizeof(float));
    return n;
}

cudaError_t fp8_product_launch(const Fp8ProductArgs& a, cudaStream_t s)
{
    Params p;
    memset(&p, 0, sizeof(p));
    const bool decode = a.T <= kDecodeTokens;
    // Rows of y that do not begin on 16 bytes go to the kernel that writes single values: the pairs write by
    // tensor copies (4000 x 4001 x 2048 onto an fp32 residual 123 us, x 4000 with the pairs 62).
    const bool ragged = a.mode == FP8_DENSE && a.N % (a.y_bf16 ? 8 : 4) != 0;
    const bool mid = !decode && (ragged || mid_batch(a.mode, a.T, a.k, a.E, a.H));
    // rows of a token box (1: rows gathered one by one)
    const int box = mid ? 16 : !decode ? 128 : a.mode == FP8_DOWN ? 1 : 16;
    uint8_t* gathered = a.scratch + partial_bytes(a.T);
    bool ok = true;
    if (a.mode == FP8_DENSE) {
        p.K = a.K;
        p.rows = a.N;
        ok &= weight_map(&p.w[0], a.w, a.K, a.N, 1, (uint64_t)a.K * a.N);
        p.ws[0] = a.wscale;
        ok &= token_map(&p.x[0], a.x, a.K, a.T, box);
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
        if (gu && !decode) {
            ok &= token_map(&p.x[0], gathered, p.K, (uint64_t)a.T * a.k, box);
            ok &= token_map(&p.x[1], a.x, p.K, a.T, box);
        } else {
            ok &= token_map(&p.x[0], a.x, p.K, gu ? a.T : (uint64_t)a.T * (a.k + a.n_shared), box);
        }
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
    p.slices = 1;
    if (a.mode == FP8_DENSE && !decode) {
        // Fewer tiles than half of the pairs: equal slices of K, at least 4 K steps each, and a
        // second launch that adds them up on every SM.  (Joining parts as the last one arrives
        // leaves that to one pair per tile: 77 x 576 x 6144 took 24 us so.)
        const int ctas = a.num_sms < kFp8Ctas ? a.num_sms : kFp8Ctas, pairs = mid ? ctas : ctas / 2;
        const int64_t tiles = (int64_t)(mid ? (a.T + 63) / 64 : (a.T + 255) / 256) * p.rb;
        if (2 * tiles <= pairs) {
            const int most = p.kb / 4, fit = pairs / (int)tiles;
            p.slices = most < 2 ? 1 : most < fit ? most : fit;
        }
        p.pitch = (a.N + 3) / 4 * 4;
        const int es = a.y_bf16 ? 2 : 4;
        if (!mid && p.slices > 1) ok &= out_map(&p.out, p.partial, 4, p.pitch, a.T, p.slices);
        if (!mid && p.slices == 1) {
            ok &= out_map(&p.out, a.y, es, a.N, a.T, 1);
            if (a.residual) ok &= out_map(&p.res, a.residual, es, a.N, a.T, 1);
        }
        if (!ok) return cudaErrorInvalidValue;
    }
    auto product = [&]() {
        return decode ? fp8_decode_launch(a.mode, p, a.num_sms, s)
               : mid  ? fp8_mid_launch(a.mode, p, a.num_sms, s)
                      : fp8_pair_launch(a.mode, p, a.num_sms, s);
    };
    if (a.mode == FP8_GATE_UP && !decode) {
        const int64_t rows = (int64_t)a.T * a.k;
        const int blocks = (int)(rows + 7 < (int64_t)8 * a.num_sms * 8 ? (rows + 7) / 8 : (int64_t)a.num_sms * 8);
        float* scales = reinterpret_cast<float*>(gathered + up((size_t)rows * a.H));
        p.xs = scales;
        p.xs_shared = a.xs;
        const cudaError_t e = launch_early<fp8_gather_kernel>(
            blocks, 256, 0, s, a.T * a.k, a.k, a.E, a.H / 16, p.kb, a.n_union, a.offsets, a.assign,
            reinterpret_cast<const uint4*>(a.x), a.xs, reinterpret_cast<uint4*>(gathered), scales, a.status);
        if (e != cudaSuccess) return e;
    }
    p.wts = a.wts;
    if (p.slices > 1) {
        const cudaError_t e = product();
        if (e != cudaSuccess) return e;
        const int64_t work = (int64_t)a.T * (p.pitch / 4);
        const int blocks = (int)(work + 255 < (int64_t)256 * a.num_sms * 8 ? (work + 255) / 256 : (int64_t)a.num_sms * 8);
        const float* part = p.partial;
        if (a.y_bf16)
            return launch_early<fp8_join_kernel<__nv_bfloat16>>(blocks, 256, 0, s, a.T, a.N, p.pitch, p.slices, part,
                                                                reinterpret_cast<const __nv_bfloat16*>(a.residual),
                                                                reinterpret_cast<__nv_bfloat16*>(a.y));
        return launch_early<fp8_join_kernel<float>>(blocks, 256, 0, s, a.T, a.N, p.pitch, p.slices, part,
                                                    reinterpret_cast<const float*>(a.residual), reinterpret_cast<float*>(a.y));
    }
    if (a.mode != FP8_DOWN || decode) return product();
    uint8_t* at = a.scratch + partial_bytes(a.T);
    p.z_row = reinterpret_cast<int32_t*>(at);
    p.z = reinterpret_cast<float*>(at + up((size_t)a.T * a.k * 4));
    if (!out_map(&p.out, p.z, 4, a.H, (uint64_t)a.T * (a.k + a.n_shared), 1)) return cudaErrorInvalidValue;
    const size_t words = up((size_t)a.T * a.k * 4) / 16;
    cudaError_t e = launch_early<fp8_clear_kernel>((int)((words + 255) / 256), 256, 0, s, words,
                                                   reinterpret_cast<uint4*>(p.z_row));
    if (e != cudaSuccess) return e;
    e = product();
    if (e != cudaSuccess) return e;
    const int64_t work = (int64_t)a.T * (a.H / 4);
    const int blocks = (int)(work + 255 < (int64_t)256 * a.num_sms * 8 ? (work + 255) / 256 : (int64_t)a.num_sms * 8);
    return launch_early<fp8_combine_kernel>(blocks, 256, 0, s, a.T, a.k, a.H, a.n_shared, (const float*)p.z,
                                            (const int32_t*)p.z_row, a.wts, reinterpret_cast<const float*>(a.residual),
                                            reinterpret_cast<float*>(a.y));
}

}  // namespace coli
