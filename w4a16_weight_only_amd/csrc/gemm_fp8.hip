// gemm_fp8.hip -- out = A B^T for e4m3 operands with a scale per block of 128.
//
//   out[m][n] = sum_b sa[m][b] * sb[n / 128][b] * sum_{k in block b} a[m][k] * b[n][k]
//
// One v_mfma_f32_16x16x128_f8f6f4 covers one block of 128 along K: products
// and the sum over the block are taken by the matrix core, and its fp32 result
// enters the running fp32 sums through one multiply-add per element with the
// block's sa * sb.  The operands' roles are swapped (weights are the rows of
// the 16 x 16 tile), so a lane's four results are four consecutive n of one m:
// it needs one sa and stores 8 bytes.
//
// Rounding: the instruction's own sums of eight consecutive k cut each product
// below 2^-14 of the binade of the largest of the eight (measured on MI355X,
// alike for the 16x16x32 e4m3 instruction of half the rate): at most 7 * 2^-14
// of that product, far below what e4m3 operands already lost (2^-4 each), and
// the price of running at the 8-bit rate.  All else is fp32.
//
// Within a block, lane (r, g) takes bytes 16g .. 16g + 15 and 64 + 16g .. of
// its row for both operands (any order of k is the same sum).
#include "device.h"
#include "layer.h"

namespace w4a16 {
namespace {

__device__ __forceinline__ f32x4 mfma_block(i32x8 a, i32x8 b) {
    // both operands e4m3 (format code 0), unscaled
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// A lane's 32 bytes of the block that starts at column k0 of a row of K.
__device__ __forceinline__ i32x8 load_block(const uint8_t *row, int k0, int g, int K) {
    const u32x4 zero{0u, 0u, 0u, 0u};
    const int ka = k0 + 16 * g, kb = ka + 64;
    const u32x4 lo = ka < K ? *reinterpret_cast<const u32x4 *>(row + ka) : zero;
    const u32x4 hi = kb < K ? *reinterpret_cast<const u32x4 *>(row + kb) : zero;
    return join(lo, hi);
}

__device__ __forceinline__ void store4(uint16_t *out, int64_t m, int n, int N, bool wide, const f32x4 &v) {
    uint16_t *p = out + m * N + n;
    if (wide && n + 4 <= N) {
        u32x2 w;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[j] = (uint32_t)f32_to_f16_bits(v[2 * j]) | ((uint32_t)f32_to_f16_bits(v[2 * j + 1]) << 16);
        *reinterpret_cast<u32x2 *>(p) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < N) p[j] = f32_to_f16_bits(v[j]);
    }
}

// 16 columns and 16 * MT rows per workgroup; W waves take blocks of K in turn
// and meet in LDS, in wave order.
template <int MT, int W>
__global__ __launch_bounds__(64 * W) void gemm_fp8_row_kernel(const uint8_t *__restrict__ a, const float *__restrict__ sa,
                                                              const uint8_t *__restrict__ b, const float *__restrict__ sb,
                                                              int M, int K, int N, uint16_t *__restrict__ out) {
    __shared__ f32x4 sh[W][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
    const int nb = (K + kFp8Block - 1) / kFp8Block;
    const uint8_t *brow = b + (size_t)(n0 + r < N ? n0 + r : N - 1) * K;
    const float *sbp = sb + (size_t)(n0 / kFp8Block) * nb;
    const uint8_t *arow[MT];
    const float *sap[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + 16 * i + r < M ? m0 + 16 * i + r : M - 1;
        arow[i] = a + (size_t)m * K;
        sap[i] = sa + (size_t)m * nb;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int kb = wave; kb < nb; kb += W) {
        const i32x8 bf = load_block(brow, kb * kFp8Block, g, K);
        const float s = sbp[kb];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const f32x4 p = mfma_block(bf, load_block(arow[i], kb * kFp8Block, g, K));
            const float f = s * sap[i][kb];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(p[j], f, acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sh[wave][i][lane] = acc[i];
    __syncthreads();
    const bool wide = (N & 3) == 0;
    for (int x = threadIdx.x; x < 64 * MT; x += 64 * W) {
        const int i = x >> 6, l = x & 63, m = m0 + 16 * i + (l & 15), n = n0 + 4 * (l >> 4);
        f32x4 v = sh[0][i][l];
#pragma unroll
        for (int w = 1; w < W; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += sh[w][i][l][j];
        if (m < M) store4(out, m, n, N, wide, v);
    }
}

}  // namespace

hipError_t launch_gemm_fp8(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, int64_t M, int64_t K,
                           int64_t N, uint16_t *out, hipStream_t stream) {
    const unsigned tn = (unsigned)((N + 15) / 16);
    if (M <= 16)
        gemm_fp8_row_kernel<1, 8><<<dim3(tn, 1), dim3(512), 0, stream>>>(a, sa, b, sb, (int)M, (int)K, (int)N, out);
    else
        gemm_fp8_row_kernel<4, 8><<<dim3(tn, (unsigned)((M + 63) / 64)), dim3(512), 0, stream>>>(a, sa, b, sb, (int)M, (int)K,
                                                                                               (int)N, out);
    return hipGetLastError();
}

}  // namespace w4a16
