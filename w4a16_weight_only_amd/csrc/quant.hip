// quant.hip -- residual + RMS norm and SwiGLU, with 8-bit outputs that carry a
// scale per row and block of 128 columns (what the 8-bit linear reads).
//
//   add_rmsnorm  h = x + r;  y = w * h / sqrt(mean(h^2) + eps)
//   quant        t = x, or silu(x[:, :K]) * x[:, K:]
//   8 bits       s = max(amax, 2^-40) / 448 per block;  code = e4m3(t * (448 / amax))
//
// Both are bound by HBM: each input is read once into registers and each
// output written once.  The sum h stays in fp32 for the norm (its fp16
// rounding is only the copy that the residual stream keeps), and so does y
// until its one rounding, to fp16 or to e4m3.  Measured on MI355X: 8192 x 4096
// to 8 bits 36 us (236 MB), SwiGLU of 4097 x 12800 36 us (264 MB), both above the
// 4.9 TB/s of a 2 GiB copy, as the cache behind HBM holds part of them; three
// rows 2.4 us, a launch and one load's latency.  A block of 128 columns is 16
// lanes of 8, so its maximum is four lane exchanges inside a DPP row.
#include "device.h"
#include "layer.h"

namespace w4a16 {
namespace {

// Maximum over each aligned group of 16 lanes, NaN ignored unless alone.
__device__ __forceinline__ float row16_max(float v) {
    v = fmaxf(v, dpp_f32<0x128>(v));  // row_ror:8
    v = fmaxf(v, dpp_f32<0x124>(v));  // row_ror:4
    v = fmaxf(v, dpp_f32<0x122>(v));  // row_ror:2
    v = fmaxf(v, dpp_f32<0x121>(v));  // row_ror:1
    return v;
}

__device__ __forceinline__ u32x4 load16(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

__device__ __forceinline__ void unpack(const u32x4 &v, float (&t)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = f16_bits_to_f32((v[e >> 1] >> (16 * (e & 1))) & 0xffffu);
}

__device__ __forceinline__ u32x4 pack16(const float (&t)[8]) {
    u32x4 o;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        o[w] = (uint32_t)f32_to_f16_bits(t[2 * w]) | ((uint32_t)f32_to_f16_bits(t[2 * w + 1]) << 16);
    return o;
}

// Quantises this lane's 8 values with the scale of its 16-lane block; every
// lane of the block must take part (lanes past the row's end with zeros).
// The floor of 2^-40 keeps the reciprocal finite and a zero block's codes
// zero; it is 2^-16 of the smallest fp16 value, so nothing that fp16 could
// hold is lost to it.
__device__ __forceinline__ u32x2 quantise8(const float (&t)[8], float &scale) {
    float m = 0x1p-40f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, __builtin_fabsf(t[e]));
    m = row16_max(m);
    scale = m / 448.0f;
    const float inv = 448.0f / m;
    float c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = t[e] * inv;
    return u32x2{pack_fp8x4(c[0], c[1], c[2], c[3]), pack_fp8x4(c[4], c[5], c[6], c[7])};
}

// One workgroup of W waves per row, V vectors of 8 per lane (width <= 512 * W
// * V).  `sum` may be x or r itself: a thread reads all of its elements before
// it writes any, and no other thread touches them.
template <int W, int V, bool FP8>
__global__ __launch_bounds__(64 * W) void add_rmsnorm_kernel(const uint16_t *x, int64_t ldx, const uint16_t *r,
                                                             int64_t ldr, const uint16_t *__restrict__ w, float eps,
                                                             int width, uint16_t *sum, uint16_t *__restrict__ y,
                                                             uint8_t *__restrict__ y8, float *__restrict__ scales) {
    __shared__ float sh[W];
    const int64_t row = blockIdx.x;
    const int nvec = width >> 3;
    const u32x4 zero{0u, 0u, 0u, 0u};
    u32x4 xv[V], rv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = threadIdx.x + j * 64 * W;
        xv[j] = i < nvec ? load16(x + row * ldx + 8 * i) : zero;
        rv[j] = r && i < nvec ? load16(r + row * ldr + 8 * i) : zero;
    }
    float t[V][8], ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float a[8], b[8];
        unpack(xv[j], a);
        unpack(rv[j], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[j][e] = a[e] + b[e];
            ss = __builtin_fmaf(t[j][e], t[j][e], ss);
        }
        const int i = threadIdx.x + j * 64 * W;
        if (sum && i < nvec) *reinterpret_cast<u32x4 *>(sum + row * width + 8 * i) = pack16(t[j]);
    }
    ss = wave_sum(ss, threadIdx.x & 63);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) ss += sh[i];
    }
    const float inv = 1.0f / sqrtf(opaque(ss / (float)width) + eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = threadIdx.x + j * 64 * W;
        const bool in = i < nvec;
        float g[8];
        if (w) {
            unpack(in ? load16(w + 8 * i) : zero, g);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = 1.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) t[j][e] = t[j][e] * inv * g[e];
        if constexpr (FP8) {
            float s;
            const u32x2 c = quantise8(t[j], s);
            if (in) {
                *reinterpret_cast<u32x2 *>(y8 + row * width + 8 * i) = c;
                if ((i & 15) == 0) scales[row * ((width + kFp8Block - 1) / kFp8Block) + (i >> 4)] = s;
            }
        } else {
            if (in) *reinterpret_cast<u32x4 *>(y + row * width + 8 * i) = pack16(t[j]);
        }
    }
}

// 256 threads quantise 2048 columns of a row.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void quant_kernel(const uint16_t *__restrict__ x, int64_t ldx, int K, int chunks,
                                                    uint8_t *__restrict__ y8, float *__restrict__ scales) {
    const int64_t row = blockIdx.x / (unsigned)chunks;
    const int i = (int)(blockIdx.x % (unsigned)chunks) * 256 + threadIdx.x, nvec = K >> 3;
    const bool in = i < nvec;
    const u32x4 zero{0u, 0u, 0u, 0u};
    const uint16_t *xr = x + row * ldx + 8 * i;
    const u32x4 a = in ? load16(xr) : zero;
    float t[8];
    unpack(a, t);
    if constexpr (SWIGLU) {
        const u32x4 b = in ? load16(xr + K) : zero;
        float u[8];
        unpack(b, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = silu_mul(t[e], u[e]);
    }
    float s;
    const u32x2 c = quantise8(t, s);
    if (in) {
        *reinterpret_cast<u32x2 *>(y8 + row * K + 8 * i) = c;
        if ((i & 15) == 0) scales[row * ((K + kFp8Block - 1) / kFp8Block) + (i >> 4)] = s;
    }
}

}  // namespace

hipError_t launch_add_rmsnorm(const uint16_t *x, int64_t ldx, const uint16_t *r, int64_t ldr, const uint16_t *w,
                              float eps, int64_t M, int64_t width, uint16_t *sum, uint16_t *y, uint8_t *y8,
                              float *scales, hipStream_t stream) {
    const int64_t nvec = width / 8;
#define W4A16_NORM(W, V)                                                                                             \
    do {                                                                                                             \
        if (y8)                                                                                                      \
            add_rmsnorm_kernel<W, V, true><<<dim3((unsigned)M), dim3(64 * W), 0, stream>>>(                          \
                x, ldx, r, ldr, w, eps, (int)width, sum, y, y8, scales);                                             \
        else                                                                                                         \
            add_rmsnorm_kernel<W, V, false><<<dim3((unsigned)M), dim3(64 * W), 0, stream>>>(                         \
                x, ldx, r, ldr, w, eps, (int)width, sum, y, y8, scales);                                             \
    } while (0)
    if (nvec <= 64) W4A16_NORM(1, 1);
    else if (nvec <= 256) W4A16_NORM(4, 1);
    else if (nvec <= 512) W4A16_NORM(8, 1);
    else if (nvec <= 1024) W4A16_NORM(16, 1);
    else if (nvec <= 2048) W4A16_NORM(16, 2);
    else W4A16_NORM(16, 4);
#undef W4A16_NORM
    return hipGetLastError();
}

hipError_t launch_quant_fp8(bool swiglu, const uint16_t *x, int64_t ldx, int64_t M, int64_t K, uint8_t *y8,
                            float *scales, hipStream_t stream) {
    const int chunks = (int)((K + 2047) / 2048);
    const dim3 grid((unsigned)(M * chunks));
    if (swiglu) quant_kernel<true><<<grid, dim3(256), 0, stream>>>(x, ldx, (int)K, chunks, y8, scales);
    else quant_kernel<false><<<grid, dim3(256), 0, stream>>>(x, ldx, (int)K, chunks, y8, scales);
    return hipGetLastError();
}

}  // namespace w4a16
