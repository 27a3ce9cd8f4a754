// kv_append.hip -- writes a call's keys and values into the paged 8-bit cache.
//
// A page of one key/value head holds its tokens' codes and one scale for keys
// and one for values, each a power of two 2^e:
//   e = clamp(ceil(log2(amax / 448)), -15, 8) over the page's tokens,
// never below the e that earlier tokens of the page already have.  Powers of
// two lose no precision against a free scale (e4m3 is a floating format) and
// make two things exact: a page whose scale grows has its old codes' exponents
// shifted, with a rounding only where they fall below e4m3's normal range; and
// every dequantised value is an fp16 value (at e >= -15 its last bit is worth
// at least 2^-24, and at e = 8 codes stop at 240, 61440), so attention feeds
// the matrix cores with no further rounding.  Infinities and NaN are stored as
// NaN and do not enter amax.
//
// Keys are stored [page, dim], values transposed [dim, page]: each is then the
// order in which attention's matrix instructions take 16 bytes per lane.
//
// One workgroup owns one (page, head) of K or of V, so no two touch the same
// scale.  It needs the new rows twice, for amax and for the codes: the second
// time from registers where they fit (64 tokens of 128 dims), else read again
// (from L2).  Prompts are bound by HBM (41697 rows of 8 heads of 128: 59 us, 256 MB,
// 4.3 TB/s) after the chain of dependent loads ahead of a workgroup's first row
// (offsets, length, page: 1000 rows take 7.5 us, 12720 rows 21 us for 78 MB), single
// tokens by that chain alone (64: 4.4 us).
#include "device.h"
#include "layer.h"

namespace w4a16 {
namespace {

__device__ __forceinline__ float finite_abs(float x) {
    const float a = __builtin_fabsf(x);
    return a < __builtin_inff() ? a : 0.f;  // NaN and infinities: 0
}

// x / 2^e as e4m3 input: saturated where e is the largest (61440 = 240 * 2^8,
// the largest code whose value fp16 holds), NaN for infinities.
__device__ __forceinline__ float scaled(float x, float inv, bool top) {
    float s = x * inv;
    if (top) s = __builtin_fabsf(s) < __builtin_inff() ? fminf(fmaxf(s, -240.f), 240.f) : s;
    return __builtin_fabsf(s) <= 448.f ? s : __builtin_nanf("");
}

__device__ __forceinline__ float fp8_value(uint32_t code) {
    return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

constexpr int kTurn = 64;  // tokens transposed at a time

template <int THREADS>
__global__ __launch_bounds__(THREADS) void kv_append_kernel(const uint16_t *__restrict__ kin, int64_t ldk,
                                                            const uint16_t *__restrict__ vin, int64_t ldv,
                                                            CacheArgs c, SeqArgs s) {
    __shared__ float sh[THREADS / 64];
    const int page = 1 << c.page_shift, D = c.dim, head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    // Work item -> (sequence, one of the pages its rows fall into).  Sequence
    // b's items start at floor(rows[b] / page) + 2b, which leaves room for its
    // floor(n / page) + 2 or fewer pages.
    const int64_t id = blockIdx.x;
    int b;
    int64_t first_id;
    if (!s.rows) {
        b = (int)id;
        first_id = id;
    } else {
        auto start = [&](int i) {
            int r = s.rows[i];
            r = r < 0 ? 0 : r > s.T ? s.T : r;
            return (int64_t)(r >> c.page_shift) + 2 * (int64_t)i;
        };
        b = find_sequence(s.B, id, start);
        first_id = start(b);
    }
    int r0, n;
    sequence_rows(s, b, r0, n);
    const int64_t len = s.lens[b];
    const int64_t begin = len - n < 0 ? 0 : len - n;  // first position written
    const int64_t pg = (begin >> c.page_shift) + (id - first_id);
    const int64_t p0 = pg << c.page_shift;
    const int64_t lo = p0 > begin ? p0 : begin, hi = p0 + page < len ? p0 + page : len;
    if (n == 0 || lo >= hi || pg >= s.max_pages) return;
    const int64_t pid = s.table[(int64_t)b * s.max_pages + pg];
    if (pid < 0 || pid >= c.pages) return;
    const int a = (int)(lo - p0), m = (int)(hi - lo);  // tokens a .. a + m of the page
    const int64_t row = r0 + (lo - (len - n));         // the first one's input row
    const uint16_t *in = (is_v ? vin : kin) + (size_t)head * D;
    const int64_t ld = is_v ? ldv : ldk;
    const size_t slot = (size_t)pid * c.heads + head;
    uint8_t *codes = (is_v ? c.v : c.k) + slot * page * D;
    uint8_t *scale = (is_v ? c.v_scale : c.k_scale) + slot;

    // 16-byte vectors: vector i is columns 8 (i % vpr) of the page's new token
    // i / vpr, vpr = D / 8 a power of two.  Up to four per thread (64 tokens of
    // 128 dims) stay in registers between the two uses, else they are read
    // again.
    const int vshift = D == 64 ? 3 : D == 128 ? 4 : 5, vectors = m << vshift, vmask = (1 << vshift) - 1;
    const bool hold = vectors <= 4 * THREADS && a + m <= (a & ~15) + kTurn;
    auto load = [&](int i) {
        return *reinterpret_cast<const u32x4 *>(in + (row + (i >> vshift)) * ld + 8 * (i & vmask));
    };
    float amax = 0.f;
    auto largest = [&](const u32x4 &x) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            amax = fmaxf(amax, finite_abs(f16_bits_to_f32((x[e >> 1] >> (16 * (e & 1))) & 0xffffu)));
    };
    u32x4 held[4];
    if (hold) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = threadIdx.x + k * THREADS;
            held[k] = i < vectors ? load(i) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) largest(held[k]);
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < vectors; i += THREADS) largest(load(i));
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
    if constexpr (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 64; ++i) amax = fmaxf(amax, sh[i]);
    }
    // ceil(log2(amax / 448)): 448 = 1.75 * 2^8, so the exponent goes up by one
    // where the fraction is above .75
    int e = (int)((__builtin_bit_cast(uint32_t, amax) + 0x1fffffu) >> 23) - 127 - 8;
    e = e < kKvMinExp ? kKvMinExp : e > kKvMaxExp ? kKvMaxExp : e;
    if (a > 0) {
        // earlier tokens: keep their scale, or shift their codes to the new one
        int old = (int)*scale - 127;
        old = old < kKvMinExp ? kKvMinExp : old > kKvMaxExp ? kKvMaxExp : old;
        if (old >= e) {
            e = old;
        } else {
            const float f = pow2f(old - e);
            for (int i = threadIdx.x; i < a * D; i += THREADS) {
                uint8_t *p = is_v ? codes + (size_t)(i / a) * page + i % a : codes + i;
                *p = (uint8_t)pack_fp8x4(fp8_value(*p) * f, 0.f, 0.f, 0.f);
            }
        }
    }
    const float inv = pow2f(-e);
    const bool top = e == kKvMaxExp;
    if constexpr (THREADS > 64) __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *scale = (uint8_t)(e + 127);
    auto codes_of = [&](const u32x4 &x) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = scaled(f16_bits_to_f32((x[j >> 1] >> (16 * (j & 1))) & 0xffffu), inv, top);
        return u32x2{pack_fp8x4(f[0], f[1], f[2], f[3]), pack_fp8x4(f[4], f[5], f[6], f[7])};
    };
    // put(i, codes) for vectors from .. to
    auto each = [&](int from, int to, auto put) __attribute__((always_inline)) {
        if (hold) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = threadIdx.x + k * THREADS;
                if (i < vectors) put(i, codes_of(held[k]));
            }
        } else {
            for (int i = from + threadIdx.x; i < to; i += THREADS) put(i, codes_of(load(i)));
        }
    };
    if (!is_v) {
        each(0, vectors, [&](int i, u32x2 o) { *reinterpret_cast<u32x2 *>(codes + (size_t)a * D + 8 * (size_t)i) = o; });
    } else if constexpr (THREADS == 64) {
        // one token: a byte of each dim's row
        each(0, vectors, [&](int i, u32x2 o) {
            const int t = i >> vshift, d = 8 * (i & vmask);
#pragma unroll
            for (int j = 0; j < 8; ++j) codes[(size_t)(d + j) * page + a + t] = (uint8_t)(o[j >> 2] >> (8 * (j & 3)));
        });
    } else {
        // Transposed through LDS, 64 tokens at a time: a thread turns 4 dims of
        // 16 tokens (16 reads of 4 bytes) into 16 bytes of each dim's row.
        __shared__ __align__(16) uint8_t tile[kTurn * (256 + 8)];
        const int stride = D + 8, qshift = vshift + 1, quads = 1 << qshift;
        for (int base = a & ~15; base < a + m; base += kTurn) {
            const int first = base > a ? base : a, end = base + kTurn < a + m ? base + kTurn : a + m;
            each((first - a) << vshift, (end - a) << vshift, [&](int i, u32x2 o) {
                *reinterpret_cast<u32x2 *>(&tile[(a - base + (i >> vshift)) * stride + 8 * (i & vmask)]) = o;
            });
            __syncthreads();
            for (int u = threadIdx.x; u < quads * ((end - base + 15) >> 4); u += THREADS) {
                const int j = u >> qshift, d = (u & (quads - 1)) * 4, t0 = base + 16 * j;
                uint32_t r[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = *reinterpret_cast<const uint32_t *>(&tile[(16 * j + k) * stride + d]);
                u32x4 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // 4 tokens x 4 dims of bytes
                    const uint32_t p0 = __builtin_amdgcn_perm(r[4 * k + 1], r[4 * k], 0x05010400u);
                    const uint32_t p1 = __builtin_amdgcn_perm(r[4 * k + 3], r[4 * k + 2], 0x05010400u);
                    const uint32_t q0 = __builtin_amdgcn_perm(r[4 * k + 1], r[4 * k], 0x07030602u);
                    const uint32_t q1 = __builtin_amdgcn_perm(r[4 * k + 3], r[4 * k + 2], 0x07030602u);
                    o[0][k] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
                    o[1][k] = __builtin_amdgcn_perm(p1, p0, 0x07060302u);
                    o[2][k] = __builtin_amdgcn_perm(q1, q0, 0x05040100u);
                    o[3][k] = __builtin_amdgcn_perm(q1, q0, 0x07060302u);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint8_t *dst = codes + (size_t)(d + x) * page + t0;
                    if (t0 >= a && t0 + 16 <= a + m) {
                        *reinterpret_cast<u32x4 *>(dst) = o[x];
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (t0 + k >= a && t0 + k < a + m) dst[k] = (uint8_t)(o[x][k >> 2] >> (8 * (k & 3)));
                    }
                }
            }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_kv_append(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const CacheArgs &c,
                            const SeqArgs &s, hipStream_t stream) {
    if (!s.rows) {
        // single tokens: one wave per (sequence, head)
        kv_append_kernel<64><<<dim3((unsigned)s.B, (unsigned)c.heads, 2), dim3(64), 0, stream>>>(k, ldk, v, ldv, c, s);
    } else {
        const unsigned ids = (unsigned)((s.T >> c.page_shift) + 2 * (int64_t)s.B);
        kv_append_kernel<256><<<dim3(ids, (unsigned)c.heads, 2), dim3(256), 0, stream>>>(k, ldk, v, ldv, c, s);
    }
    return hipGetLastError();
}

}  // namespace w4a16
