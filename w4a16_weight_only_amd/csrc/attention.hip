// attention.hip -- causal attention over the paged 8-bit cache.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale * q_i . k_j - m_i)
// over positions j <= pos_i (and j > pos_i - window), one pass over the cache
// with the running maximum m_i and sum of each row.
//
// Columns.  The rows of one sequence that share a key/value head -- its tokens
// times the query heads of the group -- are the columns c of the products
// S^T = K Q^T and O^T = V^T P^T, 16 at a time: column c is row c / group, head
// c % group.  S^T leaves the matrix cores with lane (c, g) holding four
// consecutive rows per 16 x 16 tile, and rows may stand for any tokens, so
// tile t's row 4g + i is made token 16g + 4t + i of a 64-token chunk: lane
// (c, g) then holds P for tokens 16g .. 16g + 15, which is what the second
// product takes as its operand (8 per instruction), with no exchange between
// lanes.  Each lane reads its keys and values 16 bytes at a time, and a lane's
// 16 tokens lie in one page (pages are 16 tokens or more), so one scale per
// lane dequantises them: to fp16, exactly (kv_append.hip).
//
// Rounding: q and k are exact in fp16, their products summed in fp32; the
// softmax runs in fp32; P is rounded once to fp16 for the second product
// (2^-12 of each weight at most, against 2^-12 of the result's own rounding),
// the sums of P stay unrounded in fp32, and so does O until the output.
//
// The maximum a column's weights are taken against is raised only when some
// score passes it by 2^8 (weights then stay below 2^8, far inside fp16), so
// most chunks neither exchange maxima between lanes nor rescale O.
//
// Splits: each (column tile, key/value head) is cut into pieces of `quota`
// chunks, and with few columns the four waves of a workgroup take chunks in
// turn and meet in LDS; pieces meet through the caller's workspace in a second
// kernel, in order, so results do not depend on timing.
#include "device.h"
#include "layer.h"

namespace w4a16 {
namespace {

constexpr int kChunk = 64;
constexpr float kLazy = 8.0f;  // in powers of two

struct Params {
    const uint16_t *q;
    int64_t ldq;
    CacheArgs c;
    SeqArgs s;
    int heads, group;
    float scale;  // softmax scale times log2(e)
    int window;   // 0: none
    uint16_t *out;
    float *part;  // [tiles, kv heads, splits, cols, dim], then [.., 2]
    float *ml;
    int tiles, splits, quota, cols;
};

__device__ __forceinline__ f16x8 dequant8(uint32_t a, uint32_t b, float s) {
    const f16x2 r0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, s, false);
    const f16x2 r1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, s, true);
    const f16x2 r2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, s, false);
    const f16x2 r3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, s, true);
    return f16x8{r0[0], r0[1], r1[0], r1[1], r2[0], r2[1], r3[0], r3[1]};
}

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// A scale byte as its power of two; bytes outside what the cache writer
// produces are brought into its range.
__device__ __forceinline__ float scale_of(uint8_t byte) {
    int e = (int)byte - 127;
    e = e < kKvMinExp ? kKvMinExp : e > kKvMaxExp ? kKvMaxExp : e;
    return pow2f(e);
}

// The column tile and sequence of a workgroup, computed alike by both kernels.
struct Tile {
    int b, r0, n;   // sequence, its first row and rows
    int c0, ncols;  // first column of the tile, columns of the sequence
    int first;      // position of the sequence's first row (may be negative)
    int cap;        // positions the table can hold
    int lo, hi;     // token range any of the tile's columns sees
    int split0, active;  // first chunk, and splits with work
};

__device__ __forceinline__ Tile make_tile(const Params &p, int tile) {
    Tile t;
    const int cols = p.cols;
    auto start = [&](int b) {
        int r = b;
        if (p.s.rows) {
            r = p.s.rows[b];
            r = r < 0 ? 0 : r > p.s.T ? p.s.T : r;
        }
        return (int64_t)((uint32_t)(r * p.group) / (uint32_t)cols) + b;
    };
    t.b = find_sequence(p.s.B, tile, start);
    sequence_rows(p.s, t.b, t.r0, t.n);
    t.ncols = t.n * p.group;
    const int64_t c0 = (tile - start(t.b)) * cols;  // negative only for a malformed offset table
    t.c0 = c0 < 0 || c0 >= t.ncols ? t.ncols : (int)c0;
    const int64_t len = p.s.lens[t.b] < 0 ? 0 : p.s.lens[t.b];
    t.first = (int)(len - t.n);
    t.cap = p.s.max_pages << p.c.page_shift;
    int lastc = t.c0 + cols < t.ncols ? t.c0 + cols : t.ncols;
    lastc = lastc < 1 ? 1 : lastc;
    const int64_t hi = (int64_t)t.first + (lastc - 1) / p.group + 1;
    const int64_t lo = p.window ? (int64_t)t.first + t.c0 / p.group - p.window + 1 : 0;
    t.hi = (int)(hi < 0 ? 0 : hi > t.cap ? t.cap : hi);
    t.lo = (int)(lo < 0 ? 0 : lo > t.hi ? t.hi : lo);
    t.split0 = t.lo / kChunk;
    const int chunks = t.hi > t.lo ? (t.hi + kChunk - 1) / kChunk - t.split0 : 0;
    t.active = (chunks + p.quota - 1) / p.quota;
    return t;
}

// 1 / l for a row at position pos.  A row that sees nothing is zero; one that
// sees tokens but has no weight (every score -inf) is NaN, as the formula says.
__device__ __forceinline__ float inverse(float l, int pos) {
    return l != 0.f ? 1.0f / l : pos < 0 ? 0.f : __builtin_nanf("");
}

// NT 16-column tiles per wave.  SHARED: the workgroup's four waves hold the
// same columns and take chunks in turn; otherwise wave w holds columns
// [w * 16 NT, (w + 1) * 16 NT) of the tile and walks all of its chunks.
template <int D, int NT, bool SHARED>
__global__ __launch_bounds__(256) void attention_kernel(Params p) {
    constexpr int KD = D / 64;   // 16-byte key loads per lane and 16-token tile
    constexpr int DT = D / 16;   // output tiles along dim
    __shared__ __align__(16) float lds_o[SHARED ? 4 * 16 * D : 4];
    __shared__ float lds_ml[SHARED ? 4 * 16 * 2 : 2];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, g = lane >> 4, kx = col >> 2;
    const int kvh = blockIdx.x % p.c.heads;
    const int rest = blockIdx.x / p.c.heads;
    const int split = rest % p.splits;
    const int tile = p.tiles - 1 - rest / p.splits;
    const Tile t = make_tile(p, tile);
    if (t.c0 >= t.ncols || (split > 0 && split >= t.active)) return;

    // this wave's columns and chunks
    const int wc0 = t.c0 + (SHARED ? 0 : wave * 16 * NT);
    int clo = t.split0 + split * p.quota;
    int chi = (t.hi + kChunk - 1) / kChunk;
    chi = chi < clo + p.quota ? chi : clo + p.quota;
    if (t.hi <= t.lo) chi = clo;
    int pos[NT];
    bool live[NT];
    int wcl = wc0 + 16 * NT < t.ncols ? wc0 + 16 * NT : t.ncols;  // end of the valid ones
    if (!SHARED) {
        if (wc0 >= t.ncols) return;
        const int64_t whi = (int64_t)t.first + (wcl - 1) / p.group + 1;
        const int wch = whi <= 0 ? 0 : (int)((whi + kChunk - 1) / kChunk);
        chi = chi < wch ? chi : wch;
        if (p.window) {
            const int64_t wlo = (int64_t)t.first + wc0 / p.group - p.window + 1;
            const int wcl0 = wlo <= 0 ? 0 : (int)(wlo / kChunk);
            clo = clo > wcl0 ? clo : wcl0;
        }
    }
    const int pos_min = t.first + wc0 / p.group, pos_max = t.first + (wcl - 1) / p.group;

    // Q fragments: lane (c, g) holds dims 64m + 16g .. + 15 of column c, the
    // order in which it reads keys.
    f16x8 qf[NT][2 * KD];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int cc = wc0 + 16 * n + col;
        live[n] = cc < t.ncols;
        const int i = live[n] ? cc / p.group : 0, h = live[n] ? cc - i * p.group : 0;
        pos[n] = live[n] ? t.first + i : pos_max;
        const uint16_t *src = p.q + (int64_t)(t.r0 + i) * p.ldq + (int64_t)(kvh * p.group + h) * D + 16 * g;
#pragma unroll
        for (int m = 0; m < KD; ++m)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                u32x4 v{0u, 0u, 0u, 0u};
                if (live[n]) v = *reinterpret_cast<const u32x4 *>(src + 64 * m + 8 * x);
                qf[n][2 * m + x] = __builtin_bit_cast(f16x8, v);
            }
    }

    f32x4 o[NT][DT];
    float mx[NT], sum[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        mx[n] = -__builtin_inff();
        sum[n] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const size_t page_bytes = (size_t)D << p.c.page_shift;
    const int page_mask = (1 << p.c.page_shift) - 1;
    const int32_t *table = p.s.table + (int64_t)t.b * p.s.max_pages;
    // Page of the 16-token block x of chunk c: -1 where the block lies behind
    // the tile's tokens (nothing there is read), -2 where the table's entry is
    // out of range.
    auto page_of = [&](int c, int x) {
        const int tok = c * kChunk + 16 * x;
        if (tok >= t.hi) return -1;
        const int id = table[tok >> p.c.page_shift];
        return id < 0 || id >= p.c.pages ? -2 : id;
    };
    for (int c = SHARED ? clo + wave : clo; c < chi; c += SHARED ? 4 : 1) {
        const int pk = page_of(c, kx), pv = page_of(c, g);
        const size_t sk = (size_t)(pk < 0 ? 0 : pk) * p.c.heads + kvh, sv = (size_t)(pv < 0 ? 0 : pv) * p.c.heads + kvh;
        const int offk = (c * kChunk + 16 * kx) & page_mask, offv = (c * kChunk + 16 * g) & page_mask;
        const uint8_t *kp = p.c.k + sk * page_bytes + (size_t)(offk + (col & 3)) * D + 16 * g;
        const uint8_t *vp = p.c.v + sv * page_bytes + ((size_t)col << p.c.page_shift) + offv;
        const float fk = scale_of(p.c.k_scale[sk]), fv = scale_of(p.c.v_scale[sv]);
        u32x4 kr[4][KD], vr[DT];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int m = 0; m < KD; ++m) kr[x][m] = *reinterpret_cast<const u32x4 *>(kp + (size_t)(4 * x) * D + 64 * m);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            vr[d] = *reinterpret_cast<const u32x4 *>(vp + ((size_t)(16 * d) << p.c.page_shift));

        f32x4 sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[n][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int m = 0; m < KD; ++m) {
                const f16x8 a0 = dequant8(kr[x][m][0], kr[x][m][1], fk), a1 = dequant8(kr[x][m][2], kr[x][m][3], fk);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    sc[n][x] = mfma16(a0, qf[n][2 * m], sc[n][x]);
                    sc[n][x] = mfma16(a1, qf[n][2 * m + 1], sc[n][x]);
                }
            }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][x][i] *= p.scale;

        // Chunks that some column does not see whole: masked scores are set to
        // -inf whatever they hold, a page out of range makes them NaN, and NaN
        // codes among the values are taken out, to be put back only for the
        // columns that see them.
        const int c_lo = c * kChunk, c_hi = c_lo + kChunk;
        const bool partial = c_hi - 1 > pos_min || (p.window && c_lo <= pos_max - p.window);
        bool odd = false;  // some value code was NaN
        u32x4 vnan[DT];
        if (partial || __any(pk == -2 || pv == -2)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = c_lo + 16 * g + 4 * x + i;
                        const bool seen = tok <= pos[n] && (!p.window || tok > pos[n] - p.window) && tok < t.hi;
                        sc[n][x][i] = !seen ? -__builtin_inff() : pv == -2 ? __builtin_nanf("") : sc[n][x][i];
                    }
            // tokens past the tile's last (or on a page out of range): zero codes,
            // whatever lies there (old codes may even overflow at the new scale)
            const int left = pv < 0 ? 0 : t.hi - (c_lo + 16 * g);
            uint32_t any = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = left - 4 * j;
                const uint32_t keep = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    vr[d][j] &= keep;
                    const uint32_t bad = nan_bits(vr[d][j]);
                    any |= bad;
                    vnan[d][j] = (bad >> 7) * 0x38u;  // 1.0 where the code was NaN
                    vr[d][j] &= ~((bad >> 7) * 0xffu);
                }
            }
            odd = __any(any != 0);
        }

        // Running maxima: raised when a score passes them by kLazy.
        f16x8 pf[NT][2], seen_f[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top = -__builtin_inff();
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[n][x][i]);
            if (__any(top > mx[n] + kLazy)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float m = fmaxf(mx[n], top);
                const float f = m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(mx[n] - m);
                mx[n] = m;
                sum[n] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][d][i] *= f;
            }
            const float base = mx[n] == -__builtin_inff() ? 0.f : mx[n];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(sc[n][x][i] - base);
                    sum[n] += e;
                    pf[n][x >> 1][4 * (x & 1) + i] = (f16)e;
                    if (odd) seen_f[n][x >> 1][4 * (x & 1) + i] = sc[n][x][i] == -__builtin_inff() ? (f16)0 : (f16)1;
                }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const f16x8 a0 = dequant8(vr[d][0], vr[d][1], fv), a1 = dequant8(vr[d][2], vr[d][3], fv);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n][d] = mfma16(a0, pf[n][0], o[n][d]);
                o[n][d] = mfma16(a1, pf[n][1], o[n][d]);
            }
        }
        if (odd) {
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const f16x8 a0 = dequant8(vnan[d][0], vnan[d][1], 1.f), a1 = dequant8(vnan[d][2], vnan[d][3], 1.f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    f32x4 z{0.f, 0.f, 0.f, 0.f};
                    z = mfma16(a0, seen_f[n][0], z);
                    z = mfma16(a1, seen_f[n][1], z);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (z[i] > 0.f) o[n][d][i] = __builtin_nanf("");
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        sum[n] += __shfl_xor(sum[n], 16);
        sum[n] += __shfl_xor(sum[n], 32);
        if (pos[n] >= t.cap) sum[n] = __builtin_nanf("");  // longer than its table: loud
    }

    const int64_t slot = ((int64_t)tile * p.c.heads + kvh) * p.splits + split;
    if constexpr (!SHARED) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int cc = wc0 + 16 * n + col;
            if (!live[n]) continue;
            if (t.active <= 1) {
                const int i = cc / p.group, h = cc - i * p.group;
                uint16_t *dst = p.out + ((int64_t)(t.r0 + i) * p.heads + kvh * p.group + h) * D + 4 * g;
                const float f = inverse(sum[n], t.first + i);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    u32x2 w;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        w[j] = (uint32_t)f32_to_f16_bits(o[n][d][2 * j] * f) |
                               ((uint32_t)f32_to_f16_bits(o[n][d][2 * j + 1] * f) << 16);
                    *reinterpret_cast<u32x2 *>(dst + 16 * d) = w;
                }
            } else {
                float *dst = p.part + (slot * p.cols + (cc - t.c0)) * D + 4 * g;
#pragma unroll
                for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4 *>(dst + 16 * d) = o[n][d];
                if (g == 0) {
                    p.ml[(slot * p.cols + (cc - t.c0)) * 2] = mx[n];
                    p.ml[(slot * p.cols + (cc - t.c0)) * 2 + 1] = sum[n];
                }
            }
        }
    } else {
        // The waves' pieces meet in LDS, in wave order.
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<f32x4 *>(&lds_o[(wave * 16 + col) * D + 16 * d + 4 * g]) = o[0][d];
        if (g == 0) {
            lds_ml[(wave * 16 + col) * 2] = mx[0];
            lds_ml[(wave * 16 + col) * 2 + 1] = sum[0];
        }
        __syncthreads();
        for (int x = threadIdx.x; x < 16 * D / 4; x += 256) {
            const int cc = x / (D / 4), d = (x - cc * (D / 4)) * 4;
            if (t.c0 + cc >= t.ncols) continue;
            float m = -__builtin_inff();
#pragma unroll
            for (int w = 0; w < 4; ++w) m = fmaxf(m, lds_ml[(w * 16 + cc) * 2]);
            f32x4 a{0.f, 0.f, 0.f, 0.f};
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float mw = lds_ml[(w * 16 + cc) * 2], lw = lds_ml[(w * 16 + cc) * 2 + 1];
                const float f = mw == -__builtin_inff() ? (lw == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(mw - m);
                const f32x4 v = *reinterpret_cast<const f32x4 *>(&lds_o[(w * 16 + cc) * D + d]);
                l += lw * f;
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j] = __builtin_fmaf(v[j], f, a[j]);
            }
            const int c = t.c0 + cc;
            if (t.active <= 1) {
                const int i = c / p.group, h = c - i * p.group;
                const float f = inverse(l, t.first + i);
                u32x2 w;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    w[j] = (uint32_t)f32_to_f16_bits(a[2 * j] * f) | ((uint32_t)f32_to_f16_bits(a[2 * j + 1] * f) << 16);
                *reinterpret_cast<u32x2 *>(p.out + ((int64_t)(t.r0 + i) * p.heads + kvh * p.group + h) * D + d) = w;
            } else {
                *reinterpret_cast<f32x4 *>(p.part + (slot * p.cols + cc) * D + d) = a;
                if (d == 0) {
                    p.ml[(slot * p.cols + cc) * 2] = m;
                    p.ml[(slot * p.cols + cc) * 2 + 1] = l;
                }
            }
        }
    }
}

// Joins a column tile's pieces: 16 columns per workgroup, 4 dims per thread.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(Params p) {
    const int kvh = blockIdx.x % p.c.heads, tile = blockIdx.x / p.c.heads;
    const Tile t = make_tile(p, tile);
    if (t.active <= 1) return;
    const int64_t slot = ((int64_t)tile * p.c.heads + kvh) * p.splits;
    for (int x = threadIdx.x; x < 16 * D / 4; x += 256) {
        const int cc = blockIdx.y * 16 + x / (D / 4), d = (x % (D / 4)) * 4;
        if (t.c0 + cc >= t.ncols) continue;
        float m = -__builtin_inff();
        for (int s = 0; s < t.active; ++s) m = fmaxf(m, p.ml[((slot + s) * p.cols + cc) * 2]);
        f32x4 a{0.f, 0.f, 0.f, 0.f};
        float l = 0.f;
        for (int s = 0; s < t.active; ++s) {
            const float ms = p.ml[((slot + s) * p.cols + cc) * 2], ls = p.ml[((slot + s) * p.cols + cc) * 2 + 1];
            const float f = ms == -__builtin_inff() ? (ls == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(ms - m);
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p.part + ((slot + s) * p.cols + cc) * D + d);
            l += ls * f;
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = __builtin_fmaf(v[j], f, a[j]);
        }
        const int c = t.c0 + cc, i = c / p.group, h = c - i * p.group;
        const float f = inverse(l, t.first + i);
        u32x2 w;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[j] = (uint32_t)f32_to_f16_bits(a[2 * j] * f) | ((uint32_t)f32_to_f16_bits(a[2 * j + 1] * f) << 16);
        *reinterpret_cast<u32x2 *>(p.out + ((int64_t)(t.r0 + i) * p.heads + kvh * p.group + h) * D + d) = w;
    }
}

template <int D>
hipError_t launch(const Params &p, const AttnPlan &plan, hipStream_t stream) {
    const dim3 grid((unsigned)(plan.tiles * p.c.heads * plan.splits));
    if (plan.shared) attention_kernel<D, 1, true><<<grid, dim3(256), 0, stream>>>(p);
    else if (plan.nt == 1 || D == 256) attention_kernel<D, 1, false><<<grid, dim3(256), 0, stream>>>(p);
    else attention_kernel<D, 2, false><<<grid, dim3(256), 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || plan.splits <= 1) return e;
    attention_join_kernel<D><<<dim3((unsigned)(plan.tiles * p.c.heads), (unsigned)(plan.cols / 16)), dim3(256), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(int64_t heads, int64_t kv_heads, int64_t dim, int64_t page, int64_t max_pages, int64_t B,
                        int64_t T) {
    AttnPlan p;
    const int64_t group = heads / kv_heads;
    const int64_t per = (T * group + B - 1) / B;  // columns of the average sequence
    p.shared = per <= 16;
    p.nt = p.shared || per <= 64 || dim == 256 ? 1 : 2;
    p.cols = p.shared ? 16 : 64 * p.nt;
    p.tiles = T * group / p.cols + B;
    const int64_t chunks = (max_pages * page + kChunk - 1) / kChunk;
    const int64_t wgs = p.tiles * kv_heads;
    int64_t splits = (1024 + wgs - 1) / wgs;
    const int64_t least = p.shared ? 8 : 4;  // chunks per split worth a piece of its own
    splits = splits < chunks / least ? splits : chunks / least;
    const int64_t piece = wgs * p.cols * (dim + 2);  // floats per split
    const int64_t cap = ((int64_t)256 << 20) / 4 / piece;
    splits = splits < cap ? splits : cap;
    splits = splits < 1 ? 1 : splits;
    p.quota = (int)((chunks + splits - 1) / splits);
    p.quota = p.quota < 1 ? 1 : p.quota;
    p.splits = (int)((chunks + p.quota - 1) / p.quota);
    p.splits = p.splits < 1 ? 1 : p.splits;
    p.part_floats = p.splits > 1 ? (size_t)(piece * p.splits) : 0;
    return p;
}

hipError_t launch_attention(const uint16_t *q, int64_t ldq, int heads, const CacheArgs &c, const SeqArgs &s,
                            float scale, int64_t window, uint16_t *out, float *workspace, const AttnPlan &plan,
                            hipStream_t stream) {
    Params p;
    p.q = q;
    p.ldq = ldq;
    p.c = c;
    p.s = s;
    p.heads = heads;
    p.group = heads / c.heads;
    p.scale = scale * 1.44269504088896341f;
    p.window = (int)window;
    p.out = out;
    p.tiles = (int)plan.tiles;
    p.splits = plan.splits;
    p.quota = plan.quota;
    p.cols = plan.cols;
    p.part = workspace;
    p.ml = workspace ? workspace + plan.tiles * c.heads * plan.splits * plan.cols * c.dim : nullptr;
    switch (c.dim) {
        case 64: return launch<64>(p, plan, stream);
        case 128: return launch<128>(p, plan, stream);
        case 256: return launch<256>(p, plan, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace w4a16
