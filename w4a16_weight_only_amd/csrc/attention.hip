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
// softmax runs in fp32.  For the second product the row kernel rounds P once to
// fp16 (2^-11 of each weight, as large as the result's own rounding; the sums
// take the rounded weights too, so that a row stays a mean of its values), at
// the rate of the matrix cores.  The token kernel, bound by reading the cache,
// carries each weight as two fp16 values (2^-22 of it).  Either holds weights
// below 2^-25 of the row's largest to 2^-36 of that one (kLift).  O and the sums
// of P are fp32 until the output.  Two values in the row kernel too: prompts of
// 4096 rows 850 us, 617 with one.
//
// The maximum a column's weights are taken against is raised only when some
// score passes it by 2^kLazy, so most chunks neither exchange maxima between
// lanes nor rescale O.
//
// Splits: each (column tile, key/value head) is cut into pieces of `quota`
// chunks, and with few columns the four waves of a workgroup take chunks in
// turn and meet in LDS; pieces meet through the caller's workspace in a second
// kernel, in order, so results do not depend on timing.
#include "device.h"
#include "layer.h"

#include <type_traits>

namespace w4a16 {
namespace {

constexpr int kChunk = 64;
// In powers of two: how far a score may pass the running maximum before that is
// raised, and how far above 1 a weight of the maximum itself stands.  Weights
// stay below 2^(kLazy + kLift) = 2^15, inside fp16, and keep fp16's full
// precision down to 2^-25 of the row's largest, the last of them at 2^-36: a row
// with one dominant token and a long tail under it keeps the tail.
// Measured: prompts of 4096 rows 617 us, 613 with 8 and no lift (tail lost at
// 2^-25), 8 and 7 between the two; single tokens alike.
constexpr float kLazy = 4.0f, kLift = 11.0f;
constexpr float kSteep = 0x1p20f;  // in powers of two; fp32 holds such a maximum to 2^-4

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
    int64_t first_tile;
    if (!p.s.rows) {
        const int per = (p.group + cols - 1) / cols;
        t.b = tile / per;
        first_tile = (int64_t)t.b * per;
    } else {
        auto start = [&](int b) {
            int r = p.s.rows[b];
            r = r < 0 ? 0 : r > p.s.T ? p.s.T : r;
            return (int64_t)((uint32_t)(r * p.group) / (uint32_t)cols) + b;
        };
        t.b = find_sequence(p.s.B, tile, start);
        first_tile = start(t.b);
    }
    sequence_rows(p.s, t.b, t.r0, t.n);
    t.ncols = t.n * p.group;
    const int64_t c0 = (tile - first_tile) * cols;  // negative only for a malformed offset table
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
    t.split0 = p.window ? t.lo / kChunk : 0;
    const int chunks = t.hi > t.lo ? (t.hi + kChunk - 1) / kChunk - t.split0 : 0;
    t.active = (chunks + p.quota - 1) / p.quota;
    return t;
}

// 1 / l for a row at position pos.  A row that sees nothing is zero; one that
// sees tokens but has no weight (every score -inf) is NaN, as the formula says.
__device__ __forceinline__ float inverse(float l, int pos) {
    return l != 0.f ? 1.0f / l : pos < 0 ? 0.f : __builtin_nanf("");
}

// Pages of a column tile's tokens.  lookup() gives the page of the 16-token
// block x of chunk c: -1 where the block lies behind the tile's tokens (nothing
// there is used), -2 where the table's entry is out of range; slot() a page's
// place among the cache's (page, head) pairs, page 0 for either.
struct Pages {
    const int32_t *table;
    int64_t pages;
    int heads, kvh, shift, hi, last;
    __device__ __forceinline__ Pages(const Params &p, const Tile &t, int kvh_)
        : table(p.s.table + (int64_t)t.b * p.s.max_pages), pages(p.c.pages), heads(p.c.heads), kvh(kvh_),
          shift(p.c.page_shift), hi(t.hi), last(p.s.max_pages - 1) {}
    // (The table is read at any place inside it, so that the read need not
    // wait for the sequence's length.)
    __device__ __forceinline__ int lookup(int c, int x) const {
        const int tok = c * kChunk + 16 * x, at = tok >> shift;
        const int id = table[at < last ? at : last];
        return tok >= hi ? -1 : id < 0 || id >= pages ? -2 : id;
    }
    // The same where a whole chunk lies in one page.
    __device__ __forceinline__ int lookup(int c) const { return __builtin_amdgcn_readfirstlane(lookup(c, 0)); }
    __device__ __forceinline__ size_t slot(int page) const { return (size_t)(page < 0 ? 0 : page) * heads + kvh; }
    // byte offset of block x of chunk c within its page's rows of D (keys)
    __device__ __forceinline__ int within(int c, int x) const { return (c * kChunk + 16 * x) & ((1 << shift) - 1); }
};

// NT tiles of 16 columns held by one wave: queries, running maxima, the sums of
// the weights (one more row of O, from values of one) and O, all of it fp32.
// FINE: weights enter the second product as two fp16 values, the second what
// the first left over: good to 2^-22, or where that is more to 2^-36 of the row's
// largest.
template <int D, int NT, bool FINE>
struct Columns {
    static constexpr int PARTS = FINE ? 2 : 1;
    static constexpr int KD = D / 64;  // 16-byte key pieces per lane and 16-token tile
    static constexpr int DT = D / 16;  // output tiles along dim

    int pos[NT];   // position of this lane's column
    bool live[NT];
    int pos_min, pos_max;
    f16x8 qf[NT][2 * KD];
    f32x4 o[NT][DT], l[NT];
    float mx[NT];  // of scores before their scale
    float scale, lazy;
    int window, hi;
    bool steep;  // some column's maximum is kSteep or more: only masked chunks from here on

    // Columns wc0 .. wc0 + 16 NT of the tile's sequence.  Lane (c, g) holds
    // dims 64m + 16g .. + 15 of column c's query, the order in which keys come.
    __device__ __forceinline__ void init(const Params &p, const Tile &t, int kvh, int wc0) {
        const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
        // A negative scale goes into the sign of q, so that the largest product
        // has the largest score.  (The floor keeps a scale of zero from meeting
        // the infinities of masked scores; products are below 2^40, so nothing
        // else sees it.)
        scale = fmaxf(__builtin_fabsf(p.scale), 0x1p-100f);
        lazy = kLazy / scale;
        window = p.window;
        hi = t.hi;
        steep = false;
        const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
        const int end = wc0 + 16 * NT < t.ncols ? wc0 + 16 * NT : t.ncols;
        pos_min = t.first + wc0 / p.group;
        pos_max = t.first + (end - 1) / p.group;
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
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] ^= flip;
                    qf[n][2 * m + x] = __builtin_bit_cast(f16x8, v);
                }
            mx[n] = -__builtin_inff();
            l[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int d = 0; d < DT; ++d) o[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }

    // Scores of chunk c: S^T, before the scale.  key(x, m): this lane's piece m
    // of its token of tile x.
    template <typename Key>
    __device__ __forceinline__ void scores(f32x4 (&sc)[NT][4], Key key, float fk) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < KD; ++m) {
                const u32x4 k = key(x, m);
                const f16x8 a0 = dequant8(k[0], k[1], fk), a1 = dequant8(k[2], k[3], fk);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    sc[n][x] = mfma16(a0, qf[n][2 * m], sc[n][x]);
                    sc[n][x] = mfma16(a1, qf[n][2 * m + 1], sc[n][x]);
                }
            }
        }
    }

    // The chunks [lo, hi) of [from, to) that every column sees whole.
    __device__ __forceinline__ void clean_range(int from, int to, int &lo, int &hi) const {
        const int end = pos_min < 0 ? 0 : (pos_min + 1) / kChunk;
        const int start = !window || pos_max < window ? 0 : (pos_max - window) / kChunk + 1;
        lo = start < from ? from : start > to ? to : start;
        hi = end > to ? to : end;
        hi = hi < lo ? lo : hi;
    }

    // Masked scores become -inf whatever they hold; a page out of range (of
    // this lane's tokens) makes the ones that are seen NaN.
    __device__ __forceinline__ void mask(f32x4 (&sc)[NT][4], int c, bool bad) const {
        const int tok0 = c * kChunk + 16 * ((threadIdx.x & 63) >> 4);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = tok0 + 4 * x + i;
                    const bool seen = tok <= pos[n] && (!window || tok > pos[n] - window) && tok < hi;
                    sc[n][x][i] = !seen ? -__builtin_inff() : bad ? __builtin_nanf("") : sc[n][x][i];
                }
    }

    // Weights of a chunk, as fp16.  The running maxima are raised when a score
    // passes them by kLazy after its scale.  In CLEAN chunks a weight is one fma
    // and exp2: the rounding of its base is common to the column and cancels, as
    // long as the weights stay inside fp16.  Past kSteep they might not, so there,
    // and in all other chunks, scores are taken from their maximum first.  (A
    // branch on steep in every chunk instead: prompts of 4096 rows 643 us.)
    template <bool CLEAN>
    __device__ __forceinline__ void weights(f32x4 (&sc)[NT][4], f16x8 (&pf)[NT][PARTS][2]) {
        float top[NT];
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            top[n] = -__builtin_inff();
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) top[n] = fmaxf(top[n], sc[n][x][i]);
            raise = raise || top[n] > mx[n] + lazy;
        }
        auto from_maximum = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[n][x][i] -= mx[n] == -__builtin_inff() ? 0.f : mx[n];
        };
        if (__any(raise)) {
            bool far = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                top[n] = fmaxf(top[n], __shfl_xor(top[n], 16));
                top[n] = fmaxf(top[n], __shfl_xor(top[n], 32));
                const float m = fmaxf(mx[n], top[n]);
                const float f = m == mx[n] ? 1.0f : __builtin_amdgcn_exp2f((mx[n] - m) * scale);
                mx[n] = m;
                far = far || (m != -__builtin_inff() && __builtin_fabsf(m * scale) >= kSteep);
#pragma unroll
                for (int i = 0; i < 4; ++i) l[n][i] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][d][i] *= f;
            }
            if (__any(far)) {
                steep = true;
                if constexpr (CLEAN) from_maximum();
            }
        }
        if constexpr (!CLEAN) from_maximum();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float base = mx[n] == -__builtin_inff() ? 0.f : !CLEAN || steep ? -kLift : max2(n);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][x][i], scale, -base));
                    const f16 h = (f16)e;
                    pf[n][0][x >> 1][4 * (x & 1) + i] = h;
                    if constexpr (FINE) pf[n][1][x >> 1][4 * (x & 1) + i] = (f16)(e - (float)h);
                }
        }
    }

    // O += V^T P.  value(d): this lane's 16 codes of output tile d.  CLEAN: every
    // column sees the whole chunk, and NaN among the values is every column's.
    // Otherwise codes of tokens past the tile's last (or on a page out of
    // range: left 0) count as zero, whatever lies there (old codes may even
    // overflow at the new scale), and NaN codes are taken out and put back only
    // for the columns that see them: those for which a product of ones counts.
    template <bool CLEAN, typename Value>
    __device__ __forceinline__ void values(const f32x4 (&sc)[NT][4], const f16x8 (&pf)[NT][PARTS][2], Value value, float fv,
                                           int left) {
        f16x8 ones;
#pragma unroll
        for (int j = 0; j < 8; ++j) ones[j] = (f16)1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                l[n] = mfma16(ones, pf[n][q][0], l[n]);
                l[n] = mfma16(ones, pf[n][q][1], l[n]);
            }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            u32x4 v = value(d);
            if constexpr (!CLEAN) {
                uint32_t any = 0, count[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = left - 4 * j;
                    v[j] &= n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                    const uint32_t nan = nan_bits(v[j]) >> 7;
                    any |= nan;
                    count[j] = nan * 0x38u;  // e4m3 1.0
                    v[j] &= ~(nan * 0xffu);
                }
                if (__any(any != 0)) {
                    const f16x8 a0 = dequant8(count[0], count[1], 1.f), a1 = dequant8(count[2], count[3], 1.f);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        f16x8 s0, s1;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            s0[j] = sc[n][j >> 2][j & 3] == -__builtin_inff() ? (f16)0 : (f16)1;
                            s1[j] = sc[n][2 + (j >> 2)][j & 3] == -__builtin_inff() ? (f16)0 : (f16)1;
                        }
                        f32x4 z{0.f, 0.f, 0.f, 0.f};
                        z = mfma16(a0, s0, z);
                        z = mfma16(a1, s1, z);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (z[i] > 0.f) o[n][d][i] = __builtin_nanf("");
                    }
                }
            }
            const f16x8 a0 = dequant8(v[0], v[1], fv), a1 = dequant8(v[2], v[3], fv);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                    o[n][d] = mfma16(a0, pf[n][q][0], o[n][d]);
                    o[n][d] = mfma16(a1, pf[n][q][1], o[n][d]);
                }
            }
        }
    }

    // What this lane's column takes weights against, in powers of two, and their
    // sum; NaN for a row longer than its table, and where every column saw a page
    // out of range.
    __device__ __forceinline__ float max2(int n) const { return __builtin_fmaf(mx[n], scale, -kLift); }
    __device__ __forceinline__ float total(int n, int cap, bool lost) const {
        return lost || pos[n] >= cap ? __builtin_nanf("") : l[n][0];
    }

    // One chunk.  CLEAN: as for values().  page_v: the page of this lane's 16
    // tokens.
    template <bool CLEAN, typename Key, typename Value>
    __device__ __forceinline__ void chunk(int c, Key key, float fk, Value value, float fv, int page_v) {
        f32x4 sc[NT][4];
        f16x8 pf[NT][PARTS][2];
        // matrix instructions first: the other wave of the SIMD does its softmax
        // meanwhile (prompts 627 -> 619 us)
        __builtin_amdgcn_s_setprio(1);
        scores(sc, key, fk);
        __builtin_amdgcn_s_setprio(0);
        if constexpr (!CLEAN) mask(sc, c, page_v == -2);
        weights<CLEAN>(sc, pf);
        __builtin_amdgcn_s_setprio(1);
        values<CLEAN>(sc, pf, value, fv, page_v < 0 ? 0 : hi - (c * kChunk + 16 * (int)((threadIdx.x & 63) >> 4)));
        __builtin_amdgcn_s_setprio(0);
    }
};

__device__ __forceinline__ u32x2 pack4(const f32x4 &v, float f) {
    u32x2 w;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w[j] = (uint32_t)f32_to_f16_bits(v[2 * j] * f) | ((uint32_t)f32_to_f16_bits(v[2 * j + 1] * f) << 16);
    return w;
}

// This workgroup's place in the grid: key/value heads in turn (an XCD then
// keeps to the same heads), pieces of a tile, and tiles from the last, which
// see the most tokens.
struct Place {
    int kvh, split, tile;
    __device__ __forceinline__ explicit Place(const Params &p) {
        kvh = blockIdx.x % p.c.heads;
        const int rest = blockIdx.x / p.c.heads;
        split = rest % p.splits;
        tile = p.tiles - 1 - rest / p.splits;
    }
    __device__ __forceinline__ int64_t slot(const Params &p) const {
        return ((int64_t)tile * p.c.heads + kvh) * p.splits + split;
    }
};

// Few columns (single tokens): the workgroup's waves hold the same 16
// columns and take chunks in turn, keys and values straight from memory into
// registers.  Bound by reading the cache: 48 sequences to 16384 tokens, 8 heads
// of 128, 160 us for 811 MB (5.1 TB/s; a copy of 2 GiB reaches 4.9) and 6 us for
// the join.  Short caches are bound by latency: one sequence of 64 tokens 5.4 us
// in a graph, of 256 (a chunk for each wave) 6.9, 512 8.2, 1024 12.1.  The loop
// is pipelined: a chunk's keys are requested when those of the chunk before have
// been multiplied, its values when those of the chunk before have; its pages are
// looked up one chunk earlier still.
template <int D>
__global__ __launch_bounds__(256, (D == 64 ? 3 : D == 128 ? 2 : 1)) void attention_token_kernel(Params p) {
    constexpr int W = 4;
    constexpr int KD = D / 64, DT = D / 16;
    __shared__ __align__(16) float lds_o[W * 16 * D];
    __shared__ float lds_ml[W * 16 * 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4, kx = col >> 2;
    const Place at(p);
    const Tile t = make_tile(p, at.tile);
    if (t.c0 >= t.ncols || (at.split > 0 && at.split >= t.active)) return;
    const int clo = t.split0 + at.split * p.quota;
    int chi = t.hi > t.lo ? (t.hi + kChunk - 1) / kChunk : clo;
    chi = chi < clo + p.quota ? chi : clo + p.quota;

    Columns<D, 1, true> cs;
    cs.init(p, t, at.kvh, t.c0);
    const Pages pages(p, t, at.kvh);
    const size_t page_bytes = (size_t)D << p.c.page_shift;
    u32x4 kr[4][KD], vr[DT];
    int pk = -1, pv = -1;     // pages of the chunk whose keys / values are in hand
    uint32_t bk = 0, bv = 0;  // their scale bytes
    auto load_keys = [&](int c, int page) __attribute__((always_inline)) {
        const size_t sk = pages.slot(page);
        const uint8_t *kp = p.c.k + sk * page_bytes + (size_t)(pages.within(c, kx) + (col & 3)) * D + 16 * g;
        bk = p.c.k_scale[sk];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int m = 0; m < KD; ++m) kr[x][m] = *reinterpret_cast<const u32x4 *>(kp + 4 * x * D + 64 * m);
    };
    auto load_values = [&](int c, int page) __attribute__((always_inline)) {
        const size_t sv = pages.slot(page);
        const uint8_t *vp = p.c.v + sv * page_bytes + ((size_t)col << p.c.page_shift) + pages.within(c, g);
        bv = p.c.v_scale[sv];
#pragma unroll
        for (int d = 0; d < DT; ++d) vr[d] = *reinterpret_cast<const u32x4 *>(vp + ((size_t)(16 * d) << p.c.page_shift));
    };
    int c = clo + wave, pk_next = -1, pv_next = -1;
    if (c < chi) {
        pk = pages.lookup(c, kx);
        pv = pages.lookup(c, g);
        load_keys(c, pk);
        load_values(c, pv);
        if (c + W < chi) {
            pk_next = pages.lookup(c + W, kx);
            pv_next = pages.lookup(c + W, g);
        }
    }
    bool lost = false;
    auto turn = [&](auto clean) __attribute__((always_inline)) {
        const bool more = c + W < chi;
        int pk_after = -1, pv_after = -1;
        const int page_v = pv;
        if constexpr (decltype(clean)::value) lost = lost || __any(pk == -2 || pv == -2);
        f32x4 sc[1][4];
        f16x8 pf[1][2][2];
        cs.scores(sc, [&](int x, int m) { return kr[x][m]; }, scale_of((uint8_t)bk));
        if (more) {
            load_keys(c + W, pk_next);
            if (c + 2 * W < chi) {
                pk_after = pages.lookup(c + 2 * W, kx);
                pv_after = pages.lookup(c + 2 * W, g);
            }
        }
        if constexpr (!decltype(clean)::value) cs.mask(sc, c, page_v == -2);
        cs.template weights<decltype(clean)::value>(sc, pf);
        cs.template values<decltype(clean)::value>(sc, pf, [&](int d) { return vr[d]; }, scale_of((uint8_t)bv),
                                                   page_v < 0 ? 0 : t.hi - (c * kChunk + 16 * g));
        if (more) load_values(c + W, pv_next);
        pk = pk_next;
        pv = pv_next;
        pk_next = pk_after;
        pv_next = pv_after;
    };
    int clean_lo, clean_hi;
    cs.clean_range(clo, chi, clean_lo, clean_hi);
    for (; c < clean_lo; c += W) turn(std::false_type{});
    for (; c < clean_hi && !cs.steep; c += W) turn(std::true_type{});
    for (; c < chi; c += W) turn(std::false_type{});

    // The waves' pieces meet in LDS, in wave order.
#pragma unroll
    for (int d = 0; d < DT; ++d)
        *reinterpret_cast<f32x4 *>(&lds_o[(wave * 16 + col) * D + 16 * d + 4 * g]) = cs.o[0][d];
    if (g == 0) {
        lds_ml[(wave * 16 + col) * 2] = cs.max2(0);
        lds_ml[(wave * 16 + col) * 2 + 1] = cs.total(0, t.cap, lost);
    }
    __syncthreads();
    const int64_t slot = at.slot(p);
    for (int x = threadIdx.x; x < 16 * D / 4; x += 64 * W) {
        const int cc = x / (D / 4), d = (x - cc * (D / 4)) * 4;
        if (t.c0 + cc >= t.ncols) continue;
        float m = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < W; ++w) m = fmaxf(m, lds_ml[(w * 16 + cc) * 2]);
        f32x4 a{0.f, 0.f, 0.f, 0.f};
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float mw = lds_ml[(w * 16 + cc) * 2], lw = lds_ml[(w * 16 + cc) * 2 + 1];
            const float f = mw == -__builtin_inff() ? (lw == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(mw - m);
            const f32x4 v = *reinterpret_cast<const f32x4 *>(&lds_o[(w * 16 + cc) * D + d]);
            l += lw * f;
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = __builtin_fmaf(v[j], f, a[j]);
        }
        const int c2 = t.c0 + cc;
        if (t.active <= 1) {
            const int i = c2 / p.group, h = c2 - i * p.group;
            *reinterpret_cast<u32x2 *>(p.out + ((int64_t)(t.r0 + i) * p.heads + at.kvh * p.group + h) * D + d) =
                pack4(a, inverse(l, t.first + i));
        } else {
            *reinterpret_cast<f32x4 *>(p.part + (slot * p.cols + cc) * D + d) = a;
            if (d == 0) {
                p.ml[(slot * p.cols + cc) * 2] = m;
                p.ml[(slot * p.cols + cc) * 2 + 1] = l;
            }
        }
    }
}

// Requests 16 bytes per lane from `src` into LDS at `to` + 16 * lane; there is
// no register result, and the kernel waits for its loads itself.
__device__ __forceinline__ void load_to_lds16(const uint8_t *src, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(src) : "memory", "m0");
}

// Many columns (prompts): wave w holds columns [w * 16 NT, (w + 1) * 16 NT) of
// the workgroup's 64 NT and all four walk the tile's chunks together.  A chunk
// (64 tokens of K and of V, as stored) is staged in LDS once for the four, in
// two buffers, by direct loads of whole lines; each wave converts what it reads
// to fp16 in registers.  Bound by issuing vector instructions (conversions,
// exponentials), 60% of the cycles against the matrix cores' 40%: four prompts,
// the longest 4096 rows at 6001 tokens, 32 query heads over 8 of 128 dims, 620 us
// (930 TFLOP/s; an fp16 product of 8192^3 reaches 1184).
// LDS order: a token's keys are D / 16 pieces of 16 bytes, a dim's values four
// (one per 16-token block); pieces are exchanged within their row so that the
// eight lanes of a read phase, which want the same piece of different rows,
// meet different banks.  Direct loads write in lane order, so the exchange is
// made in the lanes' addresses.
// ONE: a chunk lies in one page (pages of 64 tokens or more).
template <int D, int NT, bool ONE>
__global__ __launch_bounds__(256, (D <= 128 ? 2 : 1)) void attention_rows_kernel(Params p) {
    constexpr int PR = D / 16;             // pieces per token of keys
    constexpr int LOADS = D / 64;          // direct loads per wave of keys, and of values
    constexpr int HALF = kChunk * D;       // bytes of a chunk's keys, and of its values
    __shared__ __align__(16) uint8_t lds[2][2 * HALF];
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4, kx = col >> 2;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place at(p);
    const Tile t = make_tile(p, at.tile);
    if (t.c0 >= t.ncols || (at.split > 0 && at.split >= t.active)) return;
    const int clo = t.split0 + at.split * p.quota;
    int chi = t.hi > t.lo ? (t.hi + kChunk - 1) / kChunk : clo;
    chi = chi < clo + p.quota ? chi : clo + p.quota;

    // this wave's columns, and the chunks that any of them sees
    const int wc0 = t.c0 + wave * 16 * NT;
    const bool any_col = wc0 < t.ncols;
    Columns<D, NT, false> cs;
    cs.init(p, t, at.kvh, any_col ? wc0 : t.c0);
    const int own_hi = !any_col || cs.pos_max < 0 ? 0 : cs.pos_max / kChunk + 1;
    const int first_tok = p.window ? cs.pos_min - p.window + 1 : 0;
    const int own_lo = first_tok <= 0 ? 0 : first_tok / kChunk;

    const Pages pages(p, t, at.kvh);
    const size_t page_bytes = (size_t)D << p.c.page_shift;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&lds[0][0];
    auto key_turn = [](int row) { return PR == 4 ? ((row >> 1) & 1) | ((row >> 3) & 2) : (row & 3) | ((row >> 2) & 4); };
    // what this lane loads: keys of row krow (+ 1024 / D per load) of block
    // `wave`; values of dim vdim (+ 16 per load), block vx
    const int krow = 16 * wave + lane / PR, vdim = wave * LOADS * 16 + (lane >> 2), vx = (lane & 3) ^ ((lane >> 3) & 3);
    auto stage = [&](int c, int page_k, int page_v) __attribute__((always_inline)) {
        const uint32_t to = lds0 + (uint32_t)(c & 1) * (2 * HALF) + wave * LOADS * 1024;
        const uint8_t *kp = p.c.k + pages.slot(page_k) * page_bytes + (size_t)pages.within(c, wave) * D;
        const uint8_t *vp = p.c.v + pages.slot(page_v) * page_bytes + pages.within(c, vx);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = krow + i * (1024 / D);
            load_to_lds16(kp + (row - 16 * wave) * D + 16 * ((lane % PR) ^ key_turn(row)), to + i * 1024);
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            load_to_lds16(vp + ((size_t)(vdim + 16 * i) << p.c.page_shift), to + HALF + i * 1024);
    };

    // what it reads: keys of row 16 (col / 4) + 4x + col % 4 (all at one turn),
    // values of dim 16 d + col
    int key_at[D / 64];
#pragma unroll
    for (int m = 0; m < D / 64; ++m) key_at[m] = (16 * kx + (col & 3)) * D + 16 * ((4 * m + g) ^ key_turn(16 * kx + (col & 3)));
    const int value_at = col * 64 + 16 * (g ^ ((col >> 1) & 3));

    // Pages and scale bytes run ahead of the chunks they belong to: those that
    // this wave loads keys and values of, and those of the keys and values that
    // this lane multiplies.
    struct Ids {
        int load_k, load_v, k, v;
    };
    auto ids = [&](int c) __attribute__((always_inline)) {
        if constexpr (ONE) {
            const int id = pages.lookup(c);
            // of a chunk that ends inside the tile's tokens, blocks past them
            // count as the page's: their scores are masked
            return Ids{id, id, id, id};
        } else {
            return Ids{pages.lookup(c, wave), pages.lookup(c, vx), pages.lookup(c, kx), pages.lookup(c, g)};
        }
    };
    Ids now{-1, -1, -1, -1}, next = now;
    uint32_t bk = 0, bv = 0;
    auto scale_bytes = [&]() __attribute__((always_inline)) {
        bk = p.c.k_scale[pages.slot(next.k)];
        bv = p.c.v_scale[pages.slot(next.v)];
    };
    if (clo < chi) {
        next = ids(clo);
        stage(clo, next.load_k, next.load_v);
        scale_bytes();
        now = next;
        if (clo + 1 < chi) next = ids(clo + 1);
    }
    bool lost = false;
    auto turn = [&](int c, auto clean) __attribute__((always_inline)) {
        // chunk c has landed, and every wave is done with the other buffer
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const float fk = scale_of((uint8_t)bk), fv = scale_of((uint8_t)bv);
        const Ids cur = now;
        if (c + 1 < chi) {
            stage(c + 1, next.load_k, next.load_v);
            scale_bytes();
            now = next;
            if (c + 2 < chi) next = ids(c + 2);
        }
        const uint8_t *kb = &lds[c & 1][0], *vb = kb + HALF;
        auto key = [&](int x, int m) __attribute__((always_inline)) {
            return *reinterpret_cast<const u32x4 *>(kb + key_at[m] + 4 * x * D);
        };
        auto value = [&](int d) __attribute__((always_inline)) {
            return *reinterpret_cast<const u32x4 *>(vb + value_at + 16 * d * 64);
        };
        if constexpr (decltype(clean)::value) {
            lost = lost || (ONE ? cur.k == -2 : (bool)__any(cur.k == -2 || cur.v == -2));
            cs.template chunk<true>(c, key, fk, value, fv, cur.v);
        } else if (c >= own_lo && c < own_hi) {
            cs.template chunk<false>(c, key, fk, value, fv, cur.v);
        }
    };
    int clean_lo, clean_hi;
    cs.clean_range(clo, chi, clean_lo, clean_hi);
    if (!any_col) clean_lo = clean_hi = chi;
    int c = clo;
    for (; c < clean_lo; ++c) turn(c, std::false_type{});
    for (; c < clean_hi && !cs.steep; ++c) turn(c, std::true_type{});
    for (; c < chi; ++c) turn(c, std::false_type{});

    if (!any_col) return;
    const int64_t slot = at.slot(p);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int cc = wc0 + 16 * n + col;
        if (!cs.live[n]) continue;
        const float l = cs.total(n, t.cap, lost);
        if (t.active <= 1) {
            const int i = cc / p.group, h = cc - i * p.group;
            uint16_t *dst = p.out + ((int64_t)(t.r0 + i) * p.heads + at.kvh * p.group + h) * D + 4 * g;
            const float f = inverse(l, t.first + i);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) *reinterpret_cast<u32x2 *>(dst + 16 * d) = pack4(cs.o[n][d], f);
        } else {
            const int64_t k = slot * p.cols + (cc - t.c0);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4 *>(p.part + k * D + 16 * d + 4 * g) = cs.o[n][d];
            if (g == 0) {
                p.ml[k * 2] = cs.max2(n);
                p.ml[k * 2 + 1] = l;
            }
        }
    }
}

// Joins a column's pieces: one workgroup per column, D / 4 threads to a piece,
// the 1024 / D groups of threads taking pieces in turn and meeting in LDS, in
// order.  48 sequences to 16384 tokens: 5.6 us, bound by launch and latency.  One
// workgroup per tile left one sequence of 65536 at 61 us in both kernels, 29 now.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(Params p) {
    constexpr int TP = D / 4, GROUPS = 256 / TP;
    __shared__ f32x4 sh_o[GROUPS][TP];
    __shared__ float sh_l[GROUPS], sh_m[4];
    const int kvh = blockIdx.x % p.c.heads, tile = blockIdx.x / p.c.heads, cc = blockIdx.y;
    const Tile t = make_tile(p, tile);
    if (t.active <= 1 || t.c0 + cc >= t.ncols) return;
    const int64_t slot = ((int64_t)tile * p.c.heads + kvh) * p.splits;
    const float *ml = p.ml + (slot * p.cols + cc) * 2, *part = p.part + (slot * p.cols + cc) * D;
    float m = -__builtin_inff();
    for (int s = threadIdx.x; s < t.active; s += 256) m = fmaxf(m, ml[(int64_t)s * p.cols * 2]);
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) sh_m[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sh_m[0], sh_m[1]), fmaxf(sh_m[2], sh_m[3]));
    const int group = threadIdx.x / TP, d = threadIdx.x % TP;
    f32x4 a{0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll 4
    for (int s = group; s < t.active; s += GROUPS) {
        const float ms = ml[(int64_t)s * p.cols * 2], ls = ml[(int64_t)s * p.cols * 2 + 1];
        const f32x4 v = *reinterpret_cast<const f32x4 *>(part + (int64_t)s * p.cols * D + 4 * d);
        const float f = ms == -__builtin_inff() ? (ls == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(ms - m);
        l = __builtin_fmaf(ls, f, l);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = __builtin_fmaf(v[j], f, a[j]);
    }
    sh_o[group][d] = a;
    if (d == 0) sh_l[group] = l;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) {
        l += sh_l[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] += sh_o[k][d][j];
    }
    const int c = t.c0 + cc, i = c / p.group, h = c - i * p.group;
    *reinterpret_cast<u32x2 *>(p.out + ((int64_t)(t.r0 + i) * p.heads + kvh * p.group + h) * D + 4 * d) =
        pack4(a, inverse(l, t.first + i));
}

template <int D>
hipError_t launch(const Params &p, const AttnPlan &plan, hipStream_t stream) {
    const dim3 grid((unsigned)(plan.tiles * p.c.heads * plan.splits));
    if (plan.shared) attention_token_kernel<D><<<grid, dim3(256), 0, stream>>>(p);
    else if (plan.nt == 1 && p.c.page_shift >= 6) attention_rows_kernel<D, 1, true><<<grid, dim3(256), 0, stream>>>(p);
    else if (plan.nt == 1) attention_rows_kernel<D, 1, false><<<grid, dim3(256), 0, stream>>>(p);
    else if constexpr (D <= 128) {
        if (p.c.page_shift >= 6) attention_rows_kernel<D, 2, true><<<grid, dim3(256), 0, stream>>>(p);
        else attention_rows_kernel<D, 2, false><<<grid, dim3(256), 0, stream>>>(p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || plan.splits <= 1) return e;
    attention_join_kernel<D><<<dim3((unsigned)(plan.tiles * p.c.heads), (unsigned)plan.join_cols), dim3(256), 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(int64_t heads, int64_t kv_heads, int64_t dim, int64_t page, int64_t max_pages, int64_t B,
                        int64_t T, bool single) {
    AttnPlan p;
    const int64_t group = heads / kv_heads;
    const int64_t per = (T * group + B - 1) / B;  // columns of the average sequence
    p.shared = per <= 16;
    // Two column tiles per wave share each conversion of keys and values; one
    // gives twice the workgroups.  Measured on MI355X: 2000 rows after 6000
    // tokens (504 workgroups with two) 255 us, 328 with one; 1500 rows (376) 51
    // us, 43 with one; 1000 rows (256) 34 us, 28 with one.
    p.nt = 1;
    if (!p.shared && per > 64 && dim < 256 && (T * group / 128 + B) * kv_heads >= 400) p.nt = 2;
    p.cols = p.shared ? 16 : 64 * p.nt;
    // ragged rows: an upper bound, sequence b's tiles beginning at
    // floor(rows[b] * group / cols) + b
    p.tiles = single ? B * ((group + p.cols - 1) / p.cols) : T * group / p.cols + B;
    p.join_cols = (int)(single && group < p.cols ? group : p.cols);
    const int64_t chunks = (max_pages * page + kChunk - 1) / kChunk;
    const int64_t wgs = p.tiles * kv_heads;
    int64_t splits, least;
    if (p.shared) {
        // Pieces to about 2048 workgroups (four rounds of the chip, which evens
        // out ragged lengths), none where the tiles alone fill two.  Measured
        // on MI355X with 8 cache heads of 128 and a table as wide as the longest
        // sequence: 48 sequences to 16384 tokens 166 us (half as many pieces
        // 185, twice as many 162), one of 65536 29 us, 128 of 2000 59 us (two
        // pieces: 78); 72 of 3000 (576 tiles) 67 us, 51 whole, so the border
        // could lie lower.  A piece is at least a chunk for each wave, two
        // where there are more tiles: 4 of 2048 10.8 us (whole: 20.9), 8 of 4096
        // 17.0 us (pieces of four chunks: 18.5, whole: 41), 64 of 500 13.3 us
        // (pieces of four chunks: 23.7).  Up to 1024 tokens stay whole: a second
        // launch and its workspace cost 4 us of host time where calls are
        // launched one by one (one of 777: 12.8 us, 16.6 in pieces; one of 1024:
        // 12.6 and 17.4) and save 2.5 where they are replayed from a graph (12.7
        // and 10.2; 12.6 and 10.0).
        splits = wgs >= 1024 ? 1 : (2048 + wgs - 1) / wgs;
        least = wgs >= 64 ? 8 : chunks <= 16 ? 16 : 4;
    } else {
        // A piece of a prompt writes and reads back far more than it saves
        // once the tiles come near to filling the chip: 1000 rows (504
        // workgroups) 28 us whole, 78 in two pieces; 400 rows after 1600 tokens
        // (208) 45 us whole, 56 in two; 128 rows after 3872 (72) 34 us in seven
        // pieces, 78 whole.
        splits = wgs >= 192 ? 1 : (512 + wgs - 1) / wgs;
        least = 8;
    }
    splits = splits < chunks / least ? splits : chunks / least;
    splits = splits < 64 ? splits : 64;
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
