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

__device__ __forceinline__ void store4(uint16_t *out, int64_t m, int64_t ldo, int n, int N, bool wide, const f32x4 &v) {
    uint16_t *p = out + m * ldo + n;
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

// Few rows: 16 columns and 16 rows per workgroup of eight waves, which take
// blocks of K in turn straight from memory and meet in LDS, in wave order.
// Bound by reading the weights: with one row 4.4 TB/s on 4096 x 25600.
constexpr int kRowWaves = 8;
__global__ __launch_bounds__(64 * kRowWaves) void gemm_fp8_row_kernel(const uint8_t *__restrict__ a,
                                                                       const float *__restrict__ sa,
                                                                       const uint8_t *__restrict__ b,
                                                                       const float *__restrict__ sb, int M, int K, int N,
                                                                       uint16_t *__restrict__ out, int64_t ldo) {
    __shared__ f32x4 sh[kRowWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, m = blockIdx.y * 16 + r;
    const int nb = (K + kFp8Block - 1) / kFp8Block;
    const uint8_t *brow = b + (size_t)(n0 + r < N ? n0 + r : N - 1) * K;
    const float *sbp = sb + (size_t)(n0 / kFp8Block) * nb;
    const uint8_t *arow = a + (size_t)(m < M ? m : M - 1) * K;
    const float *sap = sa + (size_t)(m < M ? m : M - 1) * nb;
    f32x4 acc{0.f, 0.f, 0.f, 0.f};
    for (int kb = wave; kb < nb; kb += kRowWaves) {
        const f32x4 p = mfma_block(load_block(brow, kb * kFp8Block, g, K), load_block(arow, kb * kFp8Block, g, K));
        const float f = sbp[kb] * sap[kb];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = __builtin_fmaf(p[j], f, acc[j]);
    }
    sh[wave][lane] = acc;
    __syncthreads();
    if (wave != 0 || m >= M) return;
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += sh[w][lane][j];
    store4(out, m, ldo, n0 + 4 * g, N, (ldo & 3) == 0, acc);
}

// Direct loads into LDS, 16 or 4 bytes per lane: from the buffer at voff + soff
// to `to` + 16 (4) * lane.  Written as asm because the compiler makes every
// later LDS read wait for such a load, whichever bytes it reads.  There is no
// register result; the kernel waits for its loads itself (they land in order)
// before the barrier that hands a stage over.
__device__ __forceinline__ void load_to_lds16(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(voff), "s"(rsrc),
                 "s"(soff)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds4(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(to), "v"(voff), "s"(rsrc),
                 "s"(soff)
                 : "memory", "m0");
}
// Waits until at most N of the wave's loads are still on their way, and its LDS
// reads are done.
template <int N>
__device__ __forceinline__ void loads_left() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
// A byte offset past every buffer here (256 rows of at most 2^22 bytes), also
// after a wave's row offsets are added.
constexpr uint32_t kOutside = 0xc0000000u;
constexpr int64_t kTileMaxK = (int64_t)1 << 22;

// Many rows: a BN x BM tile of out (BN weight rows, BM activation rows) per
// workgroup of WN x WM waves, one block of K per step, operands and activation
// scales staged in LDS by direct loads, S - 1 steps ahead in S buffers.
// LDS holds a row's 128 bytes of the block as eight 16-byte pieces, piece c at
// place c ^ (row % 8), so the 16 rows a fragment read touches at one c cover
// all banks; the direct load writes 1 KB (eight rows) per wave in lane order,
// so the exchange is made in the lanes' global addresses.  Measured with 256 x
// 256 tiles at 8192^3: 513 us, 2140 TFLOP/s (a library product with one scale in
// all: 2448), at 1.8 - 2.1 GHz; products, adds and barriers alone, without the
// loads, take 445 us.
template <int BM, int BN, int WM, int WN, int S, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG) void gemm_fp8_tile_kernel(const uint8_t *__restrict__ a,
                                                                      const float *__restrict__ sa,
                                                                      const uint8_t *__restrict__ b,
                                                                      const float *__restrict__ sb, int M, int K, int N,
                                                                      int tiles_m, int tiles_n,
                                                                      uint16_t *__restrict__ out, int64_t ldo) {
    constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int kLoadB = BN / 8 / W, kLoadA = BM / 8 / W;  // direct loads per wave and step, and one of scales
    constexpr int kStage = (BM + BN) * kFp8Block;
    static_assert(BN % (8 * W) == 0 && BM % (8 * W) == 0, "whole loads per wave");
    static_assert(128 % (BN / WN) == 0, "one weight scale per wave");
    static_assert(KG == 1 || BM * BN * 4 <= S * kStage, "a group's sums fit its buffers");
    __shared__ __align__(16) uint8_t lds_all[KG * S * kStage];
    constexpr int kScales = BM < 64 ? 64 : BM;
    __shared__ __align__(16) float s_sa_all[KG * S * kScales];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kg = wid / W, wave = wid % W;
    const int wm = wave % WM, wn = wave / WM;
    uint8_t *lds = lds_all + kg * S * kStage;
    float *s_sa = s_sa_all + kg * S * kScales;
    // Workgroups go to the eight XCDs in turn.  Each XCD walks its own eighth of
    // the tiles, four row tiles by one column tile at a time, so that the 32
    // tiles it computes at once read 4 + 8 tiles of operands through its L2.
    const int total = tiles_m * tiles_n, per = (total + 7) / 8;
    const int order = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (order >= total || (int)(blockIdx.x >> 3) >= per) return;
    const int group = order / (4 * tiles_n), left = order - group * 4 * tiles_n;
    const int gm = tiles_m - 4 * group < 4 ? tiles_m - 4 * group : 4;
    const int m0 = (4 * group + left % gm) * BM, n0 = (left / gm) * BN;
    const int nb = (K + kFp8Block - 1) / kFp8Block;

    // Rows 0 .. BN - 1 of a stage are weights, then activations; a wave loads
    // some of each.  Rows past an operand's end read as zero.  The row is in
    // the range-checked offset, the block of K in the unchecked one.
    const int mrows = M - m0 < BM ? M - m0 : BM, nrows = N - n0 < BN ? N - n0 : BN;
    auto rsrc = [](const void *p, uint32_t bytes) {
        const uint64_t base = (uint64_t)p;
        return u32x4{(uint32_t)base, (uint32_t)(base >> 32), bytes, 0x00020000u};
    };
    const u32x4 rb = rsrc(b + (size_t)n0 * K, (uint32_t)nrows * (uint32_t)K);
    const u32x4 ra = rsrc(a + (size_t)m0 * K, (uint32_t)mrows * (uint32_t)K);
    const u32x4 rs = rsrc(sa + (size_t)m0 * nb, (uint32_t)mrows * (uint32_t)nb * 4u);
    const int piece = (lane & 7) ^ (lane >> 3);
    const uint32_t vb = (uint32_t)(wave * kLoadB * 8 + (lane >> 3)) * (uint32_t)K + 16u * piece;
    const uint32_t va = (uint32_t)(wave * kLoadA * 8 + (lane >> 3)) * (uint32_t)K + 16u * piece;
    const int srow = (wave * 64) % kScales;  // several waves may load the same scales
    const uint32_t vs = (uint32_t)(srow + lane) * (uint32_t)nb * 4u;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    const uint32_t sa0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float *)s_sa;
    // Requests this group's block of step `step` into buffer `buf`: the groups
    // take the blocks of K in turn.  Pieces past K
    // (of a short last block, or a block past the last) read as zero; a block
    // past the last is requested all the same, so that every step has the same
    // number of loads on their way and the loop no branch.
    auto stage = [&](int step, int buf) __attribute__((always_inline)) {
        const int kb = step * KG + kg;
        const bool in = (int64_t)kb * kFp8Block + 16 * piece < K;
        const uint32_t to = lds0 + (uint32_t)buf * kStage;
        // the unchecked offset stays inside the first row
        const uint32_t kc = (uint32_t)(kb < nb ? kb : nb - 1), col = kc * kFp8Block;
#pragma unroll
        for (int i = 0; i < kLoadB; ++i)
            load_to_lds16(rb, (in ? vb : kOutside) + 8u * i * (uint32_t)K, col, to + (wave * kLoadB + i) * 1024);
#pragma unroll
        for (int i = 0; i < kLoadA; ++i)
            load_to_lds16(ra, (in ? va : kOutside) + 8u * i * (uint32_t)K, col, to + BN * kFp8Block + (wave * kLoadA + i) * 1024);
        load_to_lds4(rs, kb < nb ? vs : kOutside, kc * 4u, sa0 + (uint32_t)(buf * kScales + srow) * 4u);
    };
    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nrow = n0 + wn * TN * 16;
    const float *sbp = sb + (size_t)((nrow < N ? nrow : N - 1) / kFp8Block) * nb;
    const uint32_t fo = (uint32_t)(r * kFp8Block + 16 * (g ^ (r & 7)));
    auto frag = [&](int buf, int row) __attribute__((always_inline)) {  // rows row .. row + 15
        const uint8_t *p = lds + buf * kStage + row * kFp8Block;
        return join(*reinterpret_cast<const u32x4 *>(p + fo), *reinterpret_cast<const u32x4 *>(p + (fo ^ 64u)));
    };
    const int arow = BN + wm * TM * 16, brow = wn * TN * 16;
    i32x8 bf[TN], af;
    float sf[TM];
    auto first = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < TM; ++j) sf[j] = s_sa[buf * kScales + wm * TM * 16 + r + 16 * j];
        af = frag(buf, arow);
#pragma unroll
        for (int i = 0; i < TN; ++i) bf[i] = frag(buf, brow + 16 * i);
    };
#pragma unroll
    for (int i = 0; i < S; ++i) stage(i, i);
    loads_left<(S - 1) * (kLoadA + kLoadB + 1)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    first(0);
    auto weight_scale = [&](int step) __attribute__((always_inline)) {
        const int kb = step * KG + kg;
        const float v = sbp[kb < nb ? kb : nb - 1];
        return kb < nb ? v : 0.f;
    };
    const int steps = (nb + KG - 1) / KG;
    float s = weight_scale(0), sn = weight_scale(1);
    // Products of one activation tile are added to the sums between the matrix
    // instructions of the next, so that neither unit waits for the other.
    f32x4 p[TN];
    float fp = 0.f;
    auto add = [&](int i, int j) __attribute__((always_inline)) {
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][j][x] = __builtin_fmaf(p[i][x], fp, acc[i][j][x]);
    };
#pragma unroll
    for (int i = 0; i < TN; ++i) p[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int step = 0, buf = 0; step < steps; ++step) {
        const int nbuf = buf == S - 1 ? 0 : buf + 1;
        float f[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) f[j] = s * sf[j];
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            i32x8 bc[TN];
#pragma unroll
            for (int i = 0; i < TN; ++i) bc[i] = bf[i];
            const i32x8 ac = af;
            if (j + 1 < TM) {
                af = frag(buf, arow + 16 * (j + 1));
            } else {
                // This wave has read all of its block.  Once every wave has,
                // and the next step's has landed, buffer `buf` takes the block
                // S steps on, and the next step's first fragments are read
                // under the last products of this one.
                loads_left<(S - 2) * (kLoadA + kLoadB + 1)>();
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                stage(step + S, buf);
                first(nbuf);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const f32x4 q = mfma_block(bc[i], ac);
                add(i, j == 0 ? TM - 1 : j - 1);
                p[i] = q;
                __builtin_amdgcn_sched_barrier(0);
            }
            fp = f[j];
        }
        s = sn;
        sn = weight_scale(step + 2);
        buf = nbuf;
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) add(i, TM - 1);
    loads_left<0>();  // the LDS is this workgroup's until the last load has landed
    if constexpr (KG > 1) {
        // the groups' sums meet in LDS, in order
        __syncthreads();
        f32x4 *mine = reinterpret_cast<f32x4 *>(lds) + wave * TN * TM * 64 + lane;
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) mine[(i * TM + j) * 64] = acc[i][j];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int k = 1; k < KG; ++k)
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    const f32x4 v = mine[k * (S * kStage / 16) + (i * TM + j) * 64];
#pragma unroll
                    for (int x = 0; x < 4; ++x) acc[i][j][x] += v[x];
                }
    }
    const bool wide = (ldo & 3) == 0;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int m = m0 + (wm * TM + j) * 16 + r;
        if (m >= M) continue;
#pragma unroll
        for (int i = 0; i < TN; ++i) store4(out, m, ldo, nrow + 16 * i + 4 * g, N, wide, acc[i][j]);
    }
}


template <int BM, int BN, int WM, int WN, int S, int KG>
void launch_tile(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, int64_t M, int64_t K, int64_t N,
                 uint16_t *out, int64_t ldo, hipStream_t stream) {
    const int tm = (int)((M + BM - 1) / BM), tn = (int)((N + BN - 1) / BN);
    gemm_fp8_tile_kernel<BM, BN, WM, WN, S, KG><<<dim3((unsigned)((tm * tn + 7) / 8 * 8)), dim3(64 * WM * WN * KG), 0, stream>>>(
        a, sa, b, sb, (int)M, (int)K, (int)N, tm, tn, out, ldo);
}

typedef void (*TileLauncher)(const uint8_t *, const float *, const uint8_t *, const float *, int64_t, int64_t, int64_t,
                             uint16_t *, int64_t, hipStream_t);

// The tile shapes, with the time of one step (us, measured on MI355X) where a
// CU holds one, two, .. of their workgroups; as many as its LDS and registers
// hold.
struct TileShape {
    int bm, bn, groups, resident;
    float step[4];
    TileLauncher launch;
};
const TileShape kShapes[] = {
    {32, 32, 4, 1, {.65f}, launch_tile<32, 32, 1, 2, 3, 4>},
    {32, 64, 2, 2, {.46f, .78f}, launch_tile<32, 64, 1, 4, 3, 2>},
    {32, 64, 1, 4, {.36f, .40f, .62f, .81f}, launch_tile<32, 64, 1, 4, 3, 1>},
    {64, 64, 2, 1, {.62f}, launch_tile<64, 64, 1, 4, 3, 2>},
    {64, 64, 1, 3, {.45f, .60f, .95f}, launch_tile<64, 64, 1, 4, 3, 1>},
    {64, 128, 2, 1, {.95f}, launch_tile<64, 128, 1, 4, 3, 2>},
    {64, 128, 1, 2, {.60f, .90f}, launch_tile<64, 128, 1, 4, 3, 1>},
    {128, 128, 2, 1, {1.45f}, launch_tile<128, 128, 2, 2, 2, 2>},
    {128, 256, 1, 1, {1.25f}, launch_tile<128, 256, 2, 4, 3, 1>},
    {256, 256, 1, 1, {2.0f}, launch_tile<256, 256, 2, 4, 2, 1>},
};

constexpr double kReadRate = 4.7e6;  // bytes a us

// Estimated time (us) of a shape: the busiest CU's rounds of workgroups times
// the steps of one.
double estimate(const TileShape &s, int64_t M, int64_t K, int64_t N) {
    const int64_t nb = (K + kFp8Block - 1) / kFp8Block;
    const int64_t tiles = ((M + s.bm - 1) / s.bm) * ((N + s.bn - 1) / s.bn), per_cu = (tiles + 255) / 256;
    const int64_t full = per_cu / s.resident, rest = per_cu % s.resident;
    return (double)((nb + s.groups - 1) / s.groups) *
           ((double)full * s.step[s.resident - 1] + (rest ? s.step[rest - 1] : 0.0));
}

// The shape with the least estimated time, not below the time of reading the
// operands.  Measured against all shapes at M = 1 .. 4096 of 4096 x 6144,
// 4096 x 25600 and 12800 x 4096 the choice is within 10% of the best (e.g.
// M = 64 12800 x 4096: 16 us, where the 128 x 128 tiles that win at M = 1024
// take 66).  -1: the row kernel, whose step grows with the rows it reads.
int choose(int64_t M, int64_t K, int64_t N, double *us) {
    const int64_t nb = (K + kFp8Block - 1) / kFp8Block;
    *us = 0;
    if (K > kTileMaxK) return -1;
    const double least = (double)K * (double)(N + M) / kReadRate;
    int best = -1;
    double t = 1e30;
    if (M <= 16) {
        *us = (double)((N + 4095) / 4096) * (double)((nb + 7) / 8) * (.75 + .022 * (double)M);
        t = *us < least ? least : *us;
    }
    for (int i = 0; i < (int)(sizeof(kShapes) / sizeof(kShapes[0])); ++i) {
        const double e = estimate(kShapes[i], M, K, N);
        const double score = (e < least ? least : e) + .15 * e;  // among shapes at the floor, the one with time to spare
        if (score < t) {
            t = score;
            best = i;
            *us = e;
        }
    }
    return best;
}

// Columns of the first of two launches: where the largest tiles' last round
// would leave most CUs idle, the columns of the whole rounds come first and the
// rest takes the shape of its own size.  N: one launch.  Measured with K = 4096
// N = 25600: M = 4096 (6.25 rounds) 490 us in one launch, 465 in two, M = 2048 (3.1
// rounds) 273 and 238; less than the rounds saved, as fewer busy CUs run at higher
// clocks.
int64_t first_columns(int64_t M, int64_t K, int64_t N, int shape, double us) {
    const TileShape &s = kShapes[sizeof(kShapes) / sizeof(kShapes[0]) - 1];
    if (shape != (int)(sizeof(kShapes) / sizeof(kShapes[0])) - 1) return N;
    const int64_t tm = (M + s.bm - 1) / s.bm, tn = (N + s.bn - 1) / s.bn;
    const int64_t n1 = tm * tn / 256 * 256 / tm * s.bn;
    if (n1 <= 0 || n1 >= N) return N;
    double rest;
    choose(M, K, N - n1, &rest);
    return estimate(s, M, K, n1) + rest + 4.0 < .94 * us ? n1 : N;  // a launch and its drain: about 4 us
}

void launch_one(int shape, const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, int64_t M, int64_t K,
                int64_t N, uint16_t *out, int64_t ldo, hipStream_t stream) {
    if (shape < 0)
        gemm_fp8_row_kernel<<<dim3((unsigned)((N + 15) / 16), (unsigned)((M + 15) / 16)), dim3(64 * kRowWaves), 0, stream>>>(
            a, sa, b, sb, (int)M, (int)K, (int)N, out, ldo);
    else
        kShapes[shape].launch(a, sa, b, sb, M, K, N, out, ldo, stream);
}

}  // namespace

void gemm_fp8_plan(int64_t M, int64_t K, int64_t N, int32_t *rows, int32_t *cols, int32_t *groups) {
    double us;
    const int i = choose(M, K, N, &us);
    *rows = i < 0 ? 16 : kShapes[i].bm;
    *cols = i < 0 ? 16 : kShapes[i].bn;
    *groups = i < 0 ? kRowWaves : kShapes[i].groups;
}

hipError_t launch_gemm_fp8(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, int64_t M, int64_t K,
                           int64_t N, uint16_t *out, hipStream_t stream) {
    double us;
    const int i = choose(M, K, N, &us);
    const int64_t n1 = first_columns(M, K, N, i, us);
    launch_one(i, a, sa, b, sb, M, K, n1, out, N, stream);
    if (n1 < N) {
        const int64_t nb = (K + kFp8Block - 1) / kFp8Block;
        const int j = choose(M, K, N - n1, &us);
        launch_one(j, a, sa, b + n1 * K, sb + n1 / kFp8Block * nb, M, K, N - n1, out + n1, N, stream);
    }
    return hipGetLastError();
}

}  // namespace w4a16
