// layer.h -- launch interface and device helpers of the decoder-layer
// operators in 8 bits (quant.hip, gemm_fp8.hip, kv_append.hip,
// attention.hip).  Internal to the library.
//
// 8-bit values are OCP e4m3 (largest finite value 448, one NaN code per sign,
// no infinities), the format of gfx950's conversions and matrix instructions.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

#include "w4a16.h"

namespace w4a16 {

// Records `msg` as the calling thread's last error and returns `status`
// (api.cpp; an empty message with W4A16_OK clears it).
int set_error(int status, const std::string &msg);

constexpr int kFp8Block = 128;  // columns that share one 8-bit scale
// Scale bytes of a cache page: 2^(byte - 127), byte in [112, 135].
constexpr int kKvMinExp = -15, kKvMaxExp = 8;

// Rows of a call over ragged sequences: sequence b owns rows
// [rows[b], rows[b + 1]) (rows NULL: row b), the last of its lens[b] cached
// positions.
struct SeqArgs {
    const int32_t *table;  // [B, max_pages] page numbers
    const int32_t *lens;   // [B]
    const int32_t *rows;   // [B + 1] or NULL
    int B, T, max_pages;
};

struct CacheArgs {
    uint8_t *k, *v;              // [pages, heads, page, dim], [pages, heads, dim, page]
    uint8_t *k_scale, *v_scale;  // [pages, heads]
    int64_t pages;
    int heads, dim, page_shift;
};

hipError_t launch_add_rmsnorm(const uint16_t *x, int64_t ldx, const uint16_t *r, int64_t ldr, const uint16_t *w,
                              float eps, int64_t M, int64_t width, uint16_t *sum, uint16_t *y, uint8_t *y8,
                              float *scales, hipStream_t stream);
hipError_t launch_quant_fp8(bool swiglu, const uint16_t *x, int64_t ldx, int64_t M, int64_t K, uint8_t *y8,
                            float *scales, hipStream_t stream);
hipError_t launch_gemm_fp8(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, int64_t M, int64_t K,
                           int64_t N, uint16_t *out, hipStream_t stream);
// The workgroup tile (rows x columns) and the groups K is divided among that a
// size takes.
void gemm_fp8_plan(int64_t M, int64_t K, int64_t N, int32_t *rows, int32_t *cols, int32_t *groups);
hipError_t launch_kv_append(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const CacheArgs &c,
                            const SeqArgs &s, hipStream_t stream);

// How an attention call is cut up: column tiles of `cols` (row, head) pairs of
// one sequence and key/value head, and `splits` pieces of `quota` 64-token
// chunks of the longest cache the table can hold.
struct AttnPlan {
    int nt = 1;         // 16-column tiles per wave
    bool shared = true; // a workgroup's waves share one column tile and divide its tokens
    int cols = 16;      // columns per workgroup
    int64_t tiles = 0;  // column tiles per key/value head, an upper bound
    int splits = 1;
    int quota = 0;      // chunks per split
    int join_cols = 16; // columns the pieces of a tile are joined for
    size_t part_floats = 0;  // workspace: partial outputs, then (max, sum) pairs
};
AttnPlan plan_attention(int64_t heads, int64_t kv_heads, int64_t dim, int64_t page, int64_t max_pages, int64_t B,
                        int64_t T, bool single);
hipError_t launch_attention(const uint16_t *q, int64_t ldq, int heads, const CacheArgs &c, const SeqArgs &s,
                            float scale, int64_t window, uint16_t *out, float *workspace, const AttnPlan &plan,
                            hipStream_t stream);


typedef int i32x8 __attribute__((ext_vector_type(8)));

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// Four floats to four e4m3 codes, rounded to nearest even.  Inputs are at most
// 448 in magnitude, or NaN (code 0x7f).
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// Whether any of a word's four codes is NaN (0x7f or 0xff), as a mask of the
// bytes' top bits: a byte's low seven bits plus one carry into bit 7 only at
// 0x7f.
__device__ __forceinline__ uint32_t nan_bits(uint32_t codes) {
    return ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// The largest b with start(b) <= id, for a non-decreasing start with start(0)
// = 0: which sequence a work item belongs to.
template <typename F>
__device__ __forceinline__ int find_sequence(int n, int64_t id, F start) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start(mid) <= id) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Rows of sequence b, clamped into the call's T rows (an offset table that
// runs backwards or out of range yields fewer or no rows, never a bad index).
__device__ __forceinline__ void sequence_rows(const SeqArgs &s, int b, int &r0, int &n) {
    if (!s.rows) {
        r0 = b;
        n = 1;
        return;
    }
    int a = s.rows[b], e = s.rows[b + 1];
    a = a < 0 ? 0 : a > s.T ? s.T : a;
    e = e < a ? a : e > s.T ? s.T : e;
    r0 = a;
    n = e - a;
}

}  // namespace w4a16
