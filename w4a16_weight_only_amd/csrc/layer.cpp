// layer.cpp -- C ABI of the decoder-layer operators in 8 bits: the paged
// cache's writer and attention over it, residual + RMS norm, the quantiser,
// the 8-bit linear, and the decode step that attends to a cache.  As in
// api.cpp, every argument is checked on the host before the first HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <string>
#include <vector>

#include "kernels.h"
#include "layer.h"
#include "w4a16.h"

namespace {

using namespace w4a16;

int fail(int status, const std::string &msg) { return set_error(status, msg); }
int ok() { return set_error(W4A16_OK, ""); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
    const void *p;
    size_t n;
};

bool overlaps(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Whether any output overlaps an input or another output.
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Range &i : ins)
            if (overlaps(*o, i)) return true;
        for (auto p = outs.begin(); p != o; ++p)
            if (overlaps(*o, *p)) return true;
    }
    return false;
}

struct Span {
    uintptr_t begin, end;
    bool written;
};

Range rows_range(const void *p, int64_t rows, int64_t ld, int64_t width) {
    return Range{p, rows > 0 ? (size_t)((rows - 1) * ld + width) * 2 : 0};
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxRows = (int64_t)1 << 20;  // as for w4a16_gemm
constexpr int64_t kMaxGrid = (int64_t)1 << 23;  // workgroups of 256 threads in one launch (2^32 threads at most)

int check_cache(const w4a16_kv_cache *c, CacheArgs *out) {
    if (!c) return fail(W4A16_ERR_INVALID_ARG, "cache must be non-NULL");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale)
        return fail(W4A16_ERR_INVALID_ARG, "cache with NULL codes or scales");
    if (c->pages <= 0 || c->heads <= 0 || c->page <= 0 || c->dim <= 0)
        return fail(W4A16_ERR_INVALID_ARG, "cache sizes must be positive");
    if (c->dim != 64 && c->dim != 128 && c->dim != 256)
        return fail(W4A16_ERR_UNSUPPORTED, "cache dim must be 64, 128 or 256");
    int shift = 4;
    while (shift < 8 && ((int64_t)1 << shift) != c->page) ++shift;
    if (((int64_t)1 << shift) != c->page)
        return fail(W4A16_ERR_UNSUPPORTED, "cache page must be 16, 32, 64, 128 or 256 tokens");
    if (c->heads > 1024 || c->pages > ((int64_t)1 << 31) - 1)
        return fail(W4A16_ERR_UNSUPPORTED, "cache with more than 1024 heads or 2^31 - 1 pages");
    if (!aligned16(c->k) || !aligned16(c->v))
        return fail(W4A16_ERR_UNSUPPORTED, "cache codes must be 16-byte aligned");
    *out = CacheArgs{c->k, c->v, c->k_scale, c->v_scale, c->pages, (int)c->heads, (int)c->dim, shift};
    return W4A16_OK;
}

size_t code_bytes(const CacheArgs &c) { return ((size_t)c.pages * c.heads * c.dim) << c.page_shift; }
size_t scale_bytes(const CacheArgs &c) { return (size_t)c.pages * c.heads; }

int check_sequences(const CacheArgs &c, const int32_t *table, int64_t max_pages, const int32_t *lens,
                    const int32_t *rows, int64_t B, int64_t T, SeqArgs *out) {
    if (!table || !lens) return fail(W4A16_ERR_INVALID_ARG, "block_table and lens must be non-NULL");
    if (max_pages <= 0) return fail(W4A16_ERR_INVALID_ARG, "max_pages must be positive");
    if (!rows && T != B) return fail(W4A16_ERR_INVALID_ARG, "without row offsets there is one row per sequence: T == B");
    if (T > kMaxRows || B > kMaxRows) return fail(W4A16_ERR_UNSUPPORTED, "more than 2^20 rows or sequences");
    if (max_pages > ((int64_t)1 << 26) || (max_pages << c.page_shift) > ((int64_t)1 << 30))
        return fail(W4A16_ERR_UNSUPPORTED, "block_table rows of more than 2^30 tokens");
    if (!aligned4(table) || !aligned4(lens) || !aligned4(rows))
        return fail(W4A16_ERR_UNSUPPORTED, "block_table, lens and rows must be 4-byte aligned");
    *out = SeqArgs{table, lens, rows, (int)B, (int)T, (int)max_pages};
    return W4A16_OK;
}

int hip_status(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(W4A16_ERR_HIP, std::string(what) + " launch: " + hipGetErrorString(e));
    return ok();
}

// Host part of an attention call: the plan, or why there is none.
int attention_plan(int64_t heads, const CacheArgs &c, int64_t max_pages, int64_t B, int64_t T, bool single,
                   AttnPlan *plan) {
    if (heads <= 0 || heads % c.heads != 0)
        return fail(W4A16_ERR_INVALID_ARG, "query heads must be a positive multiple of the cache's heads");
    if (heads > 1024 || T * (heads / c.heads) >= ((int64_t)1 << 30))
        return fail(W4A16_ERR_UNSUPPORTED, "more than 1024 query heads, or too many rows for 32-bit indexing");
    *plan = plan_attention(heads, c.heads, c.dim, (int64_t)1 << c.page_shift, max_pages, B, T, single);
    if (plan->tiles * c.heads * plan->splits > kMaxGrid)
        return fail(W4A16_ERR_UNSUPPORTED, "too many rows and heads for one launch");
    return W4A16_OK;
}

int check_gemm_fp8(int64_t M, int64_t K, int64_t N) {
    if (M < 0 || K <= 0 || N <= 0) return fail(W4A16_ERR_INVALID_ARG, "M must be >= 0, K and N positive");
    if (K % 16 != 0) return fail(W4A16_ERR_UNSUPPORTED, "K must be a multiple of 16");
    if (M > kMaxRows || K > ((int64_t)1 << 26) || N > ((int64_t)1 << 26))
        return fail(W4A16_ERR_UNSUPPORTED, "M above 2^20, or K or N above 2^26");
    // workgroups of the smallest tiles, and of the row kernel
    if (cdiv(M, 16) * cdiv(N, 16) > kMaxGrid * 16 || cdiv(N, 16) > kMaxGrid)
        return fail(W4A16_ERR_UNSUPPORTED, "M * N too large for one launch");
    return W4A16_OK;
}

}  // namespace

extern "C" {

int w4a16_add_rmsnorm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr, const uint16_t *weight,
                      float eps, int64_t M, int64_t width, uint16_t *sum, uint16_t *y, uint8_t *y8, float *y8_scales,
                      hipStream_t stream) {
    if (M < 0 || width <= 0) return fail(W4A16_ERR_INVALID_ARG, "M must be >= 0 and width > 0");
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(W4A16_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (M == 0) return ok();
    if (!x) return fail(W4A16_ERR_INVALID_ARG, "x must be non-NULL when M > 0");
    if ((y != nullptr) == (y8 != nullptr) || (y8 != nullptr) != (y8_scales != nullptr))
        return fail(W4A16_ERR_INVALID_ARG, "give either y, or y8 and y8_scales");
    if (width % 8 != 0 || ldx < width || ldx % 8 != 0 || (residual && (ldr < width || ldr % 8 != 0)))
        return fail(W4A16_ERR_INVALID_ARG, "width, ldx and ldr must be multiples of 8 with rows of at least width");
    if (width > kGlueMaxWidth || M > kMaxRows || ldx >= ((int64_t)1 << 31) || (residual && ldr >= ((int64_t)1 << 31)))
        return fail(W4A16_ERR_UNSUPPORTED, "width above 32768, more than 2^20 rows, or a row stride of 2^31 or more");
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(sum) || !aligned16(y) ||
        !aligned16(y8) || !aligned4(y8_scales))
        return fail(W4A16_ERR_UNSUPPORTED, "tensors must be 16-byte aligned");
    const size_t n = (size_t)M * width;
    const Range rx = rows_range(x, M, ldx, width), rr = rows_range(residual, residual ? M : 0, ldr, width),
                rw{weight, (size_t)width * 2}, ry{y, n * 2}, ry8{y8, n},
                rs8{y8_scales, (size_t)M * cdiv(width, kFp8Block) * 4}, rsum{sum, n * 2};
    // the sum may replace x or the residual in place (same rows, dense)
    const bool on_x = sum && sum == x && ldx == width, on_r = sum && sum == residual && ldr == width;
    if (clash({ry, ry8, rs8, rsum}, {rw}) || clash({ry, ry8, rs8}, {rx, rr}) || (!on_x && overlaps(rsum, rx)) ||
        (!on_r && overlaps(rsum, rr)))
        return fail(W4A16_ERR_INVALID_ARG, "outputs overlap inputs or each other (sum may be x or residual itself, dense)");
    return hip_status(launch_add_rmsnorm(x, ldx, residual, ldr, weight, eps, M, width, sum, y, y8, y8_scales, stream),
                      "norm");
}

int w4a16_quant_fp8(int act, const uint16_t *x, int64_t ldx, int64_t M, int64_t K, uint8_t *y8, float *y8_scales,
                    hipStream_t stream) {
    if (act != W4A16_ACT_NONE && act != W4A16_ACT_SWIGLU)
        return fail(W4A16_ERR_INVALID_ARG, "act must be 0 (none) or 1 (SwiGLU)");
    if (M < 0 || K <= 0) return fail(W4A16_ERR_INVALID_ARG, "M must be >= 0 and K > 0");
    if (M == 0) return ok();
    if (!x || !y8 || !y8_scales) return fail(W4A16_ERR_INVALID_ARG, "x, y8 and y8_scales must be non-NULL when M > 0");
    if (K > ((int64_t)1 << 26) || M > kMaxRows || ldx >= ((int64_t)1 << 31))
        return fail(W4A16_ERR_UNSUPPORTED, "K above 2^26, more than 2^20 rows, or a row stride of 2^31 or more");
    const int64_t width = act == W4A16_ACT_SWIGLU ? 2 * K : K;
    if (K % 8 != 0 || ldx < width || ldx % 8 != 0)
        return fail(W4A16_ERR_INVALID_ARG, "K and ldx must be multiples of 8, with rows of at least K (SwiGLU: 2K)");
    if (M * cdiv(K, 2048) > kMaxGrid) return fail(W4A16_ERR_UNSUPPORTED, "M * K too large for one launch");
    if (!aligned16(x) || !aligned16(y8) || !aligned4(y8_scales))
        return fail(W4A16_ERR_UNSUPPORTED, "x and y8 must be 16-byte aligned");
    if (clash({Range{y8, (size_t)M * K}, Range{y8_scales, (size_t)M * cdiv(K, kFp8Block) * 4}},
              {rows_range(x, M, ldx, width)}))
        return fail(W4A16_ERR_INVALID_ARG, "y8, y8_scales and x must not overlap");
    return hip_status(launch_quant_fp8(act == W4A16_ACT_SWIGLU, x, ldx, M, K, y8, y8_scales, stream), "quantiser");
}

int w4a16_gemm_fp8(const uint8_t *a, const float *a_scales, const uint8_t *b, const float *b_scales, int64_t M,
                   int64_t K, int64_t N, uint16_t *out, hipStream_t stream) {
    if (!b || !b_scales) return fail(W4A16_ERR_INVALID_ARG, "b and b_scales must be non-NULL");
    int rc = check_gemm_fp8(M, K, N);
    if (rc != W4A16_OK) return rc;
    if (M == 0) return ok();
    if (!a || !a_scales || !out) return fail(W4A16_ERR_INVALID_ARG, "a, a_scales and out must be non-NULL when M > 0");
    if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !aligned4(a_scales) || !aligned4(b_scales))
        return fail(W4A16_ERR_UNSUPPORTED, "a, b and out must be 16-byte aligned, the scales 4-byte aligned");
    const int64_t kb = cdiv(K, kFp8Block);
    if (clash({Range{out, (size_t)M * N * 2}},
              {Range{a, (size_t)M * K}, Range{b, (size_t)N * K}, Range{a_scales, (size_t)M * kb * 4},
               Range{b_scales, (size_t)cdiv(N, kFp8Block) * kb * 4}}))
        return fail(W4A16_ERR_INVALID_ARG, "out overlaps an input");
    return hip_status(launch_gemm_fp8(a, a_scales, b, b_scales, M, K, N, out, stream), "8-bit GEMM");
}

int w4a16_gemm_fp8_plan(int64_t M, int64_t K, int64_t N, int32_t *rows, int32_t *cols, int32_t *groups) {
    int rc = check_gemm_fp8(M, K, N);
    if (rc != W4A16_OK) return rc;
    int32_t r, c, g;
    gemm_fp8_plan(std::max<int64_t>(M, 1), K, N, &r, &c, &g);
    if (rows) *rows = r;
    if (cols) *cols = c;
    if (groups) *groups = g;
    return ok();
}

int w4a16_kv_append(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const w4a16_kv_cache *cache,
                    const int32_t *block_table, int64_t max_pages, const int32_t *lens, const int32_t *rows, int64_t B,
                    int64_t T, hipStream_t stream) {
    CacheArgs c;
    SeqArgs s;
    int rc = check_cache(cache, &c);
    if (rc != W4A16_OK) return rc;
    if (B < 0 || T < 0) return fail(W4A16_ERR_INVALID_ARG, "B and T must be >= 0");
    if (T > 0 && B == 0) return fail(W4A16_ERR_INVALID_ARG, "rows without sequences");
    if (T == 0) return ok();
    if (!k || !v) return fail(W4A16_ERR_INVALID_ARG, "k and v must be non-NULL when T > 0");
    if ((rc = check_sequences(c, block_table, max_pages, lens, rows, B, T, &s)) != W4A16_OK) return rc;
    const int64_t width = (int64_t)c.heads * c.dim;
    if (ldk < width || ldv < width || ldk % 8 != 0 || ldv % 8 != 0)
        return fail(W4A16_ERR_INVALID_ARG, "ldk and ldv must be multiples of 8 covering heads * dim");
    if (ldk >= ((int64_t)1 << 31) || ldv >= ((int64_t)1 << 31) || cdiv(T, (int64_t)1 << c.page_shift) + 2 * B > kMaxGrid)
        return fail(W4A16_ERR_UNSUPPORTED, "row stride or row count too large");
    if (!aligned16(k) || !aligned16(v)) return fail(W4A16_ERR_UNSUPPORTED, "k and v must be 16-byte aligned");
    const Range ck{c.k, code_bytes(c)}, cv{c.v, code_bytes(c)}, cks{c.k_scale, scale_bytes(c)}, cvs{c.v_scale, scale_bytes(c)};
    if (clash({ck, cv, cks, cvs},
              {rows_range(k, T, ldk, width), rows_range(v, T, ldv, width), Range{block_table, (size_t)B * max_pages * 4},
               Range{lens, (size_t)B * 4}, Range{rows, (size_t)(B + 1) * 4}}))
        return fail(W4A16_ERR_INVALID_ARG, "the cache's arrays overlap each other or an input");
    return hip_status(launch_kv_append(k, ldk, v, ldv, c, s, stream), "cache write");
}

size_t w4a16_attention_workspace_bytes(int64_t heads, const w4a16_kv_cache *cache, int64_t max_pages, int64_t B,
                                       int64_t T) {
    CacheArgs c;
    AttnPlan plan;
    if (B <= 0 || T <= 0 || max_pages <= 0 || B > kMaxRows || T > kMaxRows || max_pages > ((int64_t)1 << 26) ||
        check_cache(cache, &c) != W4A16_OK || attention_plan(heads, c, max_pages, B, T, false, &plan) != W4A16_OK)
        return 0;
    size_t floats = plan.part_floats;
    // one row per sequence may come with or without offsets
    if (T == B && attention_plan(heads, c, max_pages, B, T, true, &plan) == W4A16_OK)
        floats = std::max(floats, plan.part_floats);
    return floats * sizeof(float);
}

int w4a16_attention(const uint16_t *q, int64_t ldq, int64_t heads, const w4a16_kv_cache *cache,
                    const int32_t *block_table, int64_t max_pages, const int32_t *lens, const int32_t *rows, int64_t B,
                    int64_t T, float scale, int64_t window, uint16_t *out, void *workspace, size_t workspace_bytes,
                    hipStream_t stream) {
    CacheArgs c;
    SeqArgs s;
    AttnPlan plan;
    int rc = check_cache(cache, &c);
    if (rc != W4A16_OK) return rc;
    if (B < 0 || T < 0) return fail(W4A16_ERR_INVALID_ARG, "B and T must be >= 0");
    if (T > 0 && B == 0) return fail(W4A16_ERR_INVALID_ARG, "rows without sequences");
    if (!std::isfinite(scale)) return fail(W4A16_ERR_INVALID_ARG, "scale must be finite");
    if (window < 0) return fail(W4A16_ERR_INVALID_ARG, "window must be >= 0");
    if (T == 0) return ok();
    if (!q || !out) return fail(W4A16_ERR_INVALID_ARG, "q and out must be non-NULL when T > 0");
    if ((rc = check_sequences(c, block_table, max_pages, lens, rows, B, T, &s)) != W4A16_OK) return rc;
    if ((rc = attention_plan(heads, c, max_pages, B, T, !rows, &plan)) != W4A16_OK) return rc;
    const int64_t width = heads * c.dim;
    if (ldq < width || ldq % 8 != 0) return fail(W4A16_ERR_INVALID_ARG, "ldq must be a multiple of 8 covering heads * dim");
    if (ldq >= ((int64_t)1 << 31)) return fail(W4A16_ERR_UNSUPPORTED, "ldq of 2^31 or more");
    const size_t need = plan.part_floats * sizeof(float);
    if (need && (!workspace || workspace_bytes < need))
        return fail(W4A16_ERR_INVALID_ARG, "workspace smaller than w4a16_attention_workspace_bytes()");
    if (!aligned16(q) || !aligned16(out) || (need && !aligned16(workspace)))
        return fail(W4A16_ERR_UNSUPPORTED, "q, out and workspace must be 16-byte aligned");
    if (clash({Range{out, (size_t)T * width * 2}, Range{need ? workspace : nullptr, need}},
              {rows_range(q, T, ldq, width), Range{c.k, code_bytes(c)}, Range{c.v, code_bytes(c)},
               Range{c.k_scale, scale_bytes(c)}, Range{c.v_scale, scale_bytes(c)},
               Range{block_table, (size_t)B * max_pages * 4}, Range{lens, (size_t)B * 4}, Range{rows, (size_t)(B + 1) * 4}}))
        return fail(W4A16_ERR_INVALID_ARG, "out or workspace overlaps an input or each other");
    // a window that reaches past every position hides nothing
    const int64_t w = window > (max_pages << c.page_shift) ? 0 : window;
    return hip_status(launch_attention(q, ldq, (int)heads, c, s, scale, w, out, static_cast<float *>(workspace), plan, stream),
                      "attention");
}

size_t w4a16_decode_kv_workspace_bytes(int64_t M, const w4a16_linear *lin, int64_t n_layers,
                                       const w4a16_kv_cache *caches, int64_t max_pages) {
    const size_t three = w4a16_decode_workspace_bytes(M, lin, n_layers);
    if (!three || !caches || M > 8192) return 0;
    size_t attn = 0;
    for (int64_t l = 0; l < n_layers; ++l) {
        CacheArgs c;
        AttnPlan plan;
        if (max_pages <= 0 || max_pages > ((int64_t)1 << 26) || check_cache(caches + l, &c) != W4A16_OK ||
            lin[4 * l].K % c.dim != 0 || attention_plan(lin[4 * l].K / c.dim, c, max_pages, M, M, true, &plan) != W4A16_OK)
            return 0;
        attn = std::max(attn, w4a16_attention_workspace_bytes(lin[4 * l].K / c.dim, caches + l, max_pages, M, M));
    }
    return three + attn;
}

int w4a16_decode_step_kv(const w4a16_linear *lin, int64_t n_layers, const w4a16_kv_cache *caches,
                         const int32_t *block_table, int64_t max_pages, const int32_t *lens, float scale,
                         const uint16_t *x_in, uint16_t *x_out, int64_t M, void *workspace, size_t workspace_bytes,
                         hipStream_t stream) {
    if (!x_in || !x_out || !workspace) return fail(W4A16_ERR_INVALID_ARG, "x_in, x_out and workspace must be non-NULL");
    if (!lin || n_layers <= 0) return fail(W4A16_ERR_INVALID_ARG, "empty stack");
    if (!caches) return fail(W4A16_ERR_INVALID_ARG, "caches must be non-NULL");
    if (M < 1 || M > 8192) return fail(W4A16_ERR_INVALID_ARG, "M must be in [1, 8192]");
    if (!std::isfinite(scale)) return fail(W4A16_ERR_INVALID_ARG, "scale must be finite");
    const size_t three = w4a16_decode_workspace_bytes(M, lin, n_layers);
    if (!three) return fail(W4A16_ERR_INVALID_ARG, std::string("malformed stack: ") + w4a16_last_error());
    const int64_t H = lin[0].K;
    int64_t widest = 0;
    int rc;
    for (int64_t l = 0; l < n_layers; ++l) {
        CacheArgs c;
        SeqArgs s;
        if ((rc = check_cache(caches + l, &c)) != W4A16_OK) return rc;
        if (H % c.dim != 0 || lin[4 * l].N != H + 2 * (int64_t)c.heads * c.dim)
            return fail(W4A16_ERR_INVALID_ARG,
                        "the first linear's output must be queries, keys and values: hidden + 2 * cache heads * dim");
        if ((rc = check_sequences(c, block_table, max_pages, lens, nullptr, M, M, &s)) != W4A16_OK) return rc;
        for (int j = 0; j < 4; ++j) widest = std::max(widest, lin[4 * l + j].N);
    }
    const size_t need = w4a16_decode_kv_workspace_bytes(M, lin, n_layers, caches, max_pages);
    if (!need) return fail(W4A16_ERR_INVALID_ARG, std::string("malformed caches: ") + w4a16_last_error());
    if (workspace_bytes < need)
        return fail(W4A16_ERR_INVALID_ARG, "workspace smaller than w4a16_decode_kv_workspace_bytes()");
    if (M * widest >= ((int64_t)1 << 31))
        return fail(W4A16_ERR_UNSUPPORTED, "decode step too large for 32-bit kernel indexing");
    if (!aligned16(x_in) || !aligned16(x_out) || !aligned16(workspace))
        return fail(W4A16_ERR_UNSUPPORTED, "x_in, x_out and workspace must be 16-byte aligned");
    // Everything the step touches, in the order of its addresses: what it writes
    // may overlap nothing, what it only reads may (layers that share weights).
    std::vector<Span> spans;
    try {
        spans.reserve(16 * (size_t)n_layers + 5);
    } catch (const std::exception &) {
        return fail(W4A16_ERR_INVALID_ARG, "no host memory to check the memory of so many layers");
    }
    auto span = [&](const void *p, size_t n, bool written) {
        if (p && n) spans.push_back(Span{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + n, written});
    };
    if (x_in != x_out) span(x_in, (size_t)M * H * 2, false);
    span(x_out, (size_t)M * H * 2, true);
    span(workspace, need, true);
    span(block_table, (size_t)M * max_pages * 4, false);
    span(lens, (size_t)M * 4, false);
    for (int64_t l = 0; l < n_layers; ++l) {
        const w4a16_kv_cache &k = caches[l];
        const size_t n = (size_t)k.pages * k.heads * k.page * k.dim, ns = (size_t)k.pages * k.heads;
        span(k.k, n, true);
        span(k.v, n, true);
        span(k.k_scale, ns, true);
        span(k.v_scale, ns, true);
        for (int j = 0; j < 4; ++j) {
            const w4a16_linear &L = lin[4 * l + j];
            span(L.b_packed, (size_t)L.K * L.N / 2, false);
            span(L.scales, (size_t)(L.K / L.G) * L.N * 2, false);
            span(L.qzeros, (size_t)(L.K / L.G) * L.N / 2, false);
        }
    }
    std::sort(spans.begin(), spans.end(), [](const Span &a, const Span &b) { return a.begin < b.begin; });
    uintptr_t any_end = 0, written_end = 0;  // of the spans so far
    for (const Span &a : spans) {
        if (a.begin < (a.written ? any_end : written_end))
            return fail(W4A16_ERR_INVALID_ARG, "x_in, x_out, workspace, block_table, lens, the layers' caches and their "
                                               "weights must not overlap (x_out may be x_in)");
        any_end = std::max(any_end, a.end);
        if (a.written) written_end = std::max(written_end, a.end);
    }
    // Buffers: P the linears' wide outputs, Q attention and glue scratch, R the
    // hidden rows between the linears.
    const size_t buf = three / 3;
    char *base = static_cast<char *>(workspace);
    uint16_t *P = reinterpret_cast<uint16_t *>(base), *Q = reinterpret_cast<uint16_t *>(base + buf),
             *R = reinterpret_cast<uint16_t *>(base + 2 * buf);
    void *aw = base + three;
    const size_t aw_bytes = need - three;
    for (int64_t l = 0; l < n_layers; ++l) {
        const w4a16_linear *L = lin + 4 * l;
        const w4a16_kv_cache *c = caches + l;
        const int64_t NQ = L[0].N, I = L[2].N / 2, KV = c->heads * c->dim;
        if ((rc = w4a16_gemm_glue(l == 0 ? W4A16_GLUE_NONE : W4A16_GLUE_RMSNORM, l == 0 ? x_in : R, H, L, M, P, Q, buf,
                                  stream)) ||
            (rc = w4a16_kv_append(P + H, NQ, P + H + KV, NQ, c, block_table, max_pages, lens, nullptr, M, M, stream)) ||
            (rc = w4a16_attention(P, NQ, H / c->dim, c, block_table, max_pages, lens, nullptr, M, M, scale, 0, Q,
                                  aw_bytes ? aw : nullptr, aw_bytes, stream)) ||
            (rc = w4a16_gemm_glue(W4A16_GLUE_NONE, Q, H, L + 1, M, R, nullptr, 0, stream)) ||
            (rc = w4a16_gemm_glue(W4A16_GLUE_RMSNORM, R, H, L + 2, M, P, Q, buf, stream)) ||
            (rc = w4a16_gemm_glue(W4A16_GLUE_SWIGLU, P, 2 * I, L + 3, M, R, Q, buf, stream)))
            return rc;
    }
    return w4a16_rownorm(R, H, M, H, x_out, stream);
}

}  // extern "C"
