"""GPU parity of the decoder-layer operators in 8 bits against the 64-bit oracle.

Bounds are derived from the roundings each operator makes (half a step is 2^-11 for fp16, 2^-4 for e4m3, 2^-24 for
fp32) and stated where they are used; the cache writer is exact and is compared bit for bit.
"""
import sys

import numpy as np
import pytest
import torch

import oracle
import w4a16_weight_only_amd as w4
from oracle import layer as lo
from w4a16_weight_only_amd import synth

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn


def note(msg):
    print(msg, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    w4.lib()
    yield
    torch.cuda.synchronize()


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def codes_dev(x):
    return dev(x).view(FP8)


def host(t):
    torch.cuda.synchronize()
    return (t.view(torch.uint8) if t.dtype == FP8 else t).cpu().numpy()


def check(got, want, bound, what):
    got = got.astype(np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), "%s: NaN in other places" % what
    err = np.abs(got - want)[~nan]
    ratio = (err / np.broadcast_to(bound, want.shape)[~nan]).max(initial=0.0)
    note("%s max|err|=%.3g max err/bound=%.3g" % (what, err.max(initial=0.0), ratio))
    assert ratio <= 1.0, what


def check_codes(codes, scales, t, rel, what):
    """Codes and scales of rows t (64 bits) whose fp32 values are within `rel` of them.

    A scale is amax / 448, one fp32 division: within rel + 2^-23 of the exact
    one.  A code is t * (448 / amax), two more roundings, then half a step of
    e4m3 at that value (2^-4 of the value's binade, at least 2^-10)."""
    s = lo.block_scales(t)
    check(scales, s, (np.max(rel) + 2.0 ** -23) * s, what + " scales")
    c = t / lo.spread(s, t.shape[1])
    # the binade of the value as the kernel may see it, a little above the exact one
    top = np.abs(c) * (1 + 2.0 ** -12)
    half = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(top, 2.0 ** -30))), -6) - 4)
    check(lo.fp8_values(codes), c, half + np.abs(c) * (2 * rel + 2.0 ** -21), what + " codes")


# ------------------------------------------------------------------- norm ---

NORMS = [(1, 8), (3, 120), (2, 128), (5, 136), (130, 512), (7, 1000), (3, 2048), (2, 2056), (4, 4096), (3, 8200),
         (2, 16392), (2, 32768), (1200, 256)]


@pytest.mark.parametrize("M,W", NORMS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False)])
def test_add_rmsnorm(M, W, fp8, residual, weight):
    note("norm M=%d W=%d fp8=%s residual=%s weight=%s" % (M, W, fp8, residual, weight))
    g = synth.rng(W + M)
    x = synth.activations(g, M, W)
    r = (synth.activations(g, M, W) * np.float16(5)) if residual else None
    w = synth.activations(g, 1, W)[0] if weight else None
    y, h = lo.rmsnorm(x, r, w, 1e-5)
    # fp32 values of y: the mean of W squares (W * 2^-24 at most), square root, division and two products
    rel = (W / 2 + 8) * 2.0 ** -24
    if fp8:
        (codes, scales), hs = w4.w4a16_add_rmsnorm_fp8(dev(x), dev(r), dev(w), eps=1e-5)
        check_codes(host(codes), host(scales), y, rel, "norm")
    else:
        out, hs = w4.w4a16_add_rmsnorm(dev(x), dev(r), dev(w), eps=1e-5)
        check(host(out), y, np.abs(y) * (2.0 ** -11 + 2 * rel) + 2.0 ** -25, "norm")
    check(host(hs), h, np.abs(h) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25, "sum")


def test_norm_strided_and_in_place():
    g = synth.rng(11)
    M, W = 9, 264
    wide = dev(synth.activations(g, M, 1024))
    x, r = wide[:, 8:8 + W], dev(synth.activations(g, M, W))
    y, h = lo.rmsnorm(host(x), host(r), None, 1e-6)
    out, s = w4.w4a16_add_rmsnorm(x, r, sum_out=r)
    assert s is r
    check(host(out), y, np.abs(y) * (2.0 ** -11 + 2.0 ** -15) + 2.0 ** -25, "strided")
    check(host(r), h, np.abs(h) * 2.0 ** -10 + 2.0 ** -25, "in place")
    x2 = dev(host(x))
    r2 = dev(synth.activations(g, M, W))
    y2, h2 = lo.rmsnorm(host(x2), host(r2), None, 1e-6)
    out2, s2 = w4.w4a16_add_rmsnorm(x2, r2, sum_out=x2)
    assert s2 is x2
    check(host(out2), y2, np.abs(y2) * (2.0 ** -11 + 2.0 ** -15) + 2.0 ** -25, "in place of x")
    check(host(x2), h2, np.abs(h2) * 2.0 ** -10 + 2.0 ** -25, "x in place")


def test_norm_zero_rows_overflow_and_nan():
    x = np.zeros((5, 256), np.float16)
    x[1] = 65504.0
    x[2, 17] = np.nan
    x[3, 200] = np.inf
    x[4, 5] = 6e-8
    r = x.copy()
    r[2:4] = 1.0
    (codes, scales), h = w4.w4a16_add_rmsnorm_fp8(dev(x), dev(r), eps=1e-6)
    c, s, h = host(codes), host(scales), host(h)
    assert (c[0] == 0).all() and np.all(s[0] == np.float32(2.0 ** -40) / np.float32(448))
    assert (lo.fp8_values(c[1]) == 448).all() and np.isposinf(h[1]).all()   # the sum leaves fp16's range, its norm does not
    assert np.isnan(lo.fp8_values(c[2])[:, None] * s[2]).all()
    # by the formula: infinity over infinity where the infinity is, zero elsewhere
    v = lo.fp8_values(c[3])
    assert np.isnan(v[200]) and (np.delete(v, 200) == 0).all() and np.isfinite(s[3]).all()
    assert lo.fp8_values(c[4])[5] == 448 and (np.delete(c[4], 5) == 0).all()


# -------------------------------------------------------------- quantiser ---

@pytest.mark.parametrize("M,K", [(1, 8), (2, 128), (3, 136), (1, 1000), (33, 2048), (5, 2056), (2, 12800), (700, 64)])
@pytest.mark.parametrize("act", [w4.ACT_NONE, w4.ACT_SWIGLU])
def test_quant_fp8(M, K, act):
    note("quant M=%d K=%d act=%d" % (M, K, act))
    g = synth.rng(M * K + act)
    width = 2 * K if act else K
    x = (synth.activations(g, M, width + 16) * np.float16(3))
    t = lo.swiglu(x[:, :width]) if act else x[:, :width].astype(np.float64)
    # silu on the hardware exponential: its argument g log2(e) carries 2^-23 of |g|, the rest a few roundings
    rel = (np.abs(x[:, :K]).astype(np.float64) * 1.5 + 12) * 2.0 ** -23 if act else 0.0
    codes, scales = w4.w4a16_quant_fp8(dev(x)[:, :width], act=act)
    check_codes(host(codes), host(scales), t, rel, "quant")


def test_quant_special_values():
    x = np.zeros((4, 256), np.float16)
    x[1, :128] = 2.0 ** -24
    x[2, 3], x[2, 130] = np.nan, 7.0
    x[3, 3], x[3, 130] = -np.inf, -65504.0
    codes, scales = w4.w4a16_quant_fp8(dev(x))
    c, s = lo.fp8_values(host(codes)), host(scales)
    assert (c[0] == 0).all() and (c[1, :128] == 448).all() and (c[1, 128:] == 0).all()
    assert np.isnan(c[2, 3]) and np.isfinite(np.delete(c[2], 3)).all() and c[2, 130] == 448
    assert np.isnan((c[3, :128] * s[3, 0])).all() and c[3, 130] == -448 and s[3, 1] == np.float32(65504) / np.float32(448)
    # silu's ends: -inf gate gives 0 * up, a large gate is passed on
    y = np.zeros((1, 16), np.float16)
    y[0, :4], y[0, 8:12] = [-65504, 60000, 2, -2], [1, 1, 1, 1]
    codes, scales = w4.w4a16_quant_fp8(dev(y), act=w4.ACT_SWIGLU)
    v = lo.fp8_values(host(codes))[0] * host(scales)[0, 0]
    # code 448 times the scale: one reciprocal (2^-23) and one division (2^-24) away from 60000
    assert v[0] == 0 and abs(v[1] - 60000) <= 60000 * 2.0 ** -22


# ------------------------------------------------------------------- GEMM ---

GEMMS = [(1, 16, 1), (1, 112, 3), (2, 128, 16), (5, 144, 17), (16, 256, 100), (17, 1024, 128), (33, 2064, 130),
         (64, 384, 1000), (65, 512, 256), (130, 640, 264), (3, 12800, 128), (1, 4096, 6144), (128, 256, 384),
         (200, 1040, 520), (257, 144, 777), (300, 2048, 1024), (512, 128, 512), (1, 128, 40000), (1000, 400, 72)]
# one size at least for every tile shape, with ragged rows, columns and blocks (their outputs are sampled)
SHAPES = {(16, 16, 8): (5, 4112, 4090), (32, 32, 4): (30, 2000, 3000), (32, 64, 2): (60, 1424, 6100), (32, 64, 1): (1, 272, 18000),
          (64, 64, 2): (125, 1296, 6000), (64, 64, 1): (97, 272, 12000), (64, 128, 2): (190, 2064, 6001),
          (64, 128, 1): (190, 272, 13000), (128, 128, 2): (100, 1936, 18000),
          (128, 256, 1): (1000, 1680, 5000), (256, 256, 1): (2010, 1168, 6100)}


def gemm_inputs(M, K, N, seed):
    g = synth.rng(seed)
    a = lo.fp8_codes(np.clip(g.standard_normal((M, K)) * 100, -448, 448))
    b = lo.fp8_codes(np.clip(g.standard_normal((N, K)) * 100, -448, 448))
    sa = ((g.random((M, lo.blocks(K))) + 0.5) / 100).astype(np.float32)
    sb = ((g.random((lo.blocks(N), lo.blocks(K))) + 0.5) / (100 * np.sqrt(K))).astype(np.float32)
    return a, sa, b, sb


def gemm_bound(want, err):
    # the oracle's bound of the sums, then one rounding to fp16
    return np.abs(want) * 2.0 ** -11 + err * (1 + 2.0 ** -11) + 2.0 ** -25


@pytest.mark.parametrize("M,K,N", GEMMS)
def test_gemm_fp8(M, K, N):
    note("gemm_fp8 M=%d K=%d N=%d" % (M, K, N))
    a, sa, b, sb = gemm_inputs(M, K, N, M + 7 * K + 31 * N)
    want, err = lo.gemm_fp8(a, sa, b, sb)
    args = codes_dev(a), dev(sa), codes_dev(b), dev(sb)
    out = host(w4.w4a16_gemm_fp8(*args))
    check(out, want, gemm_bound(want, err), "gemm_fp8")
    assert np.array_equal(out, host(w4.w4a16_gemm_fp8(*args))), "not the same twice"


# sizes that are cut in two launches along N (the last round of 256 x 256 tiles would be mostly empty)
TWO_LAUNCHES = [(2048, 2048, 25590), (2040, 1936, 25600)]


@pytest.mark.parametrize("shape,size", list(SHAPES.items()) + [((256, 256, 1), x) for x in TWO_LAUNCHES])
def test_gemm_fp8_tile_shapes(shape, size):
    """Every tile shape: some rows in full (the first, the last and some between), against the oracle and, exactly, with
    integers whose sums are exact."""
    M, K, N = size
    assert w4.w4a16_gemm_fp8_plan(M, K, N) == shape
    note("gemm_fp8 %s M=%d K=%d N=%d" % (shape, M, K, N))
    a, sa, b, sb = gemm_inputs(M, K, N, M + K + N)
    rows = np.unique(np.linspace(0, M - 1, 9).astype(int))
    bd, sbd = codes_dev(b), dev(sb)
    out = host(w4.w4a16_gemm_fp8(codes_dev(a), dev(sa), bd, sbd))
    want, err = lo.gemm_fp8(a[rows], sa[rows], b, sb)
    check(out[rows], want, gemm_bound(want, err), "rows")
    g = synth.rng(5)
    ai, bi = g.integers(-2, 3, (M, K)), g.integers(-2, 3, (N, K))
    sa, sb = (2.0 ** g.integers(-1, 2, s.shape).astype(np.float32) for s in (sa, sb))
    out = host(w4.w4a16_gemm_fp8(codes_dev(lo.fp8_codes(ai.astype(np.float64))), dev(sa),
                                 codes_dev(lo.fp8_codes(bi.astype(np.float64))), dev(sb)))
    fa = torch.from_numpy((ai * lo.spread(sa.astype(np.float64), K))).cuda()
    fb = torch.from_numpy((bi * lo.spread(np.repeat(sb.astype(np.float64), 128, 0)[:N], K))).cuda()
    # sums of at most 5000 quarters of integers up to 16 are exact in fp32, their fp16 roundings compared bit for bit
    assert np.array_equal(out, host((fa @ fb.t().contiguous()).half()))


@pytest.mark.parametrize("M,K,N", [(1, 272, 40), (20, 272, 40), (300, 272, 300)])
def test_gemm_fp8_exact_integers(M, K, N):
    """Small integers and power-of-two scales: every product and sum is exact, so the output is, and an index that
    strays by one shows."""
    g = synth.rng(5)
    ai, bi = g.integers(-3, 4, (M, K)), g.integers(-3, 4, (N, K))
    a, b = lo.fp8_codes(ai.astype(np.float64)), lo.fp8_codes(bi.astype(np.float64))
    sa = (2.0 ** g.integers(-1, 2, (M, lo.blocks(K)))).astype(np.float32)
    sb = (2.0 ** g.integers(-1, 2, (lo.blocks(N), lo.blocks(K)))).astype(np.float32)
    want, _ = lo.gemm_fp8(a, sa, b, sb)
    assert np.array_equal(host(w4.w4a16_gemm_fp8(codes_dev(a), dev(sa), codes_dev(b), dev(sb))), want.astype(np.float16))


def test_gemm_fp8_rows_past_the_tiles_offsets():
    """K above 2^22, where every M takes the row kernel."""
    M, K, N = 20, (1 << 22) + 16, 40
    assert w4.w4a16_gemm_fp8_plan(M, K, N) == (16, 16, 8)
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, b = ((torch.rand(r, K, generator=gen, device="cuda") < 0.01).to(FP8) for r in (M, N))
    ones = (torch.ones(r, lo.blocks(K), device="cuda") for r in (M, 1))
    sa, sb = ones
    want = a.double() @ b.double().t().contiguous()          # counts of about 400: exact in fp16
    assert np.array_equal(host(w4.w4a16_gemm_fp8(a, sa, b, sb)), host(want.half()))


@pytest.mark.parametrize("M", [2, 40, 260])
def test_gemm_fp8_nan_stays_in_its_row_and_column(M):
    K, N = 256, 272
    a, sa, b, sb = gemm_inputs(M, K, N, 9)
    a[1, 200] = 0x7F
    b[130, 7] = 0xFF
    want, err = lo.gemm_fp8(a, sa, b, sb)
    assert np.isnan(want).sum() == M + N - 1
    check(host(w4.w4a16_gemm_fp8(codes_dev(a), dev(sa), codes_dev(b), dev(sb))), want, gemm_bound(want, err) + 1, "nan")


def test_gemm_fp8_subnormals_and_overflow():
    K = 128
    a = np.full((1, K), 0x01, np.uint8)          # 2^-9
    b = np.stack([np.full(K, 0x01, np.uint8), np.full(K, 0x7E, np.uint8)])
    sa, sb = np.ones((1, 1), np.float32), np.ones((1, 1), np.float32)
    out = host(w4.w4a16_gemm_fp8(codes_dev(a), dev(sa), codes_dev(b), dev(sb)))
    assert out[0, 0] == np.float16(128 * 2.0 ** -18) and out[0, 1] == np.float16(128 * 448 * 2.0 ** -9)
    big = host(w4.w4a16_gemm_fp8(codes_dev(b[1:]), dev(sa), codes_dev(b), dev(sb)))
    assert np.isposinf(big[0, 1])


# ------------------------------------------------------------------ cache ---

def empty_cache(P, H, page, D, g=None):
    """A cache whose unused slots hold old codes (NaN among them) and old scales."""
    g = g or synth.rng(1)
    c = dict(k=g.integers(0, 256, (P, H, page, D), dtype=np.uint8), v=g.integers(0, 256, (P, H, D, page), dtype=np.uint8),
             k_scale=g.integers(112, 136, (P, H), dtype=np.uint8), v_scale=g.integers(112, 136, (P, H), dtype=np.uint8))
    return c


def cache_dev(c):
    return {n: dev(x).view(FP8) if n in ("k", "v") else dev(x) for n, x in c.items()}


def one_nan(codes):
    """Codes with NaN's two signs made one: which of them a NaN is stored as is not defined."""
    return np.where((codes & 0x7F) == 0x7F, np.uint8(0x7F), codes)


def check_cache(got, want, what):
    for n in want:
        a, b = host(got[n]), want[n]
        if n in ("k", "v"):
            a, b = one_nan(a), one_nan(b)
        at = np.argwhere(a != b)
        assert len(at) == 0, "%s: %s differs at %s: %d, not %d" % (what, n, at[0], a[tuple(at[0])], b[tuple(at[0])])


def make_table(g, lens, page, extra=2):
    """Pages in random order; entries past a sequence's last page are out of range, so that a read shows."""
    per = [-(-max(int(n), 0) // page) for n in lens]
    P = sum(per) + extra
    order, at = g.permutation(P), 0
    table = np.full((len(lens), max(max(per), 1)), 1 << 30, np.int32)
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    return table, P


def both_append(k, v, c, cd, table, lens, rows):
    lo.kv_append(k, v, c, table, lens, rows)
    w4.w4a16_kv_append(dev(k), dev(v), cd, dev(table), dev(np.asarray(lens, np.int32)),
                       None if rows is None else dev(np.asarray(rows, np.int32)))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2), (256, 1)])
def test_append_prompts_then_tokens(page, D, H):
    note("append page=%d D=%d H=%d" % (page, D, H))
    g = synth.rng(page + D)
    counts = [1, page, page + 1, 3 * page - 1, 0, 40]
    steps = 5
    lens = np.array(counts)
    table, P = make_table(g, lens + 2 * page + steps, page)
    c = empty_cache(P, H, page, D, g)
    cd = cache_dev(c)
    rows = np.concatenate([[0], np.cumsum(counts)])
    T = int(rows[-1])
    both_append(synth.activations(g, T, H * D), synth.activations(g, T, H * D) * np.float16(0.01), c, cd, table, lens, rows)
    check_cache(cd, c, "prompt")
    # a second piece of each prompt, starting inside a page, with larger and smaller values
    more = np.array([page + 3, 2, 1, page, 5, 0])
    lens = lens + more
    rows = np.concatenate([[0], np.cumsum(more)])
    both_append(synth.activations(g, int(rows[-1]), H * D) * np.float16(100),
                synth.activations(g, int(rows[-1]), H * D) * np.float16(1e-3), c, cd, table, lens, rows)
    check_cache(cd, c, "second piece")
    for i in range(steps):  # single tokens, growing
        lens = lens + 1
        f = np.float16(4.0 ** (i - 2))
        both_append(synth.activations(g, len(lens), H * D) * f, synth.activations(g, len(lens), H * D) * f, c, cd, table,
                    lens, None)
        check_cache(cd, c, "token %d" % i)


def test_append_special_values():
    H, page, D = 2, 16, 64
    g = synth.rng(4)
    c = empty_cache(4, H, page, D, g)
    cd = cache_dev(c)
    table = np.array([[2, 0]], np.int32)
    x = synth.activations(g, 20, H * D)
    x[0, 3], x[1, 4], x[2, 5] = np.nan, np.inf, -np.inf
    x[16:] = 0
    x[3, 70] = 65504
    y = np.full((20, H * D), 2.0 ** -24, np.float16)
    y[5, 10] = -65504
    both_append(x, y, c, cd, table, [20], [0, 20])
    check_cache(cd, c, "special")
    # all of a page not finite
    z = np.full((1, H * D), np.nan, np.float16)
    both_append(z, -z, c, cd, np.array([[1, 3]], np.int32), [1], None)
    check_cache(cd, c, "nan")


def test_append_skips_what_has_no_place():
    """Rows before position 0, positions past the table, pages out of range: nothing else is written."""
    H, page, D = 1, 16, 64
    g = synth.rng(6)
    c = empty_cache(6, H, page, D, g)
    cd = cache_dev(c)
    table = np.array([[0, 1], [2, -1], [6, 3], [4, 5]], np.int32)
    counts = [10, 30, 40, 60]
    lens = [4, 30, 30, 60]       # 6 rows before position 0; a page -1; a page past the pool; 28 positions past the table
    rows = np.concatenate([[0], np.cumsum(counts)])
    k, v = synth.activations(g, 140, H * D), synth.activations(g, 140, H * D)
    both_append(k, v, c, cd, table, lens, rows)
    check_cache(cd, c, "skips")
    both_append(k[:4], v[:4], c, cd, table, [0, 17, 1, -5], None)
    check_cache(cd, c, "tokens")


def test_append_strided_rows():
    H, page, D = 2, 64, 128
    g = synth.rng(8)
    c = empty_cache(3, H, page, D, g)
    cd = cache_dev(c)
    qkv = synth.activations(g, 70, 5 * H * D)
    table = np.array([[2, 0]], np.int32)
    k, v = qkv[:, H * D:2 * H * D], qkv[:, 3 * H * D:4 * H * D]
    lo.kv_append(k, v, c, table, [100], [0, 70])
    q = dev(qkv)
    w4.w4a16_kv_append(q[:, H * D:2 * H * D], q[:, 3 * H * D:4 * H * D], cd, dev(table), dev(np.array([100], np.int32)),
                       dev(np.array([0, 70], np.int32)))
    check_cache(cd, c, "strided")


# -------------------------------------------------------------- attention ---

def attention_case(g, lens, counts, H, group, D, page, extra_rows=0, heavy=False, width=None):
    """Cache of sequences of `lens` tokens, queries for the last `counts` of each."""
    table, P = make_table(g, lens, page)
    if width is not None:
        table = np.concatenate([table, np.full((len(lens), width - table.shape[1]), -7, np.int32)], 1)
    c = empty_cache(P, H, page, D, g)
    n = np.maximum(np.asarray(lens), 0)
    rows = np.concatenate([[0], np.cumsum(n)])
    k, v = synth.activations(g, int(rows[-1]), H * D), synth.activations(g, int(rows[-1]), H * D)
    if heavy:
        k[:, ::7] *= np.float16(6)
    lo.kv_append(k, v, c, table, n, rows)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = synth.activations(g, int(off[-1]) + extra_rows, H * group * D)
    return q, c, table, np.asarray(lens, np.int32), off


def run_attention(q, c, table, lens, off, scale, window=0, qd=None, cd=None, workspace=None):
    fill = np.float16(-77.0)
    out = torch.full(q.shape, float(fill), dtype=torch.float16, device="cuda")
    w4.w4a16_attention(dev(q) if qd is None else qd, cache_dev(c) if cd is None else cd, dev(table), dev(lens),
                       None if off is None else dev(off), scale=scale, window=window, out=out, workspace=workspace)
    want = np.full(q.shape, float(fill))
    bound = lo.attention(q, c, table, lens, off, scale, window, want)
    return host(out), want, bound


ATTENTION = [
    # lens, rows per sequence, kv heads, group, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([0, 1, 15, 16, 17], [1] * 5, 2, 4, 128, 16),
    ([63, 64, 65, 129, 700], [1] * 5, 2, 3, 128, 32),
    ([300, 5, 1000], [1] * 3, 1, 8, 256, 64),
    ([513, 100], [1] * 2, 4, 1, 64, 128),
    ([257, 900], [1] * 2, 1, 20, 128, 256),
    ([40, 100], [2, 3], 2, 5, 64, 16),           # a few tokens each
    ([77, 33, 5], [77, 33, 5], 2, 2, 128, 16),   # prompts
    ([200, 130, 64, 1], [100, 2, 64, 1], 1, 4, 64, 32),
    ([150], [150], 1, 2, 256, 64),
    ([300, 10], [280, 10], 2, 1, 128, 64),
    ([90, 0, 70], [30, 4, 0], 1, 7, 128, 16),    # an empty sequence with rows, and one without
    ([3, 2], [5, 2], 1, 4, 64, 16),              # rows before position 0
    ([420], [400], 1, 4, 128, 128),
]


@pytest.mark.parametrize("case", range(len(ATTENTION)))
@pytest.mark.parametrize("window", [0, 1, 50])
def test_attention(case, window):
    lens, counts, H, group, D, page = ATTENTION[case]
    note("attention case=%d window=%d %s" % (case, window, ATTENTION[case]))
    g = synth.rng(100 + case)
    q, c, table, lens, off = attention_case(g, lens, counts, H, group, D, page, extra_rows=3)
    got, want, bound = run_attention(q, c, table, lens, off, D ** -0.5, window)
    check(got, want, np.where(bound == 0, 1e-30, bound), "attention")
    if all(n == 1 for n in counts):
        n = len(counts)
        got1, want1, bound1 = run_attention(q[:n], c, table, lens, None, D ** -0.5, window)
        check(got1, want1, np.where(bound1 == 0, 1e-30, bound1), "single rows")


@pytest.mark.parametrize("D,page,window", [(64, 16, 0), (64, 64, 60), (128, 64, 0), (128, 16, 60), (128, 256, 0)])
def test_attention_many_tiles(D, page, window):
    """Enough workgroups for the kernel that holds two column tiles per wave: many heads, of which some are compared; one
    sequence has a page out of range and NaN among its values."""
    H, group, lens, counts = 128, 2, [150, 330, 190], [150, 70, 190]
    g = synth.rng(D + page)
    q, c, table, lens, off = attention_case(g, lens, counts, H, group, D, page, extra_rows=1)
    table[2, 100 // page] = -3
    pid, slot = table[1, 20 // page], 20 % page
    c["v"][pid, 5, 7, slot] = 0x7F
    out = torch.full(q.shape, -77.0, dtype=torch.float16, device="cuda")
    w4.w4a16_attention(dev(q), cache_dev(c), dev(table), dev(lens), dev(off), window=window, out=out)
    out = host(out)
    assert (out[-1] == -77).all()
    for h in (0, 5, 70, 127):
        sub = {n: x[:, h:h + 1] for n, x in c.items()}
        cols = slice(h * group * D, (h + 1) * group * D)
        want = np.full((q.shape[0], group * D), -77.0)
        bound = lo.attention(q[:, cols], sub, table, lens, off, D ** -0.5, window, want)
        bound[np.isnan(bound)] = 1.0
        check(out[:, cols], want, np.where(bound == 0, 1e-30, bound), "head %d" % h)


@pytest.mark.parametrize("lens,counts,H,group,D,page,width", [
    ([5000, 64, 1, 3000, 0], [1] * 5, 1, 4, 128, 64, 200), ([2500, 130], [1, 1], 1, 16, 64, 16, 300),
    ([3000], [9], 1, 8, 128, 32, 120), ([1200, 700], [40, 30], 1, 2, 128, 64, 60), ([900], [1], 1, 6, 256, 128, 16)])
@pytest.mark.parametrize("window", [0, 700])
def test_attention_split(lens, counts, H, group, D, page, width, window):
    """Long tables: the work is cut along the tokens and joined."""
    g = synth.rng(7)
    q, c, table, lens, off = attention_case(g, lens, counts, H, group, D, page, heavy=True, width=width)
    assert w4.w4a16_attention_workspace_bytes(H * group, cache_dev(c), width, len(lens), len(q)) > 0
    got, want, bound = run_attention(q, c, table, lens, off, 1.5 * D ** -0.5, window)
    check(got, want, np.where(bound == 0, 1e-30, bound), "split")


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("counts", [[1, 1], [60, 20]])
def test_attention_scales(scale, counts):
    """Flat, reversed and peaked softmaxes (a peaked one raises the running maximum many times)."""
    g = synth.rng(17)
    q, c, table, lens, off = attention_case(g, [400, 90], counts, 2, 2, 64, 32, heavy=True)
    got, want, bound = run_attention(q, c, table, lens, off, scale)
    check(got, want, bound, "scale %g" % scale)


def test_attention_rising_scores():
    """Scores that grow along the cache by far more than the running maximum's slack, and fall again."""
    H, D, page, n = 1, 64, 16, 320
    c = empty_cache(20, H, page, D)
    ramp = np.concatenate([np.linspace(0, 200, n // 2), np.linspace(200, -100, n // 2)])
    k = np.zeros((n, D), np.float16)
    k[:, 0] = ramp
    v = synth.activations(synth.rng(3), n, D)
    table = np.arange(20, dtype=np.int32)[None, ::-1].copy()
    lo.kv_append(k, v, c, table, [n], [0, n])
    q = np.zeros((n, 2 * D), np.float16)
    q[:, 0], q[:, D] = 1.0, -1.0
    off = np.array([0, n], np.int32)
    got, want, bound = run_attention(q, c, table, np.array([n], np.int32), off, 1.0)
    check(got, want, bound, "ramp")


@pytest.mark.parametrize("counts", [[1], [33], [200]])
def test_attention_strided_queries(counts):
    g = synth.rng(23)
    H, group, D, page = 2, 4, 128, 64
    q, c, table, lens, off = attention_case(g, [260], counts, H, group, D, page)
    wide = torch.full((q.shape[0], q.shape[1] + 72), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 16:16 + q.shape[1]] = dev(q)
    got, want, bound = run_attention(q, c, table, lens, off, D ** -0.5, qd=wide[:, 16:16 + q.shape[1]])
    check(got, want, bound, "strided")


@pytest.mark.parametrize("counts,window", [([1], 0), ([1], 20), ([50], 0), ([50], 20), ([200], 0), ([200], 64)])
def test_attention_nan_reaches_exactly_the_rows_that_see_it(counts, window):
    g = synth.rng(29)
    H, group, D, page, n = 2, 2, 64, 32, 230
    q, c, table, lens, off = attention_case(g, [n], counts, H, group, D, page)
    # a value code, a key code, in different heads; and a query
    pid, slot = table[0, 195 // page], 195 % page
    c["v"][pid, 0, 11, slot] = 0x7F
    pid, slot = table[0, 215 // page], 215 % page
    c["k"][pid, 1, slot, 5] = 0xFF
    q[0, 3 * D + 1] = np.nan
    got, want, bound = run_attention(q, c, table, lens, off, D ** -0.5, window)
    bound[np.isnan(bound)] = 1.0
    check(got, want, bound, "nan")


@pytest.mark.parametrize("counts", [[1], [30], [120]])
def test_attention_stale_codes_beyond_fp16(counts):
    """Old codes of 448 in unused slots of pages whose scale is the largest (they would stand for 114688): not read."""
    g = synth.rng(30)
    H, D, page, n = 2, 64, 64, 130
    table = np.array([[2, 0, 1]], np.int32)
    c = empty_cache(4, H, page, D, g)
    c["k"][:], c["v"][:], c["k_scale"][:], c["v_scale"][:] = 0x7E, 0xFE, 135, 135
    k, v = synth.activations(g, n, H * D), synth.activations(g, n, H * D)
    v[::8] = 65504
    lo.kv_append(k, v, c, table, [n], [0, n])
    assert (c["v_scale"][[2, 0, 1]] == 135).all()
    q = synth.activations(g, counts[0], 2 * H * D)
    got, want, bound = run_attention(q, c, table, np.array([n], np.int32), np.array([0, counts[0]], np.int32), 0.125)
    check(got, want, bound, "stale")


def test_attention_bad_pages_and_lengths_are_nan():
    g = synth.rng(31)
    H, group, D, page = 1, 2, 64, 16
    q, c, table, lens, off = attention_case(g, [40, 40, 40, 40], [1, 1, 30, 1], H, group, D, page)
    table[0, 1] = -1
    table[2, 2] = c["k"].shape[0]     # seen from position 32 on
    lens[3] = 100                     # past the table
    got, want, bound = run_attention(q, c, table, lens, off, D ** -0.5)
    assert np.isnan(want[0]).all() and not np.isnan(want[1]).any() and np.isnan(want[-1]).all()
    bound[np.isnan(bound)] = 1.0
    check(got, want, bound, "bad pages")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("counts", [[1, 1], [100, 90]])
def test_attention_bad_pages_and_nan_in_whole_chunks(page, counts):
    """The same far behind the rows, in chunks that every row of a tile sees whole."""
    g = synth.rng(33)
    H, group, D, n = 2, 2, 64, 700
    q, c, table, lens, off = attention_case(g, [n, n], counts, H, group, D, page)
    table[0, 70 // page] = -5
    pid, slot = table[1, 200 // page], 200 % page
    c["v"][pid, 0, 3, slot] = 0x7F
    pid, slot = table[1, 330 // page], 330 % page
    c["k"][pid, 1, slot, 9] = 0x7F
    got, want, bound = run_attention(q, c, table, lens, off, D ** -0.5)
    assert np.isnan(want[:counts[0]]).all() and 0 < np.isnan(want[counts[0]:]).mean() < 1
    bound[np.isnan(bound)] = 1.0
    check(got, want, bound, "whole chunks")


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace from the allocator, give what they give alone."""
    g = synth.rng(35)
    jobs = []
    for i in range(2):
        q, c, table, lens, off = attention_case(g, [3000 + 500 * i, 700], [1, 1], 1, 4, 128, 64, width=80)
        args = dev(q), cache_dev(c), dev(table), dev(lens)
        jobs.append((args, host(w4.w4a16_attention(*args))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[] for _ in jobs]
    for _ in range(20):
        for s, (args, _), o in zip(streams, jobs, outs):
            with torch.cuda.stream(s):
                o.append(w4.w4a16_attention(*args))
    torch.cuda.synchronize()
    for (_, want), got in zip(jobs, outs):
        assert all(np.array_equal(host(x), want) for x in got)


def test_attention_infinite_query_is_nan():
    g = synth.rng(37)
    q, c, table, lens, off = attention_case(g, [30, 30], [1, 1], 1, 1, 64, 16)
    q[0, 0] = np.inf
    out = host(w4.w4a16_attention(dev(q), cache_dev(c), dev(table), dev(lens)))
    assert np.isnan(out[0]).all() and np.isfinite(out[1]).all()


def test_attention_malformed_offsets_stay_in_bounds():
    """Offset tables that start late, run backwards or past the rows: no fault, and other rows as they were."""
    g = synth.rng(41)
    q, c, table, lens, off = attention_case(g, [60, 60, 60], [20, 20, 20], 1, 2, 64, 16)
    cd, qd = cache_dev(c), dev(q)
    want = np.zeros(q.shape)
    lo.attention(q, c, table, lens, off, 0.125, 0, want)
    for rows in ([10, 20, 40, 60], [0, 20, 10, 500], [-5, 20, 40, 60], [60, 40, 20, 0]):
        out = torch.full(q.shape, -77.0, dtype=torch.float16, device="cuda")
        w4.w4a16_attention(qd, cd, dev(table), dev(lens), dev(np.array(rows, np.int32)), scale=0.125, out=out)
        torch.cuda.synchronize()
    late = torch.full(q.shape, -77.0, dtype=torch.float16, device="cuda")
    w4.w4a16_attention(qd, cd, dev(table), dev(lens), dev(np.array([20, 20, 40, 60], np.int32)), scale=0.125, out=late)
    late = host(late)
    assert (late[:20] == -77).all() and np.abs(late[20:] - want[20:]).max() < 0.01


def test_cache_past_4_gib():
    """Pages whose bytes lie past 32-bit offsets: the same results as from a small pool."""
    H, D, page, n = 1, 128, 64, 200
    g = synth.rng(47)
    pages = 600_000                                           # 4.9 GB of keys, as much of values
    k, v = synth.activations(g, n, D), synth.activations(g, n, D)
    lens, rows = dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32))
    outs = []
    for pool, ids in ((pages, [599_999, 3, 524_288, 524_289]), (5, [4, 3, 0, 1])):
        c = w4.w4a16_kv_cache(pool, H, page, D)
        table = dev(np.array([ids], np.int32))
        w4.w4a16_kv_append(dev(k), dev(v), c, table, lens, rows)
        q = dev(synth.activations(synth.rng(48), n, 4 * D))
        outs.append((host(w4.w4a16_attention(q, c, table, lens, rows)), host(w4.w4a16_attention(q[-1:], c, table, lens)),
                     host(c["k"][ids].contiguous()), host(c["v_scale"][ids].contiguous())))
    assert all(np.array_equal(a, b) for a, b in zip(*outs)) and np.abs(outs[0][0]).max() > 0


def test_attention_results_repeat():
    g = synth.rng(43)
    q, c, table, lens, off = attention_case(g, [900, 400], [1, 1], 2, 4, 128, 64, width=100)
    cd, a = cache_dev(c), (dev(q), dev(table), dev(lens))
    outs = [host(w4.w4a16_attention(a[0], cd, a[1], a[2])) for _ in range(4)]
    assert all(np.array_equal(outs[0], o) for o in outs)


# --------------------------------------------------------------- together ---

def quant_weights(g, N, K):
    w = g.standard_normal((N, K)) / np.sqrt(K)
    sb = np.stack([[max(np.abs(w[i:i + 128, j:j + 128]).max(), 1e-12) / 448 for j in range(0, K, 128)]
                   for i in range(0, N, 128)]).astype(np.float32)
    full = np.repeat(np.repeat(sb, 128, 0)[:N], 128, 1)[:, :K]
    return lo.fp8_codes(np.clip(w / full, -448, 448)), sb


def test_layer_in_8_bits():
    """A pre-norm decoder layer on the operators, as a server runs it: a prompt for each sequence, then single tokens.
    Every stage is checked against the oracle on the values the stage before it produced."""
    Hd, heads, kvh, D, I, page = 256, 4, 2, 64, 384, 16
    g = synth.rng(51)
    NQ = Hd + 2 * kvh * D
    lin = {n: quant_weights(g, N, K) for n, N, K in (("qkv", NQ, Hd), ("o", Hd, Hd), ("gu", 2 * I, Hd), ("down", Hd, I))}
    lind = {n: (codes_dev(a), dev(b)) for n, (a, b) in lin.items()}
    w1, w2 = (synth.activations(g, 1, Hd)[0] * np.float16(0.1) + np.float16(1) for _ in range(2))
    table, P = make_table(g, [60, 35], page)
    c = empty_cache(P, kvh, page, D, g)
    cd = cache_dev(c)

    def linear(name, codes, scales):
        out = w4.w4a16_gemm_fp8(codes, scales, *lind[name])
        want, err = lo.gemm_fp8(host(codes), host(scales), *lin[name])
        check(host(out), want, gemm_bound(want, err), name)
        return out

    def layer(x, lens, rows):
        (n8, ns), h = w4.w4a16_add_rmsnorm_fp8(x, None, dev(w1))
        y, _ = lo.rmsnorm(host(x), None, w1, 1e-6)
        check_codes(host(n8), host(ns), y, (Hd / 2 + 8) * 2.0 ** -24, "norm 1")
        qkv = linear("qkv", n8, ns)
        k, v = qkv[:, Hd:Hd + kvh * D], qkv[:, Hd + kvh * D:]
        rd = None if rows is None else dev(np.asarray(rows, np.int32))
        ld = dev(np.asarray(lens, np.int32))
        w4.w4a16_kv_append(k, v, cd, dev(table), ld, rd)
        lo.kv_append(host(k), host(v), c, table, lens, rows)
        check_cache(cd, c, "cache")
        att = w4.w4a16_attention(qkv[:, :Hd], cd, dev(table), ld, rd)
        want = np.zeros((x.shape[0], Hd))
        bound = lo.attention(host(qkv[:, :Hd]), c, table, lens, rows, D ** -0.5, 0, want)
        check(host(att), want, bound, "attention")
        a8, as_ = w4.w4a16_quant_fp8(att)
        check_codes(host(a8), host(as_), host(att).astype(np.float64), 0.0, "quant")
        o = linear("o", a8, as_)
        (m8, ms), h2 = w4.w4a16_add_rmsnorm_fp8(o, h, dev(w2))
        y, hh = lo.rmsnorm(host(o), host(h), w2, 1e-6)
        check_codes(host(m8), host(ms), y, (Hd / 2 + 8) * 2.0 ** -24, "norm 2")
        check(host(h2), hh, np.abs(hh) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25, "residual")
        gu = linear("gu", m8, ms)
        d8, ds = w4.w4a16_quant_fp8(gu, act=w4.ACT_SWIGLU)
        gh = host(gu)
        check_codes(host(d8), host(ds), lo.swiglu(gh), (np.abs(gh[:, :I]).astype(np.float64) * 1.5 + 12) * 2.0 ** -23, "swiglu")
        return linear("down", d8, ds), h2

    lens = np.array([50, 21])
    layer(dev(synth.activations(g, 71, Hd)), lens, np.array([0, 50, 71]))
    for _ in range(4):
        lens = lens + 1
        layer(dev(synth.activations(g, 2, Hd)), lens, None)


def step_inputs(M, layers, lens, page=16, H=256, kvh=2, D=64, I=384, G=64):
    g = synth.rng(61)
    stack, table = [], None
    for l in range(layers):
        for K, N in synth.stack_linear_shapes(H, H + 2 * kvh * D, I):
            stack.append(dict(b_packed=synth.packed_words(g, K, N // 8), scales=synth.scales(g, K // G, N, K), qzeros=None,
                              G=G, zp_bias=8))
    table, P = make_table(g, np.asarray(lens) + 8, page)
    caches = [empty_cache(P, kvh, page, D, g) for _ in range(layers)]
    rows = np.concatenate([[0], np.cumsum(lens)])
    for c in caches:
        lo.kv_append(synth.activations(g, int(rows[-1]), kvh * D), synth.activations(g, int(rows[-1]), kvh * D), c, table,
                     np.asarray(lens), rows)
    sd = [dict(L, b_packed=dev(L["b_packed"]), scales=dev(L["scales"])) for L in stack]
    return stack, sd, table, caches, synth.activations(g, M, H)


@pytest.mark.parametrize("M", [1, 2, 5, 20])
def test_decode_step_kv(M):
    """The step is the composition its header gives, bit for bit, and follows the oracle's linears and attention."""
    H, kvh, D, layers = 256, 2, 64, 2
    lens = [(i * 37) % 90 for i in range(M)]
    stack, sd, table, caches, x = step_inputs(M, layers, lens)
    now = np.asarray(lens, np.int32) + 1
    a, b = [cache_dev(c) for c in caches], [cache_dev(c) for c in caches]
    out = w4.w4a16_decode_step_kv(sd, a, dev(table), dev(now), dev(x))
    r, xin = None, dev(x)
    for l in range(layers):
        L = sd[4 * l:4 * l + 4]
        qkv = w4.w4a16_gemm_glue(w4.GLUE_NONE if l == 0 else w4.GLUE_RMSNORM, xin if l == 0 else r, L[0])
        w4.w4a16_kv_append(qkv[:, H:H + kvh * D], qkv[:, H + kvh * D:], b[l], dev(table), dev(now))
        att = w4.w4a16_attention(qkv[:, :H], b[l], dev(table), dev(now))
        want = np.zeros((M, H))
        host_cache = {n: host(t) for n, t in b[l].items()}
        bound = lo.attention(host(qkv[:, :H]), host_cache, table, now, None, D ** -0.5, 0, want)
        check(host(att), want, bound, "attention %d" % l)
        r = w4.w4a16_gemm_glue(w4.GLUE_NONE, att, L[1])
        want = oracle.gemm(host(att), stack[4 * l + 1]["b_packed"], stack[4 * l + 1]["scales"], None, 64, 8).astype(np.float64)
        check(host(r), want, 1e-2 * np.maximum(1, np.abs(want)), "o %d" % l)
        gu = w4.w4a16_gemm_glue(w4.GLUE_RMSNORM, r, L[2])
        r = w4.w4a16_gemm_glue(w4.GLUE_SWIGLU, gu, L[3])
    want = host(w4.w4a16_rownorm(r))
    assert np.array_equal(host(out), want)
    for ca, cb in zip(a, b):
        for n in ca:
            assert np.array_equal(host(ca[n]), host(cb[n]))
    same = dev(x)  # in place, twice on the same state: the same token is written again
    w4.w4a16_decode_step_kv(sd, a, dev(table), dev(now), same, out=same)
    assert np.array_equal(host(same), want)


def test_captured_step_replays_beside_eager_work():
    """Attention, its cache write, the norms and 8-bit linears in two captured graphs with new inputs at each replay,
    between them eager calls that use the same tensors' values."""
    H, group, D, page, B = 2, 4, 64, 16, 3
    g = synth.rng(71)
    W = H * D
    table, P = make_table(g, [400, 90, 40], page)
    lens0 = np.array([380, 70, 20], np.int32)
    c = empty_cache(P, H, page, D, g)
    n = np.concatenate([[0], np.cumsum(lens0)])
    lo.kv_append(synth.activations(g, int(n[-1]), W), synth.activations(g, int(n[-1]), W), c, table, lens0, n)
    wq, wd = quant_weights(g, (group + 2) * W, 256), quant_weights(g, 256, group * W)
    wq, wd = (codes_dev(wq[0]), dev(wq[1])), (codes_dev(wd[0]), dev(wd[1]))
    norm_w = dev(synth.activations(g, 1, 256)[0])
    td = dev(table)

    def work(s):
        (a, sa), h = w4.w4a16_add_rmsnorm_fp8(s["x"], s["r"], norm_w)
        qkv = w4.w4a16_gemm_fp8(a, sa, *wq)
        w4.w4a16_kv_append(qkv[:, group * W:(group + 1) * W], qkv[:, (group + 1) * W:], s["cache"], td, s["lens"])
        att = w4.w4a16_attention(qkv[:, :group * W], s["cache"], td, s["lens"])
        return w4.w4a16_gemm_fp8(*w4.w4a16_quant_fp8(att), *wd), h

    def state(seed):
        gg = synth.rng(seed)
        return dict(x=dev(synth.activations(gg, B, 256)), r=dev(synth.activations(gg, B, 256)), lens=dev(lens0),
                    cache=cache_dev(c))

    s1, s2, eager = state(1), state(2), state(3)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for s in (s1, s2):
            work(s)
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=stream):
                s["out"] = work(s)
            graphs.append(gr)
    torch.cuda.synchronize()
    for i in range(4):
        for s, gr in ((s1, graphs[0]), (s2, graphs[1])):
            gg = synth.rng(90 + i)
            for t in (s, eager):
                t["x"].copy_(dev(synth.activations(synth.rng(90 + i), B, 256)))
                t["r"].copy_(dev(synth.activations(synth.rng(190 + i), B, 256)))
                t["lens"].copy_(dev(lens0 + 1 + i))
            for n in eager["cache"]:
                eager["cache"][n].copy_(s["cache"][n])
            torch.cuda.synchronize()
            gr.replay()
            want, hw = work(eager)
            torch.cuda.synchronize()
            assert np.array_equal(host(s["out"][0]), host(want)) and np.array_equal(host(s["out"][1]), host(hw)), i
            for n in eager["cache"]:
                assert np.array_equal(host(s["cache"][n]), host(eager["cache"][n]))


def test_side_stream():
    """Calls follow torch's current stream: a producer on a side stream is waited for by stream order alone."""
    g = synth.rng(81)
    q, c, table, lens, off = attention_case(g, [200, 300], [1, 1], 1, 4, 128, 64)
    want = host(w4.w4a16_attention(dev(q), cache_dev(c), dev(table), dev(lens)))
    cd, t, l = cache_dev(c), dev(table), dev(lens)
    src = dev(q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = torch.zeros_like(src)
        for _ in range(50):
            x = x * 0.5
        x = x + src
        out = w4.w4a16_attention(x, cd, t, l)
    s.synchronize()
    assert np.array_equal(host(out), want)


def test_python_binding_refuses_gpu_tensors():
    g = synth.rng(83)
    q, c, table, lens, off = attention_case(g, [20, 30], [1, 1], 1, 2, 64, 16)
    cd, qd, t, l = cache_dev(c), dev(q), dev(table), dev(lens)
    with pytest.raises(ValueError):
        w4.w4a16_attention(qd.t().contiguous().t(), cd, t, l)            # columns are not contiguous
    with pytest.raises(ValueError):
        w4.w4a16_attention(qd[:, :96], cd, t, l)                         # not whole heads
    with pytest.raises(ValueError):
        w4.w4a16_attention(qd, cd, t, l[:1])
    with pytest.raises(ValueError):
        w4.w4a16_attention(qd, cd, t, l, rows=dev(np.array([0, 1], np.int32)))
    with pytest.raises(TypeError):
        w4.w4a16_attention(qd, cd, t, l.long())
    with pytest.raises(ValueError):
        w4.w4a16_attention(qd, cd, t.cpu(), l)
    with pytest.raises(ValueError):
        w4.w4a16_attention(qd, dict(cd, v=cd["k"]), t, l)
    with pytest.raises(w4.W4A16Error):
        w4.w4a16_attention(qd, cd, t, l, scale=float("nan"))
    with pytest.raises(w4.W4A16Error):
        w4.w4a16_attention(qd, cd, t, l, window=-3)
    with pytest.raises(w4.W4A16Error):
        w4.w4a16_attention(qd[:, :128].expand(2, 128).as_strided((2, 128), (0, 1)), cd, t, l)  # rows on top of each other
    with pytest.raises(ValueError):
        w4.w4a16_kv_append(qd[:, :32], qd[:, :32], cd, t, l)
    x = dev(synth.activations(g, 4, 64))
    with pytest.raises(w4.W4A16Error):
        w4.w4a16_add_rmsnorm(x[:, :60])
    with pytest.raises(w4.W4A16Error):
        w4.w4a16_add_rmsnorm(x, out=x)
    with pytest.raises(ValueError):
        w4.w4a16_add_rmsnorm(x, x[:2])
    with pytest.raises(ValueError):
        w4.w4a16_quant_fp8(x[:, :63], act=w4.ACT_SWIGLU)
    a, s = w4.w4a16_quant_fp8(x)
    with pytest.raises(ValueError):
        w4.w4a16_gemm_fp8(a, s, a, s)                                    # weight scales are per 128 rows
    with pytest.raises(w4.W4A16Error):
        w4.w4a16_gemm_fp8(a[:, :24].contiguous(), s, a[:, :24].contiguous(), s[:1])
