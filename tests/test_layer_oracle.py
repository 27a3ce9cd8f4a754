"""Pins of the 64-bit oracle of the decoder-layer operators (no GPU): the e4m3 codec against hand values and torch's
CPU conversion, the cache's scale rule against its definition, attention and the block-scaled product against direct
sums."""
import numpy as np
import pytest
import torch

from oracle import layer as lo
from tests._fixtures import cancelling_case, sink_case


def test_e4m3_hand_values():
    for code, value in ((0x00, 0.0), (0x80, -0.0), (0x01, 2.0 ** -9), (0x07, 7 * 2.0 ** -9), (0x08, 2.0 ** -6),
                        (0x38, 1.0), (0x3C, 1.5), (0x7E, 448.0), (0xFE, -448.0)):
        assert lo.VALUES[code] == value
        assert lo.fp8_codes(np.array([value]))[0] == code
    assert np.isnan(lo.VALUES[0x7F]) and np.isnan(lo.VALUES[0xFF])
    # ties go to the even fraction: 1.0625 lies between 1.0 (even) and 1.125
    assert lo.VALUES[lo.fp8_codes(np.array([1.0625]))[0]] == 1.0
    assert lo.VALUES[lo.fp8_codes(np.array([1.1875]))[0]] == 1.25
    assert lo.VALUES[lo.fp8_codes(np.array([2.0 ** -10]))[0]] == 0.0
    assert lo.VALUES[lo.fp8_codes(np.array([3 * 2.0 ** -10]))[0]] == 2.0 ** -8


def test_e4m3_matches_torch_conversion():
    g = np.random.default_rng(1)
    x = np.concatenate([g.standard_normal(20000) * 60, g.standard_normal(20000) * 0.01,
                        (lo.VALUES[:0x7E] + lo.VALUES[1:0x7F]) / 2, lo.VALUES[:0x7F]]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn)
    assert np.array_equal(lo.fp8_codes(x), want.view(torch.uint8).numpy())
    assert np.array_equal(lo.fp8_values(lo.fp8_codes(x)), want.double().numpy())


@pytest.mark.parametrize("amax,e", [(0.0, -15), (448 * 2.0 ** -15, -15), (448 * 2.0 ** -15 + 2.0 ** -16, -14),
                                    (1.75, -8), (1.751953125, -7), (448.0, 0), (448.25, 1), (57344.0, 7),
                                    (57376.0, 8), (65504.0, 8)])
def test_page_exponent(amax, e):
    assert lo.page_exponent(np.array([0.0, -amax, np.nan, np.inf])) == e


def test_cache_values_are_fp16():
    # every value the cache stands for survives a round trip through fp16
    for e in range(lo.MIN_EXP, lo.MAX_EXP + 1):
        v = lo.VALUES[np.isfinite(lo.VALUES)] * 2.0 ** e
        if e == lo.MAX_EXP:
            v = v[np.abs(v) <= 61440]
        assert np.array_equal(v.astype(np.float16).astype(np.float64), v)
    top = lo.cache_codes(np.array([65504.0, -65504.0, np.inf, np.nan]), lo.MAX_EXP)
    assert np.array_equal(lo.fp8_values(top[:2]), [240, -240]) and np.isnan(lo.fp8_values(top[2:])).all()


def test_gemm_fp8_direct_sum():
    g = np.random.default_rng(2)
    M, K, N = 3, 272, 130
    a, b = g.integers(0, 0x7F, (M, K)).astype(np.uint8), g.integers(0, 0x7F, (N, K)).astype(np.uint8)
    sa, sb = g.random((M, 3)), g.random((2, 3))
    got, _ = lo.gemm_fp8(a, sa, b, sb)
    for m, n in ((0, 0), (2, 129), (1, 127), (1, 128)):
        want = sum(lo.VALUES[a[m, k]] * sa[m, k // 128] * lo.VALUES[b[n, k]] * sb[n // 128, k // 128] for k in range(K))
        assert abs(got[m, n] - want) < 1e-9 * max(1, abs(want))


def _cache(P, H, page, D):
    return dict(k=np.zeros((P, H, page, D), np.uint8), v=np.zeros((P, H, D, page), np.uint8),
                k_scale=np.full((P, H), 112, np.uint8), v_scale=np.full((P, H), 112, np.uint8))


def test_append_then_attention_uniform_weights():
    """Equal keys: attention is the running mean of the values (which are exact in the cache)."""
    H, D, page, n = 2, 64, 16, 37
    g = np.random.default_rng(3)
    k = np.ones((n, H * D), np.float16)
    v = g.integers(-8, 9, (n, H * D)).astype(np.float16)
    c = _cache(5, H, page, D)
    table = np.array([[3, 0, 4]], np.int32)
    lo.kv_append(k, v, c, table, [n], [0, n])
    q = g.standard_normal((n, 2 * H * D)).astype(np.float16)
    out = np.zeros(q.shape)
    lo.attention(q, c, table, [n], [0, n], 0.125, 0, out)
    for h in range(2 * H):
        vh = v[:, (h // 2) * D:(h // 2 + 1) * D].astype(np.float64)
        want = np.cumsum(vh, 0) / np.arange(1, n + 1)[:, None]
        assert np.abs(out[:, h * D:(h + 1) * D] - want).max() < 1e-12
    # token by token gives the same cache where scales do not change
    c2 = _cache(5, H, page, D)
    for i in range(n):
        lo.kv_append(k[i:i + 1], v[i:i + 1], c2, table, [i + 1], None)
    K1, V1 = lo.cache_values(c, [3, 0, 4], 1)
    K2, V2 = lo.cache_values(c2, [3, 0, 4], 1)
    assert np.array_equal(K1[:n], K2[:n]) and np.array_equal(V1[:n], V2[:n])


def test_append_grows_a_page_scale():
    c = _cache(1, 1, 16, 64)
    table = np.array([[0]], np.int32)
    lo.kv_append(np.full((1, 64), 1.0, np.float16), np.full((1, 64), 3.0, np.float16), c, table, [1], None)
    assert int(c["k_scale"][0, 0]) - 127 == -8 and int(c["v_scale"][0, 0]) - 127 == -7
    lo.kv_append(np.full((1, 64), 1000.0, np.float16), np.full((1, 64), 0.5, np.float16), c, table, [2], None)
    assert int(c["k_scale"][0, 0]) - 127 == 2 and int(c["v_scale"][0, 0]) - 127 == -7
    K, V = lo.cache_values(c, [0], 0)
    assert np.array_equal(K[:2, 0], [1.0, 1024.0 if abs(1000 - 1024) < abs(1000 - 960) else 960.0])
    assert np.array_equal(V[:2, 0], [3.0, 0.5])


def held(p, lift, parts):
    """Weights p (the largest 1) as fp16 values 2^lift up, in one part or two."""
    e = (p * 2.0 ** lift).astype(np.float32)
    h = e.astype(np.float16)
    low = (e - h.astype(np.float32)).astype(np.float16).astype(np.float64) if parts == 2 else 0.0
    return h.astype(np.float64) + low


def rebuilt(q, c, table, lens, off, lift, parts):
    """Attention of one head with a scale of 1 over weights held in fp16, rounded to fp16 at the end."""
    out = np.zeros(q.shape)
    for b, (r0, n) in enumerate(lo.sequence_rows(off, lens)):
        K, V = lo.cache_values(c, table[b], 0)
        for i in range(n):
            seen = int(lens[b]) - n + i + 1
            s = K[:seen] @ q[r0 + i].astype(np.float64)
            w = held(np.exp(s - s.max()), lift, parts)
            out[r0 + i] = w @ V[:seen] / w.sum()
    return out.astype(np.float16)


@pytest.mark.parametrize("parts", [1, 2])
def test_attention_bound_tells_a_lost_tail(parts):
    """Weights that stand at 1 lose what lies 2^-25 below the largest, and the bound refuses that; 2^11 up they keep it."""
    case = sink_case(3000, 12, 17.4, True)
    want = np.zeros(case[0].shape)
    bound = lo.attention(*case, 1.0, 0, want, parts=parts)
    for lift, kept in ((0, False), (11, True)):
        over = np.abs(rebuilt(*case, lift, parts) - want) / bound
        assert (over.max() <= 1.0) == kept, (lift, over.max())


def test_attention_bound_tells_weights_of_one_part_from_two():
    q, c, table, lens = cancelling_case()
    want = np.zeros(q.shape)
    bound = lo.attention(q, c, table, lens, None, 1.0, 0, want, parts=2)
    for parts in (1, 2):
        over = np.abs(rebuilt(q, c, table, lens, None, 11, parts) - want) / bound
        assert (over.max() <= 1.0) == (parts == 2), (parts, over.max())
