"""GPU checks of how attention holds its softmax weights: long tails under one dominant token, scores far
beyond fp32's whole numbers, values that cancel, and calls that mix prompts with single tokens.

Bounds are the oracle's, with each weight as one fp16 value (2^-11 of it) where a call has more than 16 rows and heads
per sequence and key/value head on average, and as two (2^-22) otherwise.
"""
import numpy as np
import pytest

from oracle import layer as lo
from tests._fixtures import cancelling_case, sink_case
from tests.test_gpu_layer import attention_case, check, gpu, run_attention  # noqa: F401  (gpu is a fixture)
from w4a16_weight_only_amd import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,gap", [(300, 17.4), (20000, 17.4), (20000, 20.0)])
@pytest.mark.parametrize("rows,together", [(24, True), (8, False), (3, True)])
def test_tail_under_a_dominant_token(n, gap, rows, together):
    q, c, table, lens, off = sink_case(n, rows, gap, together)
    want = np.zeros(q.shape)
    bound = lo.attention(q, c, table, lens, off, 1.0, 0, want, parts=1 if rows > 16 else 2)
    got, _, _ = run_attention(q, c, table, lens, off, 1.0)
    check(got, want, bound, "tail n=%d gap=%g rows=%d" % (n, gap, rows))


@pytest.mark.parametrize("n,counts,width", [(300, [1], None), (3000, [1], 60), (300, [200], None), (300, [9], None)])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_scores_beyond_whole_numbers(n, counts, width, scale):
    """Scores of about 2^30, of which fp32 holds no fraction: the softmax picks each row's largest."""
    D = 64
    g = synth.rng(91)
    q, c, table, lens, off = attention_case(g, [n], counts, 1, 1, D, 64, width=width)
    k, v = (np.clip(g.standard_normal((n, D)) * f, -60000, 60000).astype(np.float16) for f in (16000, 1))
    lo.kv_append(k, v, c, table, [n], [0, n])
    q = np.clip(g.standard_normal(q.shape) * 16000, -60000, 60000).astype(np.float16)
    got, _, _ = run_attention(q, c, table, lens, off, scale)
    K, V = lo.cache_values(c, table[0, :-(-n // 64)], 0)
    assert np.isfinite(got).all()
    for i, row in enumerate(got):
        seen = n - len(got) + i + 1
        s = scale * (K[:seen] @ q[i].astype(np.float64))
        first, second = np.sort(s)[:-3:-1]
        # fp32 sums of D products are good to D 2^-24 of the magnitudes summed
        apart = 2 * (D + 8) * 2.0 ** -24 * (np.abs(K[:seen]) @ np.abs(q[i].astype(np.float64))).max() + 40
        assert first > 2.0 ** 28
        if first - second > apart:
            assert np.array_equal(row, V[s.argmax()].astype(np.float16)), "row %d" % i


@pytest.mark.parametrize("n,counts,width", [(700, [1], None), (3000, [1], 60), (700, [500], None), (700, [9], None)])
def test_scores_that_grow_beyond_whole_numbers(n, counts, width):
    """Small scores, then ones of 2^17, of 2^24 and of 2^30 along the cache: rows that end among the first follow the
    softmax, the others pick their largest."""
    D = 64
    g = synth.rng(93)
    q, c, table, lens, off = attention_case(g, [n], counts, 1, 1, D, 64, width=width)
    size = np.repeat([0.002, 2.0, 250.0, 16000.0], -(-n // 4))[:n, None]
    k, v = (np.clip(g.standard_normal((n, D)) * f, -60000, 60000).astype(np.float16) for f in (size, 1))
    lo.kv_append(k, v, c, table, [n], [0, n])
    q = np.clip(g.standard_normal(q.shape) * 16000, -60000, 60000).astype(np.float16)
    q[:n // 4] *= np.float16(0.01)
    got, want, bound = run_attention(q, c, table, lens, off, 1.0)
    check(got, want, bound, "growing")
    K, V = lo.cache_values(c, table[0, :-(-n // 64)], 0)
    picked = 0
    for i, row in enumerate(got):
        seen = n - len(got) + i + 1
        s = K[:seen] @ q[i].astype(np.float64)
        first, second = np.sort(s)[:-3:-1]
        if first - second > 2 * (D + 8) * 2.0 ** -24 * (np.abs(K[:seen]) @ np.abs(q[i].astype(np.float64))).max() + 40:
            assert np.array_equal(row, V[s.argmax()].astype(np.float16)), "row %d" % i
            picked += 1
    assert picked > 0


def test_single_tokens_carry_their_weights_in_two_parts():
    q, c, table, lens = cancelling_case()
    want = np.zeros(q.shape)
    bound = lo.attention(q, c, table, lens, None, 1.0, 0, want, parts=2)
    got, _, _ = run_attention(q, c, table, lens, None, 1.0)
    check(got, want, bound, "cancelling")


@pytest.mark.parametrize("lens,counts", [([3000, 700, 40], [1, 60, 1]), ([900] * 6 + [64], [1] * 6 + [40]), ([900] * 6 + [64], [1] * 6 + [12]),
                                         ([2, 2000, 130], [2, 1, 130])])
@pytest.mark.parametrize("window", [0, 100])
def test_prompts_beside_single_tokens(lens, counts, window):
    """One call over both, single tokens over long caches among them.  All of it is held as the call's average sequence is:
    up to 16 rows and heads to a key/value head in two fp16 values per weight, else in one."""
    g = synth.rng(97)
    q, c, table, lens, off = attention_case(g, lens, counts, 2, 4, 64, 32, extra_rows=2, heavy=True, width=100)
    few = -(-len(q) * 4 // len(lens)) <= 16
    want = np.full(q.shape, -77.0)
    bound = lo.attention(q, c, table, lens, off, 0.125, window, want, parts=2 if few else 1)
    got, _, _ = run_attention(q, c, table, lens, off, 0.125, window)
    check(got, want, np.where(bound == 0, 1e-30, bound), "mixed")
