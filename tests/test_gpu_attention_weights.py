"""GPU checks of how attention holds its softmax weights: long tails under one dominant token.

Bounds are the oracle's, with each weight as one fp16 value (2^-11 of it) where a call has more than 16 rows and heads
per sequence and key/value head on average, and as two (2^-22) otherwise.
"""
import numpy as np
import pytest

from oracle import layer as lo
from tests._fixtures import sink_case
from tests.test_gpu_layer import check, gpu, run_attention  # noqa: F401  (gpu is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,gap", [(300, 17.4), (20000, 17.4), (20000, 20.0)])
@pytest.mark.parametrize("rows,together", [(24, True), (8, False), (3, True)])
def test_tail_under_a_dominant_token(n, gap, rows, together):
    q, c, table, lens, off = sink_case(n, rows, gap, together)
    want = np.zeros(q.shape)
    bound = lo.attention(q, c, table, lens, off, 1.0, 0, want, parts=1 if rows > 16 else 2)
    got, _, _ = run_attention(q, c, table, lens, off, 1.0)
    check(got, want, bound, "tail n=%d gap=%g rows=%d" % (n, gap, rows))
