"""Test-side helpers: golden-file parsing and input construction.

Packing an integer matrix into words is how a test *builds* an input from a
rule; the golden hand cases fix the nibble order independently of it.
"""
import os

import numpy as np

from oracle import layer as lo
from w4a16_weight_only_amd import synth

GOLDEN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "golden")


def read_cases(fname):
    cases, cur = [], None
    with open(os.path.join(GOLDEN, fname)) as f:
        for line in f:
            line = line.strip()
            if not line or line.startswith("#"):
                continue
            key, _, rest = line.partition(" ")
            if key == "case":
                cur = {"name": rest, "src": [], "dst": []}
            elif key == "end":
                cases.append(cur)
                cur = None
            elif key in ("src", "dst"):
                cur[key].append([int(w, 16) for w in rest.split()])
            else:
                cur[key] = rest
    return cases


def words(hexlist):
    return np.array([int(w, 16) for w in hexlist.split()], dtype=np.uint32).view(np.int32)


def pack_rows(q):
    """int matrix [R, C] with entries 0..15 -> int32 [R, C/8], nibble j = column 8w+j."""
    q = np.asarray(q, dtype=np.uint32)
    R, C = q.shape
    assert C % 8 == 0
    out = np.zeros((R, C // 8), dtype=np.uint32)
    for j in range(8):
        out |= (q[:, j::8] & 0xF) << np.uint32(4 * j)
    return out.view(np.int32)


def unpack_rows(w):
    """Inverse of pack_rows."""
    w = np.asarray(w).view(np.uint32)
    R, C8 = w.shape
    q = np.zeros((R, C8 * 8), dtype=np.int64)
    for j in range(8):
        q[:, j::8] = (w >> np.uint32(4 * j)) & 0xF
    return q



def oracle_gemm_columns(a, b_kn8, scales, qzeros, G, zp_bias=8):
    """The oracle's full product over column slices on the host's cores
    (identical to one oracle.gemm call)."""
    import oracle
    return oracle.gemm_columns(a, b_kn8, scales, qzeros, G, zp_bias)


def sink_case(n, rows, gap, together):
    """Keys that score about 0 but for one that stands `gap` above them, with values of zero there: every output is the
    tail's.  Rows with gaps from gap - 8 to gap, in one sequence or each in its own over the same pages."""
    D, page = 64, 64
    g = synth.rng(n + rows)
    pages = -(-n // page)
    c = dict(k=np.zeros((pages, 1, page, D), np.uint8), v=np.zeros((pages, 1, D, page), np.uint8),
             k_scale=np.full((pages, 1), 112, np.uint8), v_scale=np.full((pages, 1), 112, np.uint8))
    k = (g.standard_normal((n, D)) * 0.05).astype(np.float16)
    v = g.integers(1, 9, (n, D)).astype(np.float16)
    k[:, 0] = 0
    k[7], v[7] = 0, 0
    k[7, 0] = 1
    lo.kv_append(k, v, c, np.arange(pages)[None], [n], [0, n])
    q = g.standard_normal((rows, D)).astype(np.float16)
    q[:, 0] = np.linspace(gap - 8, gap, rows)
    if together:
        return q, c, np.arange(pages, dtype=np.int32)[None], np.array([n], np.int32), np.array([0, rows], np.int32)
    return q, c, np.tile(np.arange(pages, dtype=np.int32), (rows, 1)), np.full(rows, n, np.int32), None


def cancelling_case(B=64):
    """Two tokens whose weighted values all but cancel: the output is what the weights' rounding leaves, far above its
    own fp16 rounding."""
    D, page = 64, 16
    c = dict(k=np.zeros((B, 1, page, D), np.uint8), v=np.zeros((B, 1, D, page), np.uint8),
             k_scale=np.full((B, 1), 112, np.uint8), v_scale=np.full((B, 1), 112, np.uint8))
    k, v = np.zeros((2 * B, D), np.float16), np.ones((2 * B, D), np.float16)
    k[1::2, 0] = 1
    v[1::2] = -np.tile([1.125, 1.25, 1.375, 1.5], D // 4)
    table, lens = np.arange(B, dtype=np.int32)[:, None], np.full(B, 2, np.int32)
    lo.kv_append(k, v, c, table, lens, np.arange(0, 2 * B + 1, 2))
    q = np.zeros((B, D), np.float16)
    q[:, 0] = -np.log(np.tile([1.125, 1.25, 1.375, 1.5], B // 4)) + np.linspace(-1e-3, 1e-3, B)
    return q, c, table, lens
