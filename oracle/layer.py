"""Plain 64-bit forms of the decoder-layer operators in 8 bits (numpy).

Written from the formulas in include/w4a16.h; nothing is shared with the GPU
path.  8-bit tensors are uint8 codes; `fp8_values` and `fp8_codes` are the
format's definition (OCP e4m3: sign, 4 exponent bits with bias 7, 3 fraction
bits; 0x7f is NaN; no infinities; largest value 448).
"""
import numpy as np

BLOCK = 128
MIN_EXP, MAX_EXP = -15, 8


def _table():
    c = np.arange(256)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v[(c & 0x7F) == 0x7F] = np.nan
    return sign * v


VALUES = _table()


def fp8_values(codes):
    return VALUES[np.asarray(codes)]


def fp8_codes(x):
    """Nearest codes of x (|x| rounding to at most 448, or NaN), ties to even."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0)
    step = np.rint(a / 2.0 ** (e - 3))           # 0..16 steps of the binade
    up = step == 16
    e, step = np.where(up, e + 1, e), np.where(up, 8.0, step)
    code = np.where(step >= 8, ((e + 7).astype(np.int64) << 3) + step.astype(np.int64) - 8, step.astype(np.int64))
    assert code.max(initial=0) <= 0x7E, "value beyond 448"
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def blocks(n):
    return -(-n // BLOCK)


def block_scales(t):
    """max(amax, 2^-40) / 448 per row and block of 128 columns."""
    return np.stack([np.maximum(np.abs(t[:, i:i + BLOCK]).max(1), 2.0 ** -40) for i in range(0, t.shape[1], BLOCK)],
                    1) / 448.0


def spread(scales, width):
    """Block scales [R, blocks] repeated over their columns: [R, width]."""
    return np.repeat(scales, BLOCK, axis=1)[:, :width]


def rmsnorm(x, residual, weight, eps):
    """(y, h) in 64 bits."""
    h = x.astype(np.float64) + (0.0 if residual is None else residual.astype(np.float64))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return (y if weight is None else y * weight.astype(np.float64)), h


def swiglu(x):
    K = x.shape[1] // 2
    g, u = x[:, :K].astype(np.float64), x[:, K:].astype(np.float64)
    return g / (1 + np.exp(-g)) * u


def gemm_fp8(a, sa, b, sb):
    """(product, bound of a kernel's error before its last rounding), 64 bits.

    The 8-bit matrix instructions of gfx950 add products in groups of eight
    consecutive k, each product cut below 2^-14 of the binade of the group's
    largest (measured: beside 448 * 448 = 1.53 * 2^17, products of 2^3 count in
    full and products of 2^2 not at all), so a group is off by less than
    7 * 2^-14 of its largest product.  Everything after that is fp32: at most
    (K + 8) * 2^-24 of the sum of magnitudes."""
    K, N = a.shape[1], b.shape[0]
    A = fp8_values(a) * spread(sa.astype(np.float64), K)
    B = fp8_values(b) * spread(np.repeat(sb.astype(np.float64), BLOCK, axis=0)[:N], K)
    P, Q = np.nan_to_num(np.abs(A)).astype(np.float32), np.nan_to_num(np.abs(B)).astype(np.float32)
    largest = np.zeros((len(A), N), np.float32)
    for k in range(0, K, 8):
        m = P[:, k, None] * Q[None, :, k]
        for j in range(k + 1, min(k + 8, K)):
            np.maximum(m, P[:, j, None] * Q[None, :, j], out=m)
        largest += m
    bound = 7 * 2.0 ** -14 * 1.001 * largest.astype(np.float64) + (K + 8) * 2.0 ** -24 * (P.astype(np.float64) @ Q.T)
    return A @ B.T, bound


def sequence_rows(rows, lens):
    """[(first row, count)] per sequence."""
    if rows is None:
        return [(b, 1) for b in range(len(lens))]
    return [(int(rows[b]), int(rows[b + 1] - rows[b])) for b in range(len(lens))]


def page_exponent(x):
    """clamp(ceil(log2(amax / 448)), -15, 8) over finite values, by exact comparison."""
    f = np.abs(x[np.isfinite(x)])
    amax = float(f.max()) if f.size else 0.0
    e = MIN_EXP
    while e < MAX_EXP and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def cache_codes(x, e):
    s = np.asarray(x, dtype=np.float64) / 2.0 ** e
    s = np.where(np.isfinite(s), s, np.nan)
    if e == MAX_EXP:
        s = np.clip(s, -240.0, 240.0)
    return fp8_codes(s)


def kv_append(k, v, cache, table, lens, rows):
    """In place on a dict of uint8 arrays k [P, H, page, D], v [P, H, D, page],
    k_scale, v_scale [P, H]."""
    P, H, page, D = cache["k"].shape
    for b, (r0, n) in enumerate(sequence_rows(rows, lens)):
        begin = max(0, int(lens[b]) - n)
        for pg in range(begin // page, -(-int(lens[b]) // page)):
            if n == 0 or pg >= table.shape[1] or not 0 <= table[b, pg] < P:
                continue
            pid, p0 = int(table[b, pg]), pg * page
            lo, hi = max(p0, begin), min(p0 + page, int(lens[b]))
            at = r0 + lo - (int(lens[b]) - n)
            for x, codes, scale in ((k, cache["k"], cache["k_scale"]),
                                    (v, cache["v"].transpose(0, 1, 3, 2), cache["v_scale"])):
                for h in range(H):
                    t = x[at:at + hi - lo, h * D:(h + 1) * D].astype(np.float64)
                    e = page_exponent(t)
                    if lo > p0:
                        old = min(max(int(scale[pid, h]) - 127, MIN_EXP), MAX_EXP)
                        if e > old:
                            codes[pid, h, :lo - p0] = fp8_codes(fp8_values(codes[pid, h, :lo - p0]) * 2.0 ** (old - e))
                        e = max(e, old)
                    scale[pid, h] = e + 127
                    codes[pid, h, lo - p0:hi - p0] = cache_codes(t, e)


def cache_values(cache, pids, h):
    """(K, V) of the pages in order: [tokens, D] each."""
    ks = 2.0 ** (cache["k_scale"][pids, h].astype(np.float64) - 127)
    vs = 2.0 ** (cache["v_scale"][pids, h].astype(np.float64) - 127)
    K = fp8_values(cache["k"][pids, h]) * ks[:, None, None]
    V = fp8_values(cache["v"][pids, h]) * vs[:, None, None]
    D = K.shape[-1]
    return K.reshape(-1, D), V.transpose(0, 2, 1).reshape(-1, D)


def attention(q, cache, table, lens, rows, scale, window, out, parts=1):
    """Writes 64-bit results over `out` [T, heads * D] (other rows stay) and
    returns the error bound of fp32 scores and fp16 weights next to it:

      weights   each is held as one fp16 value, 2^-11 of it, or with parts = 2
                as two, 2^-22 of it, in the sum it is divided by as well; or,
                where it is small, half of fp16's smallest step, 2^-25.
                Weights stand 2^11 above their maximum's 1 (which is at most the
                row's largest), so that is 2^-36;
      scores    D products summed in fp32, then one multiplication and one
                subtraction: (D + 8) * 2^-24 of the magnitudes summed, twice over
                for the weight and for the sum it is divided by; exp2 itself
                2^-22;
      sums      of n weights and weighted values, n * 2^-24 each at most (counted
                with parts = 2; less than the weights' own roundings otherwise);
      output    one rounding to fp16: 2^-11, or 2^-25 absolute."""
    D, (P, H, page, _) = cache["k"].shape[3], cache["k"].shape
    heads = q.shape[1] // D
    bound = np.zeros_like(out)
    for b, (r0, n) in enumerate(sequence_rows(rows, lens)):
        if n == 0:
            continue
        L = int(lens[b])
        npg = -(-max(L, 0) // page)
        pids = table[b, :npg].astype(np.int64)
        cap = table.shape[1] * page
        for h in range(H):
            K, V = cache_values(cache, np.where((pids >= 0) & (pids < P), pids, 0), h)
            bad = np.repeat((pids < 0) | (pids >= P), page)
            for g in range(heads // H):
                col = slice((h * (heads // H) + g) * D, (h * (heads // H) + g + 1) * D)
                for i in range(n):
                    pos = L - n + i
                    if pos < 0:
                        out[r0 + i, col] = 0.0
                        continue
                    lo = max(0, pos - window + 1) if window else 0
                    qi = q[r0 + i, col].astype(np.float64)
                    if pos >= cap or bad[lo:pos + 1].any():
                        out[r0 + i, col] = np.nan
                        continue
                    k, v = K[lo:pos + 1], V[lo:pos + 1]
                    s = scale * (k @ qi)
                    p = np.exp(s - s.max())
                    l = p.sum()
                    out[r0 + i, col] = (p @ v) / l
                    mag = np.abs(scale) * (np.abs(k) @ np.abs(qi)).max() + np.abs(s).max()
                    rel = 2.0 ** -11 if parts == 1 else 2.0 ** -21 + 2 * len(p) * 2.0 ** -24
                    rel += 2 * ((D + 8) * 2.0 ** -24 * mag + 2.0 ** -22)
                    bound[r0 + i, col] = (2.0 ** -11 * np.abs(out[r0 + i, col]) + rel * (p @ np.abs(v)) / l +
                                          2 * len(p) * 2.0 ** -36 * np.nanmax(np.abs(v)) / l + 2.0 ** -25)
    return bound
