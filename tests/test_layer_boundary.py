"""Refusals of the decoder-layer operators, at the C ABI and the Python binding (no GPU: every call here is rejected,
or returns as a no-op, before any HIP call)."""
import ctypes
import glob
import os
import re

import pytest
import torch

import w4a16_weight_only_amd as w4
from tests.test_boundary import INVALID, OK, UNSUPPORTED, lib  # noqa: F401  (lib is a fixture)

# Distinct, 16-byte-aligned fake device addresses (never dereferenced).
X, R, W, S, Y, Y8, YS, TB, LN, RW, KC, VC, KS, VS, WS = (0x10_0000_0000 + i * 0x10_0000_0000 for i in range(15))


def P(x):
    return None if x is None else ctypes.c_void_p(x)


def norm(lib, x=X, ldx=256, r=R, ldr=256, w=W, eps=1e-6, M=4, width=256, s=S, y=Y, y8=None, ys=None):  # noqa: F811
    return lib.w4a16_add_rmsnorm(P(x), ldx, P(r), ldr, P(w), eps, M, width, P(s), P(y), P(y8), P(ys), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(M=-1), INVALID), (dict(width=0), INVALID), (dict(width=252), INVALID),
    (dict(ldx=248), INVALID), (dict(ldx=260), INVALID), (dict(ldr=248), INVALID), (dict(ldr=257), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(y=None), INVALID), (dict(y8=Y8, ys=YS), INVALID), (dict(y=None, y8=Y8), INVALID),
    (dict(y=None, ys=YS), INVALID), (dict(ys=YS), INVALID),
    (dict(width=32776, ldx=32776, ldr=32776), UNSUPPORTED), (dict(M=(1 << 20) + 1), UNSUPPORTED),
    (dict(ldx=1 << 31), UNSUPPORTED),
    (dict(x=X + 8), UNSUPPORTED), (dict(w=W + 2), UNSUPPORTED), (dict(s=S + 4), UNSUPPORTED),
    (dict(y=X), INVALID), (dict(y=R + 512), INVALID), (dict(y=W), INVALID), (dict(s=W), INVALID), (dict(s=Y), INVALID),
    (dict(s=X + 512), INVALID), (dict(s=X, ldx=264), INVALID), (dict(s=R, ldr=512), INVALID),
    (dict(y=None, y8=Y8, ys=Y8 + 16), INVALID), (dict(y=None, y8=X, ys=YS), INVALID),
])
def test_norm_rejects(lib, kw, status):  # noqa: F811
    assert norm(lib, **kw) == status
    assert lib.w4a16_last_error().decode() != ""


def test_norm_noop(lib):  # noqa: F811
    assert norm(lib, M=0) == OK
    assert norm(lib, M=0, x=None, y=None) == OK


def quant(lib, act=0, x=X, ldx=256, M=4, K=256, y8=Y8, ys=YS):  # noqa: F811
    return lib.w4a16_quant_fp8(act, P(x), ldx, M, K, P(y8), P(ys), None)


@pytest.mark.parametrize("kw,status", [
    (dict(act=2), INVALID), (dict(act=-1), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(K=252), INVALID),
    (dict(x=None), INVALID), (dict(y8=None), INVALID), (dict(ys=None), INVALID), (dict(ldx=248), INVALID),
    (dict(ldx=260), INVALID), (dict(act=1), INVALID), (dict(act=1, ldx=504), INVALID),
    (dict(x=X + 2), UNSUPPORTED), (dict(y8=Y8 + 8), UNSUPPORTED), (dict(ys=YS + 2), UNSUPPORTED),
    (dict(M=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 26) + 8, ldx=1 << 27), UNSUPPORTED),
    (dict(M=1 << 20, K=1 << 16, ldx=1 << 16), UNSUPPORTED),
    (dict(y8=X), INVALID), (dict(ys=X + 256), INVALID), (dict(ys=Y8), INVALID),
])
def test_quant_rejects(lib, kw, status):  # noqa: F811
    assert quant(lib, **kw) == status
    assert lib.w4a16_last_error().decode() != ""


def gemm(lib, a=X, sa=S, b=W, sb=R, M=4, K=256, N=256, out=Y):  # noqa: F811
    return lib.w4a16_gemm_fp8(P(a), P(sa), P(b), P(sb), M, K, N, P(out), None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(b=None), INVALID), (dict(sb=None), INVALID),
    (dict(out=None), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID),
    (dict(K=264), UNSUPPORTED), (dict(K=(1 << 26) + 16), UNSUPPORTED), (dict(N=(1 << 26) + 1), UNSUPPORTED),
    (dict(M=(1 << 20) + 1), UNSUPPORTED), (dict(a=X + 8), UNSUPPORTED), (dict(b=W + 4), UNSUPPORTED),
    (dict(out=Y + 2), UNSUPPORTED), (dict(sa=S + 2), UNSUPPORTED), (dict(sb=R + 1), UNSUPPORTED),
    (dict(out=X), INVALID), (dict(out=W + 16), INVALID), (dict(out=S), INVALID), (dict(out=R), INVALID),
])
def test_gemm_fp8_rejects(lib, kw, status):  # noqa: F811
    assert gemm(lib, **kw) == status
    assert lib.w4a16_last_error().decode() != ""


def test_gemm_fp8_plan(lib):  # noqa: F811
    # few rows and long K: the row kernel; then tiles, divided along K where they are few
    assert w4.w4a16_gemm_fp8_plan(1, 12800, 4096) == (16, 16, 8)
    assert w4.w4a16_gemm_fp8_plan(64, 12800, 4096) == (32, 32, 4)
    assert w4.w4a16_gemm_fp8_plan(256, 12800, 4096) == (64, 64, 2)
    assert w4.w4a16_gemm_fp8_plan(4096, 4096, 25600) == (256, 256, 1)
    assert w4.w4a16_gemm_fp8_plan(1 << 20, 1 << 23, 64) == (16, 16, 8)  # rows past the tiles' 32-bit offsets
    for sizes, status in (((4, 264, 8), UNSUPPORTED), ((-1, 256, 8), INVALID), ((1 << 20, 256, 1 << 24), UNSUPPORTED)):
        with pytest.raises(w4.W4A16Error) as e:
            w4.w4a16_gemm_fp8_plan(*sizes)
        assert e.value.status == status


def test_gemm_fp8_noop(lib):  # noqa: F811
    assert gemm(lib, M=0, a=None, sa=None, out=None) == OK
    assert gemm(lib, M=0, b=None) == INVALID


def cache(**kw):
    c = dict(k=KC, v=VC, k_scale=KS, v_scale=VS, pages=10, heads=2, page=64, dim=128)
    c.update(kw)
    return w4.KVCache(*c.values())


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID),
    (dict(pages=0), INVALID), (dict(heads=0), INVALID), (dict(page=-16), INVALID), (dict(dim=0), INVALID),
    (dict(dim=96), UNSUPPORTED), (dict(dim=512), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=512), UNSUPPORTED), (dict(heads=1025), UNSUPPORTED), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(k=KC + 8), UNSUPPORTED), (dict(v=VC + 1), UNSUPPORTED),
]


def append(lib, c=None, k=X, ldk=256, v=R, ldv=256, tb=TB, mp=4, ln=LN, rw=RW, B=3, T=7):  # noqa: F811
    c = c or cache()
    return lib.w4a16_kv_append(P(k), ldk, P(v), ldv, ctypes.byref(c), P(tb), mp, P(ln), P(rw), B, T, None)


@pytest.mark.parametrize("kw,status", [(dict(c=cache(**c)), s) for c, s in BAD_CACHES] + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ldk=248), INVALID), (dict(ldv=260), INVALID),
    (dict(tb=None), INVALID), (dict(ln=None), INVALID), (dict(mp=0), INVALID), (dict(mp=1 << 40), UNSUPPORTED),
    (dict(mp=1 << 25), UNSUPPORTED), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(B=0), INVALID),
    (dict(rw=None), INVALID), (dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(B=(1 << 20) + 1), UNSUPPORTED),
    (dict(ldk=1 << 31), UNSUPPORTED), (dict(k=X + 8), UNSUPPORTED), (dict(v=R + 2), UNSUPPORTED),
    (dict(tb=TB + 2), UNSUPPORTED), (dict(ln=LN + 1), UNSUPPORTED), (dict(rw=RW + 2), UNSUPPORTED),
    (dict(c=cache(v=KC + 4096)), INVALID), (dict(c=cache(k_scale=KC)), INVALID), (dict(c=cache(v_scale=KS + 8)), INVALID),
    (dict(k=KC), INVALID), (dict(v=VC), INVALID), (dict(tb=KC + 64), INVALID), (dict(ln=KS), INVALID),
    (dict(rw=VS + 4), INVALID),
])
def test_append_rejects(lib, kw, status):  # noqa: F811
    assert append(lib, **kw) == status
    assert lib.w4a16_last_error().decode() != ""


def test_append_noop(lib):  # noqa: F811
    assert append(lib, T=0, k=None, v=None) == OK
    assert append(lib, T=0, B=0, k=None, v=None) == OK


def attention(lib, c=None, q=X, ldq=512, heads=4, tb=TB, mp=4, ln=LN, rw=RW, B=3, T=7, scale=0.1, window=0, out=Y,
              ws=WS, wsb=1 << 30):  # noqa: F811
    c = c or cache()
    return lib.w4a16_attention(P(q), ldq, heads, ctypes.byref(c), P(tb), mp, P(ln), P(rw), B, T, scale, window, P(out),
                               P(ws), wsb, None)


LONG = 4096  # pages per sequence: enough for the call to be split


@pytest.mark.parametrize("kw,status", [(dict(c=cache(**c)), s) for c, s in BAD_CACHES] + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(ldq=504), INVALID), (dict(ldq=516), INVALID),
    (dict(heads=3), INVALID), (dict(heads=0), INVALID), (dict(heads=-2), INVALID), (dict(heads=1026), UNSUPPORTED),
    (dict(tb=None), INVALID), (dict(ln=None), INVALID), (dict(mp=0), INVALID), (dict(mp=1 << 25), UNSUPPORTED),
    (dict(B=0), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(rw=None), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID),
    (dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(T=1 << 20, heads=1024, c=cache(heads=1)), UNSUPPORTED),
    (dict(ldq=1 << 31), UNSUPPORTED), (dict(q=X + 8), UNSUPPORTED), (dict(out=Y + 2), UNSUPPORTED),
    (dict(mp=LONG, ws=None), INVALID), (dict(mp=LONG, wsb=64), INVALID), (dict(mp=LONG, ws=WS + 4), UNSUPPORTED),
    (dict(out=X), INVALID), (dict(out=KC), INVALID), (dict(out=VC + 16), INVALID), (dict(out=KS), INVALID),
    (dict(out=TB), INVALID), (dict(mp=LONG, ws=Y), INVALID), (dict(mp=LONG, ws=X), INVALID),
    (dict(mp=LONG, ws=KC), INVALID),
])
def test_attention_rejects(lib, kw, status):  # noqa: F811
    assert attention(lib, **kw) == status
    assert lib.w4a16_last_error().decode() != ""


def test_attention_workspace_and_noop(lib):  # noqa: F811
    c = ctypes.byref(cache())
    size = lib.w4a16_attention_workspace_bytes
    assert size(4, c, LONG, 3, 7) > 0
    assert size(4, c, 1, 3, 3) == 0                      # one page each: nothing to split
    assert size(3, c, LONG, 3, 7) == 0 and size(4, c, LONG, 0, 7) == 0 and size(4, None, LONG, 3, 7) == 0
    assert size(4, ctypes.byref(cache(dim=96)), LONG, 3, 7) == 0
    assert attention(lib, T=0, q=None, out=None, ws=None) == OK
    assert attention(lib, T=0, B=0, q=None, out=None) == OK


def _stack(H=128, KV=128, I=256, G=32, layers=2):
    arr = (w4.Linear * (4 * layers))()
    for l in range(layers):
        for j, (k, n) in enumerate([(H, H + 2 * KV), (H, H), (H, 2 * I), (I, H)]):
            arr[4 * l + j] = w4.Linear(W + 0x100_0000 * (4 * l + j), S + 0x100_0000 * (4 * l + j), None, k, n, G, 8)
    return arr


def _caches(**kw):
    cs = (w4.KVCache * 2)()
    for l in range(2):
        cs[l] = cache(k=KC + l * 0x1000_0000, v=VC + l * 0x1000_0000, k_scale=KS + l * 0x1000_0000,
                      v_scale=VS + l * 0x1000_0000, heads=2, dim=64, **kw)
    return cs


def _same_cache_twice():
    cs = _caches()
    cs[1] = cs[0]
    return cs


def step(lib, stack=None, caches=None, tb=TB, mp=4, ln=LN, scale=0.1, x=X, y=Y, M=3, ws=WS, wsb=1 << 30, layers=2):  # noqa: F811
    s = ctypes.cast(stack if stack is not None else _stack(), ctypes.c_void_p)
    c = ctypes.cast(caches if caches is not None else _caches(), ctypes.c_void_p)
    return lib.w4a16_decode_step_kv(s, layers, c, P(tb), mp, P(ln), scale, P(x), P(y), M, P(ws), wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(layers=0), INVALID),
    (dict(M=0), INVALID), (dict(M=8193), INVALID), (dict(scale=float("nan")), INVALID), (dict(tb=None), INVALID),
    (dict(ln=None), INVALID), (dict(mp=0), INVALID), (dict(wsb=1000), INVALID), (dict(stack=_stack(KV=192)), INVALID),
    (dict(caches=_caches(page=24)), UNSUPPORTED), (dict(x=X + 2), UNSUPPORTED), (dict(ws=WS + 8), UNSUPPORTED),
    (dict(ws=X), INVALID), (dict(ws=KC), INVALID), (dict(y=VC), INVALID), (dict(y=X + 256), INVALID),
    (dict(y=LN), INVALID), (dict(caches=_same_cache_twice()), INVALID),
    (dict(tb=WS), INVALID), (dict(ln=WS), INVALID), (dict(tb=KC), INVALID), (dict(ln=KS), INVALID),
])
def test_decode_step_kv_rejects(lib, kw, status):  # noqa: F811
    assert step(lib, **kw) == status
    assert lib.w4a16_last_error().decode() != ""


@pytest.mark.parametrize("kw", [
    dict(ws=W + 0x100_0000 * 5), dict(ws=W + 0x100_0000 * 7 + 64), dict(ws=S + 0x100_0000), dict(y=W + 0x100_0000 * 4),
    dict(y=S + 0x100_0000 * 7), dict(weights=KC + 0x2000),
])
def test_decode_step_kv_rejects_written_memory_over_weights(lib, kw):  # noqa: F811
    """Before anything is launched: a step refused half way would have written its tokens to some of the caches."""
    stack, kw = _stack(), dict(kw)
    stack[6].b_packed = kw.pop("weights", stack[6].b_packed)
    assert step(lib, stack=stack, **kw) == INVALID
    assert "overlap" in lib.w4a16_last_error().decode()


def test_decode_step_kv_workspace(lib):  # noqa: F811
    s, c = ctypes.cast(_stack(), ctypes.c_void_p), ctypes.cast(_caches(), ctypes.c_void_p)
    three = lib.w4a16_decode_workspace_bytes(3, s, 2)
    one = ctypes.byref(_caches()[0])
    size = lib.w4a16_decode_kv_workspace_bytes
    assert size(3, s, 2, c, 1) == three
    assert size(3, s, 2, c, LONG) == three + lib.w4a16_attention_workspace_bytes(2, one, LONG, 3, 3)
    assert size(0, s, 2, c, 1) == 0 and size(3, s, 2, None, 1) == 0 and size(3, s, 2, c, 0) == 0


def test_python_binding_refuses(lib):  # noqa: F811
    x = torch.zeros(2, 256, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        w4.w4a16_add_rmsnorm(x)
    with pytest.raises(TypeError):
        w4.w4a16_quant_fp8(x.float())
    with pytest.raises(TypeError):
        w4.w4a16_gemm_fp8(x, x, x, x)
    with pytest.raises(ValueError):
        w4.w4a16_attention(x[0], {}, None, None)
    c = w4.w4a16_kv_cache(2, 1, 16, 64, device="cpu")
    assert c["k"].shape == (2, 1, 16, 64) and c["v"].shape == (2, 1, 64, 16) and int(c["k_scale"][0, 0]) == 112
    with pytest.raises(ValueError, match="GPU"):
        w4.w4a16_kv_append(x, x, c, None, None)
    # elements between a strided workspace's own would be overwritten
    assert w4._scratch(None) == (None, 0) and w4._scratch(x)[1] == 1024
    with pytest.raises(ValueError, match="contiguous"):
        w4._scratch(x[:, ::2])


def test_python_binding_checks_the_stacks_scales():
    """The library reads K/G rows of N scales from an address; a smaller tensor there would be read past its end."""
    def linear(scales, qzeros=None, G=32):
        return dict(b_packed=torch.zeros(128, 16, dtype=torch.int32), scales=torch.zeros(scales, dtype=torch.float16),
                    qzeros=None if qzeros is None else torch.zeros(qzeros, dtype=torch.int32), G=G, zp_bias=8)

    w4._check_linear_shapes([linear((4, 128)), linear((4, 128), (4, 16))])
    for bad in (linear((3, 128)), linear((4, 120)), linear((4, 128), (4, 15)), linear((4, 128), (1, 16)),
                linear((4, 128), G=64), linear((4, 128), G=0)):
        with pytest.raises(ValueError, match="linear 1"):
            w4._check_linear_shapes([linear((4, 128)), bad])


def test_inline_assembly_declares_what_it_writes():
    """Every block that sets m0 tells the compiler so, and every block that loads names memory."""
    blocks = []
    for path in glob.glob(os.path.join(os.path.dirname(w4.__file__), "csrc", "*")):
        with open(path) as f:
            blocks += re.findall(r"\basm\s+volatile\s*\((.*?)\);\n", f.read(), re.S)
    setters = [b for b in blocks if "s_mov_b32 m0" in b]
    assert setters and all('"m0"' in b.rsplit(":", 1)[1] for b in setters)
    assert all('"memory"' in b.rsplit(":", 1)[1] for b in blocks if "_load_" in b)
