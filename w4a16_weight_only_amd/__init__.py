"""W4A16 weight-only-quantized linear layer for MI355X (gfx950).

Thin Python binding over the C ABI in ``include/w4a16.h`` (``libw4a16.so``,
built in-tree by ``python -m w4a16_weight_only_amd.build``).  The functions here
only check and marshal arguments -- dtype, shape, contiguity, device -- and pass
raw device pointers plus torch's current HIP stream to the library; every step
of the computation runs in the library's HIP kernels.  There is no fallback: if
the library is missing or the tensors are not on the GPU, the call raises.

    out = w4a16_gemm(a, b_packed, scales, qzeros, G, zp_bias=8)
    dst = w4a16_repack(src_nk8, K)
    y   = w4a16_decode_step(stack, x)

The operators around the linears of a decoder layer, in 8 bits (OCP e4m3):

    cache = w4a16_kv_cache(pages, heads, page, dim)
    w4a16_kv_append(k, v, cache, block_table, lens, rows)
    out = w4a16_attention(q, cache, block_table, lens, rows)
    (codes, scales), x = w4a16_add_rmsnorm_fp8(x, residual, weight)
    codes, scales = w4a16_quant_fp8(gate_up, ACT_SWIGLU)
    out = w4a16_gemm_fp8(codes, scales, w_codes, w_scales)
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "W4A16Error", "lib", "w4a16_gemm", "w4a16_gemm_noalloc", "w4a16_repack", "w4a16_repack_scales", "w4a16_decode_step",
    "w4a16_decode_workspace_bytes", "w4a16_gemm_glue", "w4a16_gemm_glue_workspace_bytes", "w4a16_rownorm",
    "w4a16_gemm_plan", "w4a16_set_tuning", "w4a16_release", "Linear", "STATUS",
    "GLUE_NONE", "GLUE_RMSNORM", "GLUE_SWIGLU",
    "w4a16_add_rmsnorm", "w4a16_add_rmsnorm_fp8", "w4a16_quant_fp8", "w4a16_gemm_fp8",
    "w4a16_gemm_fp8_plan", "w4a16_kv_cache",
    "w4a16_kv_append", "w4a16_attention", "w4a16_attention_workspace_bytes", "w4a16_decode_step_kv",
    "w4a16_decode_kv_workspace_bytes", "KVCache", "ACT_NONE", "ACT_SWIGLU",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a16.so")

STATUS = {0: "W4A16_OK", 1: "W4A16_ERR_INVALID_ARG", 2: "W4A16_ERR_UNSUPPORTED",
          3: "W4A16_ERR_HIP", 4: "W4A16_ERR_WORKSPACE"}
GLUE_NONE, GLUE_RMSNORM, GLUE_SWIGLU = 0, 1, 2
ACT_NONE, ACT_SWIGLU = 0, 1


class W4A16Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), message))
        self.status = status


class Linear(ctypes.Structure):
    """Mirror of ``w4a16_linear`` (host struct holding device pointers)."""
    _fields_ = [("b_packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("qzeros", ctypes.c_void_p), ("K", ctypes.c_int64), ("N", ctypes.c_int64),
                ("G", ctypes.c_int64), ("zp_bias", ctypes.c_int32)]


class KVCache(ctypes.Structure):
    """Mirror of ``w4a16_kv_cache`` (host struct holding device pointers)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page", ctypes.c_int64), ("dim", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libw4a16.so with argument types declared (raises if unbuilt)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libw4a16.so is not built; run `python -m w4a16_weight_only_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    L.w4a16_status_string.restype = ctypes.c_char_p
    L.w4a16_status_string.argtypes = [ctypes.c_int]
    L.w4a16_last_error.restype = ctypes.c_char_p
    L.w4a16_last_error.argtypes = []
    L.w4a16_repack.restype = ctypes.c_int
    L.w4a16_repack.argtypes = [P, P, I64, I64, P]
    L.w4a16_repack_scales.restype = ctypes.c_int
    L.w4a16_repack_scales.argtypes = [P, P, I64, I64, P]
    L.w4a16_gemm.restype = ctypes.c_int
    L.w4a16_gemm.argtypes = [P, P, P, P, I64, I64, I64, I64, I32, P, P]
    L.w4a16_gemm_noalloc.restype = ctypes.c_int
    L.w4a16_gemm_noalloc.argtypes = [P, P, P, P, I64, I64, I64, I64, I32, P, P]
    L.w4a16_decode_workspace_bytes.restype = SZ
    L.w4a16_decode_workspace_bytes.argtypes = [I64, P, I64]
    L.w4a16_decode_step.restype = ctypes.c_int
    L.w4a16_decode_step.argtypes = [P, I64, P, P, I64, P, SZ, P]
    L.w4a16_gemm_glue_workspace_bytes.restype = SZ
    L.w4a16_gemm_glue_workspace_bytes.argtypes = [ctypes.c_int, I64, P]
    L.w4a16_gemm_glue.restype = ctypes.c_int
    L.w4a16_gemm_glue.argtypes = [ctypes.c_int, P, I64, P, I64, P, P, SZ, P]
    L.w4a16_rownorm.restype = ctypes.c_int
    L.w4a16_rownorm.argtypes = [P, I64, I64, I64, P, P]
    L.w4a16_gemm_plan.restype = ctypes.c_int
    L.w4a16_gemm_plan.argtypes = [I64, I64, I64, I64, ctypes.POINTER(ctypes.c_int32),
                                  ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int64)]
    L.w4a16_release.restype = ctypes.c_int
    L.w4a16_release.argtypes = []
    L.w4a16_set_tuning.restype = ctypes.c_int
    L.w4a16_set_tuning.argtypes = [ctypes.c_char_p]
    F32 = ctypes.c_float
    L.w4a16_add_rmsnorm.restype = ctypes.c_int
    L.w4a16_add_rmsnorm.argtypes = [P, I64, P, I64, P, F32, I64, I64, P, P, P, P, P]
    L.w4a16_quant_fp8.restype = ctypes.c_int
    L.w4a16_quant_fp8.argtypes = [ctypes.c_int, P, I64, I64, I64, P, P, P]
    L.w4a16_gemm_fp8.restype = ctypes.c_int
    L.w4a16_gemm_fp8.argtypes = [P, P, P, P, I64, I64, I64, P, P]
    L.w4a16_gemm_fp8_plan.restype = ctypes.c_int
    L.w4a16_gemm_fp8_plan.argtypes = [I64, I64, I64] + [ctypes.POINTER(ctypes.c_int32)] * 3
    L.w4a16_kv_append.restype = ctypes.c_int
    L.w4a16_kv_append.argtypes = [P, I64, P, I64, P, P, I64, P, P, I64, I64, P]
    L.w4a16_attention_workspace_bytes.restype = SZ
    L.w4a16_attention_workspace_bytes.argtypes = [I64, P, I64, I64, I64]
    L.w4a16_attention.restype = ctypes.c_int
    L.w4a16_attention.argtypes = [P, I64, I64, P, P, I64, P, P, I64, I64, F32, I64, P, P, SZ, P]
    L.w4a16_decode_kv_workspace_bytes.restype = SZ
    L.w4a16_decode_kv_workspace_bytes.argtypes = [I64, P, I64, P, I64]
    L.w4a16_decode_step_kv.restype = ctypes.c_int
    L.w4a16_decode_step_kv.argtypes = [P, I64, P, P, I64, P, F32, P, P, I64, P, SZ, P]
    _lib = L
    return L


def _check(rc: int) -> None:
    if rc != 0:
        raise W4A16Error(rc, lib().w4a16_last_error().decode())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_ptr(dev):
    torch = _torch()
    return torch.cuda.current_stream(dev).cuda_stream


def _dev_tensor(t, name, dtype, ndim):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is dtype and t.dim() == ndim and t.is_cuda and t.is_contiguous():
        return t
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != ndim:
        raise ValueError("%s must be %d-D, got shape %s" % (name, ndim, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def w4a16_gemm(a, b_packed, scales, qzeros=None, G=128, zp_bias=8, out=None):
    """out[M, N] fp16 = a[M, K] . ((q - z) * s) with b_packed int32 [K, N/8],
    scales fp16 [K/G, N], qzeros int32 [K/G, N/8] or None (z = zp_bias)."""
    torch = _torch()
    _dev_tensor(a, "a", torch.float16, 2)
    _dev_tensor(b_packed, "b_packed", torch.int32, 2)
    _dev_tensor(scales, "scales", torch.float16, 2)
    M, K = a.shape
    N = b_packed.shape[1] * 8
    if b_packed.shape[0] != K:
        raise ValueError("b_packed must be [K, N/8] = [%d, *], got %s" % (K, tuple(b_packed.shape)))
    if G <= 0 or K % G != 0 or tuple(scales.shape) != (K // G, N):
        raise ValueError("scales must be [K/G, N] = [%d, %d], got %s" % (K // max(G, 1), N, tuple(scales.shape)))
    if qzeros is not None:
        _dev_tensor(qzeros, "qzeros", torch.int32, 2)
        if tuple(qzeros.shape) != (K // G, N // 8):
            raise ValueError("qzeros must be [K/G, N/8] = [%d, %d]" % (K // G, N // 8))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=a.device)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N] = [%d, %d]" % (M, N))
    _check(lib().w4a16_gemm(a.data_ptr(), b_packed.data_ptr(), scales.data_ptr(),
                            None if qzeros is None else qzeros.data_ptr(), M, K, N, G, zp_bias,
                            out.data_ptr(), _stream_ptr(a.device)))
    return out


def w4a16_gemm_noalloc(a, b_packed, scales, qzeros, G, zp_bias, out):
    """w4a16_gemm into a caller-allocated `out`, with the library's split-K
    scratch in its fixed per-GPU array: no allocation at all."""
    torch = _torch()
    _dev_tensor(a, "a", torch.float16, 2)
    _dev_tensor(b_packed, "b_packed", torch.int32, 2)
    _dev_tensor(scales, "scales", torch.float16, 2)
    _dev_tensor(out, "out", torch.float16, 2)
    M, K = a.shape
    N = b_packed.shape[1] * 8
    if b_packed.shape[0] != K or tuple(scales.shape) != (K // G, N) or tuple(out.shape) != (M, N):
        raise ValueError("shapes do not match a [M, K], b_packed [K, N/8], scales [K/G, N], out [M, N]")
    if qzeros is not None:
        _dev_tensor(qzeros, "qzeros", torch.int32, 2)
        if tuple(qzeros.shape) != (K // G, N // 8):
            raise ValueError("qzeros must be [K/G, N/8]")
    _check(lib().w4a16_gemm_noalloc(a.data_ptr(), b_packed.data_ptr(), scales.data_ptr(),
                                    None if qzeros is None else qzeros.data_ptr(), M, K, N, G, zp_bias,
                                    out.data_ptr(), _stream_ptr(a.device)))
    return out


def w4a16_repack(src_nk8, K, out=None):
    """Checkpoint int32 [N, K/8] -> kernel layout int32 [K, N/8] (bit-exact)."""
    torch = _torch()
    _dev_tensor(src_nk8, "src_nk8", torch.int32, 2)
    N = src_nk8.shape[0]
    if src_nk8.shape[1] * 8 != K:
        raise ValueError("src_nk8 must be [N, K/8] with K = %d" % K)
    if out is None:
        out = torch.empty((K, N // 8), dtype=torch.int32, device=src_nk8.device)
    else:
        _dev_tensor(out, "out", torch.int32, 2)
    _check(lib().w4a16_repack(src_nk8.data_ptr(), out.data_ptr(), K, N, _stream_ptr(src_nk8.device)))
    return out


def w4a16_repack_scales(src_ng, out=None):
    """Checkpoint group scales fp16 [N, K/G] -> kernel layout fp16 [K/G, N]
    (bit-exact transpose)."""
    torch = _torch()
    _dev_tensor(src_ng, "src_ng", torch.float16, 2)
    N, Gn = src_ng.shape
    if out is None:
        out = torch.empty((Gn, N), dtype=torch.float16, device=src_ng.device)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
        if tuple(out.shape) != (Gn, N):
            raise ValueError("out must be [K/G, N] = [%d, %d]" % (Gn, N))
    _check(lib().w4a16_repack_scales(src_ng.data_ptr(), out.data_ptr(), Gn, N, _stream_ptr(src_ng.device)))
    return out


def _linear_array(stack):
    """stack: list of dicts with b_packed, scales, qzeros (or None), G, zp_bias."""
    torch = _torch()
    arr = (Linear * len(stack))()
    for i, L in enumerate(stack):
        b, s, qz = L["b_packed"], L["scales"], L.get("qzeros")
        _dev_tensor(b, "b_packed", torch.int32, 2)
        _dev_tensor(s, "scales", torch.float16, 2)
        if qz is not None:
            _dev_tensor(qz, "qzeros", torch.int32, 2)
        arr[i] = Linear(b.data_ptr(), s.data_ptr(), None if qz is None else qz.data_ptr(),
                        b.shape[0], b.shape[1] * 8, L["G"], L.get("zp_bias", 8))
    return arr


def w4a16_decode_workspace_bytes(M, stack):
    if len(stack) % 4 != 0 or not stack:
        raise ValueError("stack must hold 4 linears per layer")
    arr = _linear_array(stack)
    return int(lib().w4a16_decode_workspace_bytes(M, ctypes.cast(arr, ctypes.c_void_p), len(stack) // 4))


def w4a16_decode_step(stack, x, out=None, workspace=None):
    """One decode step through len(stack)//4 layers; x fp16 [M, H] on the GPU."""
    torch = _torch()
    _dev_tensor(x, "x", torch.float16, 2)
    if len(stack) % 4 != 0 or not stack:
        raise ValueError("stack must hold 4 linears per layer")
    M = x.shape[0]
    arr = _linear_array(stack)
    nl = len(stack) // 4
    need = int(lib().w4a16_decode_workspace_bytes(M, ctypes.cast(arr, ctypes.c_void_p), nl))
    if need == 0:
        raise ValueError("malformed stack (shapes do not chain)")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty_like(x)
    _check(lib().w4a16_decode_step(ctypes.cast(arr, ctypes.c_void_p), nl, x.data_ptr(), out.data_ptr(), M,
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream_ptr(x.device)))
    return out


def _one_linear(linear):
    arr = _linear_array([linear])
    return arr, ctypes.cast(arr, ctypes.c_void_p)


def w4a16_gemm_glue_workspace_bytes(glue, M, linear):
    _keep, ptr = _one_linear(linear)
    return int(lib().w4a16_gemm_glue_workspace_bytes(glue, M, ptr))


def w4a16_gemm_glue(glue, x, linear, ldx=None, out=None, workspace=None):
    """One linear on glue-transformed rows of x (fp16 [M, ldx] on the GPU):
    GLUE_NONE out = x . W, GLUE_RMSNORM out = rn(x[:, :K]) . W, GLUE_SWIGLU
    out = rn(silu(x[:, :K]) * x[:, K:2K]) . W; `linear` is a dict like the
    decode stack's entries."""
    torch = _torch()
    _dev_tensor(x, "x", torch.float16, 2)
    M = x.shape[0]
    ldx = x.shape[1] if ldx is None else ldx
    keep, ptr = _one_linear(linear)
    N = keep[0].N
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x.device)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N] = [%d, %d]" % (M, N))
    need = int(lib().w4a16_gemm_glue_workspace_bytes(glue, M, ptr))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wptr = None if workspace is None else workspace.data_ptr()
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().w4a16_gemm_glue(glue, x.data_ptr(), ldx, ptr, M, out.data_ptr(), wptr, wbytes,
                                 _stream_ptr(x.device)))
    return out


def w4a16_rownorm(x, width=None, out=None):
    """y = rn(x[:, :width]) (fp16 [M, width]) for fp16 rows x on the GPU."""
    torch = _torch()
    _dev_tensor(x, "x", torch.float16, 2)
    M, ldx = x.shape
    width = ldx if width is None else width
    if out is None:
        out = torch.empty((M, width), dtype=torch.float16, device=x.device)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
    _check(lib().w4a16_rownorm(x.data_ptr(), ldx, M, width, out.data_ptr(), _stream_ptr(x.device)))
    return out


def w4a16_gemm_plan(M, K, N, G):
    """(path, splits, grid) the library would use: path 1 = GEMV, 2 = MFMA."""
    path, splits, grid = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    _check(lib().w4a16_gemm_plan(M, K, N, G, ctypes.byref(path), ctypes.byref(splits), ctypes.byref(grid)))
    return path.value, splits.value, grid.value


def w4a16_set_tuning(spec=None):
    """Replace the planner's tuning overrides ("key=value,..."; None restores
    the defaults)."""
    _check(lib().w4a16_set_tuning(spec.encode() if spec else None))


def w4a16_release():
    _check(lib().w4a16_release())


# ------------------------------------------- decoder-layer operators, 8 bits ---

def _row_tensor(t, name):
    """Row stride of fp16 rows with unit stride along the last dimension."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != torch.float16:
        raise TypeError("%s must be torch.float16, got %s" % (name, t.dtype))
    if t.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    ld, unit = t.stride()
    rows, width = t.shape
    if unit != 1 and width > 1:
        raise ValueError("%s must have unit stride along its last dimension" % name)
    return ld if rows > 1 else width


def _same_device(first, *others):
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("a tensor is on %s, not on %s like the first" % (t.device, first.device))


def _scratch(workspace):
    """(pointer, bytes) of a caller's workspace, or of none."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _launch(first, fn, *args):
    """fn(*args, stream) on the first tensor's device and torch's current stream there."""
    torch = _torch()
    dev = first.get_device()
    # the current stream's handle without a Stream object around it
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != 0:
        _check(rc)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _blocks(n):
    return -(-n // 128)


def _norm_args(x, residual, weight, sum_out):
    torch = _torch()
    ldx = _row_tensor(x, "x")
    M, W = x.shape
    ldr = 0
    if residual is not None:
        ldr = _row_tensor(residual, "residual")
        if tuple(residual.shape) != (M, W):
            raise ValueError("residual must be [M, width] = [%d, %d]" % (M, W))
    if weight is not None:
        _dev_tensor(weight, "weight", torch.float16, 1)
        if weight.shape[0] != W:
            raise ValueError("weight must be [width] = [%d]" % W)
    if sum_out is None:
        if residual is not None:
            sum_out = torch.empty((M, W), dtype=torch.float16, device=x.device)
    else:
        _dev_tensor(sum_out, "sum_out", torch.float16, 2)
        if tuple(sum_out.shape) != (M, W):
            raise ValueError("sum_out must be [M, width] = [%d, %d]" % (M, W))
    _same_device(x, residual, weight, sum_out)
    return ldx, ldr, M, W, sum_out


def w4a16_add_rmsnorm(x, residual=None, weight=None, eps=1e-6, out=None, sum_out=None):
    """(y, h): h = x + residual and y = weight * h / sqrt(mean(h^2) + eps), fp16
    rows [M, width].  sum_out receives h; it may be x or residual itself (the
    residual stream updated in place).  Without a residual and sum_out, h is x."""
    torch = _torch()
    ldx, ldr, M, W, sum_out = _norm_args(x, residual, weight, sum_out)
    if out is None:
        out = torch.empty((M, W), dtype=torch.float16, device=x.device)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
        if tuple(out.shape) != (M, W):
            raise ValueError("out must be [M, width] = [%d, %d]" % (M, W))
        _same_device(x, out)
    _launch(x, lib().w4a16_add_rmsnorm, x.data_ptr(), ldx, _ptr(residual), ldr, _ptr(weight), eps, M, W,
            _ptr(sum_out), out.data_ptr(), None, None)
    return out, x if sum_out is None else sum_out


def _codes_out(out, M, K, dev):
    """Output tensors of a quantising call: e4m3 [M, K] and fp32 [M, ceil(K/128)]."""
    torch = _torch()
    if out is None:
        return (torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev),
                torch.empty((M, _blocks(K)), dtype=torch.float32, device=dev))
    codes, scales = out
    _dev_tensor(codes, "codes", torch.float8_e4m3fn, 2)
    _dev_tensor(scales, "scales", torch.float32, 2)
    if tuple(codes.shape) != (M, K) or tuple(scales.shape) != (M, _blocks(K)):
        raise ValueError("out must be codes [%d, %d] and scales [%d, %d]" % (M, K, M, _blocks(K)))
    return codes, scales


def w4a16_add_rmsnorm_fp8(x, residual=None, weight=None, eps=1e-6, out=None, sum_out=None):
    """((codes, scales), h): as w4a16_add_rmsnorm, with y in e4m3 [M, width] and a
    scale fp32 [M, ceil(width/128)] per row and block of 128 columns."""
    ldx, ldr, M, W, sum_out = _norm_args(x, residual, weight, sum_out)
    codes, scales = _codes_out(out, M, W, x.device)
    _same_device(x, codes, scales)
    _launch(x, lib().w4a16_add_rmsnorm, x.data_ptr(), ldx, _ptr(residual), ldr, _ptr(weight), eps, M, W,
            _ptr(sum_out), None, codes.data_ptr(), scales.data_ptr())
    return (codes, scales), x if sum_out is None else sum_out


def w4a16_quant_fp8(x, act=ACT_NONE, out=None):
    """(codes, scales) of fp16 rows x: ACT_NONE quantises x [M, K], ACT_SWIGLU
    silu(x[:, :K]) * x[:, K:] of x [M, 2K], to e4m3 [M, K] with a scale fp32
    [M, ceil(K/128)] per row and block of 128 columns."""
    ldx = _row_tensor(x, "x")
    M, K = x.shape
    if act == ACT_SWIGLU:
        if K % 2:
            raise ValueError("SwiGLU takes rows of gate and up halves, got width %d" % K)
        K //= 2
    codes, scales = _codes_out(out, M, K, x.device)
    _same_device(x, codes, scales)
    _launch(x, lib().w4a16_quant_fp8, act, x.data_ptr(), ldx, M, K, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def w4a16_gemm_fp8(a, a_scales, b, b_scales, out=None):
    """out[M, N] fp16 = A . B^T with A = a (e4m3 [M, K]) scaled by a_scales (fp32
    [M, ceil(K/128)]) and B = b (e4m3 [N, K]) scaled by b_scales (fp32
    [ceil(N/128), ceil(K/128)])."""
    torch = _torch()
    _dev_tensor(a, "a", torch.float8_e4m3fn, 2)
    _dev_tensor(a_scales, "a_scales", torch.float32, 2)
    _dev_tensor(b, "b", torch.float8_e4m3fn, 2)
    _dev_tensor(b_scales, "b_scales", torch.float32, 2)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("b must be [N, K] = [*, %d], got %s" % (K, tuple(b.shape)))
    if tuple(a_scales.shape) != (M, _blocks(K)):
        raise ValueError("a_scales must be [M, ceil(K/128)] = [%d, %d]" % (M, _blocks(K)))
    if tuple(b_scales.shape) != (_blocks(N), _blocks(K)):
        raise ValueError("b_scales must be [ceil(N/128), ceil(K/128)] = [%d, %d]" % (_blocks(N), _blocks(K)))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=a.device)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
        if tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N] = [%d, %d]" % (M, N))
    _same_device(a, a_scales, b, b_scales, out)
    _launch(a, lib().w4a16_gemm_fp8, a.data_ptr(), a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(), M, K,
            N, out.data_ptr())
    return out


def w4a16_gemm_fp8_plan(M, K, N):
    """(rows, cols, groups): the workgroup tile and the wave groups dividing K that
    w4a16_gemm_fp8 takes for a size (of its first launch, where it needs two)."""
    r, c, g = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().w4a16_gemm_fp8_plan(M, K, N, ctypes.byref(r), ctypes.byref(c), ctypes.byref(g)))
    return r.value, c.value, g.value


def w4a16_kv_cache(pages, heads, page, dim, device="cuda"):
    """An empty paged 8-bit key/value cache: a dict of k e4m3 [pages, heads, page,
    dim], v e4m3 [pages, heads, dim, page] (transposed in each page), and k_scale
    and v_scale uint8 [pages, heads] (scale 2^(byte - 127))."""
    torch = _torch()
    return dict(k=torch.zeros((pages, heads, page, dim), dtype=torch.float8_e4m3fn, device=device),
                v=torch.zeros((pages, heads, dim, page), dtype=torch.float8_e4m3fn, device=device),
                k_scale=torch.full((pages, heads), 112, dtype=torch.uint8, device=device),
                v_scale=torch.full((pages, heads), 112, dtype=torch.uint8, device=device))


def _cache_struct(cache):
    torch = _torch()
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    _dev_tensor(k, "cache k", torch.float8_e4m3fn, 4)
    _dev_tensor(v, "cache v", torch.float8_e4m3fn, 4)
    _dev_tensor(ks, "cache k_scale", torch.uint8, 2)
    _dev_tensor(vs, "cache v_scale", torch.uint8, 2)
    P, H, page, D = k.shape
    if tuple(v.shape) != (P, H, D, page) or tuple(ks.shape) != (P, H) or tuple(vs.shape) != (P, H):
        raise ValueError("cache must hold k [pages, heads, page, dim], v [pages, heads, dim, page] and scales "
                         "[pages, heads]")
    _same_device(k, v, ks, vs)
    return KVCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), P, H, page, D)


def _sequence_args(block_table, lens, rows, T):
    torch = _torch()
    _dev_tensor(block_table, "block_table", torch.int32, 2)
    _dev_tensor(lens, "lens", torch.int32, 1)
    B = lens.shape[0]
    if block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages] with B = %d" % B)
    if rows is not None:
        _dev_tensor(rows, "rows", torch.int32, 1)
        if rows.shape[0] != B + 1:
            raise ValueError("rows must be [B + 1] = [%d]" % (B + 1))
    elif T != B:
        raise ValueError("without rows there is one row per sequence: %d rows, %d sequences" % (T, B))
    return B, block_table.shape[1]


def w4a16_kv_append(k, v, cache, block_table, lens, rows=None):
    """Writes fp16 rows k and v [T, heads*dim] (any row stride) to the cache as the
    last positions of sequences of lens[b] tokens: sequence b's rows are
    rows[b]..rows[b+1] (rows None: row b), position p goes to slot p % page of
    page block_table[b, p // page].  Returns the cache."""
    ldk, ldv = _row_tensor(k, "k"), _row_tensor(v, "v")
    c = _cache_struct(cache)
    T, W = k.shape
    if W != c.heads * c.dim or tuple(v.shape) != (T, W):
        raise ValueError("k and v must be [T, heads*dim] = [*, %d], got %s and %s"
                         % (c.heads * c.dim, tuple(k.shape), tuple(v.shape)))
    B, width = _sequence_args(block_table, lens, rows, T)
    _same_device(k, v, cache["k"], block_table, lens, rows)
    _launch(k, lib().w4a16_kv_append, k.data_ptr(), ldk, v.data_ptr(), ldv, ctypes.byref(c),
            block_table.data_ptr(), width, lens.data_ptr(), _ptr(rows), B, T)
    return cache


def w4a16_attention_workspace_bytes(heads, cache, max_pages, B, T):
    c = _cache_struct(cache)
    return int(lib().w4a16_attention_workspace_bytes(heads, ctypes.byref(c), max_pages, B, T))


def w4a16_attention(q, cache, block_table, lens, rows=None, scale=None, window=0, out=None, workspace=None):
    """Causal attention of fp16 rows q [T, heads*dim] (any row stride) over the
    cache; sequences as for w4a16_kv_append, whose rows are in the cache already.
    scale defaults to 1/sqrt(dim); window > 0 keeps each row's last `window`
    positions.  Returns fp16 [T, heads*dim]; rows past rows[-1] are not written."""
    torch = _torch()
    ldq = _row_tensor(q, "q")
    c = _cache_struct(cache)
    T, W = q.shape
    if W == 0 or W % (c.heads * c.dim):
        raise ValueError("q must be [T, heads*dim] with heads a multiple of %d and dim %d, got %s"
                         % (c.heads, c.dim, tuple(q.shape)))
    heads = W // c.dim
    B, width = _sequence_args(block_table, lens, rows, T)
    if out is None:
        out = torch.empty((T, W), dtype=torch.float16, device=q.device)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
        if tuple(out.shape) != (T, W):
            raise ValueError("out must be [T, heads*dim] = [%d, %d]" % (T, W))
    ref = ctypes.byref(c)
    if workspace is None:
        need = lib().w4a16_attention_workspace_bytes(heads, ref, width, B, T)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _same_device(q, cache["k"], block_table, lens, rows, out, workspace)
    _launch(q, lib().w4a16_attention, q.data_ptr(), ldq, heads, ref, block_table.data_ptr(), width,
            lens.data_ptr(), _ptr(rows), B, T, c.dim ** -0.5 if scale is None else scale, window, out.data_ptr(),
            *_scratch(workspace))
    return out


def _check_linear_shapes(stack):
    """Scales and zeros of the size the kernels read (the library sees only their addresses)."""
    for i, L in enumerate(stack):
        (K, words), G, qz = L["b_packed"].shape, L["G"], L.get("qzeros")
        groups = K // G if G > 0 else 0
        if tuple(L["scales"].shape) != (groups, words * 8):
            raise ValueError("scales of linear %d must be [K/G, N] = [%d, %d], got %s"
                             % (i, groups, words * 8, tuple(L["scales"].shape)))
        if qz is not None and tuple(qz.shape) != (groups, words):
            raise ValueError("qzeros of linear %d must be [K/G, N/8] = [%d, %d], got %s" % (i, groups, words, tuple(qz.shape)))


def _decode_kv_args(stack, caches, M, max_pages):
    if len(stack) % 4 != 0 or not stack:
        raise ValueError("stack must hold 4 linears per layer")
    if len(caches) != len(stack) // 4:
        raise ValueError("caches must hold one cache per layer")
    arr = _linear_array(stack)
    _check_linear_shapes(stack)
    carr = (KVCache * len(caches))(*[_cache_struct(c) for c in caches])
    lp, cp = ctypes.cast(arr, ctypes.c_void_p), ctypes.cast(carr, ctypes.c_void_p)
    need = int(lib().w4a16_decode_kv_workspace_bytes(M, lp, len(caches), cp, max_pages))
    return arr, carr, lp, cp, need


def w4a16_decode_kv_workspace_bytes(M, stack, caches, max_pages):
    return _decode_kv_args(stack, caches, M, max_pages)[4]


def w4a16_decode_step_kv(stack, caches, block_table, lens, x, scale=None, out=None, workspace=None):
    """One decode step of len(stack)//4 layers with attention over one cache per
    layer: x fp16 [M, H] holds one token for each of M sequences, lens their
    lengths with it."""
    torch = _torch()
    _dev_tensor(x, "x", torch.float16, 2)
    M = x.shape[0]
    _, width = _sequence_args(block_table, lens, None, M)
    arr, carr, lp, cp, need = _decode_kv_args(stack, caches, M, width)
    if x.shape[1] != arr[0].K:
        raise ValueError("x must be [M, H] = [%d, %d]" % (M, arr[0].K))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty_like(x)
    else:
        _dev_tensor(out, "out", torch.float16, 2)
        if out.shape != x.shape:
            raise ValueError("out must be [M, H] = [%d, %d]" % tuple(x.shape))
    _same_device(x, block_table, lens, out, workspace, *[t for L in stack for t in (L["b_packed"], L["scales"], L.get("qzeros"))],
                 *[c["k"] for c in caches])
    _launch(x, lib().w4a16_decode_step_kv, lp, len(caches), cp, block_table.data_ptr(), width, lens.data_ptr(),
            carr[0].dim ** -0.5 if scale is None else scale, x.data_ptr(), out.data_ptr(), M,
            *_scratch(workspace))
    return out
