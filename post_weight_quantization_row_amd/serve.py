"""Python binding of libqrow.so's serving operators (argument marshalling
only): 8-bit rows with one scale each and their products
(include/serve/qrow_i8.h), the norm that makes such rows
(include/serve/qrow_norm.h), a paged 8-bit key/value cache and attention over
it (include/serve/qrow_kv8.h), a mixture of experts (include/serve/qrow_moe.h).

Every function has the name of the C entry point it calls and takes torch
tensors that live on the GPU; all arithmetic runs in the library's HIP
kernels, on the device of the tensors and the stream given (torch's current
one by default). There is no CPU fallback: without the built library or a GPU
the calls raise.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import qrow
from .qrow import QR_BF16, QR_F32, _check

# Every symbol the headers under include/serve/ declare.
EXPORTS = ("qr_i8_row_bytes", "qr_quantize_rows_i8", "qr_matmul_i8", "qr_kv8_code_bytes", "qr_kv8_append",
           "qr_kv8_read", "qr_attention_kv8_workspace_bytes", "qr_attention_kv8", "qr_matmul_i8_ex", "qr_norm_rows_i8",
           "qr_moe_route_workspace_bytes", "qr_moe_route", "qr_moe_i8_workspace_bytes", "qr_moe_i8")
HEAD_DIMS = (64, 128, 256)
BLOCK_TOKENS = (32, 64, 128)
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # QR_ACT_*
SCORES = {"softmax": 0, "sigmoid": 1}                                 # QR_SCORE_*
MOE_MAX_EXPERTS, MOE_MAX_TOP_K, MOE_MAX_PAIRS = 1024, 64, 8192

_DTYPES = {torch.float32: QR_F32, torch.bfloat16: QR_BF16}
_lib = None


class _Kv8(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("kd", C.c_void_p), ("vd", C.c_void_p),
                ("n_blocks", C.c_int64), ("n_heads", C.c_int64), ("head_dim", C.c_int64),
                ("block_tokens", C.c_int64)]


class _I8Epilogue(C.Structure):
    _fields_ = [("act", C.c_int64), ("up", C.c_void_p), ("upd", C.c_void_p), ("up_bias", C.c_void_p),
                ("residual", C.c_void_p), ("residual_stride", C.c_int64)]


class _Moe(C.Structure):
    _fields_ = [("gate", C.c_void_p), ("up", C.c_void_p), ("down", C.c_void_p), ("gated", C.c_void_p),
                ("upd", C.c_void_p), ("downd", C.c_void_p), ("n_experts", C.c_int64), ("n_in", C.c_int64),
                ("n_mid", C.c_int64), ("expert_rows", C.c_int64)]


def load_library():
    """libqrow.so with the serving entry points declared."""
    global _lib
    if _lib is None:
        L = qrow.load_library()
        vp, i64, i32, cache = C.c_void_p, C.c_int64, C.c_int, C.POINTER(_Kv8)
        L.qr_i8_row_bytes.argtypes = [i64]
        L.qr_quantize_rows_i8.argtypes = [i32, vp, i64, i64, i64, vp, vp, vp]
        L.qr_matmul_i8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i64, vp]
        L.qr_kv8_code_bytes.argtypes = [cache]
        rows = [cache, i32, vp, vp, i64, i64, i64, i64, vp, vp, vp, i64, vp]
        L.qr_kv8_append.argtypes = rows
        L.qr_kv8_read.argtypes = rows
        L.qr_attention_kv8_workspace_bytes.argtypes = [cache, i64, i64, i64, i64]
        L.qr_attention_kv8.argtypes = [cache, i32, vp, i64, i64, i64, i64, vp, vp, vp, i64, C.c_float, i64, vp, i64,
                                       vp, C.c_size_t, vp]
        L.qr_matmul_i8_ex.argtypes = [vp, vp, vp, vp, vp, C.POINTER(_I8Epilogue), i64, i64, i64, i32, vp, i64, vp]
        L.qr_norm_rows_i8.argtypes = [i32, vp, i64, vp, i64, i32, vp, C.c_double, i64, i64, vp, i64, vp, i64, vp, vp, vp]
        L.qr_moe_route_workspace_bytes.argtypes = [i64, i64, i64]
        L.qr_moe_route.argtypes = [i32, vp, i64, i32, vp, vp, i64, i64, i64, i64, i32, i32, C.c_float, vp, vp, vp,
                                   C.c_size_t, vp]
        L.qr_moe_i8_workspace_bytes.argtypes = [C.POINTER(_Moe), i64, i64]
        L.qr_moe_i8.argtypes = [C.POINTER(_Moe), vp, vp, vp, vp, i64, i64, i32, vp, i64, i32, vp, i64, vp, C.c_size_t, vp]
        for name in ("qr_i8_row_bytes", "qr_kv8_code_bytes", "qr_attention_kv8_workspace_bytes",
                     "qr_moe_route_workspace_bytes", "qr_moe_i8_workspace_bytes"):
            getattr(L, name).restype = C.c_size_t
        for name in ("qr_quantize_rows_i8", "qr_matmul_i8", "qr_kv8_append", "qr_kv8_read", "qr_attention_kv8",
                     "qr_matmul_i8_ex", "qr_norm_rows_i8", "qr_moe_route", "qr_moe_i8"):
            getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


# The checks below read each property once and build nothing: a decode step
# makes many small calls, and their time on the host counts.

# The handle of a device's current stream. The public call builds an object for
# it first: 1.9 us a call, against 0.1 us.
_current_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _device(t, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return t.device


def _on(t, name: str, device):
    """Refuses anything but a tensor in the memory of `device`: the kernels
    take raw device addresses, and another one would reach a kernel as one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.device != device:
        raise TypeError(f"{name} is on {t.device}, not on {device}")


def _dtype_id(t: torch.Tensor, name: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return d


def _call(device, stream, fn, *args):
    """fn(*args, stream) with `device` current, as a launch on its stream
    needs; stream None is torch's current one on the device."""
    if stream is None:
        handle = _current_stream(device.index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == device.index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != 0:
        _check(rc)


def _new(shape, dtype, device, stream):
    """A new tensor for a call on `stream`: from that stream's memory, so that
    neither what ran on the block before nor what gets it next overlaps the
    call."""
    if stream is None:
        if len(shape) <= 2:   # (with its strides a tensor is made faster: 1.0 us, 1.4 without)
            return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=device)
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _given(t, name: str, shape, dtype, device):
    _on(t, name, device)
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


# --------------------------------------------------------------------------
# 8-bit rows and their product (include/serve/qrow_i8.h)

I8_MAX_IN = 131072


def qr_i8_row_bytes(n_per_row: int) -> int:
    return int(load_library().qr_i8_row_bytes(n_per_row))


def qr_quantize_rows_i8(x: torch.Tensor, codes=None, scales=None, stream=None):
    """Quantizes the rows of x ([n_rows, n_per_row] fp32/bf16, elements of a
    row adjacent, rows any stride apart) to 8 bits with one scale per row:
    tokens and weight channels alike. Returns (codes int8 [n_rows,
    qr_i8_row_bytes(n_per_row)], scales fp32 [n_rows])."""
    device = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    src = _dtype_id(x, "x")
    n_rows, n = x.shape
    stride, step = x.stride()
    if n > 1 and step != 1:
        raise ValueError("the elements of a row of x must be adjacent")
    if n_rows <= 1:
        stride = n
    elif stride < n:
        raise ValueError("the rows of x must not overlap")
    # (outside 1 .. I8_MAX_IN the library refuses the call)
    row_bytes = (n + 127) // 128 * 128 if 0 < n <= I8_MAX_IN else 0
    if codes is None:
        codes = _new((n_rows, row_bytes), torch.int8, device, stream)
    else:
        _given(codes, "codes", (n_rows, row_bytes), torch.int8, device)
    if scales is None:
        scales = _new((n_rows,), torch.float32, device, stream)
    else:
        _given(scales, "scales", (n_rows,), torch.float32, device)
    _call(device, stream, load_library().qr_quantize_rows_i8, src, x.data_ptr(), n_rows, n, stride, codes.data_ptr(),
          scales.data_ptr())
    return codes, scales


def _i8_rows(codes, scales, name, row_bytes, device):
    _on(codes, name, device)
    _on(scales, name + "d", device)
    n = codes.shape[0] if codes.dim() == 2 else -1
    if codes.shape != (n, row_bytes) or codes.dtype != torch.int8 or not codes.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int8 [n, {row_bytes}] tensor (qr_i8_row_bytes of n_in)")
    if scales.shape != (n,) or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError(f"{name}d must be a contiguous float32 tensor with one scale per row of {name}")
    return n


def qr_matmul_i8(w: torch.Tensor, wd: torch.Tensor, x: torch.Tensor, xd: torch.Tensor, n_in: int, bias=None,
                 dtype=torch.bfloat16, out=None, stream=None):
    """y [n_tok, n_out] = (x * xd) @ (w * wd).T + bias for rows of 8-bit codes
    w [n_out, qr_i8_row_bytes(n_in)] and x [n_tok, ...] with their scales wd
    and xd (qr_quantize_rows_i8); bias fp32 [n_out] or None. y has `dtype`
    (float32 or bfloat16), or is `out`, whose rows may be strided."""
    device = _device(w, "w")
    if not 0 < n_in <= I8_MAX_IN:
        raise ValueError(f"n_in must be in 1..{I8_MAX_IN}")
    row_bytes = (n_in + 127) // 128 * 128
    n_out = _i8_rows(w, wd, "w", row_bytes, device)
    n_tok = _i8_rows(x, xd, "x", row_bytes, device)
    if bias is not None:
        _given(bias, "bias", (n_out,), torch.float32, device)
    if out is None:
        out = _new((n_tok, n_out), dtype, device, stream)
        stride = n_out
    else:
        _on(out, "out", device)
        if out.shape != (n_tok, n_out) or (n_out > 1 and out.stride(1) != 1):
            raise ValueError("out must be [n_tok, n_out] with adjacent elements in a row")
        stride = out.stride(0) if n_tok > 1 else n_out
        if stride < n_out:
            raise ValueError("the rows of out must not overlap")
    dst = _dtype_id(out, "out")
    _call(device, stream, load_library().qr_matmul_i8, w.data_ptr(), wd.data_ptr(), x.data_ptr(), xd.data_ptr(),
          None if bias is None else bias.data_ptr(), n_out, n_tok, n_in, dst, out.data_ptr(), stride)
    return out


def _rows(x, name, n_rows, n, device, dtype=None):
    """Stride of the rows of x [n_rows, n] (of `dtype`), the elements of a row
    adjacent, any stride between rows that do not overlap."""
    _on(x, name, device)
    if x.shape != (n_rows, n) or (dtype is not None and x.dtype != dtype):
        raise ValueError(f"{name} must be [{n_rows}, {n}]" + (f" of {dtype}" if dtype is not None else ""))
    stride, step = x.stride()
    if n > 1 and step != 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent")
    if n_rows <= 1:
        return n
    if stride < n:
        raise ValueError(f"the rows of {name} must not overlap")
    return stride


def _out_type(out, dtype):
    """(torch type, the library's number for it) of an output: that of `out`, or
    `dtype` for a new one."""
    dtype = dtype if out is None else out.dtype
    d = _DTYPES.get(dtype)
    if d is None:
        raise TypeError(f"the output must be float32 or bfloat16, got {dtype}")
    return dtype, d


def _choice(value, table, name):
    got = table.get(value)
    if got is None:
        raise ValueError(f"{name} must be one of {tuple(table)}")
    return got


def qr_matmul_i8_ex(w: torch.Tensor, wd: torch.Tensor, x: torch.Tensor, xd: torch.Tensor, n_in: int, bias=None,
                    act: str = "none", up=None, upd=None, up_bias=None, residual=None, dtype=torch.bfloat16, out=None,
                    stream=None):
    """qr_matmul_i8 with an epilogue: act((x * xd) @ (w * wd).T + bias), times
    the same product with up, upd and up_bias (a gated projection) where `up`
    is given, plus `residual` ([n_tok, n_out] of the output's type, rows any
    stride apart; it may be `out` itself). act: a key of ACTS."""
    device = _device(w, "w")
    if not 0 < n_in <= I8_MAX_IN:
        raise ValueError(f"n_in must be in 1..{I8_MAX_IN}")
    row_bytes = (n_in + 127) // 128 * 128
    n_out = _i8_rows(w, wd, "w", row_bytes, device)
    n_tok = _i8_rows(x, xd, "x", row_bytes, device)
    if bias is not None:
        _given(bias, "bias", (n_out,), torch.float32, device)
    e = _I8Epilogue(_choice(act, ACTS, "act"))
    if up is not None:
        if _i8_rows(up, upd, "up", row_bytes, device) != n_out:
            raise ValueError("up must have as many rows as w")
        e.up, e.upd = up.data_ptr(), upd.data_ptr()
        if up_bias is not None:
            _given(up_bias, "up_bias", (n_out,), torch.float32, device)
            e.up_bias = up_bias.data_ptr()
    elif upd is not None or up_bias is not None:
        raise ValueError("upd and up_bias need up")
    stride = n_out if out is None else _rows(out, "out", n_tok, n_out, device)
    dtype, dst = _out_type(out, dtype)
    if residual is not None:
        e.residual_stride = _rows(residual, "residual", n_tok, n_out, device, dtype)
        e.residual = residual.data_ptr()
    if out is None:
        out = _new((n_tok, n_out), dtype, device, stream)
    _call(device, stream, load_library().qr_matmul_i8_ex, w.data_ptr(), wd.data_ptr(), x.data_ptr(), xd.data_ptr(),
          None if bias is None else bias.data_ptr(), C.byref(e), n_out, n_tok, n_in, dst, out.data_ptr(), stride)
    return out


# --------------------------------------------------------------------------
# the norm that makes 8-bit rows (include/serve/qrow_norm.h)

def qr_norm_rows_i8(x: torch.Tensor, weight=None, eps: float = 1e-6, residual=None, total=None, y=None, codes=None,
                    scales=None, stream=None):
    """Root-mean-square norm of the rows of x ([n_rows, n] fp32/bf16, rows any
    stride apart), after `residual` (same type and shape) has been added, into
    8-bit rows as qr_quantize_rows_i8 makes them. weight: fp32/bf16 [n] or None
    for ones.

    Returns (codes, scales, total, y): total holds x + residual (None without a
    residual; given, it may be x or residual itself), y the normed rows in the
    type of x (None unless y is True or a tensor to be filled)."""
    device = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    src = _dtype_id(x, "x")
    n_rows, n = x.shape
    xs = _rows(x, "x", n_rows, n, device)
    wtype = src
    if weight is not None:
        _on(weight, "weight", device)
        wtype = _dtype_id(weight, "weight")
        if weight.shape != (n,) or (n > 1 and weight.stride(0) != 1):
            raise ValueError(f"weight must be a contiguous tensor of shape ({n},)")
    rs = ts = ys = 0
    if residual is not None:
        rs = _rows(residual, "residual", n_rows, n, device, x.dtype)
        ts = n if total is None else _rows(total, "total", n_rows, n, device, x.dtype)
    elif total is not None:
        raise ValueError("total needs a residual")
    if y is not None and y is not True and y is not False:
        ys = _rows(y, "y", n_rows, n, device, x.dtype)
    # (outside 1 .. I8_MAX_IN the library refuses the call)
    row_bytes = (n + 127) // 128 * 128 if 0 < n <= I8_MAX_IN else 0
    if codes is not None:
        _given(codes, "codes", (n_rows, row_bytes), torch.int8, device)
    if scales is not None:
        _given(scales, "scales", (n_rows,), torch.float32, device)
    if codes is None:
        codes = _new((n_rows, row_bytes), torch.int8, device, stream)
    if scales is None:
        scales = _new((n_rows,), torch.float32, device, stream)
    if residual is not None and total is None:
        total = _new((n_rows, n), x.dtype, device, stream)
    if y is True:
        y, ys = _new((n_rows, n), x.dtype, device, stream), n
    elif y is False:
        y = None
    _call(device, stream, load_library().qr_norm_rows_i8, src, x.data_ptr(), xs,
          None if residual is None else residual.data_ptr(), rs, wtype, None if weight is None else weight.data_ptr(),
          eps, n_rows, n, None if total is None else total.data_ptr(), ts, None if y is None else y.data_ptr(), ys,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales, total, y


# --------------------------------------------------------------------------
# a mixture of experts (include/serve/qrow_moe.h)

def _scratch(workspace, need, device, stream):
    """(pointer, bytes) of the caller's workspace, or of a new one; and the
    tensor, which has to live until the call is made."""
    if workspace is not None:
        _on(workspace, "workspace", device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if not need:
        return None, 0, None
    workspace = _new((need,), torch.uint8, device, stream)
    return workspace.data_ptr(), need, workspace


def qr_moe_route_workspace_bytes(n_experts: int, n_tok: int, n_in: int) -> int:
    return int(load_library().qr_moe_route_workspace_bytes(n_experts, n_tok, n_in))


def qr_moe_route(x: torch.Tensor, w: torch.Tensor, top_k: int, score: str = "softmax", bias=None, renorm: bool = True,
                 factor: float = 1.0, ids=None, weights=None, workspace=None, stream=None):
    """The top_k experts of every row of x ([n_tok, n_in] fp32/bf16, rows any
    stride apart) by the router rows w ([n_experts, n_in] fp32/bf16) and their
    weights: (ids int32 [n_tok, top_k], weights fp32 [n_tok, top_k]), in new
    tensors or in those given. score: a key of SCORES; bias fp32 [n_experts] or
    None takes part in the choice alone (-inf: never chosen; ids are -1 where
    no expert is left). workspace: a CUDA tensor of at least
    qr_moe_route_workspace_bytes bytes, or None to have one allocated here."""
    device = _device(x, "x")
    _on(w, "w", device)
    if x.dim() != 2 or w.dim() != 2 or not w.is_contiguous():
        raise ValueError("x must be [n_tok, n_in], w a contiguous [n_experts, n_in]")
    src, wtype = _dtype_id(x, "x"), _dtype_id(w, "w")
    n_tok, n_in = x.shape
    n_experts = w.shape[0]
    if w.shape[1] != n_in:
        raise ValueError("x and w must have rows of one length")
    xs = _rows(x, "x", n_tok, n_in, device)
    if bias is not None:
        _given(bias, "bias", (n_experts,), torch.float32, device)
    if not 0 < top_k <= MOE_MAX_TOP_K:
        raise ValueError(f"top_k must be in 1..{MOE_MAX_TOP_K}")
    shape = (n_tok, top_k)
    score = _choice(score, SCORES, "score")
    if ids is not None:
        _given(ids, "ids", shape, torch.int32, device)
    if weights is not None:
        _given(weights, "weights", shape, torch.float32, device)
    lib = load_library()
    need = 0 if workspace is not None else lib.qr_moe_route_workspace_bytes(n_experts, n_tok, n_in)
    ws, ws_bytes, workspace = _scratch(workspace, need, device, stream)
    if ids is None:
        ids = _new(shape, torch.int32, device, stream)
    if weights is None:
        weights = _new(shape, torch.float32, device, stream)
    _call(device, stream, lib.qr_moe_route, src, x.data_ptr(), xs, wtype, w.data_ptr(),
          None if bias is None else bias.data_ptr(), n_experts, n_tok, n_in, top_k, score, bool(renorm),
          factor, ids.data_ptr(), weights.data_ptr(), ws, ws_bytes)
    return ids, weights


class MoeExperts:
    """The experts' 8-bit weights (qr_quantize_rows_i8 of their rows), checked
    once here; the tensors must not be resized afterwards.

    gate, up      int8 [n_experts, n_mid, qr_i8_row_bytes(n_in)], each contiguous
                  or both halves of one [n_experts, 2 * n_mid, ...] tensor
    gated, upd    fp32 [n_experts, n_mid], likewise
    down, downd   int8 [n_experts, n_in, qr_i8_row_bytes(n_mid)], fp32 [n_experts, n_in]
    """

    __slots__ = ("gate", "gated", "up", "upd", "down", "downd", "n_experts", "n_in", "n_mid", "device", "_c")

    def __init__(self, gate, gated, up, upd, down, downd, n_in: int, n_mid: int):
        device = _device(gate, "gate")
        for t, name in ((gated, "gated"), (up, "up"), (upd, "upd"), (down, "down"), (downd, "downd")):
            _on(t, name, device)
        if not (0 < n_in <= I8_MAX_IN and 0 < n_mid <= I8_MAX_IN):
            raise ValueError(f"n_in and n_mid must be in 1..{I8_MAX_IN}")
        n = gate.shape[0] if gate.dim() == 3 else 0
        if not 0 < n <= MOE_MAX_EXPERTS:
            raise ValueError(f"gate must be [n_experts, n_mid, row bytes] of 1..{MOE_MAX_EXPERTS} experts")
        in_bytes, mid_bytes = (n_in + 127) // 128 * 128, (n_mid + 127) // 128 * 128
        rows = gate.stride(0) // in_bytes if n > 1 else n_mid
        for t, s, name in ((gate, gated, "gate"), (up, upd, "up")):
            if (t.shape != (n, n_mid, in_bytes) or t.dtype != torch.int8 or s.shape != (n, n_mid)
                    or s.dtype != torch.float32 or t.stride(2) != 1 or (n_mid > 1 and t.stride(1) != in_bytes)
                    or (n_mid > 1 and s.stride(1) != 1) or rows < n_mid
                    or (n > 1 and (t.stride(0) != rows * in_bytes or s.stride(0) != rows))):
                raise ValueError(f"{name} must be int8 [n_experts, n_mid, {in_bytes}] with float32 scales [n_experts, "
                                 "n_mid], rows adjacent, experts as far apart in gate, up and their scales")
        if (down.shape != (n, n_in, mid_bytes) or down.dtype != torch.int8 or downd.shape != (n, n_in)
                or downd.dtype != torch.float32 or not down.is_contiguous() or not downd.is_contiguous()):
            raise ValueError(f"down must be a contiguous int8 [n_experts, n_in, {mid_bytes}] with float32 scales "
                             "[n_experts, n_in]")
        self.gate, self.gated, self.up, self.upd, self.down, self.downd = gate, gated, up, upd, down, downd
        self.n_experts, self.n_in, self.n_mid, self.device = n, n_in, n_mid, device
        self._c = _Moe(gate.data_ptr(), up.data_ptr(), down.data_ptr(), gated.data_ptr(), upd.data_ptr(),
                       downd.data_ptr(), n, n_in, n_mid, rows)


def _experts(experts, device):
    if not isinstance(experts, MoeExperts):
        raise TypeError("experts must be MoeExperts")
    if experts.device != device:
        raise TypeError(f"the experts are on {experts.device}, not on {device}")
    return experts._c


def qr_moe_i8_workspace_bytes(experts: MoeExperts, n_tok: int, top_k: int) -> int:
    return int(load_library().qr_moe_i8_workspace_bytes(C.byref(_experts(experts, experts.device)), n_tok, top_k))


def qr_moe_i8(x: torch.Tensor, xd: torch.Tensor, experts: MoeExperts, ids: torch.Tensor, weights: torch.Tensor,
              act: str = "silu", residual=None, dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """The experts of a few tokens: y [n_tok, n_in] = sum over a token's slots of
    weights * down(act(gate(x)) * up(x)), plus `residual` ([n_tok, n_in] of the
    output's type, rows any stride apart; it may be `out` itself). x and xd:
    8-bit rows [n_tok, qr_i8_row_bytes(n_in)] and their scales; ids int32 and
    weights fp32 [n_tok, top_k] as qr_moe_route gives them (an id outside
    0..n_experts-1 is no expert). y has `dtype` (float32 or bfloat16), or is
    `out`, whose rows may be strided. workspace: a CUDA tensor of at least
    qr_moe_i8_workspace_bytes bytes, or None to have one allocated here."""
    device = _device(x, "x")
    c = _experts(experts, device)
    n_in = experts.n_in
    n_tok = _i8_rows(x, xd, "x", (n_in + 127) // 128 * 128, device)
    _on(ids, "ids", device)
    if ids.dim() != 2 or ids.shape[0] != n_tok or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 [n_tok, top_k] tensor")
    top_k = ids.shape[1]
    _given(weights, "weights", ids.shape, torch.float32, device)
    stride = n_in if out is None else _rows(out, "out", n_tok, n_in, device)
    dtype, dst = _out_type(out, dtype)
    res, rs = None, 0
    if residual is not None:
        rs = _rows(residual, "residual", n_tok, n_in, device, dtype)
        res = residual.data_ptr()
    act = _choice(act, ACTS, "act")
    lib = load_library()
    need = 0 if workspace is not None else lib.qr_moe_i8_workspace_bytes(C.byref(c), n_tok, top_k)
    ws, ws_bytes, workspace = _scratch(workspace, need, device, stream)
    if out is None:
        out = _new((n_tok, n_in), dtype, device, stream)
    _call(device, stream, lib.qr_moe_i8, C.byref(c), x.data_ptr(), xd.data_ptr(), ids.data_ptr(), weights.data_ptr(),
          n_tok, top_k, act, res, rs, dst, out.data_ptr(), stride, ws, ws_bytes)
    return out


# --------------------------------------------------------------------------
# the paged 8-bit cache and attention over it (include/serve/qrow_kv8.h)

class Kv8Cache:
    """The arrays of a paged 8-bit cache (layouts in qrow_kv8.h), checked once
    here; they must not be resized afterwards.

    k   int8 [n_blocks, n_heads, block_tokens, head_dim]
    v   int8 [n_blocks, n_heads, block_tokens/32, head_dim/2, 4, 2, 8]
    kd, vd  fp32 [n_blocks, n_heads]
    """

    __slots__ = ("k", "v", "kd", "vd", "n_blocks", "n_heads", "head_dim", "block_tokens", "device", "_c")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, kd: torch.Tensor, vd: torch.Tensor):
        device = _device(k, "k")
        for t, name in ((v, "v"), (kd, "kd"), (vd, "vd")):
            _on(t, name, device)
        if k.dim() != 4:
            raise ValueError("k must be [n_blocks, n_heads, block_tokens, head_dim]")
        nb, h, bt, d = k.shape
        if d not in HEAD_DIMS or bt not in BLOCK_TOKENS:
            raise ValueError(f"head_dim must be one of {HEAD_DIMS}, block_tokens one of {BLOCK_TOKENS}")
        if (k.dtype != torch.int8 or v.dtype != torch.int8 or kd.dtype != torch.float32 or vd.dtype != torch.float32
                or v.shape != (nb, h, bt // 32, d // 2, 4, 2, 8) or kd.shape != (nb, h) or vd.shape != (nb, h)
                or not all(t.is_contiguous() for t in (k, v, kd, vd))):
            raise ValueError("the cache's tensors must have the types and shapes that kv8_cache gives them")
        self.k, self.v, self.kd, self.vd = k, v, kd, vd
        self.n_blocks, self.n_heads, self.block_tokens, self.head_dim, self.device = nb, h, bt, d, device
        self._c = _Kv8(k.data_ptr(), v.data_ptr(), kd.data_ptr(), vd.data_ptr(), nb, h, d, bt)

    def __iter__(self):
        return iter((self.k, self.v, self.kd, self.vd))


def kv8_cache(n_blocks: int, n_heads: int, head_dim: int, block_tokens: int, device) -> Kv8Cache:
    """A cache of n_blocks blocks (its contents need no clearing: what a
    sequence's blocks hold is set when their tokens are appended)."""
    if head_dim not in HEAD_DIMS or block_tokens not in BLOCK_TOKENS:
        raise ValueError(f"head_dim must be one of {HEAD_DIMS}, block_tokens one of {BLOCK_TOKENS}")
    empty = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=device)
    return Kv8Cache(empty((n_blocks, n_heads, block_tokens, head_dim), torch.int8),
                    empty((n_blocks, n_heads, block_tokens // 32, head_dim // 2, 4, 2, 8), torch.int8),
                    empty((n_blocks, n_heads), torch.float32), empty((n_blocks, n_heads), torch.float32))


def _cache(cache, device):
    if not isinstance(cache, Kv8Cache):
        raise TypeError("cache must be a Kv8Cache")
    if cache.device != device:
        raise TypeError(f"the cache is on {cache.device}, not on {device}")
    return cache._c


def _batch(cu, kv_len, table, device):
    _on(cu, "cu", device)
    _on(kv_len, "kv_len", device)
    _on(table, "table", device)
    if kv_len.dim() != 1 or table.dim() != 2:
        raise ValueError("kv_len must be [n_seq], table [n_seq, table_width]")
    n_seq, width = table.shape
    if (cu.shape != (n_seq + 1,) or kv_len.shape[0] != n_seq
            or not (cu.dtype == kv_len.dtype == table.dtype == torch.int32)
            or not (cu.is_contiguous() and kv_len.is_contiguous() and table.is_contiguous())):
        raise ValueError("cu, kv_len and table must be contiguous int32 tensors [n_seq + 1], [n_seq] and "
                         "[n_seq, table_width]")
    return n_seq, width


def _heads(x, name, n_tok, n_heads, head_dim, device):
    """Stride of the tokens of x [n_tok, n_heads, head_dim], the heads of a
    token adjacent."""
    _on(x, name, device)
    if x.shape != (n_tok, n_heads, head_dim):
        raise ValueError(f"{name} must be [{n_tok}, {n_heads}, {head_dim}]")
    stride, head_step, step = x.stride()
    if step != 1 or (n_heads > 1 and head_step != head_dim):
        raise ValueError(f"the heads of a token of {name} must be adjacent")
    if n_tok <= 1:
        return n_heads * head_dim
    if stride % 8 or stride < n_heads * head_dim:
        raise ValueError(f"the tokens of {name} must be a multiple of 8 elements apart and not overlap")
    return stride


def qr_kv8_append(cache: Kv8Cache, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor,
                  table: torch.Tensor, stream=None) -> Kv8Cache:
    """Writes the keys and values k and v ([n_tok, n_heads, head_dim]
    fp32/bf16, tokens any multiple of 8 elements apart) into the cache, in
    place: rows cu[s] .. cu[s+1]-1 are the last tokens of sequence s, which
    holds kv_len[s] tokens with them, in the blocks table[s]."""
    device = _device(k, "k")
    c = _cache(cache, device)
    n_seq, width = _batch(cu, kv_len, table, device)
    src = _dtype_id(k, "k")
    n_tok = k.shape[0] if k.dim() else 0
    ks = _heads(k, "k", n_tok, cache.n_heads, cache.head_dim, device)
    vs = _heads(v, "v", n_tok, cache.n_heads, cache.head_dim, device)
    if v.dtype != k.dtype:
        raise ValueError("k and v must have one type")
    _call(device, stream, load_library().qr_kv8_append, C.byref(c), src, k.data_ptr(), v.data_ptr(), ks, vs, n_tok,
          n_seq, cu.data_ptr(), kv_len.data_ptr(), table.data_ptr(), width)
    return cache


def qr_kv8_read(cache: Kv8Cache, cu: torch.Tensor, kv_len: torch.Tensor, table: torch.Tensor, n_tok: int,
                dtype=torch.float32, k=None, v=None, stream=None):
    """The values that the cache holds for the rows that cu, kv_len and table
    describe (as in qr_kv8_append): (k, v), each [n_tok, n_heads, head_dim] of
    `dtype`, or written into the tensors given. n_tok is the number of rows
    (at least cu[n_seq]; rows from there on are left as they were)."""
    device = _device(cu, "cu")
    c = _cache(cache, device)
    n_seq, width = _batch(cu, kv_len, table, device)
    shape = (n_tok, cache.n_heads, cache.head_dim)
    if k is None:
        k = _new(shape, dtype, device, stream)
    if v is None:
        v = _new(shape, dtype, device, stream)
    ks = _heads(k, "k", *shape, device)
    vs = _heads(v, "v", *shape, device)
    dst = _dtype_id(k, "k")
    if v.dtype != k.dtype:
        raise ValueError("k and v must have one type")
    _call(device, stream, load_library().qr_kv8_read, C.byref(c), dst, k.data_ptr(), v.data_ptr(), ks, vs, n_tok, n_seq,
          cu.data_ptr(), kv_len.data_ptr(), table.data_ptr(), width)
    return k, v


def qr_attention_kv8_workspace_bytes(cache: Kv8Cache, n_q_heads: int, n_tok: int, n_seq: int,
                                     table_width: int) -> int:
    return int(load_library().qr_attention_kv8_workspace_bytes(C.byref(_cache(cache, cache.device)), n_q_heads, n_tok, n_seq, table_width))


def qr_attention_kv8(q: torch.Tensor, cache: Kv8Cache, cu: torch.Tensor, kv_len: torch.Tensor, table: torch.Tensor,
                     scale=None, window: int = 0, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Causal attention of the rows q ([n_tok, n_q_heads, head_dim] fp32/bf16)
    over their sequences' cached tokens; cu, kv_len and table as in
    qr_kv8_append, scale 1/sqrt(head_dim) by default, window 0 or the number
    of last tokens that a row sees. workspace: a CUDA uint8 tensor of at least
    qr_attention_kv8_workspace_bytes bytes, or None to have one allocated
    here. out must not overlap q. Rows from cu[n_seq] on are left as they were
    in `out` (undefined in a new one)."""
    device = _device(q, "q")
    c = _cache(cache, device)
    n_seq, width = _batch(cu, kv_len, table, device)
    src = _dtype_id(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [n_tok, n_q_heads, head_dim]")
    n_tok, n_q, dim = q.shape
    qs = _heads(q, "q", n_tok, n_q, cache.head_dim, device)
    if out is None:
        out = _new((n_tok, n_q, dim), q.dtype, device, stream)
        os_ = n_q * dim
    else:
        os_ = _heads(out, "out", n_tok, n_q, dim, device)
        if out.dtype != q.dtype:
            raise ValueError("out must have the type of q")
    lib = load_library()
    ws, ws_bytes = None, 0
    if workspace is not None:
        _on(workspace, "workspace", device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        ws_bytes = lib.qr_attention_kv8_workspace_bytes(C.byref(c), n_q, n_tok, n_seq, width)
        if ws_bytes:
            workspace = _new((ws_bytes,), torch.uint8, device, stream)
            ws = workspace.data_ptr()
    _call(device, stream, lib.qr_attention_kv8, C.byref(c), src, q.data_ptr(), qs, n_q, n_tok, n_seq, cu.data_ptr(),
          kv_len.data_ptr(), table.data_ptr(), width, dim ** -0.5 if scale is None else scale, window, out.data_ptr(),
          os_, ws, ws_bytes)
    return out
