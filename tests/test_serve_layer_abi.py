"""The C-ABI of the 8-bit layer's operators (norm, product with epilogue,
router, experts) on the CPU: sizes are right, and bad arguments are refused
before anything touches the GPU (no compute calls here)."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from post_weight_quantization_row_amd import serve
from post_weight_quantization_row_amd.qrow import qr_last_error
from test_abi import _DeviceStandIn
from test_serve_abi import FAKE, ROOT

P = C.c_void_p
NAN, INF = float("nan"), float("inf")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no GPU can reach them")
DEVICE = -5                      # a call that nothing is wrong with gets as far as the (absent) device


@pytest.fixture(scope="module")
def lib():
    return serve.load_library()


def test_headers_compile_as_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "qrow.h"\n#include "serve/qrow_i8.h"\n#include "serve/qrow_norm.h"\n'
                   '#include "serve/qrow_moe.h"\n'
                   "int main(void) { return sizeof(qr_i8_epilogue) != 48 || sizeof(qr_moe) != 80 || QR_ACT_GELU_TANH != 4\n"
                   "  || QR_SCORE_SIGMOID != 1 || QR_MOE_MAX_EXPERTS != 1024 || QR_MOE_MAX_TOP_K != 64\n"
                   "  || QR_MOE_MAX_PAIRS != 8192; }\n")
    exe = str(tmp_path / "h")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", exe, str(src)],
                   check=True)
    assert subprocess.run([exe]).returncode == 0
    assert C.sizeof(serve._I8Epilogue) == 48 and C.sizeof(serve._Moe) == 80
    assert (serve.MOE_MAX_EXPERTS, serve.MOE_MAX_TOP_K, serve.MOE_MAX_PAIRS) == (1024, 64, 8192)


# --------------------------------------------------------------------------
# the norm

def norm_call(lib, src=1, x=0x100000, xs=64, r=0x200000, rs=64, wt=1, w=0x300000, eps=1e-6, rows=4, n=64, s=0x400000,
              ss=64, y=0x500000, ys=64, c=0x600000, d=0x700000):
    return lib.qr_norm_rows_i8(src, P(x), xs, P(r), rs, wt, P(w), eps, rows, n, P(s), ss, P(y), ys, P(c), P(d), None)


def test_norm_refusals(lib):
    call = lambda **kw: norm_call(lib, **kw)
    assert call(src=2) == -1 and call(wt=2) == -1 and call(src=-1) == -1
    assert call(n=0) == -2 and call(n=131073, xs=2 ** 18, rs=2 ** 18, ss=2 ** 18, ys=2 ** 18) == -2
    for eps in (-1e-9, NAN, INF):
        assert call(eps=eps) == -2
    assert call(rows=-1) == -2
    for s in ("xs", "rs", "ss", "ys"):
        assert call(**{s: 63}) == -2 and call(**{s: 2 ** 62}) == -4
    assert call(rows=2 ** 24) == -4
    assert call(rows=0, x=None, r=None, s=None, y=None, c=None, d=None) == 0
    assert call(r=None) == -3 and call(s=None) == -3 and "both" in qr_last_error()
    for a in ("x", "c", "d"):
        assert call(**{a: None}) == -3
    for a in "xrswy":
        assert call(**{a: 0x900001}) == -3
    assert call(c=0x900008) == -3 and call(d=0x900002) == -3
    assert call(src=0, x=0x900002) == -3 and call(wt=0, w=0x900002) == -3


@no_gpu
def test_norm_overlaps(lib):
    call = lambda **kw: norm_call(lib, **kw)
    assert call() == DEVICE and call(r=None, s=None, y=None, w=None) == DEVICE
    # in place
    for kw in (dict(s=0x100000), dict(s=0x200000), dict(y=0x100000), dict(y=0x200000), dict(s=0x200000, y=0x100000)):
        assert call(**kw) == DEVICE, kw
    # outputs over each other, or over an input but not in its place (rows of 128 bytes)
    for kw in (dict(y=0x400000), dict(s=0x100000, y=0x100000), dict(s=0x100080), dict(s=0x100000, ss=72), dict(y=0x200010),
               dict(y=0x1fffa0), dict(s=0x300000), dict(y=0x300000 - 128), dict(c=0x100000), dict(c=0x4001f0), dict(d=0x5001f0),
               dict(c=0x300040), dict(d=0x300040), dict(d=0x6001f0), dict(d=0x200000)):
        assert call(**kw) == -3 and "overlap" in qr_last_error(), kw
    # a single row's stride does not matter; neighbours do not overlap
    assert call(rows=1, s=0x100000, ss=999) == DEVICE
    assert call(s=0x100200, y=0x100400, c=0x100600, d=0x100800) == DEVICE
    # columns of one buffer, rows apart
    assert call(xs=256, rs=256, ss=256, ys=256, r=0x100080, s=0x100100, y=0x100180) == DEVICE
    assert call(xs=256, rs=256, ss=256, ys=256, r=0x100080, s=0x1000fe, y=0x100180) == -3


@no_gpu
def test_a_range_between_rows(lib):
    """codes (4 rows of 128 bytes) and scales against rows that lie apart: by brute force."""
    for row_step in (128, 160, 1024, 4096):
        for at in range(-544, 5 * row_step, 16):
            c = 0x100000 + at
            met = any(0x100000 + i * row_step < c + 512 and c < 0x100000 + i * row_step + 128 for i in range(4))
            rc = norm_call(lib, xs=row_step // 2, c=c)
            assert rc == (-3 if met else DEVICE), (row_step, at)


# --------------------------------------------------------------------------
# the product with an epilogue

def ex_call(lib, e=None, w=FAKE, wd=FAKE, x=FAKE, xd=FAKE, bias=None, n_out=8, n_tok=4, n_in=64, dst=0, y=FAKE, ys=8, **kw):
    if e is None:
        d = dict(act=2, up=0x10000, upd=0x10000, up_bias=None, residual=None, residual_stride=0)
        d.update(kw)
        e = serve._I8Epilogue(*[d[n] for n, _ in serve._I8Epilogue._fields_])
    return lib.qr_matmul_i8_ex(w, wd, x, xd, bias, C.byref(e), n_out, n_tok, n_in, dst, y, ys, None)


def test_product_refusals(lib):
    call = lambda **kw: ex_call(lib, **kw)
    assert call(dst=2) == -1 and call(act=5) == -1 and call(act=-1) == -1
    assert call(n_in=0) == -2 and call(n_in=131073) == -2
    assert call(n_out=-1) == -2 and call(n_tok=-1) == -2 and call(ys=7) == -2
    assert call(residual=0x90000, residual_stride=7) == -2
    assert call(n_out=0, w=None) == 0 and call(n_tok=0, x=None, y=None) == 0
    assert call(n_out=2 ** 30, ys=2 ** 30) == -4 and call(n_tok=2 ** 31) == -4
    assert call(residual=0x90000, residual_stride=2 ** 62) == -4
    for name in ("w", "wd", "x", "xd", "y"):
        assert call(**{name: None}) == -3
    assert call(upd=None) == -3 and call(up=0x10008) == -3 and call(upd=0x10001) == -3 and call(up_bias=0x10002) == -3
    assert call(residual=0x90001, residual_stride=8) == -3
    assert lib.qr_matmul_i8_ex(FAKE, FAKE, FAKE, FAKE, None, None, 8, 4, 0, 0, FAKE, 8, None) == -2


@no_gpu
def test_product_overlaps(lib):
    y = 0x1000000
    call = lambda r, rs, ys=8, n_tok=4: ex_call(lib, y=P(y), ys=ys, residual=y + r, residual_stride=rs, n_tok=n_tok)
    assert call(0, 8) == DEVICE and call(0, 99, n_tok=1) == DEVICE and call(4 * 32, 8) == DEVICE
    assert call(32, 16, 16) == DEVICE                       # side by side
    for r, rs, ys in ((0, 9, 8), (4, 8, 8), (-4, 8, 8), (32, 8, 8), (28, 16, 16), (96, 8, 8)):
        assert call(r, rs, ys) == -3 and "overlap" in qr_last_error(), (r, rs, ys)
    # a call whose epilogue holds nothing, and one without
    assert ex_call(lib, act=0, up=None) == DEVICE
    assert lib.qr_matmul_i8_ex(FAKE, FAKE, FAKE, FAKE, None, None, 8, 4, 64, 0, P(y), 8, None) == DEVICE


# --------------------------------------------------------------------------
# the router

def route_call(lib, src=0, x=FAKE, xs=64, wt=0, w=FAKE, bias=None, e=16, t=4, n=64, k=2, score=0, renorm=1, factor=1.0,
               ids=FAKE, weights=FAKE, ws=FAKE, wb=1 << 30):
    return lib.qr_moe_route(src, x, xs, wt, w, bias, e, t, n, k, score, renorm, factor, ids, weights, ws, wb, None)


def test_route_refusals(lib):
    call = lambda **kw: route_call(lib, **kw)
    assert call(src=2) == -1 and call(wt=-1) == -1 and call(score=2) == -1
    assert call(e=0) == -2 and call(e=1025) == -2 and call(n=0) == -2 and call(n=131073, xs=2 ** 18) == -2
    assert call(k=0) == -2 and call(k=17) == -2 and call(e=1000, k=65) == -2
    assert call(t=-1) == -2 and call(xs=63) == -2 and call(factor=NAN) == -2 and call(factor=INF) == -2
    assert call(t=0, x=None, ws=None, wb=0) == 0
    assert call(t=2 ** 22) == -4 and call(xs=2 ** 62) == -4
    for a in ("x", "w", "ids", "weights", "ws"):
        assert call(**{a: None}) == -3
        assert call(**{a: P(0x10001)}) == -3
    assert call(bias=P(0x10002)) == -3 and call(ws=P(0x10080)) == -3
    need = lib.qr_moe_route_workspace_bytes(16, 4, 64)
    assert need >= 16 * 4 * 8 and call(wb=need - 1) == -2
    for args in ((0, 4, 64), (1025, 4, 64), (16, -1, 64), (16, 2 ** 22, 64), (16, 4, 0), (16, 4, 131073), (16, 0, 64)):
        assert lib.qr_moe_route_workspace_bytes(*args) == 0


# --------------------------------------------------------------------------
# the experts

def moe(**kw):
    d = dict(gate=0x10000, up=0x10000, down=0x10000, gated=0x10000, upd=0x10000, downd=0x10000, n_experts=8, n_in=64,
             n_mid=100, expert_rows=100)
    d.update(kw)
    return serve._Moe(*[d[n] for n, _ in serve._Moe._fields_])


def moe_call(lib, m=None, x=0x1000000, xd=0x2000000, ids=0x3000000, weights=0x4000000, t=4, k=2, act=2, r=None, rs=64,
             dst=0, y=0x5000000, ys=64, ws=0x6000000, wb=1 << 30):
    return lib.qr_moe_i8(C.byref(m or moe()), P(x), P(xd), P(ids), P(weights), t, k, act, P(r), rs, dst, P(y), ys, P(ws),
                         wb, None)


BAD = [dict(n_experts=0), dict(n_experts=1025), dict(n_in=0), dict(n_in=131073), dict(n_mid=0), dict(n_mid=131073),
       dict(expert_rows=99), dict(expert_rows=2 ** 62)]


def test_experts_refusals(lib):
    call = lambda **kw: moe_call(lib, **kw)
    assert lib.qr_moe_i8(None, FAKE, FAKE, FAKE, FAKE, 4, 2, 2, None, 0, 0, FAKE, 64, FAKE, 1 << 30, None) == -2
    for bad in BAD:
        assert call(m=moe(**bad)) == -2
        assert lib.qr_moe_i8_workspace_bytes(C.byref(moe(**bad)), 4, 2) == 0
    assert lib.qr_moe_i8_workspace_bytes(None, 4, 2) == 0
    assert call(dst=2) == -1 and call(act=5) == -1 and call(act=-1) == -1
    assert call(k=0) == -2 and call(k=65) == -2 and call(t=-1) == -2 and call(ys=63) == -2 and call(r=0x7000000, rs=63) == -2
    assert call(t=0, x=None, y=None, ws=None) == 0
    assert call(t=4097) == -4 and call(ys=2 ** 62) == -4 and call(r=0x7000000, rs=2 ** 62) == -4
    for a in ("x", "xd", "ids", "weights", "y", "ws"):
        assert call(**{a: None}) == -3
        assert call(**{a: 0x7000001}) == -3
    for a in ("gate", "up", "down", "gated", "upd", "downd"):
        assert call(m=moe(**{a: None})) == -3
        assert call(m=moe(**{a: 0x10001})) == -3
    assert call(x=0x7000008) == -3 and call(ws=0x7000080) == -3 and call(r=0x7000001) == -3
    # two blocks of 64 codes and a row of four scales a pair
    need = lib.qr_moe_i8_workspace_bytes(C.byref(moe()), 4, 2)
    assert need >= 8 * 2 * (64 + 4) and call(wb=need - 1) == -2
    for t, k in ((4, 0), (4, 65), (-1, 2), (4097, 2), (0, 2)):
        assert lib.qr_moe_i8_workspace_bytes(C.byref(moe()), t, k) == 0


@no_gpu
def test_experts_overlaps(lib):
    call = lambda **kw: moe_call(lib, **kw)
    y = 0x5000000
    assert call() == DEVICE and call(t=4096) == DEVICE
    assert call(r=y) == DEVICE and call(r=y, rs=99, t=1) == DEVICE and call(r=y + 256, rs=128, ys=128) == DEVICE
    for kw in (dict(r=y, rs=72), dict(r=y + 4), dict(r=y - 256), dict(x=y), dict(x=y - 496), dict(xd=y + 1020), dict(ids=y + 16),
               dict(weights=y - 28), dict(ws=y), dict(ws=y + 768)):
        assert call(**kw) == -3 and "overlap" in qr_last_error(), kw
    # between the rows of y
    assert call(ys=256, xd=y + 256, ids=y + 512, weights=y + 1024 + 256) == DEVICE


@no_gpu
def test_experts_workspace_overlaps(lib):
    """Choices that change under the call would part the waves of a workgroup."""
    m, ws = moe(), 0x7000000
    need = lib.qr_moe_i8_workspace_bytes(C.byref(m), 4, 2)
    call = lambda **kw: moe_call(lib, ws=ws, **kw)
    assert call() == DEVICE and call(ids=ws + need, weights=ws - 32, x=ws - 512 - 32, r=ws + need + 32) == DEVICE
    for kw in (dict(ids=ws + need - 4), dict(ids=ws - 28), dict(weights=ws), dict(x=ws - 496), dict(xd=ws + 4), dict(r=ws + need - 4),
               dict(r=ws - 1020)):
        assert call(**kw) == -3 and "workspace must not overlap" in qr_last_error(), kw


# --------------------------------------------------------------------------
# the binding

class _NoCompute:
    """Stands in for the loaded library: a call that would launch work fails
    the test."""

    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self._real, name)
        raise AssertionError(f"{name} was called with a bad argument")


def test_binding_refuses_wrong_tensors(lib, monkeypatch):
    monkeypatch.setattr(serve, "_lib", _NoCompute(lib))
    dev, host = _DeviceStandIn.make, torch.zeros
    z = lambda *s, dt=torch.float32: dev(torch.zeros(s, dtype=dt))
    i32 = lambda *s: z(*s, dt=torch.int32)
    i8 = lambda *s: z(*s, dt=torch.int8)
    x, w = i8(4, 128), i8(8, 128)
    ex = lambda *a, **kw: serve.qr_matmul_i8_ex(w, z(8), x, z(4), 100, *a, **kw)
    rows, router = z(4, 64), z(16, 64)
    parts = lambda **kw: {**dict(gate=i8(3, 70, 128), gated=z(3, 70), up=i8(3, 70, 128), upd=z(3, 70),
                                 down=i8(3, 100, 128), downd=z(3, 100), n_in=100, n_mid=70), **kw}
    layer = serve.MoeExperts(**parts())
    both = host((3, 140, 128), dtype=torch.int8), host(3, 140)
    first, last = [dev(t[:, :70]) for t in both], [dev(t[:, 70:]) for t in both]
    halves = serve.MoeExperts(**parts(gate=first[0], up=last[0], gated=first[1], upd=last[1]))
    assert layer._c.expert_rows == 70 and halves._c.expert_rows == 140
    assert halves._c.up - halves._c.gate == 70 * 128 and halves._c.upd - halves._c.gated == 280
    mo = lambda *a, **kw: serve.qr_moe_i8(x, z(4), layer, *(a or (i32(4, 2), z(4, 2))), **kw)
    types = [
        lambda: serve.qr_norm_rows_i8(host(4, 64)),
        lambda: serve.qr_norm_rows_i8(z(4, 64, dt=torch.float16)),
        lambda: serve.qr_norm_rows_i8(rows, host(64)),
        lambda: serve.qr_norm_rows_i8(rows, z(64, dt=torch.float16)),
        lambda: serve.qr_norm_rows_i8(rows, residual=host(4, 64)),
        lambda: serve.qr_norm_rows_i8(rows, residual=rows, total=host(4, 64)),
        lambda: serve.qr_norm_rows_i8(rows, y=host(4, 64)),
        lambda: serve.qr_norm_rows_i8(rows, codes=host((4, 128), dtype=torch.int8)),
        lambda: ex(up=host((8, 128), dtype=torch.int8), upd=z(8)),
        lambda: ex(up=w, upd=host(8)),
        lambda: ex(up=w, upd=None),
        lambda: ex(residual=host(4, 8)),
        lambda: ex(out=host(4, 8)),
        lambda: ex(bias=host(8)),
        lambda: serve.qr_moe_route(host(4, 64), router, 2),
        lambda: serve.qr_moe_route(rows, host(16, 64), 2),
        lambda: serve.qr_moe_route(rows, z(16, 64, dt=torch.float16), 2),
        lambda: serve.qr_moe_route(rows, router, 2, bias=host(16)),
        lambda: serve.qr_moe_route(rows, router, 2, ids=host((4, 2), dtype=torch.int32)),
        lambda: serve.qr_moe_route(rows, router, 2, workspace=host(1 << 16, dtype=torch.uint8)),
        lambda: serve.MoeExperts(**parts(gate=host((3, 70, 128), dtype=torch.int8))),
        lambda: serve.MoeExperts(**parts(downd=host(3, 100))),
        lambda: serve.qr_moe_i8(x, z(4), tuple(parts().values()), i32(4, 2), z(4, 2)),
        lambda: serve.qr_moe_i8(x, host(4), layer, i32(4, 2), z(4, 2)),
        lambda: mo(host((4, 2), dtype=torch.int32), z(4, 2)),
        lambda: mo(i32(4, 2), host(4, 2)),
        lambda: mo(residual=host(4, 100)),
        lambda: mo(out=host(4, 100)),
        lambda: mo(dtype=torch.float16),
        lambda: mo(workspace=host(1 << 16, dtype=torch.uint8)),
    ]
    for i, f in enumerate(types):
        with pytest.raises(TypeError):
            f()
            raise AssertionError(i)
    values = [
        lambda: serve.qr_norm_rows_i8(z(64)),
        lambda: serve.qr_norm_rows_i8(dev(host(64, 4).t())),
        lambda: serve.qr_norm_rows_i8(dev(host(1, 64).expand(4, 64))),
        lambda: serve.qr_norm_rows_i8(rows, z(63)),
        lambda: serve.qr_norm_rows_i8(rows, dev(host(128)[::2])),
        lambda: serve.qr_norm_rows_i8(rows, residual=z(4, 63)),
        lambda: serve.qr_norm_rows_i8(rows, residual=z(4, 64, dt=torch.bfloat16)),
        lambda: serve.qr_norm_rows_i8(rows, residual=rows, total=z(3, 64)),
        lambda: serve.qr_norm_rows_i8(rows, total=rows),
        lambda: serve.qr_norm_rows_i8(rows, y=z(4, 64, dt=torch.bfloat16)),
        lambda: serve.qr_norm_rows_i8(rows, y=dev(host(1, 64).expand(4, 64))),
        lambda: serve.qr_norm_rows_i8(rows, codes=i8(4, 64)),
        lambda: serve.qr_norm_rows_i8(rows, scales=z(5)),
        lambda: ex(act="swish"),
        lambda: ex(up=i8(7, 128), upd=z(7)),
        lambda: ex(up=i8(8, 64), upd=z(8)),
        lambda: ex(upd=z(8)),
        lambda: ex(up_bias=z(8)),
        lambda: ex(up=w, upd=z(8), up_bias=z(7)),
        lambda: ex(residual=z(4, 7)),
        lambda: ex(residual=z(4, 8)),                        # bf16 out, fp32 residual
        lambda: ex(out=z(4, 7)),
        lambda: ex(out=dev(host(8, 4).t())),
        lambda: ex(out=z(4, 8), residual=dev(host(1, 8).expand(4, 8))),
        lambda: serve.qr_matmul_i8_ex(w, z(8), x, z(4), 0),
        lambda: serve.qr_moe_route(z(64), router, 2),
        lambda: serve.qr_moe_route(rows, z(16, 63), 2),
        lambda: serve.qr_moe_route(rows, dev(host(64, 16).t()), 2),
        lambda: serve.qr_moe_route(rows, router, 0),
        lambda: serve.qr_moe_route(rows, router, 65),
        lambda: serve.qr_moe_route(rows, router, 2, score="tanh"),
        lambda: serve.qr_moe_route(rows, router, 2, bias=z(15)),
        lambda: serve.qr_moe_route(rows, router, 2, ids=i32(4, 3)),
        lambda: serve.qr_moe_route(rows, router, 2, weights=z(4, 2, dt=torch.float64)),
        lambda: serve.qr_moe_route(rows, router, 2, workspace=dev(torch.zeros(1 << 17, dtype=torch.uint8)[::2])),
        lambda: serve.MoeExperts(**parts(n_in=0)),
        lambda: serve.MoeExperts(**parts(n_in=200)),
        lambda: serve.MoeExperts(**parts(n_mid=71)),
        lambda: serve.MoeExperts(**parts(up=i8(3, 70, 256))),
        lambda: serve.MoeExperts(**parts(up=last[0])),   # gate by itself
        lambda: serve.MoeExperts(**parts(gated=first[1])),
        lambda: serve.MoeExperts(**parts(gated=z(3, 70, dt=torch.float64))),
        lambda: serve.MoeExperts(**parts(gate=i8(70, 128))),
        lambda: serve.MoeExperts(**parts(down=dev(host((3, 128, 100), dtype=torch.int8).transpose(1, 2)))),
        lambda: serve.MoeExperts(**parts(gate=i8(1025, 1, 128))),
        lambda: serve.qr_moe_i8(i8(4, 256), z(4), layer, i32(4, 2), z(4, 2)),
        lambda: serve.qr_moe_i8(x, z(3), layer, i32(4, 2), z(4, 2)),
        lambda: mo(i32(3, 2), z(3, 2)),
        lambda: mo(z(4, 2, dt=torch.int64), z(4, 2)),
        lambda: mo(i32(4, 2), z(4, 3)),
        lambda: mo(residual=z(4, 100)),
        lambda: mo(out=z(4, 99)),
        lambda: mo(act="swish"),
    ]
    for i, f in enumerate(values):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
