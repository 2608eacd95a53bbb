"""The serving headers' C-ABI on the CPU: every declared symbol is exported,
sizes are right, and bad arguments are refused before anything touches the
GPU (no compute calls here)."""
import ctypes as C
import glob
import os
import re

import pytest
import torch

from post_weight_quantization_row_amd import serve
from post_weight_quantization_row_amd.qrow import QrowError, qr_last_error
from test_abi import _DeviceStandIn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = C.c_void_p(0x10000)       # never dereferenced: calls fail first


@pytest.fixture(scope="module")
def lib():
    return serve.load_library()


def test_library_exports_every_declared_serving_function(lib):
    names = set()
    for h in glob.glob(os.path.join(ROOT, "include", "serve", "*.h")):
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names |= set(re.findall(r"\b(qr_[a-z0-9_]+)\s*\(", text))
    assert names == set(serve.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_headers_compile_as_c(tmp_path):
    import subprocess
    src = tmp_path / "h.c"
    src.write_text('#include "qrow.h"\n#include "serve/qrow_i8.h"\n#include "serve/qrow_kv8.h"\n'
                   "int main(void) { return (int)sizeof(qr_kv8) != 64; }\n")
    exe = str(tmp_path / "h")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", exe, str(src)],
                   check=True)
    assert subprocess.run([exe]).returncode == 0
    assert C.sizeof(serve._Kv8) == 64


def test_row_bytes(lib):
    assert [lib.qr_i8_row_bytes(n) for n in (1, 127, 128, 129, 131072)] == [128, 128, 128, 256, 131072]
    assert [lib.qr_i8_row_bytes(n) for n in (0, -1, 131073)] == [0, 0, 0]


def test_quantize_rows_i8_refusals(lib):
    f = lib.qr_quantize_rows_i8
    assert f(2, FAKE, 4, 64, 64, FAKE, FAKE, None) == -1
    assert f(0, FAKE, 4, 0, 64, FAKE, FAKE, None) == -2
    assert f(0, FAKE, 4, 131073, 131073, FAKE, FAKE, None) == -2
    assert f(0, FAKE, -1, 64, 64, FAKE, FAKE, None) == -2
    assert f(0, FAKE, 4, 64, 63, FAKE, FAKE, None) == -2
    assert f(0, None, 0, 64, 64, None, None, None) == 0
    assert f(0, FAKE, 2 ** 24, 64, 64, FAKE, FAKE, None) == -4
    assert f(0, FAKE, 2 ** 20, 64, 2 ** 60, FAKE, FAKE, None) == -4
    for bad in [(None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (C.c_void_p(0x10002), FAKE, FAKE),
                (FAKE, C.c_void_p(0x10008), FAKE), (FAKE, FAKE, C.c_void_p(0x10002))]:
        assert f(0, bad[0], 4, 64, 64, bad[1], bad[2], None) == -3


def test_matmul_i8_refusals(lib):
    f = lib.qr_matmul_i8

    def call(w=FAKE, wd=FAKE, x=FAKE, xd=FAKE, bias=None, n_out=8, n_tok=4, n_in=64, dst=0, y=FAKE, ys=8):
        return f(w, wd, x, xd, bias, n_out, n_tok, n_in, dst, y, ys, None)

    assert call(dst=2) == -1
    assert call(n_in=0) == -2 and call(n_in=131073) == -2
    assert call(n_out=-1) == -2 and call(n_tok=-1) == -2 and call(ys=7) == -2
    assert call(n_out=0, w=None) == 0 and call(n_tok=0, x=None, y=None) == 0
    assert call(n_out=2 ** 31, ys=2 ** 31) == -4 and call(n_tok=2 ** 31) == -4
    assert call(n_tok=2 ** 20, ys=2 ** 60) == -4
    assert call(n_out=2 ** 30, n_tok=2 ** 30, ys=2 ** 30) == -4
    for name in ("w", "wd", "x", "xd", "y"):
        assert call(**{name: None}) == -3
        assert call(**{name: C.c_void_p(0x10001)}) == -3
    assert call(bias=C.c_void_p(0x10002)) == -3
    assert call(w=C.c_void_p(0x10008)) == -3 and call(x=C.c_void_p(0x10008)) == -3


def cache(**kw):
    d = dict(k=0x10000, v=0x10000, kd=0x10000, vd=0x10000, n_blocks=8, n_heads=2, head_dim=64, block_tokens=32)
    d.update(kw)
    return serve._Kv8(*[d[n] for n, _ in serve._Kv8._fields_])


BAD_CACHES = [dict(n_blocks=-1), dict(n_blocks=2 ** 31), dict(n_heads=0), dict(n_heads=1025), dict(head_dim=96),
              dict(head_dim=0), dict(block_tokens=16), dict(block_tokens=48), dict(block_tokens=256)]


def test_code_bytes(lib):
    assert lib.qr_kv8_code_bytes(C.byref(cache())) == 8 * 2 * 32 * 64
    assert lib.qr_kv8_code_bytes(C.byref(cache(k=None, n_blocks=2 ** 31 - 1, n_heads=1024, head_dim=256,
                                               block_tokens=128))) == (2 ** 31 - 1) * 1024 * 256 * 128
    for bad in BAD_CACHES:
        assert lib.qr_kv8_code_bytes(C.byref(cache(**bad))) == 0
    assert lib.qr_kv8_code_bytes(None) == 0


@pytest.mark.parametrize("name", ["qr_kv8_append", "qr_kv8_read"])
def test_append_and_read_refusals(lib, name):
    f = getattr(lib, name)

    def call(c=None, dt=0, k=FAKE, v=FAKE, ks=128, vs=128, n_tok=4, n_seq=2, cu=FAKE, ln=FAKE, tab=FAKE, w=3):
        return f(C.byref(c or cache()), dt, k, v, ks, vs, n_tok, n_seq, cu, ln, tab, w, None)

    assert f(None, 0, FAKE, FAKE, 128, 128, 4, 2, FAKE, FAKE, FAKE, 3, None) == -2
    for bad in BAD_CACHES:
        assert call(c=cache(**bad)) == -2
    assert call(dt=2) == -1
    assert call(ks=120) == -2 and call(vs=132) == -2
    assert call(n_tok=-1) == -2 and call(n_seq=-1) == -2 and call(w=-1) == -2
    assert call(n_tok=0, k=None) == 0 and call(n_seq=0, cu=None) == 0
    assert call(n_tok=2 ** 31) == -4 and call(n_seq=2 ** 31 - 1) == -4 and call(w=2 ** 31) == -4
    assert call(n_seq=2 ** 30) == -4 and call(ks=2 ** 62) == -4
    for a in ("k", "v", "cu", "ln", "tab"):
        assert call(**{a: None}) == -3
    for a in ("k", "v"):
        assert call(**{a: C.c_void_p(0x10008)}) == -3
    for a in ("cu", "ln", "tab"):
        assert call(**{a: C.c_void_p(0x10002)}) == -3
    for a in ("k", "v", "kd", "vd"):
        assert call(c=cache(**{a: None})) == -3
        assert call(c=cache(**{a: 0x10001})) == -3
    assert "scales" in qr_last_error()


def test_attention_refusals(lib):
    f = lib.qr_attention_kv8

    def call(c=None, src=1, q=FAKE, qs=256, nq=4, n_tok=4, n_seq=2, cu=FAKE, ln=FAKE, tab=FAKE, w=3, scale=0.1,
             window=0, out=FAKE, os_=256, ws=None, wb=0):
        return f(C.byref(c or cache()), src, q, qs, nq, n_tok, n_seq, cu, ln, tab, w, scale, window, out, os_, ws, wb,
                 None)

    for bad in BAD_CACHES:
        assert call(c=cache(**bad)) == -2
    assert call(src=3) == -1
    assert call(nq=3) == -2 and call(nq=0) == -2 and call(nq=2 * 1025, qs=2 ** 20, os_=2 ** 20) == -2
    assert call(scale=float("nan")) == -2 and call(scale=float("inf")) == -2 and call(window=-1) == -2
    assert call(qs=252) == -2 and call(os_=248) == -2
    assert call(n_tok=-1) == -2 and call(n_seq=-1) == -2 and call(w=-1) == -2
    assert call(n_tok=0, q=None) == 0 and call(n_seq=0, cu=None) == 0
    assert call(n_tok=2 ** 30) == -4 and call(n_seq=2 ** 31 - 1) == -4
    for a in ("q", "out", "cu", "ln", "tab"):
        assert call(**{a: None}) == -3
    assert call(q=C.c_void_p(0x10008)) == -3 and call(cu=C.c_void_p(0x10001)) == -3
    # a call that splits its tokens needs its workspace, whole and aligned
    need = lib.qr_attention_kv8_workspace_bytes(C.byref(cache()), 4, 4, 2, 1024)
    assert need > 0
    big = dict(w=1024)
    assert call(**big) == -3 and call(ws=C.c_void_p(0x10080), wb=need, **big) == -3
    assert call(ws=FAKE, wb=need - 1, **big) == -2
    assert lib.qr_attention_kv8_workspace_bytes(C.byref(cache()), 4, 4, 2, 1) == 0
    for args in ((3, 4, 2, 1024), (4, 0, 2, 1024), (4, 4, 0, 1024), (4, 4, 2, -1), (4, 2 ** 31, 2, 4)):
        assert lib.qr_attention_kv8_workspace_bytes(C.byref(cache()), *args) == 0


class _NoCompute:
    """Stands in for the loaded library: a call that would launch work fails
    the test."""

    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        if name in ("qr_i8_row_bytes", "qr_kv8_code_bytes", "qr_attention_kv8_workspace_bytes"):
            return getattr(self._real, name)
        raise AssertionError(f"{name} was called with a bad argument")


def test_binding_refuses_wrong_tensors(lib, monkeypatch):
    monkeypatch.setattr(serve, "_lib", _NoCompute(lib))
    dev = _DeviceStandIn.make
    z = lambda *s, dt=torch.float32: dev(torch.zeros(s, dtype=dt))
    i32 = lambda *s: z(*s, dt=torch.int32)
    i8 = lambda *s: z(*s, dt=torch.int8)
    host = torch.zeros
    x, w = i8(4, 128), i8(8, 128)
    kv = serve.Kv8Cache(i8(8, 2, 32, 64), i8(8, 2, 1, 32, 4, 2, 8), z(8, 2), z(8, 2))
    cu, ln, tab = i32(3), i32(2), i32(2, 3)
    rows, q = z(4, 2, 64), z(4, 4, 64)
    tab_long = i32(2, 1024)
    types = [
        lambda: serve.qr_quantize_rows_i8(host(4, 64)),
        lambda: serve.qr_quantize_rows_i8(z(4, 64, dt=torch.float16)),
        lambda: serve.qr_quantize_rows_i8(z(4, 64), codes=host((4, 128), dtype=torch.int8)),
        lambda: serve.qr_matmul_i8(w, host(8), x, z(4), 100),
        lambda: serve.qr_matmul_i8(w, z(8), x, z(4), 100, bias=host(8)),
        lambda: serve.qr_matmul_i8(w, z(8), x, z(4), 100, out=host(4, 8)),
        lambda: serve.qr_matmul_i8(w, z(8), x, z(4), 100, out=z(4, 8, dt=torch.float16)),
        lambda: serve.qr_kv8_append(kv, rows, host(4, 2, 64), cu, ln, tab),
        lambda: serve.qr_kv8_append(kv, rows, rows, host(3, dtype=torch.int32), ln, tab),
        lambda: serve.qr_kv8_append(serve.Kv8Cache(kv.k, kv.v, kv.kd, host(8, 2)), rows, rows, cu, ln, tab),
        lambda: serve.qr_kv8_read(kv, cu, ln, tab, 4, k=host(4, 2, 64), v=rows),
        lambda: serve.qr_attention_kv8(q, kv, cu, ln, host((2, 3), dtype=torch.int32)),
        lambda: serve.qr_attention_kv8(q, tuple(kv), cu, ln, tab),
        lambda: serve.qr_attention_kv8(q, kv, cu, ln, tab, out=host(4, 4, 64)),
        lambda: serve.qr_attention_kv8(q, kv, cu, ln, tab_long, out=q, workspace=host(1 << 20, dtype=torch.uint8)),
    ]
    for f in types:
        with pytest.raises(TypeError):
            f()
    values = [
        lambda: serve.qr_quantize_rows_i8(z(64)),
        lambda: serve.qr_quantize_rows_i8(dev(host(64, 4).t())),
        lambda: serve.qr_quantize_rows_i8(dev(host(1, 64).expand(4, 64))),
        lambda: serve.qr_quantize_rows_i8(z(4, 64), codes=x, scales=z(3)),
        lambda: serve.qr_matmul_i8(w, z(8), x, z(4), 200),
        lambda: serve.qr_matmul_i8(w, z(7), x, z(4), 100),
        lambda: serve.qr_matmul_i8(z(8, 128), z(8), x, z(4), 100),
        lambda: serve.qr_matmul_i8(w, z(8), x, z(4), 100, bias=z(7)),
        lambda: serve.qr_matmul_i8(w, z(8), x, z(4), 100, out=z(4, 7)),
        lambda: serve.qr_matmul_i8(w, z(8), x, z(4), 100, out=dev(host(8, 4).t())),
        lambda: serve.kv8_cache(4, 2, 96, 32, "cpu"),
        lambda: serve.kv8_cache(4, 2, 64, 16, "cpu"),
        lambda: serve.qr_kv8_append(serve.Kv8Cache(kv.k, i8(8, 2, 32, 64), kv.kd, kv.vd), rows, rows, cu, ln, tab),
        lambda: serve.qr_kv8_append(kv, rows, rows, cu, ln, i32(3, 3)),
        lambda: serve.qr_kv8_append(kv, rows, rows, i32(2), ln, tab),
        lambda: serve.qr_kv8_append(kv, rows, rows, cu, ln, z(2, 3, dt=torch.int64)),
        lambda: serve.qr_kv8_append(kv, rows, z(5, 2, 64), cu, ln, tab),
        lambda: serve.qr_kv8_append(kv, z(4, 3, 64), rows, cu, ln, tab),
        lambda: serve.qr_kv8_append(kv, dev(host(4, 64, 2).transpose(1, 2)), rows, cu, ln, tab),
        lambda: serve.qr_kv8_append(kv, dev(host(4, 132)[:, :128].view(4, 2, 64)), rows, cu, ln, tab),
        lambda: serve.qr_kv8_read(kv, cu, ln, tab, 4, k=z(3, 2, 64), v=z(3, 2, 64)),
        lambda: serve.qr_attention_kv8(z(4, 4, 128), kv, cu, ln, tab),
        lambda: serve.qr_attention_kv8(q, kv, cu, ln, tab, out=z(4, 2, 64)),
    ]
    for f in values:
        with pytest.raises(ValueError):
            f()


def test_errors_carry_the_librarys_message(lib):
    with pytest.raises(QrowError, match="n_in"):
        from post_weight_quantization_row_amd.qrow import _check
        _check(lib.qr_matmul_i8(FAKE, FAKE, FAKE, FAKE, None, 8, 4, 0, 0, FAKE, 8, None))
