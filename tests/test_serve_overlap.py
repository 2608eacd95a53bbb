"""Tensors of the serving calls that must not share memory, on the CPU: what
overlaps is refused, what only lies side by side in one buffer is not."""
import ctypes as C

import pytest
import torch

from post_weight_quantization_row_amd import serve
from post_weight_quantization_row_amd.qrow import qr_last_error
from test_serve_abi import FAKE, cache

BASE = 0x10000000                # never dereferenced
QR_EINVAL_PTR, QR_EDEVICE = -3, -5


def overlap(n, row, a, a_stride, b, b_stride):
    """By brute force over the rows, in elements."""
    seen = set()
    for t in range(n):
        seen.update(range(a + t * a_stride, a + t * a_stride + row, 8))
    return any(i in seen for t in range(n) for i in range(b + t * b_stride, b + t * b_stride + row, 8))


def check(call, n, row, a_stride, b_stride, distance, esize):
    """b lies `distance` elements behind a."""
    rc = call(C.c_void_p(BASE), C.c_void_p(BASE + distance * esize), n, a_stride, b_stride)
    want = overlap(n, row, 0, a_stride, distance, b_stride)
    if want:
        assert rc == QR_EINVAL_PTR and "overlap" in qr_last_error()
    else:                        # nothing else is wrong with the call: it gets as far as the (absent) device
        assert rc == QR_EDEVICE
    return want


CASES = [(n, sa, sb, at) for n in (1, 2, 3, 7) for sa, sb in ((256, 256), (512, 512), (768, 768), (512, 768), (768, 264))
         for at in (0, 8, 248, 256, 264, 504, 512, 520, 1024, 1280, 1536, 3 * 768 + 248, 3 * 768 + 256, 6 * 768 + 256,
                    -8, -248, -256, -264, -512, -768 + 248, -768 - 256, -2 * 768 - 8, -6 * 768 - 256)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no GPU can reach them")
@pytest.mark.parametrize("src,esize", [(0, 4), (1, 2)])
def test_attention_refuses_an_output_over_its_queries(src, esize):
    f = serve.load_library().qr_attention_kv8

    def call(q, out, n, qs, os_):
        return f(C.byref(cache()), src, q, qs, 4, n, 2, FAKE, FAKE, FAKE, 3, 0.1, 0, out, os_, None, 0, None)

    met = [check(call, n, 256, sa, sb, at, esize) for n, sa, sb, at in CASES]
    assert any(met) and not all(met)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no GPU can reach them")
@pytest.mark.parametrize("dst,esize", [(0, 4), (1, 2)])
def test_read_refuses_keys_over_values(dst, esize):
    L = serve.load_library()

    def call(f, k, v, n, ks, vs):
        return f(C.byref(cache(n_heads=4)), dst, k, v, ks, vs, n, 2, FAKE, FAKE, FAKE, 3, None)

    met = [check(lambda *a: call(L.qr_kv8_read, *a), n, 256, sa, sb, at, esize) for n, sa, sb, at in CASES]
    assert any(met) and not all(met)
    # what is only read may be shared
    assert call(L.qr_kv8_append, C.c_void_p(BASE), C.c_void_p(BASE), 3, 256, 256) == QR_EDEVICE
