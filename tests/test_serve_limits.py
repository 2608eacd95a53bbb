"""The limits that the serving headers state, on the CPU: the largest call is
taken (it gets as far as the absent device), the next one is refused."""
import ctypes as C
import os
import re

import pytest
import torch

from post_weight_quantization_row_amd import serve
from test_serve_abi import FAKE, cache

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="made-up addresses: only where no GPU can reach them")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
QR_EOVERFLOW, QR_EDEVICE = -4, -5
FAR = C.c_void_p(1 << 60)        # so far from FAKE that the largest output cannot overlap


def header(name):
    return re.sub(r"\s*\n \*\s*", " ", open(os.path.join(ROOT, "include", "serve", name)).read())


@pytest.mark.parametrize("n_out,n_tok,rc", [
    (16 * (2 ** 23 - 1), 1, QR_EDEVICE), (16 * (2 ** 23 - 1) + 1, 1, QR_EOVERFLOW),
    (16 * (2 ** 23 - 1), 16, QR_EDEVICE), (16 * (2 ** 23 - 1) + 1, 16, QR_EOVERFLOW),
    (256 * 4095, 256 * 4097, QR_EDEVICE), (256 * 4096, 256 * 4096, QR_EOVERFLOW),
    (17, 2 ** 31 - 257, QR_EDEVICE), (17, 2 ** 31 - 256, QR_EOVERFLOW), (2 ** 31 - 257, 17, QR_EDEVICE)])
def test_product(n_out, n_tok, rc):
    text = header("qrow_i8.h")
    assert "n_out, n_tok < 2^31 - 256" in text and "ceil(n_out / 256) * ceil(n_tok / 256) < 2^24" in text
    assert "n_out <= 16 * (2^23 - 1)" in text
    f = serve.load_library().qr_matmul_i8
    assert f(FAKE, FAKE, FAKE, FAKE, None, n_out, n_tok, 64, 0, FAKE, n_out, None) == rc


@pytest.mark.parametrize("name", ["qr_kv8_append", "qr_kv8_read"])
@pytest.mark.parametrize("heads,block,n_tok,n_seq,rc", [
    (1024, 128, 128 * 16381, 1, QR_EDEVICE), (1024, 128, 128 * 16382, 1, QR_EOVERFLOW),
    (1024, 32, 1, 8191, QR_EDEVICE), (1024, 32, 1, 8192, QR_EOVERFLOW),
    (1, 32, 32 * (2 ** 24 - 3), 1, QR_EDEVICE), (1, 32, 32 * (2 ** 24 - 2), 1, QR_EOVERFLOW)])
def test_append_and_read(name, heads, block, n_tok, n_seq, rc):
    assert "(n_tok / block_tokens + 2 * n_seq) * n_heads < 2^24" in header("qrow_kv8.h")
    f = getattr(serve.load_library(), name)
    c = cache(n_heads=heads, block_tokens=block)
    assert f(C.byref(c), 0, FAKE, FAR, 64 * heads, 64 * heads, n_tok, n_seq, FAKE, FAKE, FAKE, 1, None) == rc


@pytest.mark.parametrize("heads,group,n_tok,n_seq,rc", [
    (1024, 1, 8192, 8192, QR_EDEVICE), (1024, 1, 16384, 16384, QR_EOVERFLOW),
    (1024, 1, 128 * 16382, 1, QR_EDEVICE), (1024, 1, 128 * 16383, 1, QR_EOVERFLOW)])
def test_attention(heads, group, n_tok, n_seq, rc):
    text = header("qrow_kv8.h")
    assert "(n_tok * g / 128 + n_seq) * n_heads < 2^24" in text and "16 in place of 128" in text
    f = serve.load_library().qr_attention_kv8
    stride = 64 * heads * group
    assert f(C.byref(cache(n_heads=heads)), 0, FAKE, stride, heads * group, n_tok, n_seq, FAKE, FAKE, FAKE, 1, 0.1, 0,
             FAR, stride, None, 0, None) == rc
