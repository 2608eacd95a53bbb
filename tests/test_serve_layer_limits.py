"""The limits that the headers of the 8-bit layer's operators state, on the CPU:
the largest call is taken (it gets as far as the absent device), the next one is
refused."""
import ctypes as C

import pytest
import torch

from post_weight_quantization_row_amd import serve
from test_serve_limits import QR_EDEVICE, QR_EOVERFLOW, header

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="made-up addresses: only where no GPU can reach them")
P = C.c_void_p
FAR = 1 << 44                    # bytes between operands: more than the largest of them has


@pytest.mark.parametrize("src", [0, 1])
@pytest.mark.parametrize("n,rows,rc", [
    (64, 2 ** 24 - 1, QR_EDEVICE), (64, 2 ** 24, QR_EOVERFLOW), (513, 2 ** 24 - 1, QR_EDEVICE), (4097, 2 ** 24 - 1, QR_EDEVICE),
    (8192, 2 ** 24 - 1, QR_EDEVICE), (8192, 2 ** 24, QR_EOVERFLOW), (8193, 2 ** 22 - 1, QR_EDEVICE), (8193, 2 ** 22, QR_EOVERFLOW),
    (8200, 2 ** 24 - 1, QR_EOVERFLOW), (131072, 2 ** 22 - 1, QR_EDEVICE), (131072, 2 ** 22, QR_EOVERFLOW)])
def test_norm(n, rows, rc, src):
    assert "n_rows < 2^24, and < 2^22 where n > 8192" in header("qrow_norm.h")
    f = serve.load_library().qr_norm_rows_i8
    a = [P(i * FAR) for i in range(1, 8)]
    assert f(src, a[0], n, a[1], n, 1, a[2], 1e-6, rows, n, a[3], n, a[4], n, a[5], a[6], None) == rc
    assert f(src, a[0], n, None, 0, 1, None, 1e-6, rows, n, None, 0, None, 0, a[5], a[6], None) == rc


@pytest.mark.parametrize("n_out,n_tok,rc", [
    (2 ** 30 - 129, 17, QR_EDEVICE), (2 ** 30 - 128, 17, QR_EOVERFLOW), (16 * (2 ** 23 - 1), 1, QR_EDEVICE),
    (16 * (2 ** 23 - 1) + 1, 1, QR_EOVERFLOW), (16 * (2 ** 23 - 1), 16, QR_EDEVICE), (16 * (2 ** 23 - 1) + 1, 16, QR_EOVERFLOW),
    (128 * 4095, 256 * 4097, QR_EDEVICE), (128 * 4096, 256 * 4096, QR_EOVERFLOW), (17, 2 ** 31 - 257, QR_EDEVICE),
    (17, 2 ** 31 - 256, QR_EOVERFLOW)])
def test_gated_product(n_out, n_tok, rc):
    """Tiles of 256 weight rows hold 128 channels of a gate; few tokens go by
    channels, with a gate as without one."""
    assert "Limits: those of qr_matmul_i8, with up and more than 16 tokens those for 2 * n_out" in header("qrow_i8.h")
    e = serve._I8Epilogue(2, FAR, FAR, None, None, 0)
    f = serve.load_library().qr_matmul_i8_ex
    a = [P(i * FAR) for i in range(1, 6)]
    assert f(a[0], a[1], a[2], a[3], None, C.byref(e), n_out, n_tok, 64, 0, a[4], n_out, None) == rc


@pytest.mark.parametrize("src", [0, 1])
@pytest.mark.parametrize("experts,n_in,top_k", [(1, 1, 1), (16, 64, 2), (64, 100, 64), (1024, 40, 64), (1024, 2000, 1), (300, 131072, 8)])
def test_route(experts, n_in, top_k, src):
    assert "n_tok < 2^22" in header("qrow_moe.h")
    lib = serve.load_library()
    a = [P(i * FAR) for i in range(1, 6)]
    for n_tok, rc in ((2 ** 22 - 1, QR_EDEVICE), (2 ** 22, QR_EOVERFLOW)):
        need = lib.qr_moe_route_workspace_bytes(experts, n_tok, n_in)
        assert (need > 0) == (rc == QR_EDEVICE)
        for score in (0, 1):
            assert lib.qr_moe_route(src, a[0], n_in, src, a[1], None, experts, n_tok, n_in, top_k, score, 1, 1.0, a[2], a[3], a[4],
                                    need, None) == rc


@pytest.mark.parametrize("n_tok,top_k,rc", [(8192, 1, QR_EDEVICE), (8193, 1, QR_EOVERFLOW), (128, 64, QR_EDEVICE), (129, 64, QR_EOVERFLOW),
                                            (2730, 3, QR_EDEVICE), (2731, 3, QR_EOVERFLOW)])
@pytest.mark.parametrize("experts,n_in,n_mid", [(1, 1, 1), (1024, 131072, 131072), (256, 7168, 2048)])
def test_experts(experts, n_in, n_mid, n_tok, top_k, rc):
    assert "n_tok * top_k <= QR_MOE_MAX_PAIRS" in header("qrow_moe.h")
    lib = serve.load_library()
    m = serve._Moe(*[20 * FAR] * 6, experts, n_in, n_mid, n_mid)
    a = [P(i * FAR) for i in range(1, 8)]
    need = lib.qr_moe_i8_workspace_bytes(C.byref(m), n_tok, top_k)
    assert lib.qr_moe_i8(C.byref(m), a[0], a[1], a[2], a[3], n_tok, top_k, 2, a[4], n_in, 0, a[5], n_in, a[6], need, None) == rc
