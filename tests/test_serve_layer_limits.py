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
