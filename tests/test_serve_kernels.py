"""The kernels that the built library holds are those that a call reaches."""
import re
import shutil
import subprocess

import pytest

from post_weight_quantization_row_amd import _build, qrow


@pytest.mark.skipif(shutil.which("nm") is None, reason="no nm")
def test_choices_from_rough_logits():
    """They are taken from more than 64 + 7 top_k experts: never by the kernel for
    64 experts and fewer."""
    qrow.load_library()
    names = subprocess.run(["nm", _build.LIB], check=True, capture_output=True, text=True).stdout
    slots = lambda kernel: sorted(map(int, re.findall(rf"__device_stub__{kernel}ILi(\d+)E", names)))
    assert slots("k_route_choose") == [1, 4, 8, 16] and slots("k_route_settle") == [4, 8, 16]
