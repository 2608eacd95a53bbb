"""qr_norm_rows_i8's checks on the CPU, built with traps on signed overflow:
strides that no 64-bit number of bytes holds are refused without one."""
import ctypes as C
import os
import shutil
import signal
import subprocess

import pytest
import torch

from post_weight_quantization_row_amd import _build

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
pytestmark = [pytest.mark.skipif(shutil.which(HIPCC) is None, reason="no hipcc"),
              pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no GPU can reach them")]
# what the checks call; a launch is none here
STUBS = """
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>
void qr_clear_error() {}
int qr_fail(int code, const char*, ...) { return code; }
int qr_check_launch(const char*) { return -5; }
extern "C" size_t qr_i8_row_bytes(int64_t n) { return (size_t)((n + 127) / 128 * 128); }
"""


def call_in_child(f):
    """What f returns, in 0..255, or the signal that ended it."""
    pid = os.fork()
    if pid == 0:
        signal.signal(signal.SIGILL, signal.SIG_DFL)
        os._exit(f() & 0xff)
    status = os.waitpid(pid, 0)[1]
    return os.WEXITSTATUS(status) if os.WIFEXITED(status) else -os.WTERMSIG(status)


def test_no_stride_overflows(tmp_path):
    src = tmp_path / "stubs.hip"
    src.write_text(STUBS)
    lib = str(tmp_path / "norm.so")
    trap = ["-Xarch_host", "-fsanitize=signed-integer-overflow", "-Xarch_host", "-fsanitize-trap=signed-integer-overflow"]
    flags = [f for f in _build.HIPCC_FLAGS if f != "-O3"] + ["-O1"]
    subprocess.run([HIPCC, *flags, *trap, "-shared", "-I", _build.INCLUDE, "-o", lib, str(src),
                    os.path.join(_build.HERE, "csrc", "serve_norm.hip")], check=True, capture_output=True)
    i64, vp = C.c_int64, C.c_void_p
    f = C.CDLL(lib).qr_norm_rows_i8
    f.argtypes = [C.c_int, vp, i64, vp, i64, C.c_int, vp, C.c_double, i64, i64, vp, i64, vp, i64, vp, vp, vp]
    a = [vp(i << 44) for i in range(1, 8)]
    call = lambda src, rows, s: f(src, a[0], s[0], a[1], s[1], 1, a[2], 1e-6, rows, 64, a[3], s[2], a[4], s[3], a[5], a[6], None)
    for which in range(4):
        for src in (0, 1):
            for stride, rows, want in ((2 ** 63 - 1, 1, -4), (2 ** 62, 4, -4), (2 ** 61, 1, -4), (2 ** 40, 4, -5), (-2 ** 63, 4, -2)):
                s = [64] * 4
                s[which] = stride
                got = call_in_child(lambda: call(src, rows, s))
                assert got == (want & 0xff), (which, src, stride, rows, got)
