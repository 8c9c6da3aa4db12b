"""Calls of the 4-bit operators at the ends of what they accept, without a
GPU (as tests/test_mx_distill_host.py: fake addresses, EHIP where every check
passes)."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_mx_distill_host import B, EHIP, EINVAL, EOVERFLOW, F16, F32, ROOT, mx


@pytest.mark.parametrize("body", ["empty_workspace", "many_rows", "gradient_parts"])
def test_limits(body):
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", CUDA_VISIBLE_DEVICES="",
               ROCR_VISIBLE_DEVICES="")
    here = os.path.dirname(os.path.abspath(__file__))
    code = (f"import sys; sys.path[:0] = [{ROOT!r}, {here!r}]; import test_mx_limits_host as t; "
            f"from zero_partitioned_mixed_layout_amd import zero_shard as zs; "
            f"t.{body}(zs); print('BODY_OK')")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "BODY_OK" in r.stdout, r.stdout + r.stderr


def empty_workspace(zs):
    """A workspace of 0 bytes overlaps nothing, wherever its pointer points."""
    L = zs.lib()
    x, y = 5 * B, 7 * B

    def grad(ws, wb):
        return L.zero_mxfp4_linear_grad_input(x, F16, 5, 48, ctypes.byref(mx(zs, 48, 96)), y, F32,
                                              96, ws, wb, None)

    for at in (x + 8, y + 8, B + 64, B + (1 << 36) + 4, 9 * B):
        assert grad(at, 0) == EHIP, hex(at)
    assert grad(x + 8, 4) == EINVAL and grad(x + 2, 0) == EINVAL and grad(9 * B, 64) == EHIP


def many_rows(zs):
    """Weights of up to 2^30 rows, short ones among them, for any number of
    rows of the left operand that takes the kernels for few."""
    L = zs.lib()
    for n in ((1 << 27) - 16, (1 << 27) + 1, 1 << 28, 1 << 30):
        for k in (1, 32, 224, 256):
            nb = -(-k // 32)
            w = mx(zs, n, k, scales=B + (1 << 39))
            for m in (1, 17, 32):
                a = mx(zs, m, k, base=3 * B)
                assert n * 16 * nb < 1 << 39 and m * n * 4 < B
                assert L.zero_mxfp4_matmul(ctypes.byref(a), ctypes.byref(w), 7 * B, F32, n,
                                           None) == EHIP, (m, n, k)
                assert L.zero_mxfp4_linear(5 * B, F16, m, k, ctypes.byref(w), 7 * B, F32, n,
                                           None) == EHIP, (m, n, k)
    w = mx(zs, (1 << 30) + 1, 32, scales=B + (1 << 39))
    assert L.zero_mxfp4_linear(5 * B, F16, 1, 32, ctypes.byref(w), 7 * B, F32, 1 << 31,
                               None) == EOVERFLOW


def gradient_parts(zs):
    """The workspace is 0 where the whole sum is faster: 256 x 256 tiles that
    fill a round, and sums too short for their parts."""
    L = zs.lib()
    for m, n, k, parts in (
            # 256 x 256 tiles: one round, two thirds of one, more than one
            (4096, 4096, 4096, 1), (4096, 11_008, 4096, 1), (4096, 32_000, 4096, 1),
            (8192, 6400, 1600, 1), (8192, 32_000, 1600, 1), (4352, 4096, 2048, 1),
            (4352, 9216, 2048, 3), (4352, 11_008, 2048, 3), (8704, 32_000, 1280, 3),
            (8960, 32_000, 1280, 1), (8192, 50_257, 4096, 1),
            # 128 x 128, one a CU
            (2048, 4096, 2048, 1), (2048, 6144, 2048, 2), (2048, 32_000, 2048, 2),
            (2304, 11_008, 2304, 1),
            # 64 x 64, many and few
            (1024, 2048, 1024, 1), (512, 2048, 1600, 1), (512, 4096, 1600, 2),
            (65, 2048, 4096, 2), (65, 50_257, 1600, 10), (512, 4096, 4096, 1)):
        n_bytes = ctypes.c_uint64(7)
        assert L.zero_mxfp4_grad_workspace(m, ctypes.byref(mx(zs, n, k)),
                                           ctypes.byref(n_bytes)) == 0
        assert n_bytes.value == (parts * m * k * 4 if parts > 1 else 0), (m, n, k)
