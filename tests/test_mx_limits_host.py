"""Calls of the 4-bit operators at the ends of what they accept, without a
GPU (as tests/test_mx_distill_host.py: fake addresses, EHIP where every check
passes)."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_mx_distill_host import B, EHIP, EINVAL, F16, F32, ROOT, mx


@pytest.mark.parametrize("body", ["empty_workspace"])
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
