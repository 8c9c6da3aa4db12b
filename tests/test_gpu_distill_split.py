"""The non-finite flag of the distillation loss where a row is split over
several workgroups.  Each case prints its name before it touches the GPU."""
import numpy as np
import pytest

from test_gpu_mxfp4 import dev, say, zs  # noqa: F401

pytestmark = pytest.mark.gpu
# rows, vocabulary: split in 12 parts (rows in registers, 1024 threads), in 4 and
# in 2 (256 threads), in 4 (16 vectors a thread), in 34 (rows read twice), whole
SIZES = [(3, 50_257), (10, 20_000), (100, 9000), (60, 131_072), (1, 140_001), (300, 9000)]


def call(zs, z, idx, log2_scale, before):
    """The flag and the gradient, written over an array full of `before`."""
    import torch
    rows, V = z.shape
    k = idx.shape[1]
    grad = torch.full((rows, V), before, dtype=torch.float16, device="cuda")
    loss = torch.empty(rows, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    zs.zero_distill_loss(z, idx, torch.zeros(rows, k, device="cuda"), loss, grad,
                         loss_scale=zs.LossScale(log2_scale, device=loss.device),
                         nonfinite_flag=flag)
    return flag.item(), grad


@pytest.mark.parametrize("rows,V", SIZES)
def test_overflow_at_an_unnamed_position_raises_the_flag(zs, rows, V):
    """A softmax of 1 at one column, which the teacher does not name, times
    2^18: past fp16's 65504 there and at no other position (the 64 named ones
    get -2^18 / 64).  Whichever part writes the column, the flag is raised,
    and what the array held before does not matter."""
    import torch
    for at in np.linspace(0, V - 1, 9).astype(int):
        say(f"distill split, overflow {rows} x {V} at {at}")
        named = (at + 1 + np.arange(64) * 7) % V
        assert at not in named
        z = np.full((rows, V), -20.0, np.float32)
        z[rows - 1, at] = 0.0
        z[:rows - 1, named[0]] = 0.0    # the other rows agree with the teacher there
        idx = np.broadcast_to(named, (rows, 64)).copy()
        idx[:rows - 1, 1:] = -1
        flag, grad = call(zs, dev(z, "f16"), torch.from_numpy(idx).cuda(), 18, 0.0)
        bad = (~torch.isfinite(grad)).nonzero().cpu().numpy()
        assert bad.tolist() == [[rows - 1, at]]
        assert flag == 1, f"column {at}"


@pytest.mark.parametrize("rows,V", SIZES)
def test_old_contents_do_not_raise_the_flag(zs, rows, V):
    """A scale at which softmax(z) 2^k alone would overflow, but only at the
    position the teacher names with probability 1, where the gradient is
    small: every value written is finite, and infinities and NaN that the
    array held before leave the flag at 0."""
    import torch
    for at in np.linspace(0, V - 1, 5).astype(int):
        say(f"distill split, old contents {rows} x {V} at {at}")
        z = np.full((rows, V), -20.0, np.float32)
        z[:, at] = 0.0
        idx = torch.full((rows, 1), int(at), device="cuda")
        for before in (float("inf"), float("nan")):
            flag, grad = call(zs, dev(z, "f16"), idx, 18, before)
            assert torch.isfinite(grad).all() and flag == 0, f"column {at}"
