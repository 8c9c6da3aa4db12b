"""The 4-bit products at the largest sizes and pitches they take.  Each case
prints its name before it touches the GPU."""
import numpy as np
import pytest

import mx_reference as ref
from test_gpu_mxfp4 import check_product, dev, host, random_mx, rounded, say, zs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", (32, 200))
def test_weights_of_more_rows_than_a_launch_dimension(zs, k):
    """2^27 + 77 rows of the weight through two rows of activations: more
    workgroups of 16 columns than one dimension of a launch holds.  The weight
    repeats every 2^17 + 19 rows, so every output has a reference; the rows
    behind the last output stay."""
    import torch
    say(f"2^27 + 77 rows of {k}")
    n, period = (1 << 27) + 77, (1 << 17) + 19
    w0, wv = random_mx(zs, period, k, 3, 112, 122)
    nb = -(-k // 32)
    reps = -(-n // period)
    w = zs.MXFP4(w0.codes.repeat(reps, 1)[:n], w0.scales.repeat(reps, 1)[:n], k)
    assert tuple(w.codes.shape) == (n, 16 * nb)
    xv = rounded(np.random.default_rng(4).standard_normal((2, k)), "bf16")
    xq = zs.MXFP4.empty(2, k)
    zs.zero_mxfp4_quantize(dev(xv, "bf16"), xq)
    code, scale, _ = ref.quantize(xv)
    for name, av in (("linear", xv), ("matmul", ref.values(code, scale, k))):
        y = torch.full((3, n), 7.0, dtype=torch.bfloat16, device="cuda")
        if name == "linear":
            zs.zero_mxfp4_linear(dev(xv, "bf16"), w, y[:2])
        else:
            zs.zero_mxfp4_matmul(xq, w, y[:2])
        check_product(host(y[:2, :period]), av, wv.T, "bf16", name)
        for i in range(2):      # every repetition has the first one's bits
            whole = y[i, :n // period * period].view(-1, period)
            assert (whole == whole[0]).all()
            tail = y[i, n // period * period:]
            assert torch.equal(tail, whole[0, :tail.numel()])
        assert (y[2] == 7).all()
        del y, whole, tail
    del w
    torch.cuda.empty_cache()
