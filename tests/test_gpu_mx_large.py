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


def top_scales(zs, n, k, seed):
    """A weight with blocks of scale bytes 253 and 254 in the first, a middle
    and the last block of some rows: finite ones (codes up to 1.5 times 2^127)
    in rows 1 and n // 2, ones past 2^128 in rows 2 and n - 1.  All codes are
    positive.  (handle, fp64 values)."""
    import torch
    rng = np.random.default_rng(seed)
    nb = -(-k // 32)
    code = rng.integers(1, 8, (n, nb * 32)).astype(np.uint8)
    scale = rng.integers(112, 123, (n, nb)).astype(np.uint8)
    for row, most, byte in ((1, 3, 254), (n // 2, 5, 253), (2, 7, 254), (n - 1, 7, 253)):
        for blk in (0, nb // 2, nb - 1):
            code[row, 32 * blk:32 * blk + 32] = rng.integers(1, most + 1, 32)
            if most == 7:
                code[row, 32 * blk] = 7
            scale[row, blk] = byte
    code[:, k:] = 0
    q = zs.MXFP4(torch.from_numpy(ref.pack(code)).cuda(), torch.from_numpy(scale).cuda(), k)
    return q, ref.values(code, scale, k)


@pytest.mark.parametrize("x_name", ("f16", "bf16"))
@pytest.mark.parametrize("m,n,k", [
    # few rows, the left operand in registers: blocks that do and do not fill steps of four
    (1, 40, 256), (3, 333, 288), (16, 200, 1600), (2, 200, 1570), (20, 200, 330), (31, 77, 4096),
    # read at each step; tiles of 64
    (3, 50, 70), (40, 100, 333), (90, 150, 288), (200, 300, 1030)])
def test_scale_bytes_253_and_254(zs, x_name, m, n, k):
    """Values below 2^128 are exact in every product.  From there on a value is
    as infinite as fp32 and bfloat16 make it: bfloat16 activations above 0 give
    +infinity, whatever the number of blocks, fp16 ones something not finite,
    and no other output is touched.  The product of two 4-bit operands takes
    the value as it is."""
    import torch
    say(f"scale bytes 253, 254 {x_name} {m} {n} {k}")
    rng = np.random.default_rng(m + n + k)
    xv, dyv = (rounded((np.abs(rng.standard_normal(s)) + 0.5) * 2.0 ** -12, x_name)
               for s in ((m, k), (m, n)))
    w, wv = top_scales(zs, n, k, 7)
    huge = np.abs(wv) >= 2.0 ** 128
    fin = np.where(huge, 0.0, wv)
    y, dx = torch.empty(m, n, device="cuda"), torch.empty(m, k, device="cuda")
    zs.zero_mxfp4_linear(dev(xv, x_name), w, y)
    zs.zero_mxfp4_linear_grad_input(dev(dyv, x_name), w, dx)
    for got, a, bt, hit in ((host(y), xv, fin.T, huge.any(1)), (host(dx), dyv, fin, huge.any(0))):
        assert hit.any() and not hit.all()
        assert not np.isfinite(got[:, hit]).any()
        if x_name == "bf16":
            assert (got[:, hit] == np.inf).all()
        check_product(got[:, ~hit], a, bt[:, ~hit], "f32", "beside values past 2^128")
    xq = zs.MXFP4.empty(m, k)
    zs.zero_mxfp4_quantize(dev(xv, x_name), xq)
    code, scale, _ = ref.quantize(xv)
    zs.zero_mxfp4_matmul(xq, w, y)
    check_product(host(y), ref.values(code, scale, k), wv.T, "f32", "matmul")


@pytest.mark.parametrize("m,n,k", [(1, 1000, 4096), (5, 257, 31), (33, 1600, 160), (65, 129, 257),
                                   (130, 70, 2048), (1030, 1029, 300)])
def test_matmul_rounds_to_fp16_infinity(zs, m, n, k):
    """Operands whose sums pass fp16's range: a sum from 65520 on, where fp16
    rounds to infinity, is infinite with its sign; below it is the sum rounded
    once; within the sum's own error of 65520 the computed sum, which lies
    within that error of the exact one, may be on either side."""
    import torch
    say(f"matmul fp16 overflow {m} {n} {k}")
    a, av = random_mx(zs, m, k, 1)
    w, wv = random_mx(zs, n, k, 2, pad_codes=16 * (k % 3), pad_scales=k % 5)
    y = torch.zeros(m, n, dtype=torch.float16, device="cuda")
    zs.zero_mxfp4_matmul(a, w, y)
    got, want = host(y), av @ wv.T
    tol = (k + 8) * 2.0 ** -23 * (np.abs(av) @ np.abs(wv).T)
    over, under = np.abs(want) - tol >= 65520.0, np.abs(want) + tol < 65520.0
    assert under.any() and (over.any() or k == 31) and np.mean(over | under) > 0.98
    assert np.array_equal(got[over], np.copysign(np.inf, want[over]))
    half = ref.HALF_STEP["f16"] * (np.abs(want) + tol) + tol + ref.SMALLEST["f16"]
    fits = np.abs(got - want) <= half
    assert fits[under].all()
    near = ~over & ~under
    assert (fits | (got == np.copysign(np.inf, want)))[near].all()
