"""The tiled kernels of the 4-bit products at each of their tiles, against
64-bit products.  Output sizes end inside a tile in both directions, inner
sizes inside a block and a step.  Each case prints its name before it touches
the GPU."""
import numpy as np
import pytest

import mx_reference as ref
from test_gpu_mxfp4 import dev, dt, far_rows, in_rows, random_mx, rounded, say, zs  # noqa: F401

pytestmark = pytest.mark.gpu

# product, tile, rows, output columns, inner size
TILES = [
    ("matmul", 64, 300, 513, 1000), ("matmul", 64, 65, 129, 70),
    ("matmul", 128, 1030, 1029, 300), ("matmul", 128, 1030, 1029, 70),
    ("matmul", 256, 3001, 3003, 300), ("matmul", 256, 3001, 3003, 70),
    ("matmul", 256, 2561, 4001, 1030),
    ("linear", 64, 300, 513, 1000), ("linear", 64, 65, 8193, 33),
    ("linear", 128, 2050, 2051, 300), ("linear", 128, 2050, 2051, 33),
    ("linear", 256, 3001, 3003, 300), ("linear", 256, 3001, 3003, 33),
    ("linear", 256, 2561, 4001, 1030),
    ("grad", 64, 300, 513, 1000), ("grad", 64, 65, 8193, 33),
    ("grad", 128, 2050, 2051, 300), ("grad", 128, 2050, 2051, 33),
    ("grad", 256, 3001, 3003, 300), ("grad", 256, 3001, 3003, 33),
    ("grad", 256, 2561, 4001, 1030)]
# sums of the gradient in parts: rows, columns, weight's rows, tile, parts
PARTS = [(300, 1001, 5003, 64, 4), (1001, 1003, 4200, 64, 2), (2047, 2043, 6300, 128, 2),
         (3001, 3003, 9300, 256, 3), (3901, 3003, 49_200, 256, 2)]


def on_gpu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).cuda()


def check(got, want, mag, inner, name, what):
    """The bound of test_gpu_mxfp4.check_product: (inner + 8) 2^-23 sum |a w|
    and one rounding to the output's type."""
    import torch
    assert torch.isfinite(got).all(), what
    tol = (inner + 8) * 2.0 ** -23 * mag
    tol = tol + ref.HALF_STEP[name] * (want.abs() + tol) + ref.SMALLEST[name]
    worst = ((got.double() - want).abs() / tol).max().item()
    assert worst <= 1.0, f"{what}: error {worst:.3g} of the tolerance"


def out_like(m, c, name, pad=3, start=1):
    import torch
    return in_rows(torch.zeros(m, c, dtype=dt(name), device="cuda"), pad, start)


def marks_stand(buf, m, c, pad=3, start=1):
    assert (buf[:start] == 7).all() and (buf[start:].view(m, c + pad)[:, c:] == 7).all()


@pytest.mark.parametrize("m,n,k", [t[2:] for t in TILES if t[0] == "matmul"])
def test_matmul_tiles(zs, m, n, k):
    say(f"matmul tiles {m} {n} {k}")
    a, av = random_mx(zs, m, k, 1, 118, 126, pad_codes=16, pad_scales=1)
    w, wv = random_mx(zs, n, k, 2, 112, 120, pad_codes=32, pad_scales=3)
    av, wv = on_gpu(av), on_gpu(wv)
    want, mag = av @ wv.t(), av.abs() @ wv.abs().t()
    for name in ("f32", "f16", "bf16"):
        o, buf = out_like(m, n, name)
        zs.zero_mxfp4_matmul(a, w, o)
        check(o, want, mag, k, name, name)
        marks_stand(buf, m, n)


def with_far_blocks(w, wv, rows, blk):
    """Blocks of 2^-60 or so and of 2^20 in `rows` of w, outside fp16."""
    wv = wv.copy()
    for row, byte in zip(rows, (70, 147)):
        cols = slice(32 * blk, min(32 * blk + 32, wv.shape[1]))
        wv[row, cols] *= 2.0 ** (byte - int(w.scales[row, blk].item()))
        w.scales[row, blk] = byte
    return wv


@pytest.mark.parametrize("x_name", ("f16", "bf16"))
@pytest.mark.parametrize("m,n,k", [t[2:] for t in TILES if t[0] == "linear"])
def test_linear_tiles(zs, x_name, m, n, k):
    """Then with blocks outside fp16 and a NaN block, each in a tile of its
    own: no other output changes by a bit, and all stay in bounds."""
    import torch
    say(f"linear tiles {x_name} {m} {n} {k}")
    xv = rounded(np.random.default_rng(m + k).standard_normal((m, k)), x_name)
    x, _ = in_rows(dev(xv, x_name), 5, 3)
    w, wv = random_mx(zs, n, k, 3, 112, 122, pad_codes=16, pad_scales=2)
    xv = on_gpu(xv)
    want, mag = xv @ on_gpu(wv).t(), xv.abs() @ on_gpu(wv).abs().t()
    for name in ("f32", "f16", "bf16"):
        o, buf = out_like(m, n, name)
        zs.zero_mxfp4_linear(x, w, o)
        check(o, want, mag, k, name, name)
        marks_stand(buf, m, n)
    first, _ = out_like(m, n, "f32")
    zs.zero_mxfp4_linear(x, w, first)
    rows = (300 % n, n - 1)
    wv2 = with_far_blocks(w, wv, rows, k // 64)
    w.scales[5, (k - 1) // 32] = 255
    o, buf = out_like(m, n, "f32")
    zs.zero_mxfp4_linear(x, w, o)
    marks_stand(buf, m, n)
    assert torch.isnan(o[:, 5]).all()
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[5] = False
    w2 = on_gpu(wv2)
    check(o[:, keep], (xv @ w2.t())[:, keep], (xv.abs() @ w2.abs().t())[:, keep], k, "f32",
          "far blocks")
    if x_name == "bf16":    # no other order of the sum
        keep[list(rows)] = False
        assert torch.equal(o[:, keep], first[:, keep])


@pytest.mark.parametrize("x_name", ("f16", "bf16"))
@pytest.mark.parametrize("m,k,n", [t[2:] for t in TILES if t[0] == "grad"] +
                         [p[:3] for p in PARTS])
def test_grad_input_tiles(zs, x_name, m, k, n):
    import torch
    say(f"grad tiles {x_name} {m} {k} {n}")
    dyv = rounded(np.random.default_rng(m + n).standard_normal((m, n)).astype(np.float32), x_name)
    dy, _ = in_rows(dev(dyv, x_name), 5, 3)
    w, wv = random_mx(zs, n, k, 4, 112, 122, pad_codes=16, pad_scales=2)
    dyv, wg = on_gpu(dyv), on_gpu(wv)
    want, mag = dyv @ wg, dyv.abs() @ wg.abs()
    for name in ("f32", "f16", "bf16"):
        o, buf = out_like(m, k, name)
        zs.zero_mxfp4_linear_grad_input(dy, w, o)
        check(o, want, mag, n, name, name)
        marks_stand(buf, m, k)
    del want, mag, wg
    # in rows of the first and the last steps (and parts): blocks outside fp16
    # and one of NaN
    wv2 = with_far_blocks(w, wv, (n // 3, n - 1), k // 64)
    w.scales[0, (k - 1) // 32] = 255
    nan = torch.zeros(k, dtype=torch.bool, device="cuda")
    nan[(k - 1) // 32 * 32:] = True
    o, buf = out_like(m, k, "f32")
    zs.zero_mxfp4_linear_grad_input(dy, w, o)
    marks_stand(buf, m, k)
    assert torch.isnan(o[:, nan]).all()
    wg = on_gpu(wv2)[:, ~nan]
    check(o[:, ~nan], dyv @ wg, dyv.abs() @ wg.abs(), n, "f32", "far blocks")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n,k", [(1030, 1029, 300), (2050, 2051, 300), (3001, 3003, 300)])
def test_tiles_repeat_and_offsets_past_32_bits(zs, m, n, k):
    """Equal calls give equal bits, in a replayed graph too, and so do rows
    2^23 apart, the widest pitch that the products take."""
    import torch
    say(f"tiles, far rows {m} {n} {k}")
    rng, ld = np.random.default_rng(5), 1 << 23
    x = dev(rng.standard_normal((m, k)), "bf16")
    dy = dev(rng.standard_normal((m, n)), "f16")
    master = dev(rng.standard_normal((n, k)) * 0.02)
    w, xq = zs.MXFP4.empty(n, k), zs.MXFP4.empty(m, k)
    zs.zero_mxfp4_quantize(master, w)
    zs.zero_mxfp4_quantize(x, xq)

    def products(x, xq, dy, w, y1, y2, dx):
        zs.zero_mxfp4_matmul(xq, w, y1)
        zs.zero_mxfp4_linear(x, w, y2)
        zs.zero_mxfp4_linear_grad_input(dy, w, dx)

    want = [torch.empty(m, c, dtype=torch.bfloat16, device="cuda") for c in (n, n, k)]
    products(x, xq, dy, w, *want)
    got = [torch.empty_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        products(x, xq, dy, w, *got)
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    far = zs.MXFP4(far_rows(n, w.codes.shape[1], ld, torch.uint8),
                   far_rows(n, w.scales.shape[1], ld, torch.uint8), k)
    far.codes.copy_(w.codes)
    far.scales.copy_(w.scales)
    fq = zs.MXFP4(far_rows(m, xq.codes.shape[1], ld, torch.uint8),
                  far_rows(m, xq.scales.shape[1], ld, torch.uint8), k)
    fq.codes.copy_(xq.codes)
    fq.scales.copy_(xq.scales)
    for t in got:
        t.zero_()
    zs.zero_mxfp4_matmul(fq, far, got[0])
    del fq
    fx = far_rows(m, k, ld, x.dtype)
    fx.copy_(x)
    zs.zero_mxfp4_linear(fx, far, got[1])
    del fx
    fd = far_rows(m, n, ld, dy.dtype)
    fd.copy_(dy)
    zs.zero_mxfp4_linear_grad_input(fd, far, got[2])
    del fd
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del far
    torch.cuda.empty_cache()
