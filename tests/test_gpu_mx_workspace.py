"""The workspace that the binding takes for a gradient whose sum goes in
parts.  Each case prints its name before it touches the GPU."""
import numpy as np
import pytest

from test_gpu_mxfp4 import check_product, dev, host, random_mx, rounded, say, zs  # noqa: F401

pytestmark = pytest.mark.gpu


def test_workspace_belongs_to_the_calls_stream(zs, monkeypatch):
    """The memory goes back to torch's allocator when the call returns, so it
    has to be the call's own stream's: the default stream, as an object and as
    handle 0, another one likewise, and the current one where none is named."""
    import torch
    say("workspace streams")
    m, n, k = 5, 20_011, 160
    dyv = rounded(np.random.default_rng(1).standard_normal((m, n)), "bf16")
    w, wv = random_mx(zs, n, k, 2, 112, 122)
    dy, dx = dev(dyv, "bf16"), torch.zeros(m, k, device="cuda")
    taken, empty = [], torch.empty

    def recording(*a, **kw):
        taken.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    side, default = torch.cuda.Stream(), torch.cuda.default_stream()
    assert default.cuda_stream == 0 and side.cuda_stream != 0
    for current in (default, side):
        for stream, want in ((default, 0), (0, 0), (side, side.cuda_stream),
                             (side.cuda_stream, side.cuda_stream), (None, current.cuda_stream)):
            dx.zero_()
            torch.cuda.synchronize()
            taken.clear()
            with torch.cuda.stream(current), monkeypatch.context() as mp:
                mp.setattr(torch, "empty", recording)
                zs.zero_mxfp4_linear_grad_input(dy, w, dx, stream=stream)
                assert torch.cuda.current_stream() == current
            torch.cuda.synchronize()
            assert taken == [want]
            check_product(host(dx), dyv, wv, "f32", "gradient")
