"""What the quantiser makes of infinities and NaNs."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [2, 20])
def test_bad_weights_stay_visible(M, zeros, bad):
    """The group gets the scale NaN, so that its output is NaN; the others are as
    without it."""
    import mixture_experts_layer_fp32_gb300 as moe
    K, N, group = 256, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    W = (0.02 * torch.randn((K, N), device="cuda", generator=g)).to(torch.bfloat16)
    good = moe.quantize_w4(W, group, zeros)
    W[70, 5] = bad
    q = moe.quantize_w4(W, group, zeros)
    hit = torch.zeros_like(q.scales, dtype=torch.bool)
    hit[5, 1] = True
    assert bool(torch.isnan(q.scales[hit]).all())
    assert torch.equal(q.scales[~hit], good.scales[~hit])
    if zeros:
        assert torch.equal(q.zeros[~hit], good.zeros[~hit])
    rows = torch.arange(N, device="cuda") != 5
    assert torch.equal(q.codes[rows], good.codes[rows])
    x = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
    y, want = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    moe.linear_w4(x, q, y, moe.alloc_workspace_linear_w4(M, q))
    moe.linear_w4(x, good, want, moe.alloc_workspace_linear_w4(M, good))
    assert bool(torch.isnan(y[:, 5]).all())
    assert torch.equal(y[:, rows], want[:, rows])
