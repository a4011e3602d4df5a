"""4-bit products and experts at the ends of their shapes: rows longer than what
the split of x holds on the chip, single outputs, more rows than a launch takes,
none at all."""

import pytest
import torch

import block_cases as bc
from test_gpu_w4 import _experts, _routing, _weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 40, 16384, 128), (1, 40, 16512, 128), (3, 33, 20480, 64), (8, 16, 32800, 32),
    (9, 33, 20480, 64), (20, 24, 32800, 32), (64, 17, 65536, 128), (2, 8, 131072, 128),
    (1, 1, 32, 32), (5, 1, 1024, 64), (40, 1, 1024, 64), (7, 2, 96, 32), (33, 3, 160, 32),
    (1024, 40, 256, 64), (1025, 40, 256, 64), (1100, 300, 160, 32), (2049, 24, 128, 128)])
def test_linear_exact(M, N, K, group, zeros):
    """Whole numbers and scales that are powers of two, as in test_gpu_w4."""
    import mixture_experts_layer_fp32_gb300 as moe
    w, W = _weight((N,), K, group, zeros, M + N, exact=True)
    x = torch.randint(-2, 3, (M, K), device="cuda").to(torch.bfloat16)
    assert 2 * 15 * 4 * K < 1 << 24
    y = torch.full((M, N), float("nan"), device="cuda")
    ws = moe.alloc_workspace_linear_w4(M, w)
    ws[256:] = 255
    moe.linear_w4(x, w, y, ws)
    moe.check(ws)
    assert torch.equal(y.double(), x.double() @ W.t())


@pytest.mark.parametrize("T,h,E,k,f,group", [(1, 256, 2, 1, 20480, 128), (3, 256, 4, 2, 17024, 64),
                                             (20, 256, 2, 1, 20480, 128),
                                             (2, 17408, 2, 2, 128, 128),
                                             (40, 17408, 2, 1, 128, 32),
                                             (400, 256, 3, 3, 128, 64)])
def test_experts(T, h, E, k, f, group):
    import mixture_experts_layer_fp32_gb300 as moe
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)
    q, W = _experts(E, h, f, group, True, T + f)
    idx, prob, keep = _routing(T, E, k, T, drop=0.2)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    y = torch.full_like(x, float("nan"))
    ws = moe.alloc_workspace_experts_w4(cfg)
    ws[256:] = 255
    moe.experts_w4(cfg, x, idx, prob, keep, q, y, ws)
    moe.check(ws)
    ref, bound = bc.experts_ref(x.double(), idx.cpu(), prob.cpu(), keep.cpu(), *W)
    bc.assert_within("y", y, ref, bound, torch.bfloat16)


def test_no_tokens():
    import mixture_experts_layer_fp32_gb300 as moe
    h, E, k, f = 256, 4, 2, 128
    cfg = moe.config(T=0, h=h, E=E, k=k, f=f)
    q, _ = _experts(E, h, f, 64, False, 1)
    x = torch.empty((0, h), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((0, k), dtype=torch.int32, device="cuda")
    prob = torch.empty((0, k), device="cuda")
    ws, layer = moe.alloc_workspace_experts_w4(cfg), moe.alloc_workspace_w4(cfg)
    moe.experts_w4(cfg, x, idx, prob, None, q, x, ws)
    count = torch.full((E,), 7, dtype=torch.int32, device="cuda")
    moe.forward_w4(cfg, x, torch.randn((h, E), device="cuda"), None, None, q, x, layer,
                   tokens_per_expert=count)
    moe.check(ws)
    moe.check(layer)
    assert torch.equal(count, torch.zeros_like(count))
