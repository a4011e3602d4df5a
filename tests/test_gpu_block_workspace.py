"""A workspace made for the largest batch serves the smaller ones: the same bits
as with a workspace of their own."""

import pytest
import torch

from test_gpu_w4 import _experts, _routing, _weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,N,K", [(64, 4000, 2048), (65, 1792, 4096), (200, 640, 1024)])
def test_linear(most, N, K):
    import mixture_experts_layer_fp32_gb300 as moe
    w, _ = _weight((N,), K, 64, True, N)
    x = torch.randn((most, K), device="cuda").to(torch.bfloat16)
    ws = moe.alloc_workspace_linear_w4(most, w)
    for rows in (1, 2, 7, 8, 9, 16, 33, 64, most):
        y, own = (torch.full((rows, N), float("nan"), device="cuda") for _ in range(2))
        moe.linear_w4(x[:rows], w, y, ws)
        moe.linear_w4(x[:rows], w, own, moe.alloc_workspace_linear_w4(rows, w))
        moe.check(ws)
        assert torch.equal(y, own)


def test_experts_and_forward():
    import mixture_experts_layer_fp32_gb300 as moe
    h, E, k, f, most = 2048, 8, 2, 4096, 40
    cfg = moe.config(T=most, h=h, E=E, k=k, f=f)
    q, _ = _experts(E, h, f, 64, False, 3)
    x = torch.randn((most, h), device="cuda").to(torch.bfloat16)
    Wg = torch.randn((h, E), device="cuda")
    ws, ws_layer = moe.alloc_workspace_experts_w4(cfg), moe.alloc_workspace_w4(cfg)
    for T in (1, 2, 5, 6, 7, 8, 20, 39, 40):
        few = moe.config(T=T, h=h, E=E, k=k, f=f)
        idx, prob, _ = _routing(T, E, k, T)
        y, own, layer, layer_own = (torch.full((T, h), float("nan"), dtype=x.dtype, device="cuda")
                                    for _ in range(4))
        moe.experts_w4(few, x[:T], idx, prob, None, q, y, ws)
        moe.experts_w4(few, x[:T], idx, prob, None, q, own, moe.alloc_workspace_experts_w4(few))
        moe.forward_w4(few, x[:T], Wg, None, None, q, layer, ws_layer)
        moe.forward_w4(few, x[:T], Wg, None, None, q, layer_own, moe.alloc_workspace_w4(few))
        moe.check(ws)
        moe.check(ws_layer)
        assert torch.equal(y, own) and torch.equal(layer, layer_own)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [64, 1021, 1024])
def test_norm_backward(H, dtype):
    import mixture_experts_layer_fp32_gb300 as moe
    most = 4000
    z, dy = (torch.randn((most, H), device="cuda").to(dtype) for _ in range(2))
    mean, rstd = z.float().mean(1), torch.rsqrt(z.float().var(1) + 1e-5)
    ws = moe.alloc_workspace_norm_backward(most, H)
    for rows in (1, 151, 303, 304, 607, 608, 1215, 1216, most):
        outs = []
        for use in (ws, moe.alloc_workspace_norm_backward(rows, H)):
            dx = torch.full((rows, H), float("nan"), dtype=dtype, device="cuda")
            dw, db = (torch.full((H,), float("nan"), device="cuda") for _ in range(2))
            moe.layer_norm_backward(dy[:rows], z[:rows], None, mean[:rows], rstd[:rows], dx, dw,
                                    db, use)
            outs.append((dx, dw, db))
        assert all(torch.equal(a, c) for a, c in zip(*outs))
