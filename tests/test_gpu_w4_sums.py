"""The sums of the 4-bit products hold what fp32 holds: whole numbers, a few of
them some 2^17 times the others, whose sums stay below 2^24 and so are exact in
any order."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _weight(values, zeros, group):
    import mixture_experts_layer_fp32_gb300 as moe
    lead = values.shape[:-1] + (values.shape[-1] // group,)
    s = torch.ones(lead, dtype=torch.bfloat16, device="cuda")
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, -1)
    w = moe.W4Weight(moe.pack_w4(values), s, zeros, group=group, k=values.shape[-1])
    return w, values.double() - z


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 5, 8, 9, 20, 40, 64, 70])
def test_linear_beside_outliers(M, group, zeros):
    import mixture_experts_layer_fp32_gb300 as moe
    N, K = 304, 1024
    g = torch.Generator(device="cuda").manual_seed(M + group)

    def draw(lo, hi, shape, dtype=torch.uint8):
        return torch.randint(lo, hi, shape, dtype=dtype, device="cuda", generator=g)

    w, W = _weight(draw(0, 16, (N, K)), draw(0, 16, (N, K // group)) if zeros else None, group)
    x = draw(-3, 4, (M, K), torch.int32).double()
    x[torch.arange(M), draw(0, K, (M,), torch.int64)] = 2.0 ** 17
    assert 15 * (2 ** 17 + 3 * K) < 1 << 24
    y = torch.full((M, N), float("nan"), device="cuda")
    ws = moe.alloc_workspace_linear_w4(M, w)
    moe.linear_w4(x.to(torch.bfloat16), w, y, ws)
    moe.check(ws)
    assert torch.equal(y.double(), x @ W.t())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 3, 9, 40])
def test_experts_beside_outliers(T, group):
    """Hidden values of 2^22 in two places, which cancel, and multiples of 32 up
    to 32 x 27 elsewhere.  a is 32 or more, so that silu(a) is a."""
    import mixture_experts_layer_fp32_gb300 as moe
    E, h, f = 2, 256, 512
    g = torch.Generator(device="cuda").manual_seed(T + group)

    def draw(lo, hi, shape, dtype=torch.uint8):
        return torch.randint(lo, hi, shape, dtype=dtype, device="cuda", generator=g)

    # inputs: 32, 2^11, 2^11, then eight small whole numbers
    x = torch.zeros((T, h), device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 32.0, 2048.0, 2048.0
    x[:, 3:11] = draw(-3, 4, (T, 8), torch.int32).float()
    W1, W3 = (torch.zeros((E, f, h), dtype=torch.uint8, device="cuda") for _ in range(2))
    features = torch.arange(f, device="cuda")
    W1[:, :, 0] = 1
    W3[:, features, 3 + features % 8] = (1 + features % 9).to(torch.uint8)
    large = 5, f - 14
    for i in large:
        W1[:, i] = W3[:, i] = 0
        W1[:, i, 1] = W3[:, i, 2] = 1
    zeros2 = draw(1, 15, (E, h, f // group))
    W2 = draw(0, 16, (E, h, f))
    each = zeros2.repeat_interleave(group, -1)
    W2[:, :, large[0]] = each[:, :, large[0]] + 1
    W2[:, :, large[1]] = each[:, :, large[1]] - 1
    none = torch.zeros((E, f, h // group), dtype=torch.uint8, device="cuda")
    (q1, A), (q3, B), (q2, C) = (_weight(v, z, group) for v, z in
                                 ((W1, none), (W3, none), (W2, zeros2)))
    idx = draw(0, E, (T, 1), torch.int32)
    cfg = moe.config(T=T, h=h, E=E, k=1, f=f)
    ws = moe.alloc_workspace_experts_w4(cfg)
    y = torch.full((T, h), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.experts_w4(cfg, x.to(torch.bfloat16), idx, torch.ones((T, 1), device="cuda"), None,
                   moe.W4Experts(q1, q3, q2), y, ws)
    moe.check(ws)
    x = x.double()
    for t in range(T):
        e = int(idx[t])
        a, b = A[e] @ x[t], B[e] @ x[t]
        assert float(a.min()) >= 32
        v = a * b
        assert 15 * float(v.abs().sum()) / 32 < 1 << 24
        assert torch.equal(y[t], (C[e] @ v).to(torch.bfloat16))
