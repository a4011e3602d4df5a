"""The 4-bit products where the powers of two of x's rows reach their ends: rows
near the largest and the smallest bf16 numbers, rows with an infinity or a NaN,
in the kernels for few and for more rows and in the experts."""

import pytest
import torch

import block_cases as bc
from test_gpu_w4 import _routing

pytestmark = pytest.mark.gpu

# of a row's values; the unit of a row is clamped below 2^-112, and from 2^118 on
# it leaves no room for another factor of 2^24 in fp32
LOW = [-133, -130, -126, -120, -114, -113, -112, -111, -110, -100, -60]
HIGH = [60, 100, 103, 104, 110, 116, 117, 118, 119, 120, 125, 127]


def _weight(shape, K, group, zeros, seed, scale):
    import mixture_experts_layer_fp32_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(0, 16, shape + (K,), dtype=torch.uint8, device="cuda", generator=g)
    s = scale * (0.5 + torch.rand(shape + (K // group,), device="cuda", generator=g))
    z = None
    if zeros:
        z = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda", generator=g)
    w = moe.W4Weight(moe.pack_w4(v), s.to(torch.bfloat16), z, group=group, k=K)
    return w, bc.w4_weight_ref(w.codes, w.scales, w.zeros, group, K)


def _rows(exponents, M, K, seed):
    """Row i: normal values, cut at 1.9, times 2^exponents[i % n]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), device="cuda", generator=g).clamp(-1.9, 1.9).double()
    e = torch.tensor([exponents[i % len(exponents)] for i in range(M)], device="cuda")
    return torch.ldexp(x, e[:, None]).to(torch.bfloat16)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("exponents,scale", [(LOW, 2.0 ** 60), (HIGH, 2.0 ** -40)])
@pytest.mark.parametrize("M", [1, 4, 8, 9, 17, 33, 50, 64, 70])
def test_linear_rows_of_any_magnitude(M, exponents, scale, out, zeros):
    import mixture_experts_layer_fp32_gb300 as moe
    K, N, group = 1024, 200, 64
    for first in range(0, len(exponents), M):
        w, W = _weight((N,), K, group, zeros, M, scale)
        x = _rows(exponents[first:] + exponents[:first], M, K, M + first)
        y = torch.full((M, N), float("nan"), dtype=out, device="cuda")
        ws = moe.alloc_workspace_linear_w4(M, w)
        moe.linear_w4(x, w, y, ws)
        moe.check(ws)
        bc.assert_within("y", y, x.double() @ W.t(), bc.w4_product_bound(x.double(), W), out)


@pytest.mark.parametrize("M", [4, 20, 64, 70])
def test_linear_bad_rows_are_nan_alone(M):
    """An infinity or a NaN in a row of x makes that row of y NaN, and no other."""
    import mixture_experts_layer_fp32_gb300 as moe
    K, N = 256, 40
    w, W = _weight((N,), K, 64, False, 3, 0.004)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    x[1, 7], x[2, 200], x[M - 1, 0] = float("inf"), float("nan"), float("-inf")
    y = torch.zeros((M, N), device="cuda")
    ws = moe.alloc_workspace_linear_w4(M, w)
    moe.linear_w4(x, w, y, ws)
    moe.check(ws)
    bad = torch.zeros(M, dtype=torch.bool)
    bad[[1, 2, M - 1]] = True
    assert bool(torch.isnan(y[bad.cuda()]).all())
    good = ~bad.cuda()
    bc.assert_within("y", y[good], x[good].double() @ W.t(),
                     bc.w4_product_bound(x[good].double(), W), y.dtype)


@pytest.mark.parametrize("x_exponent,up,down", [
    (120, 2.0 ** -115, 0.004),      # x past the range of the unit; hidden values of some 2^10
    (54, 1.0, 2.0 ** -60),          # hidden values of 2^120
    (-130, 2.0 ** 122, 0.004),      # subnormal x
    (0, 2.0 ** -60, 2.0 ** 100)])   # hidden values of 2^-120
@pytest.mark.parametrize("T,E,k", [(2, 2, 1), (5, 4, 2), (24, 2, 1), (40, 2, 2)])
def test_experts_of_any_magnitude(T, E, k, x_exponent, up, down):
    import mixture_experts_layer_fp32_gb300 as moe
    h, f, group = 256, 256, 64
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)
    ws4 = [_weight((E, n), kk, group, False, i, s)
           for i, (n, kk, s) in enumerate(((f, h, up), (f, h, up), (h, f, down)))]
    q, W = moe.W4Experts(*(w for w, _ in ws4)), [m for _, m in ws4]
    idx, prob, _ = _routing(T, E, k, T)
    x = _rows([x_exponent], T, h, T)
    y = torch.full_like(x, float("nan"))
    ws = moe.alloc_workspace_experts_w4(cfg)
    moe.experts_w4(cfg, x, idx, prob, None, q, y, ws)
    moe.check(ws)
    ref, bound = bc.experts_ref(x.double(), idx.cpu(), prob.cpu(), None, *W)
    bc.assert_within("y", y, ref, bound, torch.bfloat16)


@pytest.mark.parametrize("T", [3, 40])
def test_experts_bad_rows_are_nan_alone(T):
    import mixture_experts_layer_fp32_gb300 as moe
    h, f, E, k, group = 256, 256, 2, 2, 64
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)
    ws4 = [_weight((E, n), kk, group, True, i, 0.01)
           for i, (n, kk) in enumerate(((f, h), (f, h), (h, f)))]
    q, W = moe.W4Experts(*(w for w, _ in ws4)), [m for _, m in ws4]
    idx, prob, _ = _routing(T, E, k, T)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    x[1, 9] = float("nan")
    x[T - 1, 255] = float("inf")
    y = torch.zeros_like(x)
    ws = moe.alloc_workspace_experts_w4(cfg)
    moe.experts_w4(cfg, x, idx, prob, None, q, y, ws)
    moe.check(ws)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[1, T - 1]] = True
    assert bool(torch.isnan(y[bad]).all())
    keep = (~bad).to(torch.uint8)[:, None].expand(T, k).cpu()
    ref, bound = bc.experts_ref(torch.where(bad[:, None], 0.0, x.double()), idx.cpu(), prob.cpu(),
                                keep, *W)
    bc.assert_within("y", y[~bad], ref[~bad], bound[~bad], torch.bfloat16)
