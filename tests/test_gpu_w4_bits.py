"""How many bits of x and of the experts' hidden values the 4-bit products hold,
where whole numbers keep every other rounding out."""

import pytest
import torch

import block_cases as bc

pytestmark = pytest.mark.gpu


def _one_scale(values, zeros, group):
    import mixture_experts_layer_fp32_gb300 as moe
    s = torch.ones(zeros.shape, dtype=torch.bfloat16, device="cuda")
    return moe.W4Weight(moe.pack_w4(values), s, zeros, group=group, k=values.shape[-1])


@pytest.mark.parametrize("T", [3, 6, 40, 90])
def test_hidden_values_hold_22_bits(T):
    """Two hidden values of an expert, a b and a (b + 1), are subtracted.  a and b
    are whole numbers (sums of fewer than 2^24) and a > 24, so that silu(a) is a:
    the values are known to the last bit of fp32.  Their difference may be off by
    2^-22 of each for the two fp16 numbers that hold it, by 2^-46 of the row's
    largest, and by 8 roundings of the sums."""
    import mixture_experts_layer_fp32_gb300 as moe
    E, h, f, group = 4, 256, 256, 64
    g = torch.Generator(device="cuda").manual_seed(T)

    def draw(lo, hi, shape, dtype=torch.uint8):
        return torch.randint(lo, hi, shape, dtype=dtype, device="cuda", generator=g)

    first, second = [0, 2, 5, 7], [67, 68, 70, 65]   # of an expert: every place of eight inputs
    W1, W3 = (torch.zeros((E, f, h), dtype=torch.uint8, device="cuda") for _ in range(2))
    W2 = torch.zeros((E, h, f), dtype=torch.uint8, device="cuda")
    zeros2 = torch.zeros((E, h, f // group), dtype=torch.uint8, device="cuda")
    for e in range(E):
        i, j = first[e], second[e]
        W1[e, i] = draw(0, 16, (h,))
        W1[e, j] = W1[e, i]
        W3[e, i] = draw(0, 15, (h,))
        W3[e, j] = W3[e, i]
        W3[e, j, 0] += 1                 # x[:, 0] is 1
        for n in range(h):               # + i - j, or the other way round
            plus, minus = (i, j) if n % 2 == 0 else (j, i)
            W2[e, n, plus] = 1
            gm = minus // group
            zeros2[e, n, gm] = 1         # code - 1: -1 at `minus`, 0 elsewhere
            W2[e, n, gm * group:(gm + 1) * group] = 1
            W2[e, n, minus] = 0
    zeros = torch.zeros((E, f, h // group), dtype=torch.uint8, device="cuda")
    q = moe.W4Experts(_one_scale(W1, zeros, group), _one_scale(W3, zeros, group),
                      _one_scale(W2, zeros2, group))
    x = draw(1, 256, (T, h)).to(torch.bfloat16)
    x[:, 0] = 1
    idx = draw(0, E, (T, 1), torch.int32)
    prob = torch.ones((T, 1), device="cuda")
    cfg = moe.config(T=T, h=h, E=E, k=1, f=f)
    ws = moe.alloc_workspace_experts_w4(cfg)
    y = torch.full_like(x, float("nan"))
    moe.experts_w4(cfg, x, idx, prob, None, q, y, ws)
    moe.check(ws)
    for t in range(T):
        e = int(idx[t])
        a, b = (torch.mv(W[e].double(), x[t].double())[[first[e], second[e]]] for W in (W1, W3))
        assert float(a.min()) > 24 and float(torch.maximum(a, b).max()) < 1 << 24
        v = (a.float() * b.float()).double()
        sign = torch.where(torch.arange(h, device="cuda") % 2 == 0, 1.0, -1.0).double()
        ref = sign * (v[0] - v[1])
        bound = (2.0 ** -22 + 2.0 ** -46 + 8 * bc.U) * v.sum()
        assert float(bound) < 0.75 * 2.0 ** -18 * float(v.max())   # 17 bits would not do
        bc.assert_within("y", y[t], ref, bound.expand(h), torch.bfloat16)


@pytest.mark.parametrize("M", [1, 8, 9, 40, 70])
@pytest.mark.parametrize("exponent", [-80, 0, 100])
def test_x_is_exact_down_to_2_27_of_the_rows_largest(M, exponent):
    """One value of a row is 2^27 times the others' powers of two and meets zero
    weights; the others meet whole numbers, so that every sum is exact."""
    K, N, group = 256, 48, 64
    import mixture_experts_layer_fp32_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(M)
    values = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    values[:, 0] = 0
    w = _one_scale(values, torch.zeros((N, K // group), dtype=torch.uint8, device="cuda"), group)
    small = torch.randint(128, 256, (M, K), device="cuda", generator=g).double()
    small *= torch.where(torch.rand((M, K), device="cuda", generator=g) < 0.5, 1.0, -1.0)
    x = torch.ldexp(small, torch.tensor(exponent - 27 - 7, device="cuda"))
    x[:, 0] = 2.0 ** exponent
    assert torch.equal(x, x.to(torch.bfloat16).double())
    y = torch.full((M, N), float("nan"), device="cuda")
    ws = moe.alloc_workspace_linear_w4(M, w)
    moe.linear_w4(x.to(torch.bfloat16), w, y, ws)
    moe.check(ws)
    assert 255 * 15 * K < 1 << 24
    assert torch.equal(y.double(), x @ values.double().t())
