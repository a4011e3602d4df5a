"""The operators of a decoding step at the ends of their documented sizes."""

import pytest
import torch

from decode_cases import LayerCase
from test_gpu_few import call, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(h=2 ** 21, f=8), dict(h=8, f=2 ** 21),
                                dict(h=2 ** 21, f=8, T=33, E=1, k=1),
                                dict(h=8, f=2 ** 21, T=20, E=1, k=1, fs=1000)], ids=str)
def test_layer_of_the_widest_rows(kw):
    c = LayerCase(**dict(dict(T=3, E=2, k=1, score="softmax_pre", dtype="f32"), **kw)).cuda()
    verify(c, call(c))


def test_layer_of_the_widest_experts_in_bf16():
    """2^21 hidden values of a token: the first 2^17 times 16 the same, so one sixteenth of them
    gives a sixteenth of the result."""
    import mixture_experts_layer_fp32_gb300 as moe
    T, h, f = 5, 256, 2 ** 17
    g = torch.Generator(device="cuda").manual_seed(1)
    some = lambda *s, std: torch.empty(  # noqa: E731
        s, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)
    x, Wg = some(T, h, std=1), torch.zeros(h, 1, device="cuda")
    W1, W3, W2 = some(h, f, std=h ** -0.5), some(h, f, std=h ** -0.5), some(f, h, std=f ** -0.5)
    y = []
    for n in (1, 16):
        cfg = moe.config(T=T, h=h, E=1, k=1, f=n * f)
        ws = moe.alloc_workspace_few(cfg)
        y.append(torch.empty_like(x))
        moe.forward_few(cfg, x, Wg, None, None, W1.repeat(1, n)[None], W3.repeat(1, n)[None],
                        W2.repeat(n, 1)[None], y[-1], ws)
        moe.check(ws)
    a, b = 16 * y[0].double(), y[1].double()
    # sums of 2^21 products, each step of a chain off by 2^-23 of what it has, the chains cut among
    # the blocks; one rounding to bf16 each: two of its half steps and what the sums are off
    size = float(a.abs().max())
    assert float((a - b).abs().max()) <= 2 * 2.0 ** -8 * size + 2.0 ** -23 * (2 ** 21 / 16) * size
    assert size > 1


@pytest.mark.parametrize("M", [1, 9, 20])
def test_product_with_the_most_outputs(M):
    import mixture_experts_layer_fp32_gb300 as moe
    N, K = 2 ** 28, 16
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device="cuda",  # noqa: E731
                                     generator=g)
    wq, xq = codes(N, K), codes(M, K)
    ws = torch.rand(N, device="cuda", generator=g)
    xs = torch.rand(M, device="cuda", generator=g)
    w = moe.I8Weight(wq, ws)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    room = moe.alloc_workspace_linear_i8(M, w)
    moe.linear_i8(xq, w, y, room, x_scale=xs)
    moe.check(room)
    for at in (0, 2 ** 27 - 100, N - 1000):
        part = slice(at, at + 1000)
        whole = xq.double() @ wq[part].double().t()
        assert torch.equal(y[:, part], (whole.float() * xs[:, None] * ws[part]).to(y.dtype))


@pytest.mark.parametrize("coded", [True, False])
def test_product_with_the_most_rows(coded):
    import mixture_experts_layer_fp32_gb300 as moe
    M, N, K = 2 ** 28, 3, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    wq = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    ws = torch.rand(N, device="cuda", generator=g)
    w = moe.I8Weight(wq, ws)
    if coded:
        x = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
        xs = torch.rand(M, device="cuda", generator=g)
    else:
        x, xs = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g), None
    y = torch.empty(M, N, device="cuda")
    room = moe.alloc_workspace_linear_i8(M, w)
    moe.linear_i8(x, w, y, room, x_scale=xs)
    moe.check(room)
    for at in (0, 2 ** 27 - 100, M - 1000):
        part = slice(at, at + 1000)
        xq, s = x[part], None if xs is None else xs[part]
        if not coded:
            xq, s = torch.empty_like(xq, dtype=torch.int8), torch.empty(1000, device="cuda")
            moe.quantize_rows_i8(x[part].contiguous(), xq, s)
        whole = xq.double() @ wq.double().t()
        assert torch.equal(y[part], whole.float() * s[:, None] * ws)
