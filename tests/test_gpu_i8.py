"""8-bit integers on the GPU: quantising and the product.  Both are defined to the bit: codes are
the nearest whole number of the exact quotient, sums are whole, and each rounding after them is
named; so everything here is equality, but for a bias (fma, half a step of fp32)."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def quantised(x):
    """Codes and scales by the definition, in 64 bits (a quotient of two fp32 numbers that is not
    half of an odd number is further from one than 64 bits lose)."""
    x = x.float()
    s = x.abs().amax(-1) * torch.tensor(1 / 127, dtype=torch.float32, device=x.device)
    bad = ~torch.isfinite(x).all(-1)
    safe = torch.where((s > 0) & ~bad, s, 1.0)
    q = torch.round(x.double() / safe.double()[..., None]).clamp(-127, 127)
    q = torch.where(((s > 0) & ~bad)[..., None], q, 0.0)
    return q.to(torch.int8), torch.where(bad, float("nan"), s)


def product(xq, xs, wq, ws, out, bias=None):
    whole = xq.double() @ wq.double().t()  # exact: below 2^31
    y = whole.float() * xs[:, None]
    if bias is None:
        return (y * ws).to(out)
    return y.double() * ws.double() + bias.double()


def codes(shape, seed, top=127):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top - (top == 127), top + 1, shape, dtype=torch.int8, device="cuda",
                         generator=g)


def scales(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1e-3 * (0.1 + torch.rand(n, device="cuda", generator=g))


def linear(x, wq, ws, out, x_scale=None, bias=None, workspace=None):
    import mixture_experts_layer_fp32_gb300 as moe
    w = moe.I8Weight(wq, ws)
    m, n = x.shape[0], w.n
    room = torch.full((m * n + 128,), 7.0, dtype=out, device="cuda")
    y = room[64:64 + m * n].view(m, n)
    workspace = moe.alloc_workspace_linear_i8(m, w) if workspace is None else workspace
    moe.linear_i8(x, w, y, workspace, x_scale=x_scale, bias=bias)
    moe.check(workspace)
    assert room[:64].eq(7).all() and room[64 + m * n:].eq(7).all()
    return y


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (7, 1040), (2, 4096), (5, 8208), (300, 256),
                                    (2, 131056)])
def test_quantise(rows, K, dtype):
    import mixture_experts_layer_fp32_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn(rows, K, device="cuda", generator=g)
    x[0] *= 1e-20
    x[-1, 5:9] = 100.0
    x = x.to(DT[dtype])
    q = torch.full(x.shape, 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), 7.0, device="cuda")
    moe.quantize_rows_i8(x, q, s)
    rq, rs = quantised(x)
    assert torch.equal(s, rs) and torch.equal(q, rq)
    w = moe.quantize_i8(x)
    assert torch.equal(w.codes, rq) and torch.equal(w.scales, rs)


def test_quantise_borders_and_special_values():
    """Quotients that are a half of an odd number go to the even code; zeros, the smallest and
    largest numbers, infinities and NaN."""
    import mixture_experts_layer_fp32_gb300 as moe
    K, rows = 256, 12
    half = torch.arange(-127, 128, device="cuda").float() / 2
    x = torch.zeros(rows, K, device="cuda")
    x[0, :255], x[0, 255] = half, 127.0
    x[1] = x[0] * 2.0 ** -100
    x[2] = x[0] * 2.0 ** -130                                     # a scale below the normal ones
    x[3] = x[0] * 2.0 ** -142
    x[5] = x[0] * 2.0 ** 120
    x[6, 3] = torch.finfo(torch.float32).max
    x[7, 9] = float("inf")
    x[8, 200], x[8, 1] = float("nan"), 5.0
    x[9] = 1e-45
    g = torch.Generator(device="cuda").manual_seed(1)
    x[10:] = torch.randn(2, K, device="cuda", generator=g)
    x[11, 7] = -9.0
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    moe.quantize_rows_i8(x, q, s)
    rq, rs = quantised(x)
    assert torch.equal(torch.isnan(s), torch.isnan(rs))
    assert torch.equal(s.nan_to_num(-1), rs.nan_to_num(-1))
    assert torch.equal(q, rq)
    assert int(q[0, 130]) == 2 and int(q[0, 128]) == 0            # 1.5 -> 2, 0.5 -> 0


SHAPES = [(1, 1, 16), (1, 17, 64), (1, 4096, 512), (2, 33, 48), (5, 16, 1040), (8, 100, 4112),
          (9, 40, 128), (13, 1437, 720), (16, 256, 1024), (17, 300, 2064), (31, 129, 1152),
          (33, 130, 4096), (64, 511, 1536), (65, 257, 1040), (100, 128, 8208), (129, 1000, 256),
          (200, 300, 3088), (257, 513, 1168), (300, 64, 16)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_of_codes(M, N, K, out):
    xq, wq, xs, ws = codes((M, K), M + K), codes((N, K), N), scales(M, M), scales(N, N)
    y = linear(xq, wq, ws, DT[out], x_scale=xs)
    assert torch.equal(y, product(xq, xs, wq, ws, DT[out]))


@pytest.mark.parametrize("M,N,K", [(1, 40, 131056), (20, 40, 131056), (70, 300, 16384),
                                   (300, 260, 16400)])
def test_sums_past_what_fp32_holds(M, N, K):
    """All codes at their ends: sums near 2^31."""
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wq[::2] = 127
    xq[:, 3], wq[:, 5] = 1, 1
    xs, ws = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y = linear(xq, wq, ws, torch.float32, x_scale=xs)
    assert torch.equal(y, product(xq, xs, wq, ws, torch.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES[:14])
def test_product_of_values(M, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M * N)
    x = torch.randn(M, K, device="cuda", generator=g).to(DT[dtype])
    wq, ws = codes((N, K), N), scales(N, N)
    y = linear(x, wq, ws, torch.float32)
    xq, xs = quantised(x)
    assert torch.equal(y, product(xq, xs, wq, ws, torch.float32))


@pytest.mark.parametrize("M,N,K", [(1, 33, 80), (12, 513, 1024), (150, 260, 528)])
def test_bias(M, N, K):
    xq, wq, xs, ws = codes((M, K), M + K), codes((N, K), N), scales(M, M), scales(N, N)
    g = torch.Generator(device="cuda").manual_seed(5)
    bias = torch.randn(N, device="cuda", generator=g)
    y = linear(xq, wq, ws, torch.float32, x_scale=xs, bias=bias)
    want = product(xq, xs, wq, ws, None, bias)
    assert bool(((y.double() - want).abs() <= 2.0 ** -24 * want.abs() * (1 + 1e-6) + 1e-30).all())
    y16 = linear(xq, wq, ws, torch.bfloat16, x_scale=xs, bias=bias)
    assert torch.equal(y16, y.to(torch.bfloat16))


def test_rows_that_are_not_numbers_stay_alone():
    x = torch.randn(20, 64, device="cuda")
    x[3, 5], x[17, 9] = float("inf"), float("nan")
    wq, ws = codes((50, 64), 1), scales(50, 1)
    y = linear(x, wq, ws, torch.float32)
    bad = torch.zeros(20, dtype=torch.bool)
    bad[3] = bad[17] = True
    assert torch.equal(torch.isnan(y).all(1).cpu(), bad)
    assert torch.equal(torch.isnan(y).any(1).cpu(), bad)


def test_no_rows_and_a_workspace_of_more():
    import mixture_experts_layer_fp32_gb300 as moe
    wq, ws = codes((70, 256), 1), scales(70, 1)
    w = moe.I8Weight(wq, ws)
    room = moe.alloc_workspace_linear_i8(300, w)
    for M in (300, 64, 20, 9, 1, 0):
        x = torch.randn(M, 256, device="cuda")
        y = linear(x, wq, ws, torch.float32, workspace=room)
        xq, xs = quantised(x) if M else (x, x[:, 0])
        assert M == 0 or torch.equal(y, product(xq, xs, wq, ws, torch.float32))


def test_weights_just_quantised_are_read():
    """The product follows the quantising of its weights at once, many times."""
    import mixture_experts_layer_fp32_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(1)
    W = [torch.randn(4096, 1024, device="cuda", generator=g) for _ in range(4)]
    w = moe.quantize_i8(W[0])
    for M in (1, 8, 12, 40, 200):
        xq, xs = codes((M, 1024), M), scales(M, M)
        y = torch.empty(M, 4096, device="cuda")
        ws = moe.alloc_workspace_linear_i8(M, w)
        for i in range(12):
            moe.quantize_rows_i8(W[i % 4], w.codes, w.scales)
            moe.linear_i8(xq, w, y, ws, x_scale=xs)
            got = y.clone()
            wq, wsc = quantised(W[i % 4])
            assert torch.equal(got, product(xq, xs, wq, wsc, torch.float32))


@pytest.mark.parametrize("M,N,K", [(260, 4400, 272), (1000, 700, 2000), (70, 9000, 144),
                                   (2000, 129, 400), (640, 2049, 1040)])
def test_several_rounds_of_items(M, N, K):
    xq, wq, xs, ws = codes((M, K), M + K), codes((N, K), N), scales(M, M), scales(N, N)
    y = linear(xq, wq, ws, torch.float32, x_scale=xs)
    assert torch.equal(y, product(xq, xs, wq, ws, torch.float32))


@pytest.mark.parametrize("M,K", [(1, 1024), (8, 4096), (12, 512), (50, 2048), (200, 1024)])
def test_replays_in_graphs_that_share_a_workspace(M, K):
    import mixture_experts_layer_fp32_gb300 as moe
    N = 1100
    w = moe.I8Weight(codes((N, K), N), scales(N, N))
    g = torch.Generator(device="cuda").manual_seed(M)
    xs = [torch.randn(M, K, device="cuda", generator=g) for _ in range(2)]
    ys = [torch.empty(M, N, device="cuda") for _ in range(2)]
    ws = moe.alloc_workspace_linear_i8(M, w)
    moe.linear_i8(xs[0], w, ys[0], ws)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graphs = []
    for x, y in zip(xs, ys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            moe.linear_i8(x, w, y, ws)
    for seed in range(3):
        for i in range(2):
            xs[i].copy_(torch.randn(M, K, device="cuda", generator=g))
            ys[i].fill_(float("nan"))
            graphs[i].replay()
        torch.cuda.synchronize()
        moe.check(ws)
        for x, y in zip(xs, ys):
            xq, sc = quantised(x)
            assert torch.equal(y, product(xq, sc, w.codes, w.scales, torch.float32))


def test_two_streams_at_once():
    import mixture_experts_layer_fp32_gb300 as moe
    N, K = 2000, 2048
    w = moe.I8Weight(codes((N, K), N), scales(N, N))
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = [torch.randn(M, K, device="cuda", generator=g) for M in (3, 40, 300)]
    ys = [torch.empty(x.shape[0], N, device="cuda") for x in xs]
    room = [moe.alloc_workspace_linear_i8(x.shape[0], w) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, y, ws, s in zip(xs, ys, room, streams):
            with torch.cuda.stream(s):
                moe.linear_i8(x, w, y, ws)
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        xq, sc = quantised(x)
        assert torch.equal(y, product(xq, sc, w.codes, w.scales, torch.float32))


def test_last_dimension_and_leading_ones():
    import mixture_experts_layer_fp32_gb300 as moe
    w = moe.I8Weight(codes((96, 128), 1), scales(96, 1))
    x = torch.randn(2, 3, 5, 128, device="cuda").to(torch.bfloat16)
    y = torch.empty(2, 3, 5, 96, device="cuda")
    moe.linear_i8(x, w, y, moe.alloc_workspace_linear_i8(30, w))
    xq, xs = quantised(x.view(30, 128))
    assert torch.equal(y.view(30, 96), product(xq, xs, w.codes, w.scales, torch.float32))


def test_results_past_32_bits():
    """70000 x 32768 results: the last rows' are those of a call of their own."""
    import mixture_experts_layer_fp32_gb300 as moe
    M, N, K = 70000, 32768, 48
    xq, xs, wq, ws = codes((M, K), 1), scales(M, 2), codes((N, K), 3), scales(N, 4)
    w = moe.I8Weight(wq, ws)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    workspace = moe.alloc_workspace_linear_i8(M, w)
    moe.linear_i8(xq, w, y, workspace, x_scale=xs)
    moe.check(workspace)
    for r in (0, 65535, M - 100):
        part = slice(r, r + 100)
        assert torch.equal(y[part], product(xq[part], xs[part], wq, ws, torch.bfloat16))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K,N", [(6, 512, 100), (12, 4096, 300), (150, 1040, 260)])
def test_against_the_quotient_by_127_in_64_bits(rows, K, N, dtype):
    """The scale by its own formula, max / 127: fp32's 1 / 127 and the product are off by half a
    step each, 2^-23 together.  A code is the nearest whole number over that scale, so it stands for
    its value within half a scale; 127 times 2^-22 of one more where the largest is cut to 127.  And
    so a product of values is off by no more than what the codes are, its sum's rounding to fp32 and
    the two products', half a step each."""
    import mixture_experts_layer_fp32_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(rows * K)
    x = (torch.randn(rows, K, device="cuda", generator=g) *
         torch.rand(rows, 1, device="cuda", generator=g) * 10).to(DT[dtype])
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    moe.quantize_rows_i8(x, q, s)
    exact = x.double().abs().amax(1) / 127
    assert bool(((s.double() - exact).abs() <= 2.0 ** -23 * (1 + 1e-6) * exact).all())
    most = s.double()[:, None] * (0.5 + 127 * 2.0 ** -22)
    assert bool(((q.double() * s.double()[:, None] - x.double()).abs() <= most).all())
    assert int(q.abs().amax(1).min()) == 127
    wq, ws = codes((N, K), N), scales(N, N)
    y = linear(x, wq, ws, torch.float32).double()
    W = wq.double() * ws.double()[:, None]
    want = x.double() @ W.t()
    off = most * W.abs().sum(1)
    assert bool(((y - want).abs() <= off + 3 * 2.0 ** -24 * (want.abs() + off)).all())
