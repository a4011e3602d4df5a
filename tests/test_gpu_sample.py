"""Sampling (moe_sample) against its definition in 64 bits (decode_cases).

A weight is off by 2^-18 relative at most (the difference, the quotient by the temperature of up to
30 nats where it still counts, exp: 30 * 2u + 4u = 64 u = 2^-18 = 4e-6) and a sum of them by no more,
so an answer whose borders are further away than 1e-5 of the mass has to be met exactly.  Closer
ones: top_p's border may fall on other tokens within 1e-5 of the mass, so that a running sum moves by
less than 2e-5 and its share of the total by 4e-5; the token lies between those of u - 5e-5 and
u + 5e-5.  (min_p's border is no matter of mass: rows with a weight within 1e-5 of it are left out.)"""

import numpy as np
import pytest
import torch

from decode_cases import sample_ref

pytestmark = pytest.mark.gpu
GAP = 1e-5


def run(logits, u, prob=True, **choices):
    import mixture_experts_layer_fp32_gb300 as moe
    rows = logits.shape[0]
    room = torch.full((rows + 8,), -9, dtype=torch.int32, device="cuda")
    tokens = room[4:4 + rows]
    p = torch.full((rows,), float("nan"), device="cuda") if prob else None
    moe.sample(logits, u, tokens, prob=p, **choices)
    assert room[:4].eq(-9).all() and room[4 + rows:].eq(-9).all()
    return tokens.cpu().numpy(), None if p is None else p.double().cpu().numpy()


def verify(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The answers of all rows."""
    rows = logits.shape[0]
    got, prob = run(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    each = [np.broadcast_to(v.cpu().numpy() if isinstance(v, torch.Tensor) else np.asarray(v), rows)
            for v in (temperature, top_k, top_p, min_p)]
    l, uu = logits.double().cpu().numpy(), u.double().cpu().numpy()
    for r in range(rows):
        t, k, p, m = (float(v[r]) for v in each)
        rest = np.float32(t).item(), int(k), np.float32(p).item(), np.float32(m).item()
        token, share, gap, gap_min = sample_ref(l[r], uu[r], *rest)
        if gap_min < GAP:
            continue
        if gap < GAP:
            low, high = (sample_ref(l[r], uu[r] + d, *rest)[0] for d in (-5e-5, 5e-5))
            assert low <= got[r] <= high, (r, got[r], low, high)
            continue
        assert got[r] == token, (r, got[r], token)
        assert abs(prob[r] - share) <= 2e-5 * share + 1e-9


def draw(rows, V, seed, dtype=torch.float32, std=2.5):
    g = torch.Generator().manual_seed(seed)
    l = std * torch.randn(rows, V, generator=g) + 5 * (torch.rand(rows, V, generator=g) < 8 / V)
    u = torch.rand(rows, generator=g)
    return l.to(dtype).cuda(), u.cuda()


CHOICES = [dict(), dict(temperature=0.0), dict(top_k=1), dict(temperature=0.7, top_k=40),
           dict(top_p=0.9), dict(temperature=1.5, top_p=0.5), dict(min_p=0.05),
           dict(temperature=0.5, top_k=100, top_p=0.95, min_p=0.01), dict(top_p=0.0),
           dict(min_p=1.0), dict(top_k=10 ** 6, top_p=0.999), dict(top_k=7, top_p=0.6)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", CHOICES, ids=str)
@pytest.mark.parametrize("rows,V", [(3, 1), (9, 2), (16, 33), (12, 1009), (7, 4096), (5, 8191),
                                    (4, 32001)])
def test_choices(rows, V, kw, dtype):
    logits, u = draw(rows, V, 7 * V + rows, dtype)
    verify(logits, u, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V", [(1, 151936), (2, 128000), (2, 262147)])
def test_large_vocabulary(rows, V, dtype):
    for i, kw in enumerate([dict(temperature=0.8, top_p=0.9), dict(top_k=50, top_p=0.95),
                            dict(temperature=1.2, top_k=5000), dict(min_p=0.02)]):
        logits, u = draw(rows, V, V + i, dtype)
        verify(logits, u, **kw)


def test_each_row_its_own():
    rows, V = 40, 5000
    logits, u = draw(rows, V, 5)
    g = torch.Generator().manual_seed(6)
    t = (2 * torch.rand(rows, generator=g)).cuda()
    t[::5] = 0.0
    k = torch.randint(0, 60, (rows,), generator=g, dtype=torch.int32).cuda()
    p = torch.rand(rows, generator=g).cuda()
    p[::3] = 1.0
    m = (0.2 * torch.rand(rows, generator=g)).cuda()
    verify(logits, u, temperature=t, top_k=k, top_p=p, min_p=m)


@pytest.mark.parametrize("V", [5, 3000, 70000])
def test_equal_logits_go_by_index(V):
    """All logits equal, and few values: borders inside runs of equal logits."""
    logits = torch.zeros(6, V, device="cuda")
    u = torch.tensor([0.0, 0.1, 0.33, 0.7, 0.95, 0.999], device="cuda")
    got, prob = run(logits, u)
    want = np.floor(u.double().cpu().numpy() * V).astype(int)
    assert np.array_equal(got, want) and np.allclose(prob, 1 / V, rtol=1e-6)
    k = max(1, V // 3)
    got, prob = run(logits, u, top_k=k)
    assert np.array_equal(got, np.floor(u.double().cpu().numpy() * k).astype(int))
    got, prob = run(logits, u, top_p=0.5)
    n = -(-V // 2)
    assert np.array_equal(got, np.floor(u.double().cpu().numpy() * n).astype(int))
    g = torch.Generator().manual_seed(V)
    few = torch.randint(0, 3, (8, V), generator=g).float()
    for kw in (dict(top_k=k), dict(top_p=0.3), dict(top_k=k, top_p=0.8), dict(top_p=0.97)):
        verify(few.cuda(), torch.rand(8, generator=g).cuda(), **kw)


def test_masked_and_special_values():
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    rows = torch.tensor([[-inf, -inf, -inf, -inf], [nan, nan, -inf, nan], [low, low, low, low],
                         [nan, 1.0, nan, -inf], [inf, 0.0, inf, nan], [-inf, low, 3.0, -inf],
                         [-0.0, 0.0, -0.0, -5.0]], device="cuda")
    u = torch.tensor([0.5, 0.5, 0.6, 0.9, 0.7, 0.99, 0.4], device="cuda")
    for kw in (dict(), dict(top_k=3), dict(top_p=0.99), dict(top_k=3, top_p=0.99, min_p=0.1)):
        got, prob = run(rows, u, **kw)
        assert list(got[:2]) == [-1, -1] and list(prob[:2]) == [0.0, 0.0]
        assert got[3] == 1 and got[4] == 2 and got[5] == 2
        assert got[2] == (2 if not kw else 1) or got[2] == int(0.6 * (3 if "top_k" in kw else 4))
    got, prob = run(rows, u, temperature=0.0)
    assert list(got) == [-1, -1, 0, 1, 0, 2, 0]
    # random numbers outside [0, 1), and none at all
    one = torch.zeros(4, 10, device="cuda")
    got, _ = run(one, torch.tensor([-1.0, 1.0, 2.0, nan], device="cuda"))
    assert list(got) == [0, 9, 9, 0]
    got, _ = run(one[:0], u[:0])
    assert got.size == 0


def test_choices_of_a_row_outside_their_ranges():
    inf, nan = float("inf"), float("nan")
    logits = torch.tensor([[1.0, 3.0, 2.0]], device="cuda").expand(6, 3).contiguous()
    u = torch.full((6,), 0.999, device="cuda")
    f = lambda *v: torch.tensor(v, device="cuda")  # noqa: E731
    got, _ = run(logits, u, temperature=f(-1.0, nan, inf, 0.0, 1e-30, 1.0))
    assert list(got) == [1, 1, 2, 1, 1, 2]
    got, _ = run(logits, u, top_p=f(-1.0, nan, 2.0, 0.0, 1.0, 0.1))
    assert list(got) == [1, 2, 2, 1, 2, 1]
    got, _ = run(logits, u, min_p=f(-1.0, nan, 2.0, 0.0, 1.0, 0.5))
    assert list(got) == [2, 2, 1, 2, 1, 1]
    got, _ = run(logits, u, top_k=torch.tensor([-5, 0, 1, 2, 3, 100], dtype=torch.int32,
                                               device="cuda"))
    assert list(got) == [2, 2, 1, 2, 2, 2]
    assert run(logits, u, prob=False)[1] is None


def test_a_row_alone_is_the_row_in_a_batch():
    for V in (1001, 40000):
        logits, u = draw(200, V, V)
        kw = dict(temperature=0.9, top_k=300, top_p=0.9)
        got, prob = run(logits, u, **kw)
        again, p2 = run(logits, u, **kw)
        assert np.array_equal(got, again) and np.array_equal(prob, p2)
        for r in (0, 57, 199):
            g1, p1 = run(logits[r:r + 1].clone(), u[r:r + 1].clone(), **kw)
            assert g1[0] == got[r] and p1[0] == prob[r]


def test_row_too_long_for_shared_memory():
    V = 800001
    logits, u = draw(2, V, 3, std=1.0)
    verify(logits, u, top_k=20)
    got, _ = run(logits, u, top_p=0.9)
    l = logits.double()
    order = l.sort(dim=1, descending=True, stable=True)
    w = torch.exp(order[0] - order[0][:, :1])
    cum = w.cumsum(1)
    w = w * (cum - w < 0.9 * cum[:, -1:])
    at = torch.zeros_like(w).scatter_(1, order[1], w).cumsum(1)
    for r in range(2):   # a token's share here is 1e-6: within two of it
        lo, hi = (float(at[r, max(0, int(got[r]) + d)] / at[r, -1]) for d in (-2000, 2000))
        assert lo <= float(u[r]) <= hi


def test_replays_in_a_graph_on_another_stream():
    import mixture_experts_layer_fp32_gb300 as moe
    logits, u = draw(8, 20000, 1)
    tokens = torch.zeros(8, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        moe.sample(logits, u, tokens, top_k=50, top_p=0.9)
        stream.synchronize()
        with torch.cuda.graph(g, stream=stream):
            moe.sample(logits, u, tokens, top_k=50, top_p=0.9)
    for seed in range(3):
        l2, u2 = draw(8, 20000, 10 + seed)
        logits.copy_(l2), u.copy_(u2)
        g.replay()
        torch.cuda.synchronize()
        want, _ = run(l2, u2, top_k=50, top_p=0.9)
        assert np.array_equal(tokens.cpu().numpy(), want)


def test_many_rows():
    """More rows than a grid has in one direction."""
    rows, V = 70001, 3
    logits, u = draw(rows, V, 9)
    got, _ = run(logits, u, top_k=2)
    l = logits.double()
    order = l.sort(dim=1, descending=True, stable=True)
    w = torch.exp(l - order[0][:, :1])
    w = torch.where(torch.zeros_like(w).scatter_(1, order[1][:, :2], 1.0) > 0, w, 0.0)
    cum = w.cumsum(1)
    at = u.double()[:, None] * cum[:, -1:]
    want = (cum <= at).sum(1)
    close = ((cum - at).abs() < 1e-5 * cum[:, -1:]).any(1)
    assert bool(((torch.from_numpy(got).cuda() == want) | close).all())
    assert float(close.double().mean()) < 0.01


def test_streams_at_once():
    import mixture_experts_layer_fp32_gb300 as moe
    sets = [draw(r, V, V) for r, V in ((1, 100000), (30, 4000), (64, 20000))]
    kw = dict(top_k=100, top_p=0.9, temperature=0.8)
    want = [run(l, u, **kw)[0] for l, u in sets]
    out = [torch.empty(l.shape[0], dtype=torch.int32, device="cuda") for l, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for (l, u), o, s in zip(sets, out, streams):
            with torch.cuda.stream(s):
                moe.sample(l, u, o, **kw)
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert np.array_equal(o.cpu().numpy(), w)


def test_logits_past_32_bits():
    """20000 rows of 120001: the last rows' tokens are those of a call of their own."""
    rows, V = 20000, 120001
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.empty(rows, V, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    u = torch.rand(rows, device="cuda", generator=g)
    kw = dict(temperature=0.8, top_k=50, top_p=0.9)
    got, prob = run(logits, u, **kw)
    # 2400020000 logits: the last 16 rows, and those around the 2^31st
    for r in (rows - 16, 2 ** 31 // V - 8):
        l, v = logits[r:r + 16].clone(), u[r:r + 16].clone()
        want, p = run(l, v, **kw)
        assert np.array_equal(got[r:r + 16], want) and np.array_equal(prob[r:r + 16], p)
