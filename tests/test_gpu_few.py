"""The whole layer for few tokens (moe_forward_few) against a reference in 64 bits
(decode_cases): routing exact, outputs within bounds derived there."""

import numpy as np
import pytest
import torch

from decode_cases import LayerCase, assert_close

pytestmark = pytest.mark.gpu


def call(c, y=None, ws=None, x=None):
    import mixture_experts_layer_fp32_gb300 as moe
    cfg = moe.config(T=c.T, h=c.h, E=c.E, k=c.k, f=c.f, score=c.score, dtype=c.dtype,
                     capacity_factor=c.capacity, drop_policy=c.policy,
                     min_capacity=c.min_capacity, num_groups=c.groups, group_topk=c.group_topk)
    x = c.x if x is None else x
    y = torch.full_like(c.x, float("nan")) if y is None else y
    ws = moe.alloc_workspace_few(cfg, c.fs) if ws is None else ws
    idx = torch.full((c.T, c.k), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((c.T, c.k), float("nan"), device="cuda")
    tpe = torch.full((c.E,), -7, dtype=torch.int32, device="cuda")
    moe.forward_few(cfg, x, c.Wg, c.gb, c.eb, c.W1, c.W3, c.W2, y, ws, topk_idx=idx,
                    topk_prob=prob, tokens_per_expert=tpe, shared=c.shared)
    moe.check(ws)
    return y, idx, prob, tpe, ws, cfg


def verify(c, out):
    y, idx, prob, tpe = out[:4]
    ri, rp, rt, ry, bound = c.reference()
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(tpe.cpu().numpy(), rt)
    p = prob.double().cpu().numpy()
    assert np.array_equal(p > 0, rp > 0)
    assert (np.abs(p - rp) <= 1e-5 * rp + 1e-6).all()
    assert_close(y, ry, bound, c.dt)


BF16 = [
    dict(T=1, h=256, E=1, k=1, f=128),
    dict(T=1, h=512, E=8, k=2, f=384),
    dict(T=2, h=1024, E=5, k=3, f=640),
    dict(T=7, h=768, E=12, k=4, f=256, score="sigmoid", expert_bias=True),
    dict(T=8, h=256, E=64, k=8, f=128, score="sqrtsoftplus", expert_bias=True),
    dict(T=9, h=2048, E=32, k=4, f=128, groups=8, group_topk=2),
    dict(T=17, h=512, E=256, k=8, f=256, groups=8, group_topk=4, score="sigmoid",
         expert_bias=True, fs=256),
    dict(T=31, h=256, E=4, k=1, f=1408, score="softmax_pre", capacity=1.0),
    dict(T=33, h=256, E=2, k=2, f=256, fs=384),
    dict(T=48, h=512, E=16, k=2, f=384, capacity=1.25, policy="position", fs=128),
    dict(T=64, h=256, E=8, k=8, f=128, capacity=0.5),
    dict(T=64, h=512, E=3, k=1, f=512, score="softmax_pre", fs=512),
    dict(T=64, h=256, E=100, k=8, f=128, gate_bias=False),
    dict(T=64, h=256, E=24, k=2, f=256, same=True),
    dict(T=3, h=7168, E=8, k=2, f=256),
    dict(T=5, h=256, E=4, k=2, f=8192),
]
F32 = [
    dict(T=1, h=8, E=1, k=1, f=8),
    dict(T=1, h=128, E=8, k=2, f=256),
    dict(T=3, h=24, E=7, k=2, f=40, fs=16),
    dict(T=7, h=1032, E=12, k=3, f=1416, score="sigmoid", expert_bias=True),
    dict(T=16, h=136, E=16, k=4, f=264, groups=4, group_topk=2, fs=520),
    dict(T=33, h=200, E=3, k=2, f=72, capacity=1.0),
    dict(T=64, h=512, E=5, k=1, f=520, score="softmax_pre", capacity=0.7, policy="position"),
    dict(T=64, h=64, E=256, k=8, f=16),
    dict(T=64, h=72, E=2, k=2, f=1000, fs=24),
]


@pytest.mark.parametrize("kw", BF16, ids=str)
def test_bf16(kw):
    c = LayerCase(**kw).cuda()
    verify(c, call(c))


@pytest.mark.parametrize("kw", F32, ids=str)
def test_f32(kw):
    c = LayerCase(dtype="f32", **kw).cuda()
    verify(c, call(c))


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a[:4], b[:4]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_and_a_workspace_of_more_tokens(dtype):
    """Equal bits again and again, in a workspace of 64 tokens that other calls used before."""
    import mixture_experts_layer_fp32_gb300 as moe
    kw = dict(h=512, E=16, k=4, f=640, fs=128, dtype=dtype)
    most = moe.config(T=64, h=512, E=16, k=4, f=640, dtype=dtype)
    ws = moe.alloc_workspace_few(most, 128)
    for T in (64, 1, 33, 4, 5, 9, 64, 2):
        c = LayerCase(T=T, seed=T, **kw).cuda()
        first = call(c)
        verify(c, first)
        for _ in range(3):
            assert same(first, call(c, ws=ws))


def test_a_token_alone_is_the_token_in_a_batch():
    """Its row does not depend on the others in value, but for how sums are cut: within the bounds
    of both."""
    c = LayerCase(T=12, h=512, E=8, k=2, f=384).cuda()
    y = call(c)[0]
    for t in (0, 5, 11):
        one = LayerCase(T=1, h=512, E=8, k=2, f=384).cuda()
        for n in ("Wg", "gb", "W1", "W3", "W2"):
            setattr(one, n, getattr(c, n))
        one.x = c.x[t:t + 1].clone()
        out = call(one)
        verify(one, out)
        ref, bound = one.reference()[3:]
        assert bool(((out[0].double() - y[t:t + 1].double()).abs() <=
                     2 * (bound + 2.0 ** -8 * (ref.abs() + bound))).all())


def test_output_in_place_of_the_input_and_nothing_optional():
    import mixture_experts_layer_fp32_gb300 as moe
    c = LayerCase(T=9, h=512, E=8, k=2, f=384, fs=256).cuda()
    want = call(c)[0]
    x = c.x.clone()
    cfg = moe.config(T=9, h=512, E=8, k=2, f=384)
    ws = moe.alloc_workspace_few(cfg, 256)
    moe.forward_few(cfg, x, c.Wg, c.gb, None, c.W1, c.W3, c.W2, x, ws, shared=c.shared)
    moe.check(ws)
    assert torch.equal(x, want)


def test_no_tokens():
    import mixture_experts_layer_fp32_gb300 as moe
    cfg = moe.config(T=0, h=256, E=4, k=2, f=128)
    c = LayerCase(T=1, h=256, E=4, k=2, f=128).cuda()
    none = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    tpe = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    ws = moe.alloc_workspace_few(cfg)
    moe.forward_few(cfg, none, c.Wg, None, None, c.W1, c.W3, c.W2, none, ws,
                    tokens_per_expert=tpe)
    moe.check(ws)
    assert tpe.tolist() == [0] * 4


def test_only_the_hit_experts_weights_count():
    """What is not read cannot matter: experts that nobody chose hold NaN, and so do the shared
    weights' neighbours."""
    c = LayerCase(T=3, h=256, E=32, k=2, f=256, fs=128).cuda()
    first = call(c)
    hit = set(first[1].flatten().tolist())
    for e in range(32):
        if e not in hit:
            for w in (c.W1, c.W3, c.W2):
                w[e] = float("nan")
    assert same(first, call(c))


@pytest.mark.parametrize("T", [3, 40])
def test_rows_that_are_not_numbers_stay_alone(T):
    """A token with an infinity or a NaN spoils its own row; NaN logits are reported and named."""
    import mixture_experts_layer_fp32_gb300 as moe
    for dtype in ("bf16", "f32"):
        c = LayerCase(T=T, h=256, E=4, k=2, f=256, fs=128, dtype=dtype).cuda()
        clean = call(c)[0]
        x = c.x.clone()
        x[1, 5], x[2, 9] = float("nan"), float("inf")
        cfg = moe.config(T=T, h=256, E=4, k=2, f=256, dtype=dtype)
        ws = moe.alloc_workspace_few(cfg, 128)
        y = torch.zeros_like(x)
        idx = torch.empty((T, 2), dtype=torch.int32, device="cuda")
        for _ in range(2):
            moe.forward_few(cfg, x, c.Wg, c.gb, None, c.W1, c.W3, c.W2, y, ws, topk_idx=idx,
                            shared=c.shared)
            with pytest.raises(moe.MoeError) as err:
                moe.check(ws)
            assert err.value.code == 5
        assert bool(((idx >= 0) & (idx < 4)).all())
        rest = [t for t in range(T) if t not in (1, 2)]
        assert bool(torch.isfinite(y[rest]).all())
        assert float((y[rest].double() - clean[rest].double()).abs().max()) <= 2.0 ** -6 * float(
            clean.double().abs().max())
        assert bool(torch.isnan(y[1]).all())
        assert same(call(c), (clean,))


@pytest.mark.parametrize("kw", [dict(T=1, h=512, E=8, k=2, f=384),
                                dict(T=30, h=256, E=64, k=8, f=128, fs=128)], ids=str)
def test_replays_in_graphs_that_share_a_workspace(kw):
    import mixture_experts_layer_fp32_gb300 as moe
    c = LayerCase(**kw).cuda()
    cfg = moe.config(T=c.T, h=c.h, E=c.E, k=c.k, f=c.f)
    ws = moe.alloc_workspace_few(cfg, c.fs)
    ys = [torch.empty_like(c.x) for _ in range(2)]
    xs = [c.x.clone(), c.x.flip(0).contiguous()]

    def run(i):
        moe.forward_few(cfg, xs[i], c.Wg, c.gb, None, c.W1, c.W3, c.W2, ys[i], ws,
                        shared=c.shared)

    run(0)
    torch.cuda.synchronize()
    graphs = []
    stream = torch.cuda.Stream()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            run(i)
        graphs.append(g)
    want = call(c)[0]
    for _ in range(3):
        for i in range(2):
            ys[i].fill_(float("nan"))
            graphs[i].replay()
        torch.cuda.synchronize()
        moe.check(ws)
        assert torch.equal(ys[0], want)
    c.x = xs[1]
    assert torch.equal(ys[1], call(c)[0])


def test_two_streams_at_once():
    """Two calls in flight, each with a workspace of its own, beside other work."""
    import mixture_experts_layer_fp32_gb300 as moe
    cases = [LayerCase(T=T, h=1024, E=16, k=4, f=1024, seed=T).cuda() for T in (4, 20)]
    want = [call(c)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    cfgs = [moe.config(T=c.T, h=c.h, E=c.E, k=c.k, f=c.f) for c in cases]
    wss = [moe.alloc_workspace_few(cfg) for cfg in cfgs]
    ys = [torch.empty_like(c.x) for c in cases]
    a = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        for c, cfg, ws, y, s in zip(cases, cfgs, wss, ys, streams):
            with torch.cuda.stream(s):
                moe.forward_few(cfg, c.x, c.Wg, c.gb, None, c.W1, c.W3, c.W2, y, ws)
        a = a @ a * 1e-3
    torch.cuda.synchronize()
    for y, w, ws in zip(ys, want, wss):
        moe.check(ws)
        assert torch.equal(y, w)


def test_a_workspace_that_other_entry_points_used():
    import mixture_experts_layer_fp32_gb300 as moe
    c = LayerCase(T=16, h=256, E=8, k=2, f=256).cuda()
    want = call(c)[0]
    cfg = moe.config(T=16, h=256, E=8, k=2, f=256)
    ws = torch.zeros(max(moe.workspace_size(cfg), moe.workspace_size_few(cfg)), dtype=torch.uint8,
                     device="cuda")
    y = torch.empty_like(c.x)
    for _ in range(3):
        moe.forward(cfg, c.x, c.Wg, c.gb, None, c.W1, c.W3, c.W2, y, ws)
        full = y.clone()
        moe.forward_few(cfg, c.x, c.Wg, c.gb, None, c.W1, c.W3, c.W2, y, ws)
        moe.check(ws)
        assert torch.equal(y, want)
        # the layer rounds its hidden values to bf16 in between: 2e-2 of the output's RMS
        rms = float(want.double().square().mean().sqrt())
        assert float((full.double() - want.double()).abs().max()) <= 2e-2 * rms + \
            2.0 ** -7 * float(want.double().abs().max())


def test_a_wait_that_runs_out_is_reported():
    """Counters of the workspace that say the blocks have not come: every block gives up after a
    second, and the next call is well."""
    import mixture_experts_layer_fp32_gb300 as moe
    c = LayerCase(T=5, h=256, E=4, k=2, f=128).cuda()
    cfg = moe.config(T=5, h=256, E=4, k=2, f=128)
    want = call(c)[0]
    ws = moe.alloc_workspace_few(cfg)
    ws[128:132].view(torch.int32).fill_(-1000000)
    y = torch.empty_like(c.x)
    moe.forward_few(cfg, c.x, c.Wg, c.gb, None, c.W1, c.W3, c.W2, y, ws)
    with pytest.raises(moe.MoeError) as err:
        moe.check(ws)
    assert err.value.code == 6
    moe.forward_few(cfg, c.x, c.Wg, c.gb, None, c.W1, c.W3, c.W2, y, ws)
    moe.check(ws)
    assert torch.equal(y, want)


@pytest.mark.parametrize("kw", [
    dict(T=64, h=1024, E=256, k=8, f=128),                    # some 440 tiles of 4 units
    dict(T=48, h=1024, E=256, k=8, f=128, fs=256, score="sigmoid", expert_bias=True),
    dict(T=64, h=4096, E=48, k=8, f=384, capacity=0.5),
    dict(T=64, h=1024, E=256, k=8, f=128, same=True),         # room for pieces, eight experts
    dict(T=20, h=7168, E=32, k=8, f=128, fs=1408),            # long and short tiles
], ids=str)
def test_pieces_taken_in_turn(kw):
    """Where FC2 has many tiles its stream is taken in pieces: which block has which is not the
    same from call to call, the bits are."""
    c = LayerCase(**kw).cuda()
    out = call(c)
    verify(c, out)
    for _ in range(5):
        assert same(out, call(c, ws=out[4]))


def test_weights_past_32_bits():
    """Experts that lie more than 2^31 weights from the first give what a layer of those alone
    does: scores are sigmoids, so leaving out the others changes no weight."""
    import mixture_experts_layer_fp32_gb300 as moe
    T, h, E, f = 5, 4096, 136, 4096
    g = torch.Generator(device="cuda").manual_seed(1)

    def some(*shape, std):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)

    x, y = some(T, h, std=1), []
    Wg = some(h, E, std=h ** -0.5).float()
    W1, W3 = (some(E, h, f, std=h ** -0.5) for _ in range(2))
    W2 = some(E, f, h, std=f ** -0.5)
    bias = torch.zeros(E, device="cuda")
    bias[-2:] = 10
    for first in (0, E - 2):
        cfg = moe.config(T=T, h=h, E=E - first, k=2, f=f, score="sigmoid")
        ws = moe.alloc_workspace_few(cfg)
        idx = torch.empty(T, 2, dtype=torch.int32, device="cuda")
        y.append(torch.empty(T, h, dtype=torch.bfloat16, device="cuda"))
        moe.forward_few(cfg, x, Wg[:, first:].contiguous(), None, bias[first:].clone(), W1[first:],
                        W3[first:], W2[first:], y[-1], ws, topk_idx=idx)
        moe.check(ws)
        assert bool((idx + first >= E - 2).all())
    # fp32 sums in another order, one rounding each: a step of bf16 of the largest at most
    a, b = (v.double() for v in y)
    assert float((a - b).abs().max()) <= 2.0 ** -7 * float(a.abs().max())
    assert float(a.abs().max()) > 0.1


@pytest.mark.parametrize("kw", [
    dict(T=24, h=512, E=16, k=4, f=384),               # a tile of FC1 in several blocks' runs
    dict(T=64, h=2048, E=4, k=2, f=640, fs=256),       # long tiles, many blocks to each
    dict(T=9, h=264, E=8, k=2, f=520, dtype="f32"),
], ids=str)
def test_tiles_shared_by_blocks_repeat_bit_for_bit(kw):
    """A block's last tile of FC1 is mostly finished by another one, and its own warps go on to the
    next expert's hidden values at once."""
    c = LayerCase(**kw).cuda()
    out = call(c)
    verify(c, out)
    for _ in range(60):
        assert same(out, call(c, ws=out[4]))
