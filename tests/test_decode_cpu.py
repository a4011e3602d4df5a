"""The decoding step's entry points without a GPU: what the library refuses before anything is
enqueued, workspace sizes, and what the binding refuses and hands on."""

import ctypes

import pytest
import torch

from test_block_binding_cpu import moe as recorder  # noqa: F401

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE, ODD = 0x10000, 0x10008
BIG = 1 << 40
F32, BF16, I8 = 0, 1, 2


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_fp32_gb300 import build
    build.build()
    import mixture_experts_layer_fp32_gb300 as m
    return m


def few(moe, cfg, fs=0, size=BIG, **over):
    names = ("x", "Wg", "gb", "eb", "W1", "W3", "W2", "V1", "V3", "V2", "y", "idx", "prob", "tpe",
             "ws")
    a = dict.fromkeys(names, FAKE)
    a.update(gb=None, eb=None, idx=None, prob=None, tpe=None)
    if not fs:
        a.update(V1=None, V3=None, V2=None)
    a.update(over)
    return moe.lib().moe_forward_few(ctypes.byref(cfg), fs, *(a[n] for n in names), size, None)


def test_few_refusals(moe):
    ok = moe.config(T=8, h=256, E=4, k=2, f=128)
    need = moe.workspace_size_few(ok)
    assert few(moe, ok, size=need - 1) == WORKSPACE
    for name in ("x", "Wg", "W1", "W3", "W2", "y", "ws"):
        assert few(moe, ok, **{name: None}) == INVALID
        assert few(moe, ok, **{name: ODD}) == INVALID
    for name in ("gb", "eb", "idx", "prob", "tpe"):
        assert few(moe, ok, **{name: 0x10002}) == INVALID
    for name in ("V1", "V3", "V2"):
        assert few(moe, ok, fs=128, **{name: None}) == INVALID
    assert few(moe, ok, fs=-1) == INVALID
    assert few(moe, ok, fs=64) == UNSUPPORTED          # bf16: a multiple of 128
    assert few(moe, moe.config(T=65, h=256, E=4, k=2, f=128)) == UNSUPPORTED
    assert few(moe, moe.config(T=-1, h=256, E=4, k=2, f=128)) == INVALID
    assert few(moe, moe.config(T=8, h=264, E=4, k=2, f=128)) == UNSUPPORTED
    assert few(moe, moe.config(T=8, h=264, E=4, k=2, f=12, dtype="f32")) == UNSUPPORTED
    assert few(moe, moe.config(T=8, h=264, E=4, k=5, f=16, dtype="f32")) == UNSUPPORTED
    assert few(moe, moe.config(T=8, h=264, E=257, k=5, f=16, dtype="f32")) == UNSUPPORTED
    assert few(moe, moe.config(T=8, h=1 << 22, E=4, k=2, f=16, dtype="f32")) == UNSUPPORTED
    assert few(moe, moe.config(T=8, h=1 << 21, E=256, k=2, f=1 << 21, dtype="f32")) == UNSUPPORTED
    size = ctypes.c_size_t()
    assert moe.lib().moe_workspace_size_few(ctypes.byref(ok), 0, None) == INVALID
    assert moe.lib().moe_workspace_size_few(None, 0, ctypes.byref(size)) == INVALID


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_workspace_serves_fewer_tokens(moe, dtype):
    for fs in (0, 256):
        sizes = [moe.workspace_size_few(moe.config(T=T, h=512, E=16, k=4, f=384, dtype=dtype), fs)
                 for T in range(moe.FEW_MAX_TOKENS + 1)]
        assert sizes == sorted(sizes)


def linear(moe, rows=4, N=32, K=64, xt=BF16, yt=F32, size=BIG, **over):
    a = dict(x=FAKE, xs=FAKE if xt == I8 else None, W=FAKE, ws=FAKE, bias=None, y=FAKE, room=FAKE)
    a.update(over)
    return moe.lib().moe_linear_i8(rows, N, K, a["x"], xt, a["xs"], a["W"], a["ws"], a["bias"],
                                   a["y"], yt, a["room"], size, None)


def test_linear_refusals(moe):
    for name in ("x", "W", "y", "room"):
        assert linear(moe, **{name: None}) == INVALID
        assert linear(moe, **{name: ODD}) == INVALID
    assert linear(moe, ws=None) == INVALID
    assert linear(moe, bias=0x10002) == INVALID
    assert linear(moe, xt=I8, xs=None) == INVALID
    assert linear(moe, xt=BF16, xs=FAKE) == INVALID
    assert linear(moe, xt=3) == INVALID and linear(moe, yt=I8) == INVALID
    assert linear(moe, rows=-1) == INVALID and linear(moe, N=0) == INVALID
    assert linear(moe, K=0) == INVALID
    assert linear(moe, K=72) == UNSUPPORTED and linear(moe, K=131072) == UNSUPPORTED
    assert linear(moe, size=256) == WORKSPACE
    assert linear(moe, rows=0, x=None, y=None) == OK   # nothing to do, nothing enqueued


@pytest.mark.parametrize("N,K", [(1, 16), (100, 4096), (4096, 4096), (14337, 7168), (256, 128),
                                 (300, 131056)])
def test_linear_workspace_serves_fewer_rows(moe, N, K):
    """Every smaller call fits into the workspace of the largest, and just so: the sizes that the
    calls themselves ask for."""
    def fits(rows, size):
        # y NULL is refused before the workspace is looked at, a good y after
        return moe.lib().moe_linear_i8(rows, N, K, FAKE, I8, FAKE, FAKE, FAKE, None, FAKE, 7, FAKE,
                                       size, None)
    most = 0
    for rows in list(range(0, 70)) + [100, 128, 129, 200, 256, 257, 384, 1000, 5000, 19456, 19500,
                                      40000]:
        v = ctypes.c_size_t()
        assert moe.lib().moe_workspace_size_linear_i8(rows, N, K, ctypes.byref(v)) == OK
        assert v.value >= most
        most = v.value
    assert fits(4, most) == INVALID   # (an unknown type of y: nothing is enqueued)


def quantize(moe, rows=4, K=64, dtype=F32, x=FAKE, codes=FAKE, scales=FAKE):
    return moe.lib().moe_quantize_rows_i8(rows, K, dtype, x, codes, scales, None)


def test_quantize_refusals(moe):
    for name in ("x", "codes"):
        assert quantize(moe, **{name: None}) == INVALID
        assert quantize(moe, **{name: ODD}) == INVALID
    assert quantize(moe, scales=None) == INVALID
    assert quantize(moe, dtype=I8) == INVALID and quantize(moe, rows=-1) == INVALID
    assert quantize(moe, K=24) == UNSUPPORTED and quantize(moe, K=1 << 18) == UNSUPPORTED
    assert quantize(moe, rows=0, x=None, codes=None, scales=None) == OK


def sample(moe, rows=4, V=100, dtype=F32, t=1.0, k=0, p=1.0, m=0.0, **over):
    a = dict(logits=FAKE, u=FAKE, tokens=FAKE, prob=None, each=(None,) * 4)
    a.update(over)
    c = moe._binding.SampleChoices(t, k, p, m, *a["each"])
    return moe.lib().moe_sample(rows, V, dtype, a["logits"], a["u"], ctypes.byref(c), a["tokens"],
                                a["prob"], None)


def test_sample_refusals(moe):
    for name in ("logits", "u", "tokens"):
        assert sample(moe, **{name: None}) == INVALID
    assert sample(moe, logits=ODD) == INVALID and sample(moe, prob=0x10002) == INVALID
    nan = float("nan")
    for kw in (dict(t=-0.1), dict(t=nan), dict(k=-1), dict(p=-0.1), dict(p=1.5), dict(p=nan),
               dict(m=-0.1), dict(m=1.1), dict(m=nan), dict(rows=-1), dict(V=0), dict(dtype=I8)):
        assert sample(moe, **kw) == INVALID, kw
    assert sample(moe, V=(1 << 30) + 1) == UNSUPPORTED
    for i in range(4):
        each = [None] * 4
        each[i] = 0x10001
        assert sample(moe, each=each) == INVALID
    assert moe.lib().moe_sample(1, 5, F32, FAKE, FAKE, None, FAKE, None, None) == INVALID
    assert sample(moe, rows=0, logits=None, u=None, tokens=None) == OK


# ------------------------------------------------------------------ the binding

BF = torch.bfloat16


def test_binding_few(recorder):  # noqa: F811
    m = recorder
    cfg = m.config(T=2, h=256, E=4, k=2, f=128)
    x, Wg = torch.zeros(2, 256, dtype=BF), torch.zeros(256, 4)
    W1, W2 = torch.zeros(4, 256, 128, dtype=BF), torch.zeros(4, 128, 256, dtype=BF)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    m.forward_few(cfg, x, Wg, None, None, W1, W1, W2, x, ws)
    name, args = m.calls[-1]
    assert name == "moe_forward_few" and args[1] == 0 and args[9:12] == (None,) * 3
    V = torch.zeros(256, 384, dtype=BF), torch.zeros(256, 384, dtype=BF), torch.zeros(
        384, 256, dtype=BF)
    m.forward_few(cfg, x, Wg, None, None, W1, W1, W2, x, ws, shared=V)
    assert m.calls[-1][1][1] == 384
    for bad in (dict(x=x.float()), dict(x=torch.zeros(3, 256, dtype=BF)), dict(W1=W2.float()),
                dict(W2=torch.zeros(4, 128, 128, dtype=BF)), dict(Wg=Wg.to(BF)),
                dict(shared=(V[0], V[1], V[0])), dict(topk_idx=torch.zeros(2, 2)),
                dict(topk_prob=torch.zeros(2, 3)), dict(tokens_per_expert=torch.zeros(4))):
        a = dict(x=x, Wg=Wg, gate_bias=None, expert_bias=None, W1=W1, W3=W1, W2=W2, y=x, ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            m.forward_few(cfg, **a)


def test_binding_linear_and_quantize(recorder):  # noqa: F811
    m = recorder
    w = m.I8Weight(torch.zeros(8, 32, dtype=torch.int8), torch.ones(8))
    for name in ("codes", "scales", "n", "k"):
        with pytest.raises(AttributeError):
            setattr(w, name, None)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    x, y = torch.zeros(3, 32, dtype=BF), torch.zeros(3, 8)
    m.linear_i8(x, w, y, ws)
    assert m.calls[-1][1][4] == 1
    codes = torch.zeros(3, 32, dtype=torch.int8)
    m.linear_i8(codes, w, y, ws, x_scale=torch.ones(3), bias=torch.ones(8))
    assert m.calls[-1][1][4] == 2
    for bad in (dict(x=x.half()), dict(x=torch.zeros(3, 16, dtype=BF)), dict(x=codes),
                dict(x_scale=torch.ones(3)), dict(y=torch.zeros(3, 9)), dict(y=torch.zeros(2, 8)),
                dict(y=y.half()), dict(bias=torch.ones(7)), dict(bias=torch.ones(8, dtype=BF))):
        a = dict(x=x, w=w, y=y, ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            m.linear_i8(**a)
    with pytest.raises(ValueError):
        m.linear_i8(codes, w, y, ws, x_scale=torch.ones(2))
    for c, s in ((torch.zeros(8, 32), torch.ones(8)), (torch.zeros(8, 32, dtype=torch.int8),
                                                       torch.ones(7)),
                 (torch.zeros(8, 32, dtype=torch.int8), torch.ones(8, dtype=BF)),
                 (torch.zeros(2, 8, 32, dtype=torch.int8), torch.ones(2, 8))):
        with pytest.raises(ValueError):
            m.I8Weight(c, s)
    with pytest.raises(ValueError):
        m.quantize_rows_i8(x, codes[:2], torch.ones(3))
    with pytest.raises(ValueError):
        m.quantize_rows_i8(x, codes, torch.ones(2))
    with pytest.raises(ValueError):
        m.quantize_rows_i8(x.half(), codes, torch.ones(3))


def test_binding_sample(recorder):  # noqa: F811
    m = recorder
    l, u, t = torch.zeros(3, 10), torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    m.sample(l, u, t, temperature=0.5, top_k=torch.ones(3, dtype=torch.int32), top_p=0.9)
    name, args = m.calls[-1]
    c = args[5]._obj
    assert name == "moe_sample" and args[:3] == (3, 10, 0)
    assert c.temperature == 0.5 and c.top_k == 0 and c.top_k_of and not c.top_p_of
    for bad in (dict(logits=l[0]), dict(logits=l.half()), dict(u=u[:2]), dict(u=u.double()),
                dict(tokens=t.long()), dict(prob=torch.zeros(2)), dict(top_k=torch.zeros(3)),
                dict(top_p=torch.zeros(2)), dict(min_p=torch.zeros(3, dtype=BF))):
        a = dict(logits=l, u=u, tokens=t)
        a.update(bad)
        with pytest.raises(ValueError):
            m.sample(**a)


@pytest.mark.parametrize("fs", [0, 1408])
def test_few_workspace_serves_fewer_tokens_where_pieces_begin(moe, fs):
    """From some number of tokens on there are places for more partial sums: no size is above that
    of more tokens."""
    sizes = [moe.workspace_size_few(moe.config(T=T, h=4096, E=128, k=8, f=1536), fs)
             for T in range(0, 65)]
    assert sizes == sorted(sizes)
    steps = [b - a for a, b in zip(sizes[1:], sizes[2:])]
    assert max(steps) > 2 * sorted(steps)[len(steps) // 2]  # where they begin


def test_sample_refuses_vocabularies_whose_sums_overflow(moe):
    """A weight is 2^40 at most: 2^24 of them would add up to 2^64."""
    for V in (1 << 24, (1 << 24) + 1, 1 << 30):
        assert sample(moe, V=V) == UNSUPPORTED
        assert sample(moe, V=V, rows=0, logits=None, u=None, tokens=None) == UNSUPPORTED
    assert sample(moe, V=(1 << 24) - 1, rows=0, logits=None, u=None, tokens=None) == OK


def test_binding_hands_on_no_number_cut_to_32_bits(recorder):  # noqa: F811
    """Sizes and a top-k past 32 bits: the end of the range (a size that the library refuses, a
    top-k of all tokens), not what their lowest bits say."""
    m, most = recorder, 2 ** 31 - 1
    l, u, t = torch.zeros(3, 10), torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    for k, want in ((2 ** 32 + 5, most), (2 ** 31, most), (2 ** 63 - 1, most), (most, most),
                    (-2 ** 32 + 7, -2 ** 31), (7, 7)):
        m.sample(l, u, t, top_k=k)
        assert m.calls[-1][1][5]._obj.top_k == want
    with pytest.raises(TypeError):
        m.sample(l, u, t, top_k=2.5)
    none = torch.empty(0, 2 ** 32 + 16, dtype=BF)   # no rows: no memory
    m.sample(none, u[:0], t[:0])
    assert m.calls[-1][1][1] == most
    codes = torch.empty(0, 2 ** 32 + 16, dtype=torch.int8)
    m.quantize_rows_i8(none, codes, u[:0])
    assert m.calls[-1][1][1] == most
    w = m.I8Weight(codes, u[:0])
    m.linear_i8(none, w, torch.empty(0, 0), torch.zeros(256, dtype=torch.uint8))
    assert m.calls[-1][1][:3] == (0, 0, most)
    with pytest.raises(m.MoeError):   # the real library
        m.workspace_size_linear_i8(1, w)
