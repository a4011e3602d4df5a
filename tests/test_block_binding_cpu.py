"""What the binding hands to the library, without a GPU: the library is a
recorder and host tensors stand for device tensors."""

import pytest
import torch

BF = torch.bfloat16


@pytest.fixture
def moe(monkeypatch):
    from mixture_experts_layer_fp32_gb300 import build
    build.build()
    import mixture_experts_layer_fp32_gb300 as m
    b = m._binding
    real = b.lib()

    class Recorder:
        calls = []

        def __getattr__(self, name):
            if name.startswith("moe_workspace_size"):
                return getattr(real, name)

            def call(*args):
                self.calls.append((name, args))
                return 0
            return call

    def address(t):
        if t is None:
            return None
        assert t.is_contiguous()
        return t.data_ptr()

    recorder = Recorder()
    recorder.calls = []
    monkeypatch.setattr(b, "lib", lambda: recorder)
    monkeypatch.setattr(b, "_p", address)
    monkeypatch.setattr(b, "_stream", lambda: 0)
    m.calls = recorder.calls
    yield m
    del m.calls


def _weight(moe, *shape, K, group=64, zeros=False):
    n = shape + (K // group,)
    return moe.W4Weight(torch.zeros(shape + (moe.w4_row_bytes(K),), dtype=torch.uint8),
                        torch.ones(n, dtype=BF),
                        torch.zeros(n, dtype=torch.uint8) if zeros else None, group=group, k=K)


def _pointers(arg):
    """A moe_w4 argument, by value or by reference."""
    w = getattr(arg, "_obj", arg)
    return w.codes, w.scales, w.zeros


def _linear(moe, w):
    x, y = torch.zeros((3, w.k), dtype=BF), torch.zeros((3, w.n))
    moe.linear_w4(x, w, y, torch.zeros(1 << 20, dtype=torch.uint8))
    name, args = moe.calls[-1]
    assert name == "moe_linear_w4"
    return _pointers(args[5])


def test_a_weights_tensors_cannot_be_exchanged(moe):
    w = _weight(moe, 32, K=128, zeros=True)
    for name in ("codes", "scales", "zeros", "group", "k", "n"):
        with pytest.raises(AttributeError):
            setattr(w, name, getattr(w, name))
    q = moe.W4Experts(*(_weight(moe, 2, 256, K=256) for _ in range(3)))
    for name in ("W1", "W3", "W2", "group"):
        with pytest.raises(AttributeError):
            setattr(q, name, getattr(q, name))


def test_addresses_are_read_at_each_call(moe):
    """A tensor that was given other storage is read from there."""
    w = _weight(moe, 32, K=128, zeros=True)
    assert _linear(moe, w) == (w.codes.data_ptr(), w.scales.data_ptr(), w.zeros.data_ptr())
    others = [t.clone() for t in (w.codes, w.scales, w.zeros)]
    for t, other in zip((w.codes, w.scales, w.zeros), others):
        t.set_(other)
    assert _linear(moe, w) == tuple(t.data_ptr() for t in others)


T, H, E, K, F = 6, 256, 8, 2, 128


def _layer(moe):
    q = moe.W4Experts(_weight(moe, E, F, K=H), _weight(moe, E, F, K=H), _weight(moe, E, H, K=F))
    return moe.config(T=T, h=H, E=E, k=K, f=F), q, torch.zeros(1 << 20, dtype=torch.uint8)


def _wrong(t):
    """Tensors that must not be taken in the place of t: another type, fewer and
    more values, rows of another length."""
    other = torch.int64 if t.dtype == torch.int32 else torch.float16
    short, long = t[:-1].clone(), torch.cat((t, t[:1]))
    return [t.to(other), t.double(), short, long] + ([t.t().contiguous()] if t.dim() == 2 else [])


EXPERTS = dict(x=torch.zeros((T, H), dtype=BF), topk_idx=torch.zeros((T, K), dtype=torch.int32),
               topk_prob=torch.zeros((T, K)), keep=torch.ones((T, K), dtype=torch.uint8),
               y=torch.zeros((T, H), dtype=BF))


@pytest.mark.parametrize("name", list(EXPERTS))
def test_experts_take_no_other_tensors(moe, name):
    cfg, q, ws = _layer(moe)
    for bad in _wrong(EXPERTS[name]):
        a = dict(EXPERTS, **{name: bad})
        with pytest.raises(ValueError, match=name):
            moe.experts_w4(cfg, a["x"], a["topk_idx"], a["topk_prob"], a["keep"], q, a["y"], ws)
    assert not moe.calls


@pytest.mark.parametrize("keep", [None, torch.ones((T, K), dtype=torch.uint8),
                                  torch.ones((T, K), dtype=torch.bool),
                                  torch.ones(T * K, dtype=torch.uint8)])
def test_experts_take_what_the_router_writes(moe, keep):
    cfg, q, ws = _layer(moe)
    a = EXPERTS
    moe.experts_w4(cfg, a["x"].view(2, 3, H), a["topk_idx"], a["topk_prob"], keep, q, a["y"], ws)
    name, args = moe.calls[-1]
    assert name == "moe_experts_w4" and args[1] == 64
    assert args[2:6] == (a["x"].data_ptr(), a["topk_idx"].data_ptr(), a["topk_prob"].data_ptr(),
                         None if keep is None else keep.data_ptr())
    assert [_pointers(w) for w in args[6:9]] == [_pointers(w) for w in q._pointers()]
    assert args[9:12] == (a["y"].data_ptr(), ws.data_ptr(), ws.numel())


FORWARD = dict(x=EXPERTS["x"], Wg=torch.zeros((H, E)), gate_bias=torch.zeros(E),
               expert_bias=torch.zeros(E), y=EXPERTS["y"], topk_idx=EXPERTS["topk_idx"],
               topk_prob=EXPERTS["topk_prob"],
               tokens_per_expert=torch.zeros(E, dtype=torch.int32))


@pytest.mark.parametrize("name", list(FORWARD))
def test_forward_takes_no_other_tensors(moe, name):
    cfg, q, ws = _layer(moe)

    def call(a):
        moe.forward_w4(cfg, a["x"], a["Wg"], a["gate_bias"], a["expert_bias"], q, a["y"], ws,
                       topk_idx=a["topk_idx"], topk_prob=a["topk_prob"],
                       tokens_per_expert=a["tokens_per_expert"])

    for bad in _wrong(FORWARD[name]):
        with pytest.raises(ValueError, match=name):
            call(dict(FORWARD, **{name: bad}))
    assert not moe.calls
    call(FORWARD)
    if name not in ("x", "Wg", "y"):
        call(dict(FORWARD, **{name: None}))
    assert all(n == "moe_forward_w4" for n, _ in moe.calls)
