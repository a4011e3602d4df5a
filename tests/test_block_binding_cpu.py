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
