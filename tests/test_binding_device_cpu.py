"""Tensors of another device than the current one are refused, without a GPU: a tensor that says it
lives elsewhere.  A kernel is launched on the current device, where such an address means nothing."""

import pytest
import torch


class On(torch.Tensor):
    device_index = 0

    def get_device(self):
        return self.device_index

    is_cuda = property(lambda self: self.device_index >= 0)


def on(device, *shape, dtype=torch.float32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.device_index = device
    return t


@pytest.fixture
def binding(monkeypatch):
    from mixture_experts_layer_fp32_gb300 import _binding as b
    monkeypatch.setattr(b, "_current_device", lambda: 1)
    monkeypatch.setattr(b, "_stream", lambda: 0)

    class Refused:
        def __getattr__(self, name):
            raise AssertionError("%s was reached" % name)
    monkeypatch.setattr(b, "lib", Refused)
    return b


def test_addresses_of_the_current_device_alone(binding):
    t = on(1, 4)
    assert binding._p(t) == t.data_ptr() and binding._p(None) is None
    for bad in (on(0, 4), on(2, 4), on(-1, 4), torch.zeros(4)):
        with pytest.raises(ValueError):
            binding._p(bad)
    for other in (5, "x", [t], object()):
        with pytest.raises(TypeError):
            binding._p(other)


def test_entry_points_refuse_one_tensor_of_another_device(binding, monkeypatch):
    class Reached(Exception):
        pass

    class Library:
        def __getattr__(self, name):
            def call(*args):
                raise Reached(name)
            return call
    monkeypatch.setattr(binding, "lib", Library)
    a = dict(logits=on(1, 3, 10), u=on(1, 3), tokens=on(1, 3, dtype=torch.int32), prob=on(1, 3),
             top_p=on(1, 3))
    with pytest.raises(Reached):
        binding.sample(**a)
    for name, t in a.items():
        with pytest.raises(ValueError):
            binding.sample(**dict(a, **{name: on(0, *t.shape, dtype=t.dtype)}))
    w = binding.I8Weight(on(1, 8, 32, dtype=torch.int8), on(1, 8))
    other = binding.I8Weight(on(0, 8, 32, dtype=torch.int8), on(1, 8))
    a = dict(x=on(1, 3, 32), w=w, y=on(1, 3, 8), ws=on(1, 1024, dtype=torch.uint8), bias=on(1, 8))
    with pytest.raises(Reached):
        binding.linear_i8(**a)
    for bad in (dict(x=on(0, 3, 32)), dict(w=other), dict(y=on(0, 3, 8)), dict(bias=on(2, 8)),
                dict(ws=on(0, 1024, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            binding.linear_i8(**dict(a, **bad))
