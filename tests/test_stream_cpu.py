"""Where the binding takes the current stream's handle from."""

import importlib
import types

import torch


def test_a_torch_without_the_raw_handle_takes_the_public_way(monkeypatch):
    import mixture_experts_layer_fp32_gb300._binding as b
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=1234))
    spec = importlib.util.spec_from_file_location("binding_again", b.__file__)
    again = importlib.util.module_from_spec(spec)
    again.__package__ = b.__package__
    spec.loader.exec_module(again)
    assert again._stream() == 1234
