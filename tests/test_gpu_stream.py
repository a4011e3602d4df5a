"""The handle that calls run on is the current stream's."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_handles_agree(monkeypatch):
    import mixture_experts_layer_fp32_gb300 as moe
    b = moe._binding
    for stream in (torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            assert b._stream() == stream.cuda_stream
            with monkeypatch.context() as m:
                m.setattr(b, "_raw_stream", None)
                assert b._stream() == stream.cuda_stream
