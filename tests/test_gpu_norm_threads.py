"""Calls from several host threads whose rows take the same kernel with different
amounts of shared memory."""

import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-5
ROWS, THREADS, CALLS = 8, 4, 6000


def _statuses(calls):
    """The library's calls, each over and over in THREADS threads at once,
    prepared beforehand so that they meet inside the library; the statuses seen."""
    seen, gate = set(), threading.Barrier(THREADS * len(calls))

    def go(fn, args):
        gate.wait()
        mine = set()
        for _ in range(CALLS):
            mine.add(fn(*args))
        seen.update(mine)

    threads = [threading.Thread(target=go, args=c) for c in calls for _ in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return seen


def _pointers(*tensors):
    return [ctypes.c_void_p(None if t is None else t.data_ptr()) for t in tensors]


@pytest.mark.parametrize("dtype,widths", [(torch.bfloat16, (8192, 16384)),
                                          (torch.float32, (6144, 8192))])
def test_forward_of_two_widths(dtype, widths):
    """64 and 128 KB of one instantiation, 48 and 64."""
    import mixture_experts_layer_fp32_gb300 as moe
    calls, outs = [], []
    for H in widths:
        x = torch.randn((ROWS, H), device="cuda").to(dtype)
        y, want = torch.empty_like(x), torch.empty_like(x)
        moe.layer_norm(x, None, None, EPS, want)
        cfg = moe.NormConfig(ROWS, 0.0, H, int(dtype == torch.bfloat16), 0, 0, EPS)
        args = [ctypes.byref(cfg), *_pointers(x, None, None, None, None, None, y, None, None, None)]
        calls.append((moe.lib().moe_layer_norm, args))
        outs.append((y, want, x, cfg))
    torch.cuda.synchronize()
    assert _statuses(calls) == {0}
    assert all(torch.equal(y, want) for y, want, *_ in outs)


@pytest.mark.parametrize("dtype,widths", [(torch.bfloat16, (4096, 8192)),
                                          (torch.float32, (2048, 4096))])
def test_backward_of_two_widths(dtype, widths):
    import mixture_experts_layer_fp32_gb300 as moe
    calls, outs = [], []
    for H in widths:
        z, dy = (torch.randn((ROWS, H), device="cuda").to(dtype) for _ in range(2))
        mean, rstd = z.float().mean(1), torch.rsqrt(z.float().var(1) + EPS)
        dx, want = torch.empty_like(z), torch.empty_like(z)
        ws = moe.alloc_workspace_norm_backward(ROWS, H)
        moe.layer_norm_backward(dy, z, None, mean, rstd, want, None, None, ws)
        cfg = moe.NormConfig(ROWS, 0.0, H, int(dtype == torch.bfloat16), 0, 0, EPS)
        args = [ctypes.byref(cfg), *_pointers(dy, z, None, mean, rstd, None, None, dx, None, None,
                                              None, ws), ctypes.c_size_t(ws.numel()),
                ctypes.c_void_p(None)]
        calls.append((moe.lib().moe_layer_norm_backward, args))
        outs.append((dx, want, z, dy, mean, rstd, ws, cfg))
    torch.cuda.synchronize()
    assert _statuses(calls) == {0}
    assert all(torch.equal(dx, want) for dx, want, *_ in outs)
