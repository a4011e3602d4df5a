"""The norm and its backward at the widths where the layout of a row changes:
each number of vectors to a thread with even and odd widths, the last widths that
stay on the chip, and the kernels for wider rows, against 64 bits."""

import pytest
import torch

from test_gpu_norm import DT, EPS, _check_backward, _check_forward, _inputs, _rand, _rng, _rows

pytestmark = pytest.mark.gpu

# bf16: three vectors to a thread up to 24576; fp32: four from 8193, five from
# 16385, up to 20480.  Past those, and for odd widths that touch one vector more,
# the kernel that reads a row three times.
FORWARD = [("bf16", H) for H in (16392, 20011, 24569, 24576, 24577, 24584, 32768, 33000, 65537)] + \
          [("f32", H) for H in (8193, 10001, 12288, 16379, 16384, 16388, 20473, 20480, 20484, 20485,
                                33000, 50001)]

# bf16 two, three, four vectors to a thread, then the kernel for wider rows; fp32
# two, three, four, eight
BACKWARD = [("bf16", H) for H in (8200, 9001, 10240, 12007, 12288, 15360, 16384, 16411, 18425,
                                  18432, 18433, 24001, 33000)] + \
           [("f32", H) for H in (4100, 5003, 5120, 6144, 6707, 7680, 8192, 9001, 10240, 12288,
                                 12289, 16384, 18432, 18433, 20004, 33000)]


@pytest.mark.parametrize("dtype,hidden", FORWARD)
def test_forward(dtype, hidden):
    rows = _rows(hidden)
    for param in {"f32", dtype}:
        _check_forward(rows, hidden, dtype, param, rms=False, residual=False, p=0.0)
        _check_forward(rows, hidden, dtype, param, rms=True, residual=True, p=0.3, seed=9)
        _check_forward(rows, hidden, dtype, param, rms=False, residual=True, p=0.0, bias=False)
        _check_forward(rows, hidden, dtype, param, rms=True, residual=False, p=0.0, weight=False)


@pytest.mark.parametrize("dtype,hidden", BACKWARD)
def test_backward(dtype, hidden):
    rows = _rows(hidden)
    for param in {"f32", dtype}:
        _check_backward(rows, hidden, dtype, param, rms=False, dz=False, p=None)
        _check_backward(rows, hidden, dtype, param, rms=True, dz=True, p=0.3, seed=9)
        _check_backward(rows, hidden, dtype, param, rms=False, dz=True, p=0.0, weight=False)


@pytest.mark.parametrize("dtype,hidden", [("bf16", 9001), ("bf16", 12288), ("bf16", 16411),
                                          ("bf16", 18433), ("f32", 4100), ("f32", 6707),
                                          ("f32", 9001), ("f32", 12289), ("f32", 18433)])
def test_backward_of_more_rows_than_blocks(dtype, hidden):
    """A block adds up several rows; 700 of the widest kernel's 608 blocks."""
    rows = 700 if hidden > 18432 else 400
    _check_backward(rows, hidden, dtype, "f32", rms=False, dz=True, p=0.2)


@pytest.mark.parametrize("dtype,hidden", [("bf16", 24576), ("bf16", 24577), ("f32", 16379),
                                          ("f32", 20480), ("f32", 20485)])
def test_forward_of_more_rows_than_blocks(dtype, hidden):
    _check_forward(400, hidden, dtype, "f32", rms=False, residual=True, p=0.2)


@pytest.mark.parametrize("dtype,hidden", FORWARD)
def test_forward_in_place(dtype, hidden):
    """The same bits as in buffers of their own, which test_forward compares."""
    import mixture_experts_layer_fp32_gb300 as moe
    rows, p = _rows(hidden), 0.2
    x, res, w, b = _inputs(rows, hidden, dtype, "f32", 6)
    y, z = torch.empty_like(x), torch.empty_like(x)
    moe.layer_norm(x, w, b, EPS, y, residual=res, z=z, p=p, rng=_rng())
    for y_over_x in (True, False):
        x2, r2 = x.clone(), res.clone()
        y2, z2 = (x2, r2) if y_over_x else (r2, x2)
        moe.layer_norm(x2, w, b, EPS, y2, residual=r2, z=z2, p=p, rng=_rng())
        assert torch.equal(y2, y) and torch.equal(z2, z)


@pytest.mark.parametrize("dtype,hidden", BACKWARD)
def test_backward_in_place(dtype, hidden):
    import mixture_experts_layer_fp32_gb300 as moe
    rows, p = _rows(hidden), 0.2
    z, _, w, _ = _inputs(rows, hidden, dtype, "f32", 6)
    mean, rstd = z.float().mean(1), torch.rsqrt(z.float().var(1) + EPS)
    ws = moe.alloc_workspace_norm_backward(rows, hidden)
    outs = []
    for where in ("own", "dx over dy", "dx over dz"):
        dy, dz = _rand(z.shape, DT[dtype], 7), _rand(z.shape, DT[dtype], 8)
        dx, db = {"own": (torch.empty_like(z), torch.empty_like(z)), "dx over dy": (dy, dz),
                  "dx over dz": (dz, dy)}[where]
        dw, dbias = (torch.empty(hidden, device="cuda") for _ in range(2))
        moe.layer_norm_backward(dy, z, w, mean, rstd, dx, dw, dbias, ws, dz=dz, dbranch=db, p=p,
                                rng=_rng())
        outs.append((dx, db, dw, dbias))
    for other in outs[1:]:
        assert all(torch.equal(a, c) for a, c in zip(outs[0], other))
