"""The norm, its backward and the dropout on the GPU against references in 64
bits (block_cases); the bounds there count roundings."""

import pytest
import torch

import block_cases as bc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5

# widths around the vector, warp and block sizes, odd ones among them, and past
# the widths whose rows are kept on the chip
WIDTHS = [1, 2, 3, 7, 8, 31, 64, 257, 512, 1021, 1024, 1032, 2048, 4096, 4099, 7168, 8200, 16384,
          16392, 20003]


def _rng(seed=77, offset=(1 << 35) + 5):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def _rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, device="cuda", generator=g) + shift).to(dtype)


def _rows(hidden):
    return max(3, min(700, 300000 // hidden))


def _inputs(rows, hidden, dtype, param, seed):
    x = _rand((rows, hidden), DT[dtype], seed, shift=0.5)
    res = _rand((rows, hidden), DT[dtype], seed + 1)
    w = _rand((hidden,), DT[param], seed + 2, 0.2, 1.0)
    b = _rand((hidden,), DT[param], seed + 3)
    return x, res, w, b


def _check_forward(rows, hidden, dtype, param, rms, residual, p, weight=True, bias=True, seed=1):
    import mixture_experts_layer_fp32_gb300 as moe
    x, res, w, b = _inputs(rows, hidden, dtype, param, seed)
    w, b, res = (w if weight else None), (b if bias else None), (res if residual else None)
    rng = _rng()
    y = torch.full_like(x, float("nan"))
    z = torch.full_like(x, float("nan")) if residual else None
    mean = torch.full((rows,), float("nan"), device="cuda")
    rstd = torch.full((rows,), float("nan"), device="cuda")
    moe.layer_norm(x, w, b, EPS, y, None if rms else mean, rstd, rms=rms, residual=res, z=z, p=p,
                   rng=rng)
    z64, e_z = x.double(), None
    if residual:
        a = x.double()
        if p > 0:
            a = bc.dropped(a, p, bc.keep_mask(77, (1 << 35) + 5, p, x.numel()))
        z64 = a + res.double()
        # the scaled value and the sum, one rounding each
        e_z = bc.U * (a.abs() + z64.abs())
        bc.assert_within("z", z, z64, e_z, DT[dtype])
    r = bc.norm_ref(z64, w, b, EPS, rms)
    e_y, e_mean, e_rstd = r["e_y"], r["e_mean"], r["e_rstd"]
    if residual:  # z's own error, through the norm
        mz = e_z.mean(1, keepdim=True)
        dr = r["rstd"][:, None] ** 2 * e_z.pow(2).mean(1, keepdim=True).sqrt()
        e_rstd = e_rstd + 2 * (r["rstd"][:, None] * dr.sqrt() * dr.sqrt())[:, 0]
        e_mean = e_mean + mz[:, 0]
        ww = 1.0 if w is None else w.double().abs()
        c = (z64 - r["mean"][:, None]).abs()
        e_y = e_y + ww * (r["rstd"][:, None] * (e_z + mz) + 2 * c * r["rstd"][:, None] * dr)
    bc.assert_within("y", y, r["y"], e_y, DT[dtype])
    bc.assert_within("rstd", rstd, r["rstd"], e_rstd)
    if not rms:
        bc.assert_within("mean", mean, r["mean"], e_mean)


@pytest.mark.parametrize("dtype,param", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_forward(hidden, dtype, param):
    rows = _rows(hidden)
    _check_forward(rows, hidden, dtype, param, rms=False, residual=False, p=0.0)
    _check_forward(rows, hidden, dtype, param, rms=True, residual=True, p=0.3, seed=9)


@pytest.mark.parametrize("rows", [1, 2, 5, 9, 153, 2500])
@pytest.mark.parametrize("hidden,dtype", [(64, "bf16"), (1021, "f32"), (1023, "bf16"),
                                          (2050, "bf16")])
def test_forward_rows(rows, hidden, dtype):
    _check_forward(rows, hidden, dtype, "f32", rms=False, residual=True, p=0.1)
    _check_forward(rows, hidden, dtype, "f32", rms=True, residual=True, p=0.0, bias=False)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("hidden", [96, 1025, 6000])
def test_forward_without_parameters(hidden, weight, bias):
    _check_forward(6, hidden, "bf16", "f32", rms=False, residual=False, p=0.0, weight=weight,
                   bias=bias)


def _check_backward(rows, hidden, dtype, param, rms, dz, p, weight=True, seed=1):
    import mixture_experts_layer_fp32_gb300 as moe
    z, _, w, _ = _inputs(rows, hidden, dtype, param, seed)
    w = w if weight else None
    dy = _rand((rows, hidden), DT[dtype], seed + 5)
    d = _rand((rows, hidden), DT[dtype], seed + 6) if dz else None
    f = bc.norm_ref(z.double(), w, None, EPS, rms)
    mean, rstd = f["mean"].float(), f["rstd"].float()
    rng = _rng()
    dx = torch.full_like(z, float("nan"))
    db = torch.full_like(z, float("nan")) if p is not None else None
    dw = torch.full((hidden,), float("nan"), device="cuda")
    dbias = torch.full((hidden,), float("nan"), device="cuda")
    ws = moe.alloc_workspace_norm_backward(rows, hidden)
    moe.layer_norm_backward(dy, z, w, None if rms else mean, rstd, dx, dw, dbias, ws, rms=rms,
                            dz=d, dbranch=db, p=p or 0.0, rng=rng)
    r = bc.norm_grad_ref(dy.double(), z.double(), w, mean, rstd, None if d is None else d.double(),
                         rms)
    bc.assert_within("dx", dx, r["dx"], r["e_dx"], DT[dtype])
    bc.assert_within("dweight", dw, r["dweight"], r["e_dweight"], torch.float32)
    bc.assert_within("dbias", dbias, r["dbias"], r["e_dbias"], torch.float32)
    if p is not None:
        keep = bc.keep_mask(77, (1 << 35) + 5, p, z.numel())
        ref = bc.dropped(r["dx"], p, keep)
        scale = 1 / (1 - p)
        bc.assert_within("dbranch", db, ref, scale * (r["e_dx"] + bc.U * r["dx"].abs()), DT[dtype])
        assert torch.equal(db[~keep.view(db.shape).cuda()].float(),
                           torch.zeros(int((~keep).sum()), device="cuda"))
    moe.check(ws)


@pytest.mark.parametrize("dtype,param", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_backward(hidden, dtype, param):
    rows = _rows(hidden)
    _check_backward(rows, hidden, dtype, param, rms=False, dz=False, p=None)
    _check_backward(rows, hidden, dtype, param, rms=True, dz=True, p=0.3, seed=9)


@pytest.mark.parametrize("rows", [1, 2, 5, 9, 153, 2500, 9001])
@pytest.mark.parametrize("hidden,dtype", [(64, "bf16"), (1021, "f32"), (1023, "bf16"),
                                          (2050, "bf16")])
def test_backward_rows(rows, hidden, dtype):
    _check_backward(rows, hidden, dtype, "f32", rms=False, dz=True, p=0.1)
    _check_backward(rows, hidden, dtype, "f32", rms=True, dz=False, p=0.0, weight=False)


def test_no_rows():
    import mixture_experts_layer_fp32_gb300 as moe
    x = torch.empty((0, 64), device="cuda")
    moe.layer_norm(x, None, None, EPS, x)
    moe.dropout_add(x, x, 0.0, None)
    dw = torch.full((64,), 3.0, device="cuda")
    db = torch.full((64,), 3.0, device="cuda")
    s = torch.empty((0,), device="cuda")
    moe.layer_norm_backward(x, x, None, s, s, x, dw, db, moe.alloc_workspace_norm_backward(0, 64))
    assert float(dw.abs().sum()) == 0 and float(db.abs().sum()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 255, 4096, 100003])
@pytest.mark.parametrize("p", [0.0, 1e-12, 0.1, 0.5, 1.0])
def test_dropout(n, dtype, p):
    import mixture_experts_layer_fp32_gb300 as moe
    x, res = _rand((n,), DT[dtype], 3), _rand((n,), DT[dtype], 4)
    keep = bc.keep_mask(77, (1 << 35) + 5, p, n)
    for r in (None, res):
        y = torch.full_like(x, float("nan"))
        moe.dropout_add(x, y, p, _rng(), residual=r)
        a = bc.dropped(x.double(), p, keep)
        ref = a if r is None else a + r.double()
        bc.assert_within("y", y, ref, bc.U * (a.abs() + ref.abs()), DT[dtype])


def test_dropped_infinities_and_nans_are_zero():
    import mixture_experts_layer_fp32_gb300 as moe
    n = 4096
    keep = bc.keep_mask(77, (1 << 35) + 5, 0.5, n).cuda()
    x = torch.where(torch.arange(n, device="cuda") % 2 == 0, float("inf"), float("nan"))
    y = torch.empty_like(x)
    moe.dropout_add(x, y, 0.5, _rng())
    assert torch.equal(y[~keep], torch.zeros_like(y[~keep]))
    assert not torch.isfinite(y[keep]).any()


def test_masks_agree_between_calls_and_follow_rng():
    import mixture_experts_layer_fp32_gb300 as moe
    rows, H, p = 37, 1003, 0.25
    x, res, w, b = _inputs(rows, H, "bf16", "f32", 4)
    y, z, only = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    moe.layer_norm(x, w, b, EPS, y, residual=res, z=z, p=p, rng=_rng())
    moe.dropout_add(x, only, p, _rng(), residual=res)
    assert torch.equal(z, only)
    for other in (_rng(seed=78), _rng(offset=5), _rng(seed=77 + (1 << 40)),
                  _rng(offset=(1 << 36) + 5)):
        moe.dropout_add(x, y, p, other, residual=res)
        assert not torch.equal(y, only)


def test_special_rows():
    """A constant row, a row of zeros, one huge value, an infinity, a NaN: the
    bad rows stay by themselves."""
    import mixture_experts_layer_fp32_gb300 as moe
    for H in (65, 1024, 5000):
        x = _rand((8, H), torch.float32, 5)
        x[1], x[2], x[3, 0] = 3.0, 0.0, 1e15
        x[4, H // 2], x[5, 1] = float("inf"), float("nan")
        y, ref = torch.empty_like(x), bc.norm_ref(x.double(), None, None, EPS, False)
        moe.layer_norm(x, None, None, EPS, y)
        rows = [0, 1, 2, 3, 6, 7]
        bc.assert_within("y", y[rows], ref["y"][rows], ref["e_y"][rows], torch.float32)
        assert torch.isnan(y[4]).any() and torch.isnan(y[5]).all()


@pytest.mark.parametrize("hidden", [136, 1021, 4096, 17001])
def test_in_place(hidden):
    import mixture_experts_layer_fp32_gb300 as moe
    rows, p = 11, 0.2
    x, res, w, b = _inputs(rows, hidden, "bf16", "f32", 6)
    y, z = torch.empty_like(x), torch.empty_like(x)
    moe.layer_norm(x, w, b, EPS, y, residual=res, z=z, p=p, rng=_rng())
    x2, r2 = x.clone(), res.clone()
    moe.layer_norm(x2, w, b, EPS, x2, residual=r2, z=r2, p=p, rng=_rng())
    assert torch.equal(x2, y) and torch.equal(r2, z)
    x2, r2 = x.clone(), res.clone()
    moe.layer_norm(x2, w, b, EPS, r2, residual=r2, z=x2, p=p, rng=_rng())
    assert torch.equal(r2, y) and torch.equal(x2, z)
    moe.dropout_add(x, y, p, _rng(), residual=res)
    x2 = x.clone()
    moe.dropout_add(x2, x2, p, _rng(), residual=res)
    assert torch.equal(x2, y)
    # backward: dx over dy, dbranch over dz
    f = bc.norm_ref(z.double(), w, None, EPS, False)
    mean, rstd = f["mean"].float(), f["rstd"].float()
    ws = moe.alloc_workspace_norm_backward(rows, hidden)
    outs = []
    for inplace in (False, True):
        dy, dz = _rand(x.shape, x.dtype, 7), _rand(x.shape, x.dtype, 8)
        dx, db = (dy, dz) if inplace else (torch.empty_like(x), torch.empty_like(x))
        dw, dbias = torch.empty(hidden, device="cuda"), torch.empty(hidden, device="cuda")
        moe.layer_norm_backward(dy, z, w, mean, rstd, dx, dw, dbias, ws, dz=dz, dbranch=db, p=p,
                                rng=_rng())
        outs.append((dx, db, dw, dbias))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


def test_repeats_are_equal_and_neighbours_untouched():
    """Same inputs, same bits; nothing outside the output buffers is written."""
    import mixture_experts_layer_fp32_gb300 as moe
    for rows, H, dtype in ((1300, 1021, "f32"), (700, 1027, "bf16"), (1025, 96, "bf16")):
        z, _, w, _ = _inputs(rows, H, dtype, "f32", 3)
        dy = _rand(z.shape, z.dtype, 4)
        f = bc.norm_ref(z.double(), w, None, EPS, False)
        mean, rstd = f["mean"].float(), f["rstd"].float()
        ws = moe.alloc_workspace_norm_backward(rows, H)
        seen = []
        for _ in range(3):
            room = torch.full((rows * H + 64,), 7.0, dtype=z.dtype, device="cuda")
            dx = room[32:32 + rows * H].view(rows, H)
            grads = torch.full((2, H + 64 + (-H) % 4), 7.0, device="cuda")
            dw, db = grads[0, 32:32 + H], grads[1, 32:32 + H]
            moe.layer_norm_backward(dy, z, w, mean, rstd, dx, dw, db, ws)
            y = torch.full_like(room, 7.0)
            moe.layer_norm(z, w, None, EPS, y[32:32 + rows * H].view(rows, H))
            for t in (room, y):
                assert float((t[:32] - 7).abs().max()) == 0
                assert float((t[32 + rows * H:] - 7).abs().max()) == 0
            assert float((grads[:, :32] - 7).abs().max()) == 0
            assert float((grads[:, 32 + H:] - 7).abs().max()) == 0
            seen.append((dx.clone(), dw.clone(), db.clone(), y.clone()))
        for other in seen[1:]:
            for a, c in zip(seen[0], other):
                assert torch.equal(a, c)


def test_past_32_bits():
    """A tensor of more than 2^32 elements: its last rows and their mask."""
    import mixture_experts_layer_fp32_gb300 as moe
    H, rows, p, last = 16383, 262500, 0.5, 4
    n = rows * H
    assert n > 1 << 32
    x = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    x[-last:] = _rand((last, H), torch.bfloat16, 2)
    y, z = torch.empty_like(x), torch.empty_like(x)
    res = torch.ones_like(x)
    moe.layer_norm(x, None, None, EPS, y, residual=res, z=z, p=p, rng=_rng())
    first = (n - last * H) // 4 * 4
    keep = bc.keep_mask(77, (1 << 35) + 5, p, n - first, first=first)[n - last * H - first:]
    z64 = bc.dropped(x[-last:].double(), p, keep) + 1.0
    bc.assert_within("z", z[-last:], z64, 3 * bc.U * z64.abs(), torch.bfloat16)
    del y
    moe.dropout_add(x, res, p, _rng(), residual=res)
    assert torch.equal(res, z)


def test_on_another_stream_and_in_a_graph():
    """The calls follow torch's current stream, and a captured step draws new
    masks when the offset in device memory moves on."""
    import mixture_experts_layer_fp32_gb300 as moe
    rows, H, p = 64, 2048, 0.5
    x, res, w, b = _inputs(rows, H, "bf16", "f32", 6)
    rng = _rng()
    out = {n: torch.empty_like(x) for n in ("z", "y", "dx", "db")}
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, dbias = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = moe.alloc_workspace_norm_backward(rows, H)

    def step():
        moe.layer_norm(x, w, b, EPS, out["y"], mean, rstd, residual=res, z=out["z"], p=p, rng=rng)
        moe.layer_norm_backward(out["y"], out["z"], w, mean, rstd, out["dx"], dw, dbias, ws,
                                dz=out["z"], dbranch=out["db"], p=p, rng=rng)
        rng[1:].add_(1)

    def values():
        torch.cuda.synchronize()
        return [t.clone() for t in (*out.values(), mean, rstd, dw, dbias)]

    step()
    first = values()
    step()
    second = values()
    assert not torch.equal(first[0], second[0])
    side = torch.cuda.Stream()
    rng.copy_(_rng())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    assert all(torch.equal(a, c) for a, c in zip(first, values()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng.copy_(_rng())
    for want in (first, second):
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(want, values()))


@pytest.mark.parametrize("dtype,hidden", [("bf16", 6144), ("f32", 6144), ("bf16", 6100),
                                          ("f32", 3000), ("bf16", 12288), ("f32", 12288)])
def test_shared_memory_around_48_kb(dtype, hidden):
    """Widths whose parameters take just the shared memory that a kernel has without asking."""
    rows = _rows(hidden)
    _check_forward(rows, hidden, dtype, "f32", False, True, 0.1, seed=hidden)
    _check_forward(rows, hidden, dtype, dtype, True, False, 0.0, seed=hidden)
    _check_backward(rows, hidden, dtype, "f32", False, True, 0.1, seed=hidden)
    _check_backward(rows, hidden, dtype, dtype, True, False, 0.0, seed=hidden)
