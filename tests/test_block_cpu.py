"""What surrounds the layer, without a GPU: the references that the GPU tests
use (Philox against its published vectors, the norm's gradient against
differences, the 4-bit layout against its definition), and the refusals of the
C ABI, none of which reaches the CUDA runtime."""

import ctypes

import numpy as np
import pytest
import torch

import block_cases as bc

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE, OTHER, MISALIGNED = 0x10000, 0x20000, 0x10004


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_fp32_gb300 import build
    build.build()
    import mixture_experts_layer_fp32_gb300 as m
    return m


# the known answers that are published with the generator
@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(ctr, key, want):
    assert tuple(int(v) for v in bc.philox4x32([ctr], key)[0]) == want


def test_keep_mask_rate():
    n = 1 << 18
    for p in (0.1, 0.5, 0.9):
        kept = bc.keep_mask(1234, 5678, p, n).double().mean().item()
        assert abs(kept - (1 - p)) < 5 * (p * (1 - p) / n) ** 0.5
    assert bool(bc.keep_mask(1, 2, 0.0, 64).all()) and not bool(bc.keep_mask(1, 2, 1.0, 64).any())


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("H", [1, 2, 7, 33])
def test_norm_gradient_against_differences(rms, H):
    g = torch.Generator().manual_seed(H)
    z = torch.randn(3, H, dtype=torch.float64, generator=g) + 0.5
    w = 1 + 0.3 * torch.randn(H, dtype=torch.float64, generator=g)
    b = torch.randn(H, dtype=torch.float64, generator=g)
    dy = torch.randn(3, H, dtype=torch.float64, generator=g)
    dz = torch.randn(3, H, dtype=torch.float64, generator=g)
    eps = 0.05   # so that a row of one column has a gradient too
    out = bc.norm_ref(z, w, b, eps, rms)
    got = bc.norm_grad_ref(dy, z, w, out["mean"], out["rstd"], dz, rms)

    def loss(z, w, b):
        return float((bc.norm_ref(z, w, b, eps, rms)["y"] * dy).sum() + (z * dz).sum())

    step = 1e-5
    for args, name in ((0, "dx"), (1, "dweight"), (2, "dbias")):
        base = [z, w, b]
        num = torch.zeros_like(base[args])
        for i in range(num.numel()):
            hi, lo = base[args].clone(), base[args].clone()
            hi.view(-1)[i] += step
            lo.view(-1)[i] -= step
            up, dn = list(base), list(base)
            up[args], dn[args] = hi, lo
            num.view(-1)[i] = (loss(*up) - loss(*dn)) / (2 * step)
        # the difference quotient is off by step^2 f''' / 6 and 2^-53 |f| / step
        assert torch.allclose(got[name], num, rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("K", [32, 96, 128, 160, 256, 480])
def test_w4_layout(K):
    rng = np.random.default_rng(K)
    v = rng.integers(0, 16, (2, 3, K)).astype(np.uint8)
    codes = bc.w4_pack_ref(v)
    assert codes.shape == (2, 3, -(-K // 128) * 64)
    assert np.array_equal(bc.w4_unpack_ref(codes, K), v)
    # the definition: word 4t + j holds k = 32j + 8t + i, input i in nibble i/2 + 4(i%2)
    words = codes.view("<u4")
    for k in range(K):
        j, t, i = k % 128 // 32, k % 32 // 8, k % 8
        word = words[..., k // 128 * 16 + 4 * t + j]
        assert np.array_equal((word >> (4 * (i // 2 + 4 * (i % 2)))) & 15, v[..., k])


# ------------------------------------------------------------------ refusals

def _norm(moe, **over):
    a = dict(rows=4, dropout=0.0, hidden=64, dtype=1, param_dtype=0, kind=0, eps=1e-5)
    a.update(over)
    return moe.NormConfig(*(a[f] for f, _ in moe.NormConfig._fields_))


@pytest.mark.parametrize("over,want", [
    (dict(rows=-1), INVALID), (dict(hidden=0), INVALID), (dict(hidden=-8), INVALID),
    (dict(dtype=2), INVALID), (dict(param_dtype=-1), INVALID), (dict(kind=2), INVALID),
    (dict(dropout=-0.1), INVALID), (dict(dropout=1.5), INVALID),
    (dict(dropout=float("nan")), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(dtype=0, param_dtype=1), UNSUPPORTED), (dict(hidden=(1 << 24) + 1), UNSUPPORTED),
    (dict(rows=1 << 60), UNSUPPORTED), (dict(), OK), (dict(rows=0), OK), (dict(hidden=1), OK),
])
def test_norm_config_checks(moe, over, want):
    size = ctypes.c_size_t()
    assert moe.lib().moe_workspace_size_norm_backward(ctypes.byref(_norm(moe, **over)),
                                                      ctypes.byref(size)) == want


def test_norm_refusals(moe):
    lib = moe.lib()

    def call(x=FAKE, residual=None, rng=None, weight=FAKE, bias=None, z=None, y=OTHER, mean=FAKE,
             rstd=FAKE, **over):
        return lib.moe_layer_norm(ctypes.byref(_norm(moe, **over)), x, residual, rng, weight, bias,
                                  z, y, mean, rstd, None)

    assert lib.moe_layer_norm(None, *[FAKE] * 9, None) == INVALID
    assert call(x=None) == INVALID and call(y=None) == INVALID
    for name in ("x", "residual", "weight", "bias", "y", "mean", "rstd"):
        assert call(**{name: MISALIGNED}) == INVALID, name
    assert call(z=FAKE) == INVALID                        # z without a residual
    assert call(dropout=0.1, rng=FAKE) == INVALID         # dropout without a residual
    assert call(residual=FAKE, dropout=0.1) == INVALID    # dropout without rng
    assert call(residual=FAKE, z=OTHER) == INVALID        # z and y in one buffer
    assert call(x=None, y=None, rows=0) == OK             # nothing to do, nothing enqueued


def test_norm_backward_refusals(moe):
    lib = moe.lib()
    size = ctypes.c_size_t()
    assert lib.moe_workspace_size_norm_backward(ctypes.byref(_norm(moe)), None) == INVALID
    assert lib.moe_workspace_size_norm_backward(ctypes.byref(_norm(moe)),
                                                ctypes.byref(size)) == OK

    def call(dy=FAKE, z=FAKE, weight=FAKE, mean=FAKE, rstd=FAKE, dz=None, rng=None, dx=OTHER,
             dbranch=None, dweight=FAKE, dbias=FAKE, ws=FAKE, ws_bytes=size.value, **over):
        return lib.moe_layer_norm_backward(ctypes.byref(_norm(moe, **over)), dy, z, weight, mean,
                                           rstd, dz, rng, dx, dbranch, dweight, dbias, ws,
                                           ws_bytes, None)

    for name in ("dy", "z", "mean", "rstd", "dx", "ws"):
        assert call(**{name: None}) == INVALID, name
    for name in ("dy", "z", "weight", "mean", "rstd", "dz", "dx", "dbranch", "dweight", "dbias",
                 "ws"):
        assert call(**{name: MISALIGNED}) == INVALID, name
    assert call(dbranch=OTHER) == INVALID                     # dx and dbranch in one buffer
    assert call(dbranch=FAKE, dropout=0.5) == INVALID         # no rng
    assert call(ws_bytes=size.value - 1) == WORKSPACE


def test_dropout_refusals(moe):
    lib = moe.lib()
    assert lib.moe_dropout_add(-1, 1, 0.1, FAKE, FAKE, None, FAKE, None) == INVALID
    assert lib.moe_dropout_add(8, 2, 0.1, FAKE, FAKE, None, FAKE, None) == INVALID
    assert lib.moe_dropout_add(8, 1, 1.1, FAKE, FAKE, None, FAKE, None) == INVALID
    assert lib.moe_dropout_add(8, 1, 0.1, None, FAKE, None, FAKE, None) == INVALID
    assert lib.moe_dropout_add(8, 1, 0.1, FAKE, None, None, FAKE, None) == INVALID
    assert lib.moe_dropout_add(8, 1, 0.1, FAKE, FAKE, MISALIGNED, FAKE, None) == INVALID
    assert lib.moe_dropout_add(1 << 60, 1, 0.1, FAKE, FAKE, None, FAKE, None) == UNSUPPORTED
    assert lib.moe_dropout_add(0, 1, 0.1, None, None, None, None, None) == OK


def _w4(moe, codes=FAKE, scales=FAKE, zeros=None):
    return moe._binding.W4Pointers(codes, scales, zeros)


def test_w4_refusals(moe):
    lib = moe.lib()
    size = ctypes.c_size_t()
    for rows, N, K, want in ((-1, 8, 64, INVALID), (1, 0, 64, INVALID), (1, 8, 0, INVALID),
                             (1, 8, 48, UNSUPPORTED), (1, 1, 32, OK), (0, 8, 64, OK),
                             (1 << 40, 8, 64, UNSUPPORTED)):
        assert lib.moe_workspace_size_linear_w4(rows, N, K, ctypes.byref(size)) == want
    assert lib.moe_workspace_size_linear_w4(4, 64, 256, ctypes.byref(size)) == OK
    need = size.value

    def linear(rows=4, N=64, K=256, group=64, x=FAKE, w=_w4(moe), y=FAKE, y_dtype=1, ws=FAKE,
               ws_bytes=need):
        return lib.moe_linear_w4(rows, N, K, group, x, ctypes.byref(w) if w else None, y, y_dtype,
                                 ws, ws_bytes, None)

    for over in (dict(group=48), dict(group=0), dict(x=None), dict(x=MISALIGNED), dict(y=None),
                 dict(w=None), dict(w=_w4(moe, codes=None)), dict(w=_w4(moe, scales=None)),
                 dict(w=_w4(moe, zeros=MISALIGNED)), dict(y_dtype=3), dict(ws=None)):
        assert linear(**over) == INVALID, over
    assert linear(K=96, group=64) == UNSUPPORTED
    assert linear(ws_bytes=need - 1) == WORKSPACE
    assert linear(rows=0, x=None, y=None) == OK

    assert lib.moe_quantize_w4(0, 64, 64, 64, FAKE, FAKE, FAKE, None, None) == INVALID
    assert lib.moe_quantize_w4(1, 64, 64, 16, FAKE, FAKE, FAKE, None, None) == INVALID
    assert lib.moe_quantize_w4(1, 64, 72, 64, FAKE, FAKE, FAKE, None, None) == UNSUPPORTED
    assert lib.moe_quantize_w4(1, 192, 64, 128, FAKE, FAKE, FAKE, None, None) == UNSUPPORTED
    assert lib.moe_quantize_w4(1, 64, 64, 64, None, FAKE, FAKE, None, None) == INVALID
    assert lib.moe_pack_w4(1, 8, 0, FAKE, FAKE, None) == INVALID
    assert lib.moe_pack_w4(1, 8, 32, FAKE, None, None) == INVALID


def test_experts_w4_refusals(moe):
    lib = moe.lib()
    cfg = moe.config(T=4, h=512, E=8, k=2, f=256)
    size = ctypes.c_size_t()
    assert lib.moe_workspace_size_experts_w4(ctypes.byref(cfg), ctypes.byref(size)) == OK
    need = size.value
    f32 = moe.config(T=4, h=512, E=8, k=2, f=256, dtype="f32")
    for fn in (lib.moe_workspace_size_experts_w4, lib.moe_workspace_size_w4):
        assert fn(ctypes.byref(f32), ctypes.byref(size)) == UNSUPPORTED
        assert fn(None, ctypes.byref(size)) == INVALID

    def experts(cfg=cfg, group=64, x=FAKE, idx=FAKE, prob=FAKE, keep=None, w1=_w4(moe),
                w3=_w4(moe), w2=_w4(moe), y=FAKE, ws=FAKE, ws_bytes=need):
        r = [ctypes.byref(w) if w else None for w in (w1, w3, w2)]
        return lib.moe_experts_w4(ctypes.byref(cfg), group, x, idx, prob, keep, *r, y, ws,
                                  ws_bytes, None)

    for over in (dict(group=256), dict(x=None), dict(x=MISALIGNED), dict(idx=None),
                 dict(prob=None), dict(w1=None), dict(w3=_w4(moe, codes=None)),
                 dict(w2=_w4(moe, scales=MISALIGNED)), dict(y=None), dict(ws=None)):
        assert experts(**over) == INVALID, over
    assert experts(cfg=f32) == UNSUPPORTED
    assert experts(ws_bytes=need - 1) == WORKSPACE
    assert experts(cfg=moe.config(T=0, h=512, E=8, k=2, f=256), x=None, idx=None, prob=None,
                   y=None) == OK

    assert lib.moe_workspace_size_w4(ctypes.byref(cfg), ctypes.byref(size)) == OK
    assert size.value >= need + moe.workspace_size(cfg) - 256
    r = ctypes.byref(_w4(moe))
    args = [FAKE, FAKE, None, None, r, r, r, FAKE, None, None, None, FAKE]
    assert lib.moe_forward_w4(ctypes.byref(cfg), 64, *args, size.value - 1, None) == WORKSPACE
    args[1] = None   # Wg
    assert lib.moe_forward_w4(ctypes.byref(cfg), 64, *args, size.value, None) == INVALID


def test_binding_refuses_what_does_not_fit(moe):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):       # host tensors
        moe.layer_norm(x, None, None, 1e-5, x)
    with pytest.raises(ValueError):
        moe.layer_norm(x.half(), None, None, 1e-5, x.half())
    with pytest.raises(ValueError):       # weight of another width
        moe.layer_norm(x, torch.zeros(63), None, 1e-5, x)
    with pytest.raises(ValueError):       # weight and bias of two types
        moe.layer_norm(x, torch.zeros(64), torch.zeros(64, dtype=torch.bfloat16), 1e-5, x)
    with pytest.raises(ValueError):       # no rng
        moe.dropout_add(x, x, 0.5, None)
    with pytest.raises(ValueError):       # codes of another K
        moe.W4Weight(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4).bfloat16(), group=64)
    with pytest.raises(ValueError):       # zeros of another shape
        moe.W4Weight(torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1).bfloat16(),
                     torch.zeros(8, dtype=torch.uint8), group=128)
