"""The whole layer for few tokens (moe_forward_few) against a reference in 64 bits
(decode_cases): routing exact, outputs within bounds derived there."""

import numpy as np
import pytest
import torch

from decode_cases import LayerCase, assert_close

pytestmark = pytest.mark.gpu


def call(c, y=None, ws=None, x=None):
    import mixture_experts_layer_fp32_gb300 as moe
    cfg = moe.config(T=c.T, h=c.h, E=c.E, k=c.k, f=c.f, score=c.score, dtype=c.dtype,
                     capacity_factor=c.capacity, drop_policy=c.policy,
                     min_capacity=c.min_capacity, num_groups=c.groups, group_topk=c.group_topk)
    x = c.x if x is None else x
    y = torch.full_like(c.x, float("nan")) if y is None else y
    ws = moe.alloc_workspace_few(cfg, c.fs) if ws is None else ws
    idx = torch.full((c.T, c.k), -7, dtype=torch.int32, device="cuda")
    prob = torch.full((c.T, c.k), float("nan"), device="cuda")
    tpe = torch.full((c.E,), -7, dtype=torch.int32, device="cuda")
    moe.forward_few(cfg, x, c.Wg, c.gb, c.eb, c.W1, c.W3, c.W2, y, ws, topk_idx=idx,
                    topk_prob=prob, tokens_per_expert=tpe, shared=c.shared)
    moe.check(ws)
    return y, idx, prob, tpe, ws, cfg


def verify(c, out):
    y, idx, prob, tpe = out[:4]
    ri, rp, rt, ry, bound = c.reference()
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(tpe.cpu().numpy(), rt)
    p = prob.double().cpu().numpy()
    assert np.array_equal(p > 0, rp > 0)
    assert (np.abs(p - rp) <= 1e-5 * rp + 1e-6).all()
    assert_close(y, ry, bound, c.dt)


BF16 = [
    dict(T=1, h=256, E=1, k=1, f=128),
    dict(T=1, h=512, E=8, k=2, f=384),
    dict(T=2, h=1024, E=5, k=3, f=640),
    dict(T=7, h=768, E=12, k=4, f=256, score="sigmoid", expert_bias=True),
    dict(T=8, h=256, E=64, k=8, f=128, score="sqrtsoftplus", expert_bias=True),
    dict(T=9, h=2048, E=32, k=4, f=128, groups=8, group_topk=2),
    dict(T=17, h=512, E=256, k=8, f=256, groups=8, group_topk=4, score="sigmoid",
         expert_bias=True, fs=256),
    dict(T=31, h=256, E=4, k=1, f=1408, score="softmax_pre", capacity=1.0),
    dict(T=33, h=256, E=2, k=2, f=256, fs=384),
    dict(T=48, h=512, E=16, k=2, f=384, capacity=1.25, policy="position", fs=128),
    dict(T=64, h=256, E=8, k=8, f=128, capacity=0.5),
    dict(T=64, h=512, E=3, k=1, f=512, score="softmax_pre", fs=512),
    dict(T=64, h=256, E=100, k=8, f=128, gate_bias=False),
    dict(T=64, h=256, E=24, k=2, f=256, same=True),
    dict(T=3, h=7168, E=8, k=2, f=256),
    dict(T=5, h=256, E=4, k=2, f=8192),
]
F32 = [
    dict(T=1, h=8, E=1, k=1, f=8),
    dict(T=1, h=128, E=8, k=2, f=256),
    dict(T=3, h=24, E=7, k=2, f=40, fs=16),
    dict(T=7, h=1032, E=12, k=3, f=1416, score="sigmoid", expert_bias=True),
    dict(T=16, h=136, E=16, k=4, f=264, groups=4, group_topk=2, fs=520),
    dict(T=33, h=200, E=3, k=2, f=72, capacity=1.0),
    dict(T=64, h=512, E=5, k=1, f=520, score="softmax_pre", capacity=0.7, policy="position"),
    dict(T=64, h=64, E=256, k=8, f=16),
    dict(T=64, h=72, E=2, k=2, f=1000, fs=24),
]


@pytest.mark.parametrize("kw", BF16, ids=str)
def test_bf16(kw):
    c = LayerCase(**kw).cuda()
    verify(c, call(c))


@pytest.mark.parametrize("kw", F32, ids=str)
def test_f32(kw):
    c = LayerCase(dtype="f32", **kw).cuda()
    verify(c, call(c))
