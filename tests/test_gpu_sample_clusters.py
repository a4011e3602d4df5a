"""Sampling at the borders between its forms, against the definition in 64 bits (decode_cases):
1 to 16 blocks to a row, lists and bins, held rows and rows read again.

The bounds are those of test_gpu_sample.py: a weight is off by 2^-18 at most, so that answers with
borders further away than 1e-5 of the mass are met exactly.  Closer ones: the token lies between
those of u - 5e-5 and u + 5e-5, and its probability is its own weight over a sum that the moved
border changes by 1e-5 of the mass that top_p looks at, 1e-5 / top_p of what is kept, beside the
weights' own 2^-18 on both sides: with top_p of 0.4 and more 2.5e-5 + 8e-6, below 5e-5."""

import math

import numpy as np
import pytest
import torch

from decode_cases import sample_ref

pytestmark = pytest.mark.gpu
GAP = 1e-5


def run(logits, u, **choices):
    import mixture_experts_layer_fp32_gb300 as moe
    rows = logits.shape[0]
    tokens = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((rows,), float("nan"), device="cuda")
    moe.sample(logits, u, tokens, prob=prob, **choices)
    return tokens.cpu().numpy(), prob.double().cpu().numpy()


def verify(logits, u, which, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The answers of the rows `which`."""
    assert top_p >= 0.4
    got, prob = run(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    t, p, m = (float(np.float32(v)) for v in (temperature, top_p, min_p))
    exact = 0
    for r in which:
        l, ur = logits[r].double().cpu().numpy(), float(u[r])
        token, share, gap, gap_min = sample_ref(l, ur, t, top_k, p, m)
        if gap_min < GAP:
            continue
        if gap >= GAP:
            exact += 1
            assert got[r] == token, (r, got[r], token)
            assert abs(prob[r] - share) <= 2e-5 * share + 1e-9
            continue
        low, high = (sample_ref(l, ur + d, t, top_k, p, m)[0] for d in (-5e-5, 5e-5))
        assert low <= got[r] <= high, (r, got[r], low, high)
        total = math.exp((l[token] - l.max()) / t) / share
        own = math.exp((l[got[r]] - l.max()) / t) / total
        assert abs(prob[r] - own) <= 5e-5 * own + 1e-9
    return exact


def draw(rows, V, seed, dtype, std=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.empty(rows, V, device="cuda").normal_(0, std, generator=g)
    l += 5 * (torch.rand(rows, V, device="cuda", generator=g) < 8 / V).float()
    return l.to(dtype), torch.rand(rows, device="cuda", generator=g)


CHOICES = [dict(), dict(temperature=0.7, top_k=40), dict(top_p=0.9), dict(min_p=0.02),
           dict(temperature=1.5, top_p=0.5), dict(top_k=300, top_p=0.95, min_p=0.01),
           dict(temperature=1.2, top_k=2500), dict(top_k=4000, top_p=0.6)]

# 152 SMs run 9 clusters of 16 blocks at a time, 19 of 8, 38 of 4, 76 of 2, if all of them can: so
# many rows take 16, 8, 4, 2 blocks and 1 to a row
SHAPES = [(1, 40000), (9, 33001), (12, 40000), (20, 50001), (30, 40000), (39, 20001), (60, 30000),
          (77, 9001), (200, 4097)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,V", SHAPES)
def test_rows_of_every_number_of_blocks(rows, V, dtype):
    exact = 0
    for i, kw in enumerate(CHOICES):
        logits, u = draw(rows, V, 100 * rows + i, dtype)
        exact += verify(logits, u, sorted({0, rows // 2, rows - 1}), **kw)
    assert exact > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(3, 2047), (3, 2048), (3, 2049), (100, 2048), (100, 2049),
                                    (2, 4095), (2, 4096), (2, 4097)])
def test_around_the_list(rows, V, dtype):
    """2048 tokens are sorted at once; from 4096 on a row may have two blocks."""
    for i, kw in enumerate(CHOICES + [dict(top_k=V - 1), dict(top_k=V), dict(top_k=V + 1),
                                      dict(top_k=V - 1, top_p=0.99)]):
        logits, u = draw(rows, V, 7 * V + i, dtype)
        verify(logits, u, [0, 1, rows - 1], **kw)


@pytest.mark.parametrize("std", [0.3, 2.5])
@pytest.mark.parametrize("rows,V,k", [(1, 60000, 1199), (1, 60000, 1200), (1, 60000, 1201),
                                      (100, 5000, 341), (100, 5000, 342), (60, 9000, 682),
                                      (60, 9000, 683), (4, 60000, 2047), (4, 60000, 2048),
                                      (4, 60000, 2049)])
def test_around_the_top_k_that_is_gathered(rows, V, k, std):
    """Up to 1200, and a third of the threads of a row, the largest are gathered at once."""
    for i, kw in enumerate([dict(), dict(top_p=0.9), dict(temperature=0.5, min_p=0.01)]):
        logits, u = draw(rows, V, V + k + i, torch.float32, std)
        verify(logits, u, [0, rows - 1], top_k=k, **kw)


def test_more_likely_tokens_than_the_list_holds():
    """Runs of equal logits that overfill the list: the general form takes over.  (Of n equal
    weights a top_p lies on a border or within 1/n of one, so those answers are all close ones.)"""
    g = torch.Generator(device="cuda").manual_seed(11)
    logits = torch.randint(0, 4, (3, 50000), device="cuda", generator=g).float()
    u = torch.tensor([0.05, 0.5, 0.95], device="cuda")
    for kw in (dict(top_k=50), dict(top_k=1000, top_p=0.5), dict(top_k=13000), dict(top_p=0.45)):
        exact = verify(logits, u, [0, 1, 2], **kw)
        assert exact > 0 or "top_p" in kw


def test_rows_that_are_read_again():
    """Parts of a row that shared memory does not hold: 64 x 151936 fp32 in twos, and 80 in ones."""
    for rows in (64, 80):
        logits, u = draw(rows, 151936, rows, torch.float32)
        for kw in (dict(top_k=50, top_p=0.9), dict(top_p=0.9), dict(temperature=0.8)):
            verify(logits, u, [0, rows - 1], **kw)


def test_masked_row_has_one_right_answer():
    """Four tokens of the type's lowest value, u = 0.6: the third of four, the second of three."""
    for dtype in (torch.float32, torch.bfloat16):
        low = torch.finfo(dtype).min
        rows = torch.full((3, 4), low, dtype=dtype, device="cuda")
        u = torch.full((3,), 0.6, device="cuda")
        for kw, n in ((dict(), 4), (dict(top_k=3), 3), (dict(top_p=0.99), 4), (dict(top_p=0.75), 3),
                      (dict(top_k=3, top_p=0.99, min_p=0.1), 3), (dict(min_p=1.0), 4)):
            got, prob = run(rows, u, **kw)
            assert list(got) == [int(0.6 * n)] * 3, kw
            assert np.allclose(prob, 1 / n, rtol=2.0 ** -23)
