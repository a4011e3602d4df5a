"""Sampling from rows so long and flat that the sums of weights near the numbers that hold them.
All weights are 1 here, so the answer is one of whole numbers: of n kept tokens the floor(u n)-th
(u has 24 bits and n too: u n is exact in 64-bit floating point)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
MOST = 2 ** 24 - 1   # the largest vocabulary


def draw(logits, u, **choices):
    import mixture_experts_layer_fp32_gb300 as moe
    rows = logits.shape[0]
    tokens = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((rows,), float("nan"), device="cuda")
    moe.sample(logits, u, tokens, prob=prob, **choices)
    return tokens.cpu().numpy(), prob.double().cpu().numpy()


def numbers(rows, seed):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(rows, generator=g)
    u[0], u[-1] = 0.0, 1 - 2.0 ** -24
    return u


def check(logits, n, u, **choices):
    got, prob = draw(logits, u.cuda(), **choices)
    assert np.array_equal(got, np.floor(u.double().numpy() * n).astype(np.int64))
    assert np.allclose(prob, 1 / n, rtol=2.0 ** -23, atol=0)


# A thread's 32-bit sums are of up to 4095 tokens: 4095 x 1024 tokens to a block.
@pytest.mark.parametrize("rows,V", [(80, 4095 * 1024), (80, 4095 * 1024 + 1), (80, 4096 * 1024),
                                    (80, 4096 * 1024 + 77), (40, 2 * 4096 * 1024),
                                    (40, 2 * 4095 * 1024)])
def test_flat_rows_of_long_parts(rows, V):
    """More rows than run at once with more blocks to each: parts of some 2^22 tokens."""
    logits = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    check(logits, V, numbers(rows, V))


@pytest.mark.parametrize("V", [MOST, 2 ** 23 + 1])
def test_flat_row_at_the_largest_vocabulary(V):
    logits = torch.full((3, V), -2.5, device="cuda")
    u = numbers(3, V)
    check(logits, V, u)
    check(logits, V, u, min_p=0.5)
    k = 2 ** 23 - 3
    check(logits, k, u, top_k=k)
    check(logits, -(-V // 2), u, top_p=0.5)      # the fewest that reach half of all
    check(logits, -(-k // 4), u, top_k=k, top_p=0.25)


def test_any_logits_weigh_the_same_at_an_endless_temperature():
    g = torch.Generator(device="cuda").manual_seed(3)
    V = 2 ** 23 + 12345
    logits = torch.empty(2, V, device="cuda").normal_(0, 5, generator=g)
    u = torch.tensor([0.3, 0.999])
    for t in (float("inf"), 1e30):
        check(logits, V, u, temperature=torch.full((2,), t, device="cuda"))
