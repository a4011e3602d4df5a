"""examples/sublayer.py: a decoding step with the layer for few tokens, a head in 8 bits and
sampling, against the definitions in 64 bits."""

import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from decode_cases import LayerCase, sample_ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "sublayer", os.path.join(ROOT, "examples", "sublayer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rms(z, w, eps):
    return z * (z.square().mean(1, keepdim=True) + eps).rsqrt() * w.double()


def test_decode_step_and_next_tokens():
    """The bf16 values on the way are rounded three times, by 2^-9 of their size in the mean at
    most, and the head's input to 8 bits: half a step of a 127th of its largest, about 4 of its
    own mean, 0.5 / 127 * 4 / sqrt(3) = 9e-3: together below 2e-2."""
    import mixture_experts_layer_fp32_gb300 as moe
    ex = _example()
    c = LayerCase(T=6, h=512, E=8, k=2, f=384, gate_bias=False, seed=3).cuda()
    vocabulary = 1003
    g = torch.Generator(device="cuda").manual_seed(4)
    norms = [1 + 0.1 * torch.randn(c.h, device="cuda", generator=g) for _ in range(2)]
    head = moe.quantize_i8(torch.randn(vocabulary, c.h, device="cuda", generator=g) * c.h ** -0.5)
    cfg = moe.config(T=c.T, h=c.h, E=c.E, k=c.k, f=c.f)
    decoder = ex.Decoder(cfg, c.Wg, (c.W1, c.W3, c.W2), norms, head)
    h = c.x.clone()
    logits = decoder.decode_step(h).clone()
    u = torch.rand(c.T, device="cuda", generator=g)
    choices = dict(temperature=0.7, top_k=40, top_p=0.9)
    tokens = decoder.next_tokens(u, **choices).clone()
    moe.check(decoder.ws)

    n = _rms(h.double(), norms[0], ex.EPS)
    c.x = n
    m = torch.zeros_like(n)
    prob = (n @ c.Wg.double()).gather(1, decoder.idx.long()).softmax(1)
    for t in range(c.T):
        for j in range(c.k):
            e = int(decoder.idx[t, j])
            m[t] += prob[t, j] * c.swiglu(n[t:t + 1], c.W1[e], c.W3[e], c.W2[e])[0][0]
    W = head.codes.double() * head.scales.double()[:, None]
    ref = _rms(h.double() + m, norms[1], ex.EPS) @ W.t()
    assert float((logits.double() - ref).norm() / ref.norm()) <= 2e-2
    # the tokens are those of the logits that there are
    l = logits.double().cpu().numpy()
    for t in range(c.T):
        token, _, gap, _ = sample_ref(l[t], float(u[t]), np.float32(0.7).item(), 40,
                                      np.float32(0.9).item(), 0.0)
        assert gap < 1e-5 or int(tokens[t]) == token

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decoder.decode_step(h)
        decoder.next_tokens(u, **choices)
    for _ in range(3):
        decoder.logits.fill_(float("nan"))
        decoder.tokens.fill_(-5)
        graph.replay()
        assert torch.equal(decoder.logits, logits) and torch.equal(decoder.tokens, tokens)


def test_a_step_with_4_bit_experts_and_a_head_in_8():
    """The parts can be mixed: the same head on the layer's output of either kind of experts."""
    import mixture_experts_layer_fp32_gb300 as moe
    ex = _example()
    c = LayerCase(T=3, h=256, E=4, k=2, f=256, gate_bias=False, seed=8).cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    norm = torch.ones(c.h, device="cuda")
    head = moe.quantize_i8(torch.randn(320, c.h, device="cuda", generator=g))
    cfg = moe.config(T=c.T, h=c.h, E=c.E, k=c.k, f=c.f)
    decoder = ex.Decoder(cfg, c.Wg, moe.quantize_experts_w4(c.W1, c.W3, c.W2, group=64),
                         (norm, norm), head)
    logits = decoder.decode_step(c.x)
    moe.check(decoder.ws)
    codes = torch.empty(c.T, c.h, dtype=torch.int8, device="cuda")
    scales = torch.empty(c.T, device="cuda")
    moe.quantize_rows_i8(decoder.n2, codes, scales)
    want = (codes.double() @ head.codes.double().t()).float() * scales[:, None] * head.scales
    assert torch.equal(logits, want)


def test_first_calls_are_captured():
    """A process whose first calls of the three operators are captured into a graph."""
    code = """
import torch
import mixture_experts_layer_fp32_gb300 as moe
d = dict(device="cuda")
bf = torch.bfloat16
x = torch.randn(9, 256, **d).to(bf)
Wg = torch.randn(256, 4, **d)
W = [torch.randn(4, 256, 256, **d).to(bf) * 0.1 for _ in range(3)]
cfg = moe.config(T=9, h=256, E=4, k=2, f=256)
ws = moe.alloc_workspace_few(cfg)
w = moe.I8Weight(torch.randint(-127, 128, (1000, 256), dtype=torch.int8, **d), torch.ones(1000, **d))
wl = moe.alloc_workspace_linear_i8(20, w)
x2 = torch.randn(20, 256, **d)
u = torch.rand(20, **d)
def step():
    y = torch.zeros(9, 256, dtype=bf, **d)
    moe.forward_few(cfg, x, Wg, None, None, *W, y, ws)
    logits = torch.zeros(20, 1000, **d)
    moe.linear_i8(x2, w, logits, wl)
    tokens = torch.zeros(20, dtype=torch.int32, **d)
    moe.sample(logits, u, tokens, top_k=30)
    return y, logits, tokens
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
moe.check(ws), moe.check(wl)
want = step()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert float(got[0].abs().max()) > 0 and int(got[2].max()) > 0
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
