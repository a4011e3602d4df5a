"""examples/sublayer.py: the norm, the MoE layer, the dropout and their backward
as one training step, and the 4-bit decoding step, against 64-bit autograd and
the definitions."""

import importlib.util
import os

import pytest
import torch

import block_cases as bc

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "sublayer", os.path.join(ROOT, "examples", "sublayer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _normal(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return scale * torch.randn(shape, device="cuda", generator=g)


def _close(name, got, ref, tol):
    err = float((got.double() - ref).norm() / ref.norm())
    assert err <= tol, "%s: relative error %g > %g" % (name, err, tol)


def test_train_step_gradients():
    """An fp32 step.  Every value passes fewer than ten fp32 operations that are
    off by 2^-24 each and sums of up to 1000 terms, whose roundings add up like
    the root of their number: below 10 * 32 * 2^-24 = 2e-5 in the mean."""
    import mixture_experts_layer_fp32_gb300 as moe
    ex = _example()
    T, hidden, E, k, f, p = 96, 128, 4, 2, 192, 0.25
    cfg = moe.config(T=T, h=hidden, E=E, k=k, f=f, dtype="f32")
    h = _normal(T, hidden, seed=1)
    Wg = _normal(hidden, E, seed=2, scale=0.1)
    W1, W3 = (_normal(E, hidden, f, seed=s, scale=0.1) for s in (3, 4))
    W2 = _normal(E, f, hidden, seed=5, scale=0.1)
    weight, bias = 1 + _normal(hidden, seed=6, scale=0.1), _normal(hidden, seed=7, scale=0.1)
    d_out = _normal(T, hidden, seed=8)
    rng = torch.tensor([99, 12345], dtype=torch.int64, device="cuda")
    saved, grads = moe.Buffers(cfg), moe.Grads(cfg)
    ws = moe.alloc_workspace_backward(cfg)
    out, dh, dweight, dbias = ex.train_step(
        cfg, h, d_out, (Wg, W1, W3, W2), (weight, bias), p, rng, saved, grads, ws,
        moe.alloc_workspace_norm_backward(T, hidden))
    moe.check(ws)

    leaves = [t.double().requires_grad_() for t in (h, Wg, W1, W3, W2, weight, bias)]
    h64, g64, a64, b64, c64, w64, s64 = leaves
    mu = h64.mean(1, keepdim=True)
    n = (h64 - mu) * (h64.var(1, unbiased=False, keepdim=True) + ex.EPS).rsqrt() * w64 + s64
    idx = saved.topk_idx.long()
    prob = (n @ g64).gather(1, idx).softmax(1)
    m = torch.zeros_like(n)
    for e in range(E):
        y = (torch.nn.functional.silu(n @ a64[e]) * (n @ b64[e])) @ c64[e]
        m = m + y * ((idx == e) * prob).sum(1, keepdim=True)
    mask = bc.keep_mask(99, 12345, p, h.numel()).to(h.device).view(T, hidden)
    ref = h64 + m * mask / (1 - p)
    ref.backward(d_out.double())
    _close("out", out, ref.detach(), 2e-5)
    got = (dh, grads.dWg, grads.dW1, grads.dW3, grads.dW2, dweight, dbias)
    for name, a, leaf in zip(("dh", "dWg", "dW1", "dW3", "dW2", "dweight", "dbias"), got, leaves):
        _close(name, a, leaf.grad, 2e-5)


def test_decode_step():
    """The bf16 values on the way are rounded four times, by 2^-9 of their size
    in the mean at most: 4 * 2^-9 < 1e-2."""
    import mixture_experts_layer_fp32_gb300 as moe
    ex = _example()
    T, hidden, E, k, f, vocabulary = 5, 256, 8, 2, 384, 333
    cfg = moe.config(T=T, h=hidden, E=E, k=k, f=f)
    bf = torch.bfloat16
    Wg = _normal(hidden, E, seed=11, scale=0.1)
    experts = moe.quantize_experts_w4(
        *(_normal(*s, seed=i, scale=0.1).to(bf) for i, s in
          ((12, (E, hidden, f)), (13, (E, hidden, f)), (14, (E, f, hidden)))), group=64)
    # (the quantiser takes multiples of 64 outputs only)
    g = torch.Generator(device="cuda").manual_seed(15)
    codes, zeros = (torch.randint(0, 16, (vocabulary, n), dtype=torch.uint8, device="cuda",
                                  generator=g) for n in (hidden, hidden // 64))
    scales = 0.1 + 0.1 * torch.rand(zeros.shape, device="cuda", generator=g)
    head = moe.W4Weight(moe.pack_w4(codes), scales.to(bf), zeros, group=64)
    norms = [1 + _normal(hidden, seed=s, scale=0.1) for s in (16, 17)]
    h = _normal(T, hidden, seed=18).to(bf)
    decoder = ex.Decoder(cfg, Wg, experts, norms, head)
    logits = decoder.decode_step(h).clone()
    moe.check(decoder.ws)

    def rms(z, w):
        return z * (z.square().mean(1, keepdim=True) + ex.EPS).rsqrt() * w.double()

    W = [bc.w4_weight_ref(m.codes, m.scales, m.zeros, 64, m.k)
         for m in (experts.W1, experts.W3, experts.W2, head)]
    n = rms(h.double(), norms[0])
    m, _ = bc.experts_ref(n, decoder.idx.cpu(), decoder.prob.cpu(), None, *W[:3])
    _close("probabilities", decoder.prob,
           (n @ Wg.double()).gather(1, decoder.idx.long()).softmax(1), 1e-2)
    ref = rms(h.double() + m.to(h.device), norms[1]) @ W[3].t().to(h.device)
    _close("logits", logits, ref, 1e-2)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decoder.decode_step(h)
    decoder.logits.fill_(float("nan"))
    graph.replay()
    assert torch.equal(decoder.logits, logits)
