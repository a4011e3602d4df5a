"""The feed-forward half of a transformer block around the MoE layer.

    out = h + dropout(MoE(norm(h)))

train_step runs it forward and backward: the norm, the layer's stages, the
dropout with the residual sum, and back through all of them, with the dropout's
mask drawn again from its seed and offset instead of stored.  decode_step runs
it for a few tokens with the experts in 4 bits, then the next norm (which adds
the residual as it reads it) and a head in 4 bits.

    python -m examples.sublayer      (from the root of the repository)
"""

import torch

import mixture_experts_layer_fp32_gb300 as moe

EPS = 1e-5


def train_step(cfg, h, d_out, weights, norm, p, rng, saved, grads, ws, norm_ws):
    """h, d_out [T,h] -> out and the gradients.  weights: Wg, W1, W3, W2; norm:
    weight and bias; saved: moe.Buffers; grads: moe.Grads.  Returns out, dh,
    dweight, dbias; the layer's own gradients are in `grads`."""
    Wg, W1, W3, W2 = weights
    rows, hidden = h.shape
    mean, rstd = (torch.empty(rows, device=h.device) for _ in range(2))
    n, out = torch.empty_like(h), torch.empty_like(h)
    b = saved
    moe.layer_norm(h, *norm, EPS, n, mean, rstd)
    moe.route(cfg, n, Wg, None, None, b.topk_idx, b.topk_prob, b.keep, b.tokens_per_expert, None,
              b.ws)
    moe.permute(cfg, n, b.topk_idx, b.keep, b.x_perm, b.row_map, b.expert_offsets, b.ws)
    moe.grouped_mlp(cfg, b.x_perm, b.expert_offsets, W1, W3, W2, b.h_mid, b.y_perm, b.ws)
    moe.combine(cfg, b.y_perm, b.row_map, b.topk_prob, b.y)
    moe.dropout_add(b.y, out, p, rng, residual=h)

    d_moe, dh = torch.empty_like(h), torch.empty_like(h)
    dweight, dbias = (torch.empty(hidden, device=h.device) for _ in range(2))
    moe.dropout_add(d_out, d_moe, p, rng)
    moe.backward(cfg, n, Wg, None, W1, W3, W2, b, d_moe, grads, ws)
    # the residual's gradient joins the norm's where that is written
    moe.layer_norm_backward(grads.dx, h, norm[0], mean, rstd, dh, dweight, dbias, norm_ws,
                            dz=d_out)
    return out, dh, dweight, dbias


class Decoder:
    """Buffers and 4-bit weights of decode_step for cfg's number of tokens."""

    def __init__(self, cfg, Wg, experts, norms, head):
        self.cfg, self.Wg, self.experts, self.norms, self.head = cfg, Wg, experts, norms, head
        T, hidden, k = cfg.num_tokens, cfg.hidden, cfg.topk
        self.n, self.m, self.out, self.n2 = (
            torch.empty((T, hidden), dtype=torch.bfloat16, device="cuda") for _ in range(4))
        self.logits = torch.empty((T, head.n), device="cuda")
        self.idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
        self.prob = torch.empty((T, k), device="cuda")
        self.ws = moe.alloc_workspace_w4(cfg)
        self.head_ws = moe.alloc_workspace_linear_w4(T, head)

    def decode_step(self, h):
        """h [T,h] bf16 -> logits [T, vocabulary] fp32; no allocation, so a step
        can be captured into a graph."""
        moe.layer_norm(h, self.norms[0], None, EPS, self.n, rms=True)
        moe.forward_w4(self.cfg, self.n, self.Wg, None, None, self.experts, self.m, self.ws,
                       topk_idx=self.idx, topk_prob=self.prob)
        moe.layer_norm(self.m, self.norms[1], None, EPS, self.n2, rms=True, residual=h,
                       z=self.out)
        moe.linear_w4(self.n2, self.head, self.logits, self.head_ws)
        return self.logits


def main():
    torch.manual_seed(0)
    T, hidden, E, k, f, vocabulary = 256, 512, 8, 2, 1024, 1024

    def normal(*shape, dtype=torch.bfloat16):
        return (0.02 * torch.randn(shape, device="cuda")).to(dtype)

    Wg = normal(hidden, E, dtype=torch.float32)
    W1, W3, W2 = normal(E, hidden, f), normal(E, hidden, f), normal(E, f, hidden)
    norm = torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")

    cfg = moe.config(T=T, h=hidden, E=E, k=k, f=f)
    h = torch.randn((T, hidden), device="cuda").to(torch.bfloat16)
    d_out = torch.randn((T, hidden), device="cuda").to(torch.bfloat16)
    rng = torch.tensor([1234, 0], dtype=torch.int64, device="cuda")
    grads = moe.Grads(cfg)
    ws = moe.alloc_workspace_backward(cfg)
    out, dh, dweight, dbias = train_step(
        cfg, h, d_out, (Wg, W1, W3, W2), norm, 0.1, rng, moe.Buffers(cfg), grads, ws,
        moe.alloc_workspace_norm_backward(T, hidden))
    moe.check(ws)
    print("training: |out| %.3f |dh| %.3f |dW1| %.3f |dweight| %.3f" % tuple(
        float(t.float().norm()) for t in (out, dh, grads.dW1, dweight)))

    few = moe.config(T=4, h=hidden, E=E, k=k, f=f)
    head = moe.quantize_w4(normal(hidden, vocabulary), group=64, zeros=True)
    decoder = Decoder(few, Wg, moe.quantize_experts_w4(W1, W3, W2, group=64), (norm[0], norm[0]),
                      head)
    logits = decoder.decode_step(h[:4].contiguous())
    moe.check(decoder.ws)
    print("decoding: next tokens", logits.argmax(-1).tolist())


if __name__ == "__main__":
    main()
