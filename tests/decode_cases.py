"""References in 64 bits for the operators of a decoding step (the layer for few
tokens), with the error bounds that their tests use.  Plain numpy/torch, no code
of the package.

u = 2^-24 is half a step of fp32, `half(t)` half a step of an output type."""

import math

import numpy as np
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------- the layer

class LayerCase:
    """Seeded inputs of one layer on the GPU; every token's choice of experts is
    clear of what 32-bit sums can change."""

    def __init__(self, T, h, E, k, f, dtype="bf16", score="softmax_post", groups=0, group_topk=0,
                 fs=0, capacity=0.0, policy="probs", min_capacity=0, gate_bias=True,
                 expert_bias=False, seed=0, same=False):
        self.__dict__.update({n: v for n, v in locals().items() if n != "self"})
        self.dt = torch.float32 if dtype == "f32" else torch.bfloat16
        g = torch.Generator().manual_seed(1000 * seed + 7 * T + h + E + f)
        draw = lambda shape, std: std * torch.randn(shape, generator=g)  # noqa: E731
        self.Wg = draw((h, E), h ** -0.5)
        self.gb = draw((E,), 0.5) if gate_bias else None
        self.eb = 0.2 * torch.rand(E, generator=g) - 0.1 if expert_bias else None
        x = draw((2 * T + 8, h), 1.0).to(self.dt)
        if same:  # every token the same: they all meet the same experts
            x = x[:1].expand(2 * T + 8, h).contiguous()
        clear = [t for t in range(x.shape[0]) if self.margin(x[t]) > 1e-4]
        assert len(clear) >= T
        self.x = x[clear[:T]].contiguous()
        self.W1, self.W3 = (draw((E, h, f), h ** -0.5).to(self.dt) for _ in range(2))
        self.W2 = draw((E, f, h), f ** -0.5).to(self.dt)
        self.shared = None
        if fs:
            self.shared = (draw((h, fs), h ** -0.5).to(self.dt),
                           draw((h, fs), h ** -0.5).to(self.dt),
                           draw((fs, h), fs ** -0.5).to(self.dt))

    def cuda(self):
        for n in ("x", "Wg", "gb", "eb", "W1", "W3", "W2"):
            v = getattr(self, n)
            setattr(self, n, None if v is None else v.cuda())
        if self.shared is not None:
            self.shared = tuple(v.cuda() for v in self.shared)
        return self

    def scores(self, x):
        """(scores of the weights, selection scores) of one token, float64 numpy."""
        l = (x.double() @ self.Wg.double()).cpu().numpy()
        if self.gb is not None:
            l = l + self.gb.double().cpu().numpy()
        if self.score == "softmax_pre":
            s = np.exp(l - l.max())
            s = s / s.sum()
        elif self.score == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        elif self.score == "sqrtsoftplus":
            s = np.sqrt(np.log1p(np.exp(-np.abs(l))) + np.maximum(l, 0))
        else:
            s = l
        return s, s if self.eb is None else s + self.eb.double().cpu().numpy()

    def allowed(self, sel):
        if self.groups <= 1:
            return list(range(self.E)), []
        n = self.E // self.groups
        m = self.k // self.group_topk
        top = [np.sort(sel[g * n:(g + 1) * n])[::-1][:m].sum() for g in range(self.groups)]
        best = sorted(range(self.groups), key=lambda g: (-top[g], g))
        keep = set(best[:self.group_topk])
        gap = []
        if self.group_topk < self.groups:
            gap = [top[best[self.group_topk - 1]] - top[best[self.group_topk]]]
        return [e for e in range(self.E) if e // n in keep], gap

    def margin(self, x):
        _, sel = self.scores(x)
        allowed, gaps = self.allowed(sel)
        best = sorted((-sel[e] for e in allowed))[:self.k + 1]
        return min(gaps + [b - a for a, b in zip(best, best[1:])] + [1.0])

    def route(self):
        """idx [T,k], p [T,k] float64 (0: dropped), tokens per expert."""
        T, k = self.T, self.k
        idx, p = np.zeros((T, k), np.int64), np.zeros((T, k))
        for t in range(T):
            s, sel = self.scores(self.x[t])
            idx[t] = sorted(self.allowed(sel)[0], key=lambda e: (-sel[e], e))[:k]
            v = s[idx[t]]
            if self.score == "softmax_post":
                v = np.exp(v - v[0])
                v = v / v.sum()
            elif self.score != "softmax_pre":
                v = v / (v.sum() + 1e-20)
            p[t] = v
        kept = np.ones((T, k), bool)
        if self.capacity > 0:
            cap = max(math.ceil(T * k / self.E * float(np.float32(self.capacity))),
                      self.min_capacity)
            for e in range(self.E):
                pairs = [(t, j) for t in range(T) for j in range(k) if idx[t, j] == e]
                if self.policy == "probs":
                    pairs.sort(key=lambda q: (-np.float32(p[q]), q[0]))
                for q in pairs[cap:]:
                    kept[q] = False
        p = np.where(kept, p, 0.0)
        return idx, p, np.bincount(idx[kept], minlength=self.E)

    def swiglu(self, x, W1, W3, W2):
        """(result, error bound) of one expert.  A product's sum: the tensor cores
        add 16 products (fp32: one) to a running sum and may cut instead of round,
        2u a step, and runs are added up; the terms' magnitudes bound each step."""
        step = 1 if self.dtype == "f32" else 16
        W1, W3, W2 = (w.double() for w in (W1, W3, W2))

        def product(v, W, ev):
            y = v @ W
            size = v.abs() @ W.abs()
            return y, (W.shape[0] / step + 16 + 8) * 2 * U * size + ev @ W.abs()

        a, ea = product(x, W1, torch.zeros_like(x))
        b, eb = product(x, W3, torch.zeros_like(x))
        s = a * torch.sigmoid(a)
        hid = s * b
        # |silu'| <= 1.1; exp, the quotient and the product: 8 u; two bf16 pieces: 2^-17
        eh = (1.1 * ea * (b.abs() + eb) + s.abs() * eb + 8 * U * (hid.abs() + ea * eb) +
              (0 if self.dtype == "f32" else 2.0 ** -17) * hid.abs())
        return product(hid, W2, eh)

    def reference(self):
        """idx, p, tokens per expert, y and its bound before the last rounding."""
        idx, p, tpe = self.route()
        x = self.x.double()
        y, bound = torch.zeros_like(x), torch.zeros_like(x)
        for e in sorted(set(idx[p > 0].tolist())):
            t, j = np.nonzero((idx == e) & (p > 0))
            t, w = torch.from_numpy(t).to(x.device), torch.from_numpy(p[t, j]).to(x.device)
            out, err = self.swiglu(x[t], self.W1[e], self.W3[e], self.W2[e])
            y.index_add_(0, t, w[:, None] * out)
            # the weights' own error, as the tests of the router allow it
            bound.index_add_(0, t, w[:, None] * err + (1e-5 * w[:, None] + 1e-6) * out.abs() +
                             self.k * 2 * U * (w[:, None] * out).abs())
        if self.shared is not None:
            out, err = self.swiglu(x, *self.shared)
            y = y + out
            bound = bound + err + 2 * U * y.abs()
        return idx, p, tpe, y, bound + self.k * U * y.abs()


def assert_close(got, y, bound, dtype):
    """Within the bound and half a step of the output's type."""
    limit = bound + half(dtype) * (y.abs() + bound) + 1e-30
    over = (got.double() - y).abs() / limit
    assert bool(torch.isfinite(got).all())
    assert float(over.max()) <= 1.0, "error %.2f of what is allowed" % float(over.max())


# ----------------------------------------------------------------- sampling

def sample_ref(l, u, t, top_k, top_p, min_p):
    """One row (float64 numpy logits) -> (token, its probability, the least gap between
    u or top_p and a border between two tokens, in units of the whole mass, and that
    between min_p and a weight)."""
    V = l.size
    order = sorted(range(V), key=lambda i: (-l[i], i))
    order = np.array([i for i in order if l[i] > -np.inf], dtype=np.int64)
    if order.size == 0:
        return -1, 0.0, 1.0, 1.0
    if not t > 0 or top_k == 1:
        return int(order[0]), 1.0, 1.0, 1.0
    top = l[order[0]]
    w = np.array([1.0 if l[i] == top else math.exp((l[i] - top) / t) for i in order])
    gap = gap_min = 1.0
    if top_k > 0:
        w = w[:top_k]
    if top_p < 1:
        cum = np.cumsum(w) / w.sum()
        n = int(np.argmax(cum >= top_p))
        gap = min(gap, np.abs(cum - top_p).min() if top_p > 0 else 1.0)
        w = w[:n + 1]
    if min_p > 0:
        gap_min = np.abs(w / min(min_p, 1.0) - 1)[1:].min(initial=1.0)
        w = w[np.concatenate(([True], w[1:] >= min(min_p, 1.0)))]
    kept = np.sort(order[:w.size])
    by = np.argsort(order[:w.size], kind="stable")
    share = w[by] / w.sum()
    cum = np.cumsum(share)
    u = min(max(u, 0.0), 1 - 2.0 ** -24)
    at = min(int(np.searchsorted(cum, u, side="right")), w.size - 1)
    gap = min(gap, np.abs(cum - u)[:-1].min(initial=1.0) if u > 0 else 1.0)
    return int(kept[at]), float(share[at]), gap, gap_min
