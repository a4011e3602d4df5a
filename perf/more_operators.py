"""The operators of a decoding step, as measured cases.

Three operators: the whole MoE layer for a few tokens with the layer's own weights (``layer``:
router, capacity drops, SwiGLU experts, combine, optionally a shared expert), the product in
8-bit integers with a scale for each token and output channel (``linear``: rows of bf16 or fp32
quantised in the call, or codes that are there already) and the choice of the next token from
given random numbers (``sample``: temperature, top-k, top-p, min-p).  ``run`` computes them in
plain torch operations, or through this package's entry points where ``own`` is true; ``exact``
holds the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LAYER = dict(score="softmax_post", dtype="bf16", groups=0, group_topk=0, shared=0, capacity=0.0,
             policy="probs", bias=False)


def listed():
    return [
        # decoding one token, two of eight wide experts
        dict(LAYER, name="layer one token", op="layer", tokens=1, hidden=4096, experts=8, topk=2,
             ffn=14336),
        # a few tokens of a small fp32 layer, widths that no tile divides, sigmoid scores with a
        # bias that only chooses
        dict(LAYER, name="layer few tokens fp32", op="layer", tokens=7, hidden=1032, experts=12,
             topk=3, ffn=1416, score="sigmoid", bias=True, dtype="f32"),
        # decoding of a batch, fine-grained experts: most are hit by a few tokens
        dict(LAYER, name="layer fine-grained batch", op="layer", tokens=32, hidden=4096,
             experts=128, topk=8, ffn=1536),
        # expert groups and a shared expert that every token goes through
        dict(LAYER, name="layer groups and shared expert", op="layer", tokens=8, hidden=7168,
             experts=64, topk=8, ffn=2048, score="sigmoid", bias=True, groups=8, group_topk=4,
             shared=2048),
        # one token through a square projection: latency counts
        dict(name="linear one token", op="linear", rows=1, n=4096, k=4096, x="bf16", bias=False,
             out="bf16"),
        # a few fp32 rows, an odd number of outputs, a bias, fp32 results
        dict(name="linear few tokens", op="linear", rows=13, n=14337, k=7168, x="f32", bias=True,
             out="f32"),
        # the head of a batch: a large vocabulary, codes from an earlier quantisation, fp32 logits
        dict(name="linear head of a batch", op="linear", rows=64, n=151936, k=4096, x="i8",
             bias=False, out="f32"),
        # a prompt through a wide projection: the arithmetic counts
        dict(name="linear prompt", op="linear", rows=8192, n=14336, k=4096, x="bf16", bias=False,
             out="bf16"),
        # the next token of one sequence, one set of choices
        dict(name="sample one sequence", op="sample", rows=1, vocab=128000, dtype="f32",
             temperature=0.8, top_k=0, top_p=0.9, min_p=0.0, each=False),
        # a batch whose sequences have choices of their own, some of them greedy
        dict(name="sample batch", op="sample", rows=64, vocab=151936, dtype="bf16",
             temperature=1.0, top_k=50, top_p=0.95, min_p=0.02, each=True),
        # an odd small vocabulary, nothing but the temperature
        dict(name="sample odd vocabulary", op="sample", rows=5, vocab=1009, dtype="f32",
             temperature=1.3, top_k=0, top_p=1.0, min_p=0.0, each=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer", "layer", "linear", "sample"])
    if op == "linear":
        rows, k = _log(rng, 1, 8192), _log(rng, 8, 896) * 16
        most = min(151936, (1 << 30) // k, 8192 * 14336 * 4096 // (rows * k))
        return dict(op=op, rows=rows, n=_log(rng, 64, max(64, most)), k=k,
                    x=rng.choice(["bf16", "bf16", "f32", "i8"]), bias=rng.random() < 0.4,
                    out=rng.choice(["bf16", "f32"]))
    if op == "sample":
        vocab = _log(rng, 500, 262144)
        return dict(op=op, rows=_log(rng, 1, max(1, min(512, 64 * 151936 // vocab))), vocab=vocab,
                    dtype=rng.choice(["f32", "f32", "bf16"]),
                    temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5]),
                    top_k=rng.choice([0, 0, 1, 20, 50, 1000]),
                    top_p=rng.choice([1.0, 0.5, 0.9, 0.95, 0.99]),
                    min_p=rng.choice([0.0, 0.0, 0.01, 0.1]), each=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    score = rng.choice(["softmax_post", "softmax_pre", "sigmoid", "sqrtsoftplus"])
    experts = _log(rng, 1, 128)
    topk = min(experts, rng.choice([1, 2, 4, 8]))
    groups = group_topk = 0
    if experts % 8 == 0 and experts >= 16 and topk % 2 == 0 and rng.random() < 0.3:
        groups, group_topk = experts // 8, 2
    if dtype == "bf16":
        hidden, unit = _log(rng, 1, 28) * 256, 128
    else:
        hidden, unit = _log(rng, 8, 896) * 8, 8
    most = 128 * 4096 * 1536 // (2 if dtype == "f32" else 1)
    ffn = _log(rng, 1, max(1, min(14336 // unit, most // experts // hidden // unit))) * unit
    return dict(op=op, tokens=_log(rng, 1, 64), hidden=hidden, experts=experts, topk=topk,
                ffn=ffn, score=score, dtype=dtype, groups=groups, group_topk=group_topk,
                shared=rng.choice([0, 0, _log(rng, 1, max(1, min(ffn, 4096) // unit)) * unit]),
                capacity=rng.choice([0.0, 0.0, 1.0, 1.5]),
                policy=rng.choice(["probs", "position"]),
                bias=score in ("sigmoid", "sqrtsoftplus") and rng.random() < 0.7)


# ------------------------------------------------------------------- inputs

def _normal(gen, shape, std, dtype):
    """Normal values, a part of the first dimension at a time."""
    out = torch.empty(shape, device="cuda", dtype=dtype)
    if len(shape) < 3:
        return out.copy_(std * torch.randn(shape, device="cuda", generator=gen))
    for i in range(shape[0]):
        out[i] = std * torch.randn(shape[1:], device="cuda", generator=gen)
    return out


def _logits64(x, Wg, gate_bias):
    return x.double() @ Wg.double() + gate_bias.double()


def _margin(case, logits, expert_bias):
    """How far each token is from another choice of experts, or another order of them: the least
    gap between neighbouring scores among those that decide."""
    if case["score"] == "sigmoid":
        logits = torch.sigmoid(logits) + (0 if expert_bias is None else expert_bias.double())
    elif case["score"] == "sqrtsoftplus":
        logits = torch.nn.functional.softplus(logits).sqrt()
        logits = logits + (0 if expert_bias is None else expert_bias.double())
    elif case["groups"] > 1 and case["score"] == "softmax_pre":
        logits = torch.softmax(logits, 1)
    gap = logits.new_full((logits.shape[0],), 1.0)
    if case["groups"] > 1:
        by_group = logits.view(logits.shape[0], case["groups"], -1)
        scores = by_group.topk(case["topk"] // case["group_topk"], dim=2)[0].sum(2)
        best = scores.sort(dim=1, descending=True)[0]
        g = case["group_topk"]
        if g < case["groups"]:
            gap = torch.minimum(gap, best[:, g - 1] - best[:, g])
        keep = torch.zeros_like(scores, dtype=torch.bool)
        keep.scatter_(1, scores.topk(g, dim=1)[1], True)
        logits = by_group.masked_fill(~keep[:, :, None], -1e30).flatten(1)
    best = logits.sort(dim=1, descending=True)[0][:, :case["topk"] + 1]
    if best.shape[1] > 1:
        gap = torch.minimum(gap, (best[:, :-1] - best[:, 1:]).min(dim=1)[0])
    return gap


def _prepare_layer(case, gen, st):
    T, h, E, f = (case[n] for n in ("tokens", "hidden", "experts", "ffn"))
    dt = DTYPES[case["dtype"]]
    st["Wg"] = _normal(gen, (h, E), h ** -0.5, torch.float32)
    st["gate_bias"] = _normal(gen, (E,), 0.3, torch.float32)
    st["expert_bias"] = None
    if case["bias"]:
        st["expert_bias"] = 0.2 * torch.rand(E, device="cuda", generator=gen) - 0.1
    # A token whose choice hangs on the last bits of a 32-bit sum has no one right answer: of
    # twice as many tokens, the first ones that are clear of that.
    x = _normal(gen, (2 * T + 16, h), 1.0, dt)
    gap = _margin(case, _logits64(x, st["Wg"], st["gate_bias"]), st["expert_bias"])
    order = torch.argsort((gap < 2e-5).to(torch.int8), stable=True)
    st["x"] = x[order[:T]].contiguous()
    std = h ** -0.5
    st["W1"], st["W3"] = (_normal(gen, (E, h, f), std, dt) for _ in range(2))
    st["W2"] = _normal(gen, (E, f, h), f ** -0.5, dt)
    st["shared"] = None
    if case["shared"]:
        fs = case["shared"]
        st["shared"] = (_normal(gen, (h, fs), std, dt), _normal(gen, (h, fs), std, dt),
                        _normal(gen, (fs, h), fs ** -0.5, dt))


def _prepare_sample(case, gen, st):
    rows, V = case["rows"], case["vocab"]
    logits = 2.5 * torch.randn(rows, V, device="cuda", generator=gen)
    # a few tokens that the model prefers, and some that the program has ruled out
    logits += 6 * (torch.rand(rows, V, device="cuda", generator=gen) < 20.0 / V).float()
    out = torch.rand(rows, V, device="cuda", generator=gen)
    logits = torch.where(out < 0.01, float("-inf"), logits)
    logits = torch.where(out > 0.995, torch.finfo(DTYPES[case["dtype"]]).min, logits)
    logits[:, 0] = 1.0
    logits = st["logits"] = logits.to(DTYPES[case["dtype"]])

    def each(value, low, high):
        """Rows' own values, or one for all: spread around the case's."""
        r = torch.rand(rows, dtype=torch.float64, device="cuda", generator=gen)
        if not case["each"]:
            return torch.full_like(r, value)
        return low + (high - low) * r

    t = case["temperature"]
    temperature = each(t, 0.5 * t, 1.5 * t)
    if case["each"]:
        temperature[::7] = 0.0
    temperature = temperature.float()
    k = case["top_k"]
    top_k = each(k, 1, 2 * k + 1).floor().int() if k else torch.zeros(rows, dtype=torch.int32,
                                                                     device="cuda")
    p = case["top_p"]
    top_p = each(p, 2 * p - 1, 1.0) if p < 1 else each(p, 1.0, 1.0)
    m = case["min_p"]
    min_p = each(m, 0.2 * m, 2 * m)
    # Where a border between two tokens is closer than 32-bit weights are, there is no one right
    # answer: top_p and min_p are moved to the middle between the two sums or weights on either
    # side, and of eight random numbers the one furthest from a border is taken.
    order = logits.double().sort(dim=1, descending=True, stable=True)
    z = order[0] - order[0][:, :1]
    w = torch.exp(z / torch.where(temperature > 0, temperature, 1.0).double()[:, None])
    w = torch.where((temperature > 0)[:, None], w, (torch.arange(V, device="cuda") == 0).double())
    place = torch.arange(V, device="cuda")
    if k:
        w = w * (place < top_k[:, None])
    cum = w.cumsum(1)
    total = cum[:, -1:]
    n = (cum < top_p[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    if p < 1:
        below = torch.where(n > 0, cum.gather(1, (n - 1).clamp(min=0)), 0.0)
        top_p = (0.5 * (below + cum.gather(1, n)) / total)[:, 0]
        w = w * (place <= n)
    if m:
        n = (w >= min_p[:, None]).sum(1, keepdim=True)
        above, below = w.gather(1, n - 1), w.gather(1, n.clamp(max=V - 1))
        min_p = torch.where(below > 0, (above * below).sqrt(), min_p[:, None])[:, 0]
        w = w * (place < n)
    cum = torch.zeros_like(w).scatter_(1, order[1], w).cumsum(1)
    u = torch.rand(rows, 8, dtype=torch.float64, device="cuda", generator=gen).float()
    at = u.double() * cum[:, -1:]
    right = torch.searchsorted(cum, at, right=True).clamp(max=V - 1)
    high = cum.gather(1, right) - at
    low = at - torch.where(right > 0, cum.gather(1, (right - 1).clamp(min=0)), -1.0)
    pick = torch.minimum(low, high).argmax(1, keepdim=True)
    st["u"] = u.gather(1, pick)[:, 0].contiguous()
    st["temperature"], st["top_k"] = temperature, top_k
    st["top_p"], st["min_p"] = top_p.float(), min_p.float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "layer":
        _prepare_layer(case, gen, st)
    elif case["op"] == "sample":
        _prepare_sample(case, gen, st)
    else:
        rows, n, k = case["rows"], case["n"], case["k"]
        # weights and activations as a network has them: a few features are much larger
        x = torch.randn(rows, k, device="cuda", generator=gen)
        x *= 1 + 9 * (torch.rand(k, device="cuda", generator=gen) < 0.002).float()
        st["x_scale"] = None
        if case["x"] == "i8":
            st["x"], st["x_scale"] = _quantised(x)
        else:
            st["x"] = x.to(DTYPES[case["x"]])
        st["codes"] = torch.empty((n, k), dtype=torch.int8, device="cuda")
        for i in range(0, n, 16384):
            w = torch.randn(min(16384, n - i), k, device="cuda", generator=gen)
            st["codes"][i:i + 16384] = torch.round(w.mul_(32)).clamp_(-127, 127)
        st["scales"] = (0.5 + torch.rand(n, device="cuda", generator=gen)) * (k ** -0.5 / 32)
        st["bias"] = None
        if case["bias"]:
            st["bias"] = torch.randn(n, device="cuda", generator=gen)
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a program that uses the package keeps beside its tensors: output buffers, the
    workspace and the descriptors."""
    import mixture_experts_layer_fp32_gb300 as moe
    case = st["case"]
    st["moe"] = moe
    if case["op"] == "layer":
        T, k, E = case["tokens"], case["topk"], case["experts"]
        st["cfg"] = moe.config(T=T, h=case["hidden"], E=E, k=k, f=case["ffn"],
                               score=case["score"], dtype=case["dtype"],
                               capacity_factor=case["capacity"], drop_policy=case["policy"],
                               num_groups=case["groups"], group_topk=case["group_topk"])
        st["y"] = torch.empty_like(st["x"])
        st["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["prob"] = torch.empty((T, k), device="cuda")
        st["tpe"] = torch.empty(E, dtype=torch.int32, device="cuda")
        st["ws"] = moe.alloc_workspace_few(st["cfg"], case["shared"])
    elif case["op"] == "linear":
        st["w"] = moe.I8Weight(st["codes"], st["scales"])
        st["y"] = torch.empty((case["rows"], case["n"]), device="cuda",
                              dtype=DTYPES[case["out"]])
        st["ws"] = moe.alloc_workspace_linear_i8(case["rows"], st["w"])
    else:
        st["tokens"] = torch.empty(case["rows"], dtype=torch.int32, device="cuda")
        st["prob"] = torch.empty(case["rows"], device="cuda")
        names = ("temperature", "top_k", "top_p", "min_p")
        st["choices"] = {n: st[n] if case["each"] else st[n][0].item() for n in names}
        if not case["each"]:   # rows that share their choices: one top_p and min_p would move
            for n, off in (("top_p", 1.0), ("min_p", 0.0)):
                if case["rows"] > 1 and case[n] != off:
                    st["choices"][n] = st[n]


# --------------------------------------------------------------- plain forms

def _quantised(x):
    """Rows as codes -127..127 and a scale: the largest magnitude over 127, and the nearest whole
    number of x over it (in 64 bits: a quotient next to a border)."""
    scale = x.float().abs().amax(dim=1) / 127.0
    safe = torch.where(scale > 0, scale, 1.0)
    codes = torch.round(x.double() / safe.double()[:, None]).clamp(-127, 127)
    return codes.to(torch.int8), scale


def _scores(case, logits, expert_bias):
    """(weights' scores, selection scores) of logits [T,E] in 64 bits."""
    if case["score"] == "softmax_pre":
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        s = e / e.sum(dim=1, keepdim=True)
        return s, s
    if case["score"] == "softmax_post":
        return logits, logits
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-logits))
    else:
        s = torch.sqrt(torch.clamp(logits, min=0) + torch.log1p(torch.exp(-logits.abs())))
    return s, s if expert_bias is None else s + expert_bias.double()


def _capacity(case):
    if case["capacity"] <= 0:
        return None
    return math.ceil(case["tokens"] * case["topk"] / case["experts"] * case["capacity"])


def _plain_route(st):
    case = st["case"]
    T, E, k = case["tokens"], case["experts"], case["topk"]
    s, sel = _scores(case, _logits64(st["x"], st["Wg"], st["gate_bias"]), st["expert_bias"])
    if case["groups"] > 1:
        grouped = sel.view(T, case["groups"], -1)
        best = grouped.sort(dim=2, descending=True)[0][:, :, :k // case["group_topk"]].sum(2)
        chosen = best.sort(dim=1, descending=True, stable=True)[1][:, :case["group_topk"]]
        allowed = torch.zeros(T, case["groups"], device=s.device)
        allowed.scatter_(1, chosen, 1.0)
        sel = torch.where(allowed[:, :, None] > 0, grouped, float("-inf")).reshape(T, E)
    idx = sel.sort(dim=1, descending=True, stable=True)[1][:, :k]
    p = s.gather(1, idx)
    if case["score"] == "softmax_post":
        p = torch.exp(p - p[:, :1])
        p = p / p.sum(dim=1, keepdim=True)
    elif case["score"] != "softmax_pre":
        p = p / (p.sum(dim=1, keepdim=True) + 1e-20)
    p = p.float()
    keep = torch.ones_like(idx, dtype=torch.bool)
    cap = _capacity(case)
    if cap is not None:
        e, t = idx.reshape(-1), torch.arange(T, device=s.device).repeat_interleave(k)
        q = p.reshape(-1)
        before = t[None, :] < t[:, None]
        if case["policy"] == "probs":
            before = (q[None, :] > q[:, None]) | ((q[None, :] == q[:, None]) & before)
        rank = ((e[None, :] == e[:, None]) & before).sum(dim=1)
        keep = (rank < cap).view(T, k)
        p = p * keep
    hit = (idx[:, :, None] == torch.arange(E, device=s.device)) & keep[:, :, None]
    return idx, p, hit.sum(dim=(0, 1)).to(torch.int32)


def _swiglu(x, W1, W3, W2):
    a = x @ W1.float()
    return (a / (1.0 + torch.exp(-a)) * (x @ W3.float())) @ W2.float()


def _plain_layer(st):
    case = st["case"]
    x = st["x"].float()
    idx, p, tpe = _plain_route(st)
    y = torch.zeros_like(x)
    T, k = idx.shape
    if case["experts"] <= T * k:   # by expert: its share of every token's weight
        for e in range(case["experts"]):
            share = (p * (idx == e)).sum(dim=1, keepdim=True)
            y += share * _swiglu(x, st["W1"][e], st["W3"][e], st["W2"][e])
    else:                          # by pair
        for t in range(T):
            for j in range(k):
                e = idx[t, j:j + 1]
                w = (st[n].index_select(0, e)[0] for n in ("W1", "W3", "W2"))
                y[t] += p[t, j] * _swiglu(x[t:t + 1], *w)[0]
    if st["shared"] is not None:
        y += _swiglu(x, *st["shared"])
    return dict(y=y.to(st["x"].dtype), idx=idx.to(torch.int32), prob=p, tokens_per_expert=tpe)


def _plain_linear(st):
    codes, scale = st["x"], st["x_scale"]
    if scale is None:
        codes, scale = _quantised(st["x"])
    y = codes.float() @ st["codes"].float().t()
    y = y * scale[:, None] * st["scales"]
    if st["bias"] is not None:
        y = y + st["bias"]
    return dict(y=y.to(DTYPES[st["case"]["out"]]))


def _plain_sample(st):
    logits, t = st["logits"].double(), st["temperature"].double()[:, None]
    rows, V = logits.shape
    value, order = logits.sort(dim=1, descending=True, stable=True)
    place = torch.arange(V, device=logits.device)
    z = (value - value[:, :1]) / torch.where(t > 0, t, 1.0)
    w = torch.where(t > 0, torch.exp(z), (place == 0).double())
    top_k = st["top_k"][:, None]
    w = w * ((place < top_k) | (top_k <= 0))
    before = w.cumsum(1) - w
    top_p = st["top_p"].double()[:, None]
    w = w * ((before < top_p * w.sum(1, keepdim=True)) | (top_p >= 1) | (place == 0))
    w = w * (w >= st["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, w)
    cum = w.cumsum(1)
    at = st["u"].double()[:, None] * cum[:, -1:]
    token = (cum <= at).sum(1).clamp(max=V - 1)
    prob = w.gather(1, token[:, None])[:, 0] / cum[:, -1]
    return dict(tokens=token.to(torch.int32), prob=prob.float())


def run(state):
    st = state
    op = st["case"]["op"]
    if own:
        moe = st["moe"]
        if op == "layer":
            moe.forward_few(st["cfg"], st["x"], st["Wg"], st["gate_bias"], st["expert_bias"],
                            st["W1"], st["W3"], st["W2"], st["y"], st["ws"], topk_idx=st["idx"],
                            topk_prob=st["prob"], tokens_per_expert=st["tpe"],
                            shared=st["shared"])
            return dict(y=st["y"], idx=st["idx"], prob=st["prob"], tokens_per_expert=st["tpe"])
        if op == "linear":
            moe.linear_i8(st["x"], st["w"], st["y"], st["ws"], x_scale=st["x_scale"],
                          bias=st["bias"])
            return dict(y=st["y"])
        moe.sample(st["logits"], st["u"], st["tokens"], prob=st["prob"], **st["choices"])
        return dict(tokens=st["tokens"], prob=st["prob"])
    return {"layer": _plain_layer, "linear": _plain_linear, "sample": _plain_sample}[op](st)


# ----------------------------------------------------------------- the work

def work(case):
    if case["op"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        x = {"bf16": 2, "f32": 4, "i8": 1}[case["x"]]
        return {"bytes": n * k + n * (8 if case["bias"] else 4) + m * k * x +
                m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2.0 * m * n * k}
    if case["op"] == "sample":
        count = case["rows"] * case["vocab"]
        return {"bytes": count * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * 12,
                "flops": 4.0 * count}
    T, h, E, k, f = (case[n] for n in ("tokens", "hidden", "experts", "topk", "ffn"))
    size = 2 if case["dtype"] == "bf16" else 4
    # how many experts a random routing hits, on average
    hit = E * (1.0 - (1.0 - k / E) ** T)
    cap = _capacity(case)
    pairs = T * k if cap is None else min(T * k, E * cap)
    each = 3.0 * h * f
    shared = 3.0 * h * case["shared"]
    return {"bytes": (hit * each + shared + 2 * T * h) * size + 4 * h * E + 8 * T * k,
            "flops": 2.0 * (pairs * each + T * shared + T * h * E)}


# -------------------------------------------------- the definitions in 64 bits

def _exact_layer(st):
    case = st["case"]
    T, E, k = case["tokens"], case["experts"], case["topk"]
    x = st["x"].double()
    logits = torch.einsum("th,he->te", x, st["Wg"].double()) + st["gate_bias"].double()
    l = logits.cpu().numpy()
    score = case["score"]
    if score == "softmax_pre":
        s = np.exp(l) / np.exp(l).sum(1, keepdims=True)
    elif score == "sigmoid":
        s = 0.5 * (1 + np.tanh(0.5 * l))
    elif score == "sqrtsoftplus":
        s = np.sqrt(np.logaddexp(0.0, l))
    else:
        s = l
    sel = s if st["expert_bias"] is None else s + st["expert_bias"].double().cpu().numpy()
    idx, p = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        allowed = np.arange(E)
        if case["groups"] > 1:
            each = E // case["groups"]
            top = [np.sort(sel[t, g * each:(g + 1) * each])[::-1][:k // case["group_topk"]].sum()
                   for g in range(case["groups"])]
            best = sorted(range(case["groups"]), key=lambda g: (-top[g], g))
            allowed = np.array([e for e in range(E) if e // each in
                                best[:case["group_topk"]]])
        idx[t] = sorted(allowed, key=lambda e: (-sel[t, e], e))[:k]
        v = s[t, idx[t]]
        if score == "softmax_post":
            p[t] = np.exp(v) / np.exp(v).sum()
        else:
            p[t] = v if score == "softmax_pre" else v / v.sum()
    kept = np.ones((T, k), bool)
    cap = _capacity(case)
    for e in range(E if cap is not None else 0):
        pairs = [(t, j) for t in range(T) for j in range(k) if idx[t, j] == e]
        if case["policy"] == "probs":   # equal in 32 bits: the lower token
            pairs.sort(key=lambda q: (-np.float32(p[q]), q[0]))
        for q in pairs[cap:]:
            kept[q], p[q] = False, 0.0
    y = torch.zeros_like(x)
    for e in sorted(set(idx[kept].tolist())):
        t, j = (torch.from_numpy(v).cuda() for v in np.nonzero((idx == e) & kept))
        a = x[t] @ st["W1"][e].double()
        g = x[t] @ st["W3"][e].double()
        out = (a * torch.sigmoid(a) * g) @ st["W2"][e].double()
        y.index_add_(0, t, torch.from_numpy(p).cuda()[t, j][:, None] * out)
    if st["shared"] is not None:
        W1, W3, W2 = (w.double() for w in st["shared"])
        a = x @ W1
        y += (a * torch.sigmoid(a) * (x @ W3)) @ W2
    tpe = np.bincount(idx[kept], minlength=E)
    return dict(y=y, idx=torch.from_numpy(idx.astype(np.int32)).cuda(),
                prob=torch.from_numpy(p).cuda(),
                tokens_per_expert=torch.from_numpy(tpe.astype(np.int32)).cuda())


def _exact_linear(st):
    if st["x_scale"] is not None:
        codes, scale = st["x"].double(), st["x_scale"].double()
    else:
        # codes by counting the borders below: whole numbers and a half times the scale
        x = st["x"].double()
        scale = (st["x"].float().abs().amax(dim=1) / 127.0).double()
        part = (x / scale.clamp(min=1e-300)[:, None]).clamp(-127, 127)
        low = torch.floor(part)
        over = part - low
        odd = (low % 2) != 0
        codes = low + ((over > 0.5) | ((over == 0.5) & odd)).double()
    y = torch.empty(codes.shape[0], st["codes"].shape[0], dtype=torch.float64, device="cuda")
    for i in range(0, y.shape[1], 16384):
        w = st["codes"][i:i + 16384].double() * st["scales"][i:i + 16384].double()[:, None]
        y[:, i:i + 16384] = codes @ w.t()
    y *= scale[:, None]
    if st["bias"] is not None:
        y += st["bias"].double()
    return dict(y=y)


def _exact_sample(st):
    logits = st["logits"].double().cpu().numpy()
    get = {n: st[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p",
                                                     "u")}
    rows, V = logits.shape
    tokens, probs = np.zeros(rows, np.int32), np.zeros(rows)
    for r in range(rows):
        l, t = logits[r], get["temperature"][r]
        order = np.argsort(-l, kind="stable")
        order = order[l[order] > -np.inf]
        w = np.exp((l[order] - l[order[0]]) / t) if t > 0 else np.ones(1)
        if get["top_k"][r] > 0:
            w = w[:int(get["top_k"][r])]
        if get["top_p"][r] < 1:
            reached = np.cumsum(w) >= get["top_p"][r] * w.sum()
            w = w[:int(np.argmax(reached)) + 1 if reached.any() else w.size]
        w = w[w >= get["min_p"][r]]
        kept = order[:w.size]
        by_index = np.argsort(kept)
        cum = np.cumsum(w[by_index])
        at = min(int(np.searchsorted(cum, get["u"][r] * cum[-1], side="right")), w.size - 1)
        tokens[r], probs[r] = kept[by_index[at]], w[by_index[at]] / cum[-1]
    return dict(tokens=torch.from_numpy(tokens).cuda(), prob=torch.from_numpy(probs).cuda())


def exact(case, seed):
    global own
    before, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = before
    return {"layer": _exact_layer, "linear": _exact_linear, "sample": _exact_sample}[
        case["op"]](st)
