"""The operators around and inside the MoE layer, as measured cases.

Five operators: the norm's forward pass (``norm``: layer norm or RMS norm, on its own or of
residual + dropout(branch)), its backward pass (``norm_grad``), the dropout with the residual
addition (``dropout``), the product with 4-bit weights (``linear``) and the routed SwiGLU experts
with 4-bit weights for few tokens (``experts``).  ``run`` computes them in plain torch operations,
or through this package's entry points where ``own`` is true; ``exact`` holds the definitions in
64 bits.
"""

import math

import numpy as np
import torch

own = False

# Philox4x32-10 of Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3"
# (SC 2011): the multipliers and key increments of the paper.
PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the norm before the router of one new token, after the attention's output was added
        dict(name="norm one token", op="norm", rows=1, hidden=7168, dtype="bf16", param="bf16",
             rms=True, residual=True, p=0.0),
        # the same place in training: dropout of the branch, the residual sum, the norm
        dict(name="norm dropout train", op="norm", rows=8192, hidden=4096, dtype="bf16",
             param="f32", rms=False, residual=True, p=0.1),
        # a plain fp32 layer norm over rows of an odd width
        dict(name="norm odd fp32", op="norm", rows=2999, hidden=1021, dtype="f32", param="f32",
             rms=False, residual=False, p=0.0),
        # the backward of the training case, with the gradient that arrives by the residual path
        dict(name="norm_grad dropout train", op="norm_grad", rows=16384, hidden=4096,
             dtype="bf16", param="f32", rms=False, residual=True, p=0.1),
        # the plain backward, odd width
        dict(name="norm_grad odd fp32", op="norm_grad", rows=2999, hidden=1021, dtype="f32",
             param="f32", rms=False, residual=False, p=0.0),
        # the end of the block: no norm follows in this call
        dict(name="dropout train", op="dropout", rows=32768, hidden=1024, dtype="bf16",
             residual=True, p=0.1),
        # a small odd call without a residual (also the shape of its backward)
        dict(name="dropout odd fp32", op="dropout", rows=333, hidden=257, dtype="f32",
             residual=False, p=0.5),
        # one token through a square projection: latency counts
        dict(name="linear one token", op="linear", rows=1, n=4096, k=4096, group=128, zeros=False,
             out="bf16"),
        # a few tokens, finer groups with zero points, an odd number of outputs, fp32 results
        dict(name="linear few tokens", op="linear", rows=7, n=14337, k=7168, group=64, zeros=True,
             out="f32"),
        # decoding: one token, two of eight wide experts
        dict(name="experts one token", op="experts", tokens=1, hidden=4096, experts=8, topk=2,
             ffn=14336, group=128, zeros=False, drop=0.0),
        # decoding of a batch, fine-grained experts: most are hit by one token or none
        dict(name="experts fine-grained", op="experts", tokens=16, hidden=4096, experts=128,
             topk=8, ffn=1536, group=64, zeros=False, drop=0.0),
        # decoding of a larger batch, wide experts: each is hit by many tokens
        dict(name="experts batch", op="experts", tokens=64, hidden=4096, experts=8, topk=2,
             ffn=14336, group=128, zeros=True, drop=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dropout", "linear", "experts"])
    if op in ("norm", "norm_grad", "dropout"):
        hidden = _log(rng, 48, 16384)
        if rng.random() < 0.6:
            hidden = max(64, hidden // 64 * 64)
        most = (1 << 26) if op == "norm_grad" else (1 << 25)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = _log(rng, 1, max(1, min(65536, most // hidden // (2 if dtype == "f32" else 1))))
        if op == "dropout":
            return dict(op=op, rows=rows, hidden=hidden, dtype=dtype,
                        residual=rng.random() < 0.7, p=rng.choice([0.1, 0.25, 0.5]))
        residual = rng.random() < 0.5
        return dict(op=op, rows=rows, hidden=hidden, dtype=dtype,
                    param="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]),
                    rms=rng.random() < 0.4, residual=residual,
                    p=rng.choice([0.0, 0.1, 0.3]) if residual else 0.0)
    group = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.4
    if op == "linear":
        return dict(op=op, rows=_log(rng, 1, 64), n=_log(rng, 64, 16384),
                    k=_log(rng, 2, 14336 // group) * group, group=group, zeros=zeros,
                    out=rng.choice(["bf16", "f32"]))
    experts = _log(rng, 1, 128)
    topk = min(experts, rng.choice([1, 2, 4, 8]))
    hidden = _log(rng, 1, 28) * 256
    ffn = _log(rng, 2, max(2, min(112, 470_000_000 // experts // hidden // 128))) * 128
    return dict(op=op, tokens=_log(rng, 1, 64), hidden=hidden, experts=experts, topk=topk,
                ffn=ffn, group=group, zeros=zeros, drop=rng.choice([0.0, 0.0, 0.1]))


# ------------------------------------------------------------------- inputs

def _w4(gen, experts, n, k, group, zeros):
    """A weight [experts, n, k] in 4 bits: codes in blocks of 128 along k (64 bytes each), one
    bf16 scale and, optionally, one zero point for each group."""
    blocks = -(-k // 128)
    codes = torch.randint(0, 256, (experts, n, blocks * 64), dtype=torch.uint8, device="cuda",
                          generator=gen)
    groups = (experts, n, k // group)
    scales = (0.02 / 4.6) * torch.exp(0.25 * torch.randn(groups, device="cuda", generator=gen))
    z = None
    if zeros:
        z = torch.randint(6, 10, groups, dtype=torch.uint8, device="cuda", generator=gen)
    return dict(codes=codes, scales=scales.to(torch.bfloat16), zeros=z, group=group, k=k)


def _activations(gen, rows, hidden, dtype):
    """Rows as a residual stream has them: unit scale, an offset, and a few features that are an
    order of magnitude larger than the rest."""
    x = torch.randn(rows, hidden, device="cuda", generator=gen)
    feature = 1 + 9 * (torch.rand(hidden, device="cuda", generator=gen) < 0.002).float()
    offset = 0.3 * torch.randn(rows, 1, device="cuda", generator=gen)
    return (x * feature + offset).to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "linear":
        st["x"] = torch.randn(case["rows"], case["k"], device="cuda",
                              generator=gen).to(torch.bfloat16)
        st["w"] = _w4(gen, 1, case["n"], case["k"], case["group"], case["zeros"])
    elif case["op"] == "experts":
        T, h, E, f, k = (case[n] for n in ("tokens", "hidden", "experts", "ffn", "topk"))
        st["x"] = torch.randn(T, h, device="cuda", generator=gen).to(torch.bfloat16)
        score, idx = torch.randn(T, E, device="cuda", generator=gen).topk(k, dim=1)
        st["idx"] = idx.to(torch.int32)
        st["keep"] = None
        st["prob"] = torch.softmax(score, dim=1)
        if case["drop"]:
            kept = torch.rand(T, k, device="cuda", generator=gen) >= case["drop"]
            st["keep"] = kept.to(torch.uint8)
            st["prob"] = st["prob"] * kept
        for name, n, kk in (("W1", f, h), ("W3", f, h), ("W2", h, f)):
            st[name] = _w4(gen, E, n, kk, case["group"], case["zeros"])
    else:
        rows, hidden, dtype = case["rows"], case["hidden"], case["dtype"]
        st["x"] = _activations(gen, rows, hidden, dtype)
        st["res"] = None
        if case["residual"]:
            st["res"] = _activations(gen, rows, hidden, dtype)
        # seed and offset of the generator; the offset is past 32 bits now and then
        st["rng"] = torch.randint(0, 1 << 40, (2,), dtype=torch.int64, device="cuda",
                                  generator=gen)
        if case["op"] != "dropout":
            pt = DTYPES[case["param"]]
            st["weight"] = (1 + 0.1 * torch.randn(hidden, device="cuda", generator=gen)).to(pt)
            st["bias"] = None
            if not case["rms"]:
                st["bias"] = (0.1 * torch.randn(hidden, device="cuda", generator=gen)).to(pt)
        if case["op"] == "norm_grad":
            # what the forward pass saved: the normed tensor and its statistics
            z = st["x"].float()
            mean = torch.zeros(rows, device="cuda") if case["rms"] else z.mean(dim=1)
            var = (z - mean[:, None]).square().mean(dim=1)
            st["mean"] = None if case["rms"] else mean
            st["rstd"] = torch.rsqrt(var + EPS)
            scale = 1e-3
            st["dy"] = (scale * torch.randn(rows, hidden, device="cuda",
                                            generator=gen)).to(DTYPES[dtype])
            st["dz"] = None
            if case["residual"]:
                st["dz"] = (scale * torch.randn(rows, hidden, device="cuda",
                                                generator=gen)).to(DTYPES[dtype])
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a program that uses the package keeps beside its tensors: output buffers, the
    workspace and the descriptors."""
    import mixture_experts_layer_fp32_gb300 as moe
    case, x = st["case"], st["x"]
    st["moe"] = moe

    def weight(w, squeeze=False):
        pick = (lambda t: t[0]) if squeeze else (lambda t: t)
        return moe.W4Weight(pick(w["codes"]), pick(w["scales"]),
                            None if w["zeros"] is None else pick(w["zeros"]),
                            group=w["group"], k=w["k"])

    if case["op"] == "linear":
        st["w4"] = weight(st["w"], squeeze=True)
        st["y"] = torch.empty(case["rows"], case["n"], device="cuda", dtype=DTYPES[case["out"]])
        st["ws"] = moe.alloc_workspace_linear_w4(case["rows"], st["w4"])
    elif case["op"] == "experts":
        st["cfg"] = moe.config(T=case["tokens"], h=case["hidden"], E=case["experts"],
                               k=case["topk"], f=case["ffn"])
        st["q"] = moe.W4Experts(weight(st["W1"]), weight(st["W3"]), weight(st["W2"]))
        st["y"] = torch.empty_like(x)
        st["ws"] = moe.alloc_workspace_experts_w4(st["cfg"])
    else:
        rows, hidden = x.shape
        st["y"] = torch.empty_like(x)
        if case["op"] == "norm":
            st["z"] = torch.empty_like(x) if case["residual"] else None
            st["mean"] = None if case["rms"] else torch.empty(rows, device="cuda")
            st["rstd"] = torch.empty(rows, device="cuda")
        elif case["op"] == "norm_grad":
            st["dx"] = torch.empty_like(x)
            st["dbranch"] = torch.empty_like(x) if case["p"] > 0 else None
            st["dweight"] = torch.empty(hidden, device="cuda")
            st["dbias"] = None if case["rms"] else torch.empty(hidden, device="cuda")
            st["ws"] = moe.alloc_workspace_norm_backward(rows, hidden)


# --------------------------------------------------------------- plain forms

def _philox_keep(rng, count, p):
    """Truth values [count]: element i is kept iff word i % 4 of the block with the counter
    (i // 4, offset) under the key seed is at least floor(p 2^32).  32-bit arithmetic in int64."""
    low = 0xFFFFFFFF
    block = torch.arange((count + 3) // 4, dtype=torch.int64, device=rng.device)
    seed, offset = rng[0], rng[1]
    c0, c1 = block & low, (block >> 32) & low
    c2, c3 = (offset & low).expand_as(block), ((offset >> 32) & low).expand_as(block)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * PHILOX_M[0], c2 * PHILOX_M[1]
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + PHILOX_W[0]) & low, (k1 + PHILOX_W[1]) & low
    words = torch.stack((c0, c1, c2, c3), dim=1).reshape(-1)[:count]
    return words >= int(math.floor(p * 4294967296.0))


def _dropped(x, p, rng):
    if p == 0.0:
        return x
    keep = _philox_keep(rng, x.numel(), p).view(x.shape)
    return torch.where(keep, x * (1.0 / (1.0 - p)), torch.zeros((), device=x.device))


def _unpacked(w, pick=None):
    """The weight in 32 bits, [.., n, k], of the experts `pick` (all where None)."""
    codes, scales, zeros = w["codes"], w["scales"], w["zeros"]
    if pick is not None:
        codes, scales = codes[pick], scales[pick]
        zeros = None if zeros is None else zeros[pick]
    lead = codes.shape[:-1]
    q = torch.stack((codes & 15, codes >> 4), dim=-1)
    # a block of 128: word 4t + j holds k = 32j + 8t .. +7, its nibble p the k of offset
    # 2 (p % 4) + p // 4
    q = q.reshape(*lead, -1, 4, 4, 2, 4).movedim(-4, -3).movedim(-1, -2)
    q = q.reshape(*lead, -1)[..., :w["k"]].reshape(*lead, -1, w["group"]).float()
    z = 8.0 if zeros is None else zeros.float()[..., None]
    return ((q - z) * scales.float()[..., None]).reshape(*lead, w["k"])


def _plain_norm(st):
    case = st["case"]
    z = st["x"].float()
    if st["res"] is not None:
        z = st["res"].float() + _dropped(z, case["p"], st["rng"])
    mean = torch.zeros(z.shape[0], 1, device=z.device)
    if not case["rms"]:
        mean = z.mean(dim=1, keepdim=True)
    centred = z - mean
    rstd = 1.0 / torch.sqrt((centred * centred).mean(dim=1, keepdim=True) + EPS)
    y = centred * rstd * st["weight"].float()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    out = dict(y=y.to(st["x"].dtype), rstd=rstd[:, 0])
    if not case["rms"]:
        out["mean"] = mean[:, 0]
    if st["res"] is not None:
        out["z"] = z.to(st["x"].dtype)
    return out


def _plain_norm_grad(st):
    case = st["case"]
    z, dy = st["x"].float(), st["dy"].float()
    mean = 0.0 if case["rms"] else st["mean"][:, None]
    rstd = st["rstd"][:, None]
    xhat = (z - mean) * rstd
    g = dy * st["weight"].float()
    dx = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if not case["rms"]:
        dx = dx - g.mean(dim=1, keepdim=True)
    dx = dx * rstd
    if st["dz"] is not None:
        dx = dx + st["dz"].float()
    out = dict(dx=dx.to(st["x"].dtype),
               dweight=(dy * xhat).sum(dim=0, dtype=torch.float64).float())
    if not case["rms"]:
        out["dbias"] = dy.sum(dim=0, dtype=torch.float64).float()
    if case["p"] > 0:
        out["dbranch"] = _dropped(dx, case["p"], st["rng"]).to(st["x"].dtype)
    return out


def _plain_experts(st):
    case = st["case"]
    x, idx, prob = st["x"].float(), st["idx"], st["prob"]
    y = torch.zeros_like(x)
    silu = lambda v: v / (1.0 + torch.exp(-v))  # noqa: E731
    T, k = idx.shape
    if case["experts"] <= T * k:   # by expert: its share of every token's weight
        for e in range(case["experts"]):
            share = (prob * (idx == e)).sum(dim=1, keepdim=True)
            hid = silu(x @ _unpacked(st["W1"], e).t()) * (x @ _unpacked(st["W3"], e).t())
            y += share * (hid @ _unpacked(st["W2"], e).t())
        return y.to(st["x"].dtype)
    for t in range(T):             # by pair
        for j in range(k):
            e = idx[t, j:j + 1].long()
            hid = silu(_unpacked(st["W1"], e)[0] @ x[t]) * (_unpacked(st["W3"], e)[0] @ x[t])
            y[t] += prob[t, j] * (_unpacked(st["W2"], e)[0] @ hid)
    return y.to(st["x"].dtype)


def run(state):
    st = state
    case = st["case"]
    op = case["op"]
    if own:
        moe = st["moe"]
        if op == "norm":
            moe.layer_norm(st["x"], st["weight"], st["bias"], EPS, st["y"], st["mean"],
                           st["rstd"], rms=case["rms"], residual=st["res"], z=st["z"],
                           p=case["p"], rng=st["rng"])
            out = dict(y=st["y"], rstd=st["rstd"])
            if not case["rms"]:
                out["mean"] = st["mean"]
            if st["z"] is not None:
                out["z"] = st["z"]
            return out
        if op == "norm_grad":
            moe.layer_norm_backward(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"],
                                    st["dx"], st["dweight"], st["dbias"], st["ws"],
                                    rms=case["rms"], dz=st["dz"], dbranch=st["dbranch"],
                                    p=case["p"], rng=st["rng"])
            out = dict(dx=st["dx"], dweight=st["dweight"])
            if not case["rms"]:
                out["dbias"] = st["dbias"]
            if case["p"] > 0:
                out["dbranch"] = st["dbranch"]
            return out
        if op == "dropout":
            moe.dropout_add(st["x"], st["y"], case["p"], st["rng"], residual=st["res"])
        elif op == "linear":
            moe.linear_w4(st["x"], st["w4"], st["y"], st["ws"])
        else:
            moe.experts_w4(st["cfg"], st["x"], st["idx"], st["prob"], st["keep"], st["q"],
                           st["y"], st["ws"])
        return dict(y=st["y"])
    if op == "norm":
        return _plain_norm(st)
    if op == "norm_grad":
        return _plain_norm_grad(st)
    if op == "dropout":
        y = _dropped(st["x"].float(), case["p"], st["rng"])
        if st["res"] is not None:
            y = y + st["res"].float()
        return dict(y=y.to(st["x"].dtype))
    if op == "linear":
        return dict(y=(st["x"].float() @ _unpacked(st["w"])[0].t()).to(DTYPES[case["out"]]))
    return dict(y=_plain_experts(st))


# ----------------------------------------------------------------- the work

def _hit(case):
    """How many experts the pairs of a random routing hit, on average."""
    E, pairs = case["experts"], case["tokens"] * case["topk"] * (1 - case["drop"])
    return E * (1.0 - (1.0 - case["topk"] / E) ** (pairs / case["topk"]))


def work(case):
    if case["op"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        weights = n * k / 2 + n * (k // case["group"]) * (3 if case["zeros"] else 2)
        return {"bytes": weights + m * k * 2 + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2.0 * m * n * k}
    if case["op"] == "experts":
        values = 3.0 * case["hidden"] * case["ffn"]
        each = values / 2 + values / case["group"] * (3 if case["zeros"] else 2)
        pairs = case["tokens"] * case["topk"] * (1 - case["drop"])
        return {"bytes": _hit(case) * each + case["tokens"] * case["hidden"] * 4,
                "flops": 2.0 * pairs * values}
    count = case["rows"] * case["hidden"]
    size = 2 if case["dtype"] == "bf16" else 4
    dropout = 18.0 if case["p"] > 0 else 0.0
    if case["op"] == "dropout":
        return {"bytes": count * size * (3 if case["residual"] else 2), "flops": count * dropout}
    if case["op"] == "norm":
        moved = 4 if case["residual"] else 2
        return {"bytes": count * size * moved + case["rows"] * 8, "flops": count * (8 + dropout)}
    moved = 3 + (1 if case["residual"] else 0) + (1 if case["p"] > 0 else 0)
    return {"bytes": count * size * moved + case["rows"] * 8 + case["hidden"] * 8,
            "flops": count * (14 + dropout)}


# -------------------------------------------------- the definitions in 64 bits

def _keep_numpy(rng, count, p):
    """The kept elements, from the generator's definition, in numpy's unsigned integers."""
    seed, offset = (int(v) for v in rng.cpu())
    m32 = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    ctr = np.arange((count + 3) // 4, dtype=np.uint64)
    x = [ctr & m32, ctr >> s32, np.full_like(ctr, offset & 0xFFFFFFFF),
         np.full_like(ctr, (offset >> 32) & 0xFFFFFFFF)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for r in range(10):
        k0 = np.uint64((key[0] + r * PHILOX_W[0]) & 0xFFFFFFFF)
        k1 = np.uint64((key[1] + r * PHILOX_W[1]) & 0xFFFFFFFF)
        left, right = x[0] * np.uint64(PHILOX_M[0]), x[2] * np.uint64(PHILOX_M[1])
        x = [(right >> s32) ^ x[1] ^ k0, right & m32, (left >> s32) ^ x[3] ^ k1, left & m32]
    words = np.empty((ctr.size, 4), dtype=np.uint32)
    for i in range(4):
        words[:, i] = x[i]
    kept = words.reshape(-1)[:count].astype(np.float64) / 4294967296.0
    return torch.from_numpy(kept >= math.floor(p * 4294967296.0) / 4294967296.0).cuda()


def _mask64(st, x):
    p = st["case"]["p"]
    if p == 0.0:
        return torch.ones_like(x)
    return _keep_numpy(st["rng"], x.numel(), p).view(x.shape).double() / (1.0 - p)


def _weight64(w, e):
    """Expert e's weight in 64 bits: each nibble put at its place by an index table."""
    codes = w["codes"][e].to(torch.int16)
    n, total = codes.shape[0], codes.shape[1] * 2
    value = torch.empty(n, total, dtype=torch.float64, device=codes.device)
    place = np.empty(total, dtype=np.int64)   # place[nibble] = its k
    for nib in range(128):
        word, pos = nib // 8, nib % 8
        t, j = word // 4, word % 4
        place[nib::128] = 32 * j + 8 * t + 2 * (pos % 4) + pos // 4
    place += np.arange(total, dtype=np.int64) // 128 * 128
    place = torch.from_numpy(place).to(codes.device)
    value[:, place[0::2]] = (codes % 16).double()
    value[:, place[1::2]] = (codes // 16).double()
    value = value[:, :w["k"]]
    each = lambda t: t[e].double().repeat_interleave(w["group"], dim=1)  # noqa: E731
    return (value - (8.0 if w["zeros"] is None else each(w["zeros"]))) * each(w["scales"])


def exact(case, seed):
    global own
    before, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = before
    op = case["op"]
    if op == "linear":
        return dict(y=torch.einsum("mk,nk->mn", st["x"].double(), _weight64(st["w"], 0)))
    if op == "experts":
        x = st["x"].double()
        y = torch.zeros_like(x)
        idx, prob = st["idx"].cpu().numpy(), st["prob"].double()
        for e in sorted(set(idx.reshape(-1).tolist())):
            t, j = (torch.from_numpy(v).cuda() for v in np.nonzero(idx == e))
            a = x[t] @ _weight64(st["W1"], e).t()
            b = x[t] @ _weight64(st["W3"], e).t()
            out = (a * torch.sigmoid(a) * b) @ _weight64(st["W2"], e).t()
            y.index_add_(0, t, prob[t, j][:, None] * out)
        return dict(y=y)
    x = st["x"].double()
    if op == "dropout":
        y = x * _mask64(st, x)
        return dict(y=y if st["res"] is None else y + st["res"].double())
    w = st["weight"].double()
    if op == "norm":
        z = x if st["res"] is None else st["res"].double() + x * _mask64(st, x)
        mean = z.new_zeros(z.shape[0]) if case["rms"] else z.sum(1) / z.shape[1]
        var = (z * z).sum(1) / z.shape[1] - mean * mean
        rstd = (var + EPS) ** -0.5
        y = (z - mean[:, None]) * rstd[:, None] * w
        out = dict(y=y if st["bias"] is None else y + st["bias"].double(), rstd=rstd)
        if not case["rms"]:
            out["mean"] = mean
        if st["res"] is not None:
            out["z"] = z
        return out
    # the gradient by the product with the norm's Jacobian: rstd (I - 1/H - xhat xhat^T / H)
    dy, H = st["dy"].double(), x.shape[1]
    rstd = st["rstd"].double()
    xhat = x if case["rms"] else x - st["mean"].double()[:, None]
    xhat = xhat * rstd[:, None]
    g = dy * w
    inner = torch.einsum("rh,rh->r", g, xhat) / H
    dz = g - inner[:, None] * xhat
    if not case["rms"]:
        dz = dz - (g.sum(1) / H)[:, None]
    dz = dz * rstd[:, None]
    if st["dz"] is not None:
        dz = dz + st["dz"].double()
    out = dict(dx=dz, dweight=torch.einsum("rh,rh->h", dy, xhat))
    if not case["rms"]:
        out["dbias"] = dy.sum(0)
    if case["p"] > 0:
        out["dbranch"] = dz * _mask64(st, dz)
    return out
