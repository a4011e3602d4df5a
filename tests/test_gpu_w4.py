"""4-bit weights on the GPU: quantiser, packing, product and experts against
references in 64 bits (block_cases)."""

import numpy as np
import pytest
import torch

import block_cases as bc
import synthetic
from moe_cases import gpu_config, to_dev

pytestmark = pytest.mark.gpu


def _weight(shape, K, group, zeros, seed, exact=False):
    """Random codes [*shape, K]; exact: scales that are powers of two."""
    import mixture_experts_layer_fp32_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(0, 16, shape + (K,), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.rand(shape + (K // group,), device="cuda", generator=g)
    s = 2.0 ** torch.floor(3 * s) if exact else 0.004 * (0.5 + s)
    z = None
    if zeros:
        z = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda", generator=g)
    w = moe.W4Weight(moe.pack_w4(v), s.to(torch.bfloat16), z, group=group, k=K)
    return w, bc.w4_weight_ref(w.codes, w.scales, w.zeros, group, K)


@pytest.mark.parametrize("K", [32, 96, 128, 160, 1024, 1440])
def test_pack(K):
    import mixture_experts_layer_fp32_gb300 as moe
    v = torch.randint(0, 256, (2, 5, K), dtype=torch.uint8, device="cuda")
    assert np.array_equal(moe.pack_w4(v).cpu().numpy(), bc.w4_pack_ref(v.cpu().numpy()))


def _quantize_ref(W, group, zeros):
    """The quantiser's definition, in fp32 as it is stated (numpy)."""
    W = W.float().cpu().numpy().swapaxes(-1, -2)
    g = W.reshape(W.shape[:-1] + (-1, group))
    lo = np.minimum(g.min(-1), np.float32(0))
    hi = np.maximum(g.max(-1), np.float32(0))
    s = (hi - lo) / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7)
    s = torch.from_numpy(s).to(torch.bfloat16).float().numpy()
    safe = np.where(s > 0, s, np.float32(1))
    z = np.full(s.shape, 8, np.float32)
    if zeros:
        z = np.where(s > 0, np.clip(np.rint(-lo / safe), 0, 15), 0).astype(np.float32)
    q = np.where(s[..., None] > 0, np.rint(g / safe[..., None]) + z[..., None], z[..., None])
    return np.clip(q, 0, 15).astype(np.uint8).reshape(W.shape), s, z.astype(np.uint8)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("E,K,N,group", [(1, 64, 64, 32), (3, 192, 128, 64), (2, 512, 192, 128)])
def test_quantize(E, K, N, group, zeros):
    import mixture_experts_layer_fp32_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(K)
    W = (0.02 * torch.randn((E, K, N), device="cuda", generator=g)).to(torch.bfloat16)
    W[0, :group, 3] = 0.0
    W[0, :group, 4] = 0.5      # one sign only
    q = moe.quantize_w4(W, group, zeros)
    values, s, z = _quantize_ref(W, group, zeros)
    assert np.array_equal(bc.w4_unpack_ref(q.codes.cpu().numpy(), K), values)
    assert np.array_equal(q.scales.float().cpu().numpy(), s)
    if zeros:
        assert np.array_equal(q.zeros.cpu().numpy(), z)
    # the weight is off by half a step, and by the rounding of the scale at the ends (7 or 15
    # steps, 2^-8 each) and of the zero point (half a step)
    back = bc.w4_weight_ref(q.codes, q.scales, q.zeros, group, K)
    step = q.scales.double().repeat_interleave(group, -1)
    limit = step * (0.5 + 15 * 2.0 ** -8 + (0.5 if zeros else 0))
    assert bool(((back - W.double().transpose(1, 2)).abs() <= limit + 1e-12).all())


SHAPES = [(1, 1, 32, 32), (1, 17, 64, 64), (2, 16, 128, 128), (3, 100, 480, 32), (5, 33, 192, 64),
          (8, 64, 1024, 128), (9, 130, 1152, 128), (16, 257, 2048, 64), (17, 40, 4096, 32),
          (31, 96, 640, 128), (33, 50, 14336, 128), (64, 128, 1536, 64), (65, 24, 256, 32),
          (1, 4096, 512, 128), (4, 1000, 7168, 64)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_linear_exact(M, N, K, group, zeros):
    """Whole numbers and scales that are powers of two: every sum is exact."""
    import mixture_experts_layer_fp32_gb300 as moe
    w, W = _weight((N,), K, group, zeros, M + N, exact=True)
    x = torch.randint(-2, 3, (M, K), device="cuda").to(torch.bfloat16)
    assert 2 * 15 * 4 * K < 1 << 24
    room = torch.full((M * N + 64,), 7.0, device="cuda")
    y = room[32:32 + M * N].view(M, N)
    moe.linear_w4(x, w, y, moe.alloc_workspace_linear_w4(M, w))
    assert torch.equal(y.double(), x.double() @ W.t())
    assert float((room[:32] - 7).abs().max()) == 0
    assert float((room[32 + M * N:] - 7).abs().max()) == 0


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_linear(M, N, K, group, out):
    import mixture_experts_layer_fp32_gb300 as moe
    w, W = _weight((N,), K, group, group != 64, M * N)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    y = torch.full((M, N), float("nan"), dtype=out, device="cuda")
    moe.linear_w4(x, w, y, moe.alloc_workspace_linear_w4(M, w))
    bc.assert_within("y", y, x.double() @ W.t(), bc.w4_product_bound(x.double(), W), out)
    again = torch.empty_like(y)
    moe.linear_w4(x, w, again, moe.alloc_workspace_linear_w4(M, w))
    assert torch.equal(y, again)


def test_linear_no_rows_and_special_values():
    import mixture_experts_layer_fp32_gb300 as moe
    w, W = _weight((40,), 256, 64, False, 3)
    ws = moe.alloc_workspace_linear_w4(0, w)
    moe.linear_w4(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), w,
                  torch.empty((0, 40), device="cuda"), ws)
    # an infinity or a NaN in one row of x stays in that row
    x = torch.randn((4, 256), device="cuda").to(torch.bfloat16)
    x[1, 7], x[2, 200] = float("inf"), float("nan")
    y = torch.empty((4, 40), device="cuda")
    moe.linear_w4(x, w, y, moe.alloc_workspace_linear_w4(4, w))
    rows = [0, 3]
    bc.assert_within("y", y[rows], x[rows].double() @ W.t(),
                     bc.w4_product_bound(x[rows].double(), W), torch.float32)
    assert not torch.isfinite(y[1:3]).all()


def _experts(E, h, f, group, zeros, seed):
    import mixture_experts_layer_fp32_gb300 as moe
    ws = [_weight((E, n), k, group, zeros, seed + i)
          for i, (n, k) in enumerate(((f, h), (f, h), (h, f)))]
    return moe.W4Experts(*(w for w, _ in ws)), [W for _, W in ws]


def _routing(T, E, k, seed, drop=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    score, idx = torch.randn((T, E), device="cuda", generator=g).topk(k, dim=1)
    keep = (torch.rand((T, k), device="cuda", generator=g) >= drop).to(torch.uint8)
    return idx.to(torch.int32), torch.softmax(score, 1), keep


CASES = [(1, 256, 1, 1, 128, 128), (1, 512, 8, 2, 256, 64), (2, 256, 4, 4, 384, 32),
         (5, 768, 16, 8, 128, 64), (9, 512, 3, 2, 640, 128), (33, 256, 2, 1, 256, 32),
         (64, 256, 8, 2, 1536, 128), (130, 512, 4, 2, 128, 64), (70, 256, 256, 8, 128, 32),
         (300, 256, 8, 8, 256, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,h,E,k,f,group", CASES)
def test_experts(T, h, E, k, f, group, zeros):
    import mixture_experts_layer_fp32_gb300 as moe
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)
    q, W = _experts(E, h, f, group, zeros, T + f)
    idx, prob, keep = _routing(T, E, k, T, drop=0.2)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    for kp in (None, keep):
        y = torch.full_like(x, float("nan"))
        ws = moe.alloc_workspace_experts_w4(cfg)
        ws[256:] = 255        # what scratch holds must not matter
        moe.experts_w4(cfg, x, idx, prob, kp, q, y, ws)
        moe.check(ws)
        ref, bound = bc.experts_ref(x.double(), idx.cpu(), prob.cpu(),
                                    None if kp is None else kp.cpu(), *W)
        bc.assert_within("y", y, ref, bound, torch.bfloat16)
        again = torch.empty_like(y)
        moe.experts_w4(cfg, x, idx, prob, kp, q, again, ws)
        assert torch.equal(y, again)


def test_experts_every_pair_dropped_or_on_one_expert():
    import mixture_experts_layer_fp32_gb300 as moe
    T, h, E, k, f = 40, 256, 4, 2, 256
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)
    q, W = _experts(E, h, f, 64, True, 5)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    idx, prob, _ = _routing(T, E, k, 5)
    y = torch.full_like(x, float("nan"))
    ws = moe.alloc_workspace_experts_w4(cfg)
    keep = torch.zeros((T, k), dtype=torch.uint8, device="cuda")
    moe.experts_w4(cfg, x, idx, prob, keep, q, y, ws)
    assert torch.equal(y, torch.zeros_like(y))
    keep[:, 0] = 1
    keep[7] = 0                                   # one token without a pair
    idx[:, 0] = 3
    moe.experts_w4(cfg, x, idx, prob, keep, q, y, ws)
    ref, bound = bc.experts_ref(x.double(), idx.cpu(), prob.cpu(), keep.cpu(), *W)
    bc.assert_within("y", y, ref, bound, torch.bfloat16)
    assert torch.equal(y[7], torch.zeros_like(y[7]))


def test_experts_index_out_of_range_is_reported():
    """The kernels check every id before they use it."""
    import mixture_experts_layer_fp32_gb300 as moe
    T, h, E, k, f = 6, 256, 4, 2, 128
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)
    q, W = _experts(E, h, f, 128, False, 8)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    idx, prob, _ = _routing(T, E, k, 8)
    idx[2, 1], idx[4, 0] = E, -1
    y = torch.empty_like(x)
    ws = moe.alloc_workspace_experts_w4(cfg)
    moe.experts_w4(cfg, x, idx, prob, None, q, y, ws)
    with pytest.raises(moe.MoeError) as ei:
        moe.check(ws)
    assert ei.value.code == 5
    keep = torch.ones((T, k), dtype=torch.uint8)
    keep[2, 1] = keep[4, 0] = 0
    ref, bound = bc.experts_ref(x.double(), idx.cpu(), prob.cpu(), keep, *W)
    bc.assert_within("y", y, ref, bound, torch.bfloat16)
    moe.check(ws)      # the report was taken


def test_experts_codes_past_32_bits():
    import mixture_experts_layer_fp32_gb300 as moe
    T, h, E, k, f, group = 1, 7168, 256, 2, 4864, 128
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)

    def weight(n, kk, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        codes = torch.randint(0, 256, (E, n, kk // 2), dtype=torch.uint8, device="cuda",
                              generator=g)
        assert codes.numel() > 1 << 32
        s = 0.004 * (0.5 + torch.rand((E, n, kk // group), device="cuda", generator=g))
        return moe.W4Weight(codes, s.to(torch.bfloat16), group=group, k=kk)

    q = moe.W4Experts(weight(f, h, 1), weight(f, h, 2), weight(h, f, 3))
    idx = torch.tensor([[255, 1]], dtype=torch.int32, device="cuda")
    prob = torch.tensor([[0.75, 0.25]], device="cuda")
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    y = torch.empty_like(x)
    moe.experts_w4(cfg, x, idx, prob, None, q, y, moe.alloc_workspace_experts_w4(cfg))
    pick = [255, 1]
    W = [bc.w4_weight_ref(w.codes[pick], w.scales[pick], None, group, w.k)
         for w in (q.W1, q.W3, q.W2)]
    ref, bound = bc.experts_ref(x.double(), torch.tensor([[0, 1]]), prob.cpu(), None, *W)
    bc.assert_within("y", y, ref, bound, torch.bfloat16)


@pytest.mark.parametrize("name,over", [
    ("mixtral", dict(T=3, h=512, f=256)), ("dsv3", dict(T=17, h=256, f=128)),
    ("switch", dict(T=200, h=256, f=256)), ("switch_pad", dict(T=200, h=256, f=256)),
    ("dsv3_grouped", dict(T=4, h=256, f=128))])
def test_forward_w4(name, over):
    """The layer forward with 4-bit experts: the routing of moe_route, then the
    experts over the weights that the codes stand for."""
    import mixture_experts_layer_fp32_gb300 as moe
    w = synthetic.scaled(name, seed=41, **over)
    cfg = gpu_config(w)
    d = to_dev(synthetic.generate(w, device="cpu"), "cuda:0")
    q = moe.quantize_experts_w4(d["W1"], d["W3"], d["W2"], group=64, zeros=True)
    T, k = w.T, w.k
    y = torch.full_like(d["x"], float("nan"))
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    prob = torch.empty((T, k), device="cuda")
    ws = moe.alloc_workspace_w4(cfg)
    moe.forward_w4(cfg, d["x"], d["Wg"], d["gate_bias"], d["expert_bias"], q, y, ws,
                   topk_idx=idx, topk_prob=prob)
    moe.check(ws)
    b = moe.Buffers(cfg)
    rm = b.routing_map if w.pad_to_capacity else None
    moe.route(cfg, d["x"], d["Wg"], d["gate_bias"], d["expert_bias"], b.topk_idx, b.topk_prob,
              b.keep, b.tokens_per_expert, rm, b.ws)
    assert torch.equal(idx, b.topk_idx) and torch.equal(prob, b.topk_prob)
    W = [bc.w4_weight_ref(m.codes, m.scales, m.zeros, 64, m.k) for m in (q.W1, q.W3, q.W2)]
    ref, bound = bc.experts_ref(d["x"].double(), idx.cpu(), prob.cpu(), b.keep.cpu(), *W)
    bc.assert_within("y", y, ref, bound, torch.bfloat16)
    # without the optional outputs
    y2 = torch.empty_like(y)
    moe.forward_w4(cfg, d["x"], d["Wg"], d["gate_bias"], d["expert_bias"], q, y2, ws)
    assert torch.equal(y, y2)


def test_on_another_stream_and_in_a_graph():
    import mixture_experts_layer_fp32_gb300 as moe
    T, h, E, k, f = 4, 512, 8, 2, 256
    cfg = moe.config(T=T, h=h, E=E, k=k, f=f)
    q, _ = _experts(E, h, f, 64, False, 12)
    w, _ = _weight((300,), h, 64, False, 13)
    x = torch.randn((T, h), device="cuda").to(torch.bfloat16)
    idx, prob, keep = _routing(T, E, k, 12)
    y, v = torch.empty_like(x), torch.empty((T, 300), device="cuda")
    ws, wl = moe.alloc_workspace_experts_w4(cfg), moe.alloc_workspace_linear_w4(T, w)

    def step():
        moe.experts_w4(cfg, x, idx, prob, keep, q, y, ws)
        moe.linear_w4(y, w, v, wl)

    def take():
        torch.cuda.synchronize()
        got = y.clone(), v.clone()
        y.fill_(float("nan"))
        v.fill_(float("nan"))
        torch.cuda.synchronize()
        return got

    step()
    first = take()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    assert all(torch.equal(a, c) for a, c in zip(first, take()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    take()
    graph.replay()
    assert all(torch.equal(a, c) for a, c in zip(first, take()))
    x.mul_(2)
    step()
    second = take()
    graph.replay()
    assert all(torch.equal(a, c) for a, c in zip(second, take()))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", [
    (20, 40000, 384, 128),    # more tiles than SMs, rows of an odd number of blocks
    (33, 39200, 160, 32),     # two blocks, the second a quarter full; more than 32 columns
    (64, 40001, 64, 64),      # one block, half full; an odd number of outputs
    (70, 1100, 1440, 32)])    # two chunks of rows; parts of different lengths
def test_linear_more_rows(M, N, K, group, zeros):
    import mixture_experts_layer_fp32_gb300 as moe
    w, W = _weight((N,), K, group, zeros, M + K)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    y = torch.full((M, N), float("nan"), device="cuda")
    ws = moe.alloc_workspace_linear_w4(M, w)
    moe.linear_w4(x, w, y, ws)
    moe.check(ws)
    bc.assert_within("y", y, x.double() @ W.t(), bc.w4_product_bound(x.double(), W), y.dtype)
