"""References in 64 bits for the norm, the dropout and the 4-bit products, with
the error bounds that their tests use.  Plain numpy/torch, no code of the
package.

Bounds: u = 2^-24 is half a step of fp32; `half(dtype)` is half a step of an
output type (bf16 2^-8, fp32 2^-24), relative to the value."""

import numpy as np
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------- Philox

def philox4x32(ctr, key, rounds=10):
    """ctr [n, 4], key [2] as integers -> words [n, 4] uint32."""
    x = [np.asarray(c, dtype=np.uint64) for c in np.asarray(ctr, dtype=np.uint64).T]
    k = [int(key[0]), int(key[1])]
    mask, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> s) ^ x[1] ^ np.uint64(k[0]), b & mask, (a >> s) ^ x[3] ^ np.uint64(k[1]),
             a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(x, axis=1).astype(np.uint32)


def keep_mask(seed, offset, p, n, first=0):
    """Truth values of the elements first .. first + n - 1 (first % 4 == 0)."""
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    blocks = np.arange(first // 4, (first + n + 3) // 4, dtype=np.uint64)
    ctr = np.stack([blocks & np.uint64(0xFFFFFFFF), blocks >> np.uint64(32),
                    np.full_like(blocks, offset & 0xFFFFFFFF),
                    np.full_like(blocks, offset >> 32)], axis=1)
    words = philox4x32(ctr, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)[:n]
    return torch.from_numpy(words.astype(np.uint64) >= np.uint64(int(p * 4294967296.0)))


def dropped(x, p, keep):
    """dropout's map of x (float64): the scale is rounded to fp32 as in the kernel."""
    scale = float(np.float32(1.0 / (1.0 - p))) if p < 1 else 0.0
    return torch.where(keep.view(x.shape).to(x.device), x * scale, torch.zeros_like(x))


# --------------------------------------------------------------------- norm

def depth(hidden):
    """Longest chain of additions of one row's sum: the columns of one thread
    (256 threads at least for more than 1024 columns), then the tree."""
    return 64 + hidden // 256


def norm_ref(z, weight, bias, eps, rms):
    """z float64 -> y, mean, rstd and bounds of their fp32 errors (z itself with
    an error of 3u |z| + 3u from the residual sum is the caller's to add)."""
    H = z.shape[1]
    d = depth(H) * U
    mean = torch.zeros_like(z[:, :1]) if rms else z.mean(1, keepdim=True)
    c = z - mean
    var = (c * c).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    xh = c * rstd
    w = torch.ones_like(z[0]) if weight is None else weight.double()
    b = torch.zeros_like(z[0]) if bias is None else bias.double()
    e_mean = torch.zeros_like(mean) if rms else d * z.abs().mean(1, keepdim=True)
    # each centred value is off by the mean's error and a rounding of the difference; the
    # variance by twice that against |c|, and by its own sum
    e_c = e_mean + U * c.abs()
    e_var = d * var + 2 * (c.abs() * e_c).mean(1, keepdim=True) + (e_c ** 2).mean(1, keepdim=True)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 4 * U)
    y = xh * w + b
    e_y = w.abs() * (rstd * e_c + c.abs() * e_rstd) + 4 * U * ((xh * w).abs() + b.abs())
    return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0], e_y=e_y, e_mean=e_mean[:, 0],
                e_rstd=e_rstd[:, 0])


def norm_grad_ref(dy, z, weight, mean, rstd, dz, rms):
    """All float64 (mean, rstd as stored) -> dx, dweight, dbias and their bounds."""
    rows, H = z.shape
    d = depth(H) * U
    w = torch.ones_like(z[0]) if weight is None else weight.double()
    m = torch.zeros_like(z[:, :1]) if rms else mean.double()[:, None]
    rs = rstd.double()[:, None]
    xh = (z - m) * rs
    e_xh = 3 * U * xh.abs()
    g = dy * w
    c1 = torch.zeros_like(rs) if rms else g.mean(1, keepdim=True)
    c2 = (g * xh).mean(1, keepdim=True)
    e_c1 = 0 if rms else (d + 2 * U) * g.abs().mean(1, keepdim=True)
    e_c2 = (d + 6 * U) * (g * xh).abs().mean(1, keepdim=True)
    core = g - c1 - xh * c2
    e_core = 4 * U * (g.abs() + c1.abs() + (xh * c2).abs()) + e_c1 + xh.abs() * e_c2 \
        + e_xh * c2.abs()
    dx = rs * core
    e_dx = rs * e_core + U * dx.abs()
    if dz is not None:
        dx = dx + dz
        e_dx = e_dx + U * (dx.abs() + dz.abs())
    # rows are added one after another within a block, then the blocks' sums
    n = (min(rows, 1300) + rows // 64 + 16) * U
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return dict(dx=dx, e_dx=e_dx, dweight=dw, e_dweight=(n + 4 * U) * (dy * xh).abs().sum(0),
                dbias=db, e_dbias=n * dy.abs().sum(0))


# ------------------------------------------------------------- 4-bit weights

def w4_place(nibble):
    """k of nibble 0..127 of a block (nibble = 8 word + position)."""
    word, pos = nibble // 8, nibble % 8
    return 32 * (word % 4) + 8 * (word // 4) + 2 * (pos % 4) + pos // 4


def w4_pack_ref(values):
    """values [..., N, K] uint8 (numpy) -> codes [..., N, ceil(K/128)*64]."""
    K = values.shape[-1]
    nb = -(-K // 128)
    full = np.zeros(values.shape[:-1] + (nb * 128,), dtype=np.uint8)
    full[..., :K] = values & 15
    order = np.array([w4_place(i) for i in range(128)])
    nib = full.reshape(full.shape[:-1] + (nb, 128))[..., order]
    codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
    return np.ascontiguousarray(codes.reshape(values.shape[:-1] + (nb * 64,)))


def w4_unpack_ref(codes, K):
    """codes [..., bytes] (numpy) -> values [..., K]."""
    nb = codes.shape[-1] // 64
    c = codes.reshape(codes.shape[:-1] + (nb, 64))
    nib = np.empty(c.shape[:-1] + (128,), dtype=np.uint8)
    nib[..., 0::2] = c & 15
    nib[..., 1::2] = c >> 4
    out = np.empty_like(nib)
    out[..., np.array([w4_place(i) for i in range(128)])] = nib
    return out.reshape(codes.shape[:-1] + (nb * 128,))[..., :K]


def w4_weight_ref(codes, scales, zeros, group, K):
    """Device tensors -> the weight in float64 on the same device."""
    q = torch.from_numpy(w4_unpack_ref(codes.cpu().numpy(), K)).to(codes.device).double()
    s = scales.double().repeat_interleave(group, dim=-1)
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, dim=-1)
    return (q - z) * s


def w4_product_bound(x, W):
    """Bound of the fp32 error of x W^T: the products are exact; a group's sum
    of at most 128 terms may be truncated (a whole step, 2u) at each addition,
    then the scaled group sums are added."""
    K = x.shape[-1]
    return (2 * 128 + K // 32 + 32) * U * (x.abs() @ W.abs().transpose(-1, -2))


def experts_ref(x, idx, prob, keep, W1, W3, W2):
    """x float64 [T,h]; weights float64 [E,..]; -> y and the bound of its error
    before the last rounding."""
    y, e_y = torch.zeros_like(x), torch.zeros_like(x)
    T, k = idx.shape
    for t in range(T):
        for j in range(k):
            if keep is not None and not keep[t, j]:
                continue
            e, p = int(idx[t, j]), float(prob[t, j])
            xt = x[t:t + 1]
            a, b = xt @ W1[e].t(), xt @ W3[e].t()
            ea, eb = w4_product_bound(xt, W1[e]), w4_product_bound(xt, W3[e])
            s = a * torch.sigmoid(a)
            h = s * b
            # |silu'| < 1.1; silu itself to 8 roundings, and the two bf16 parts hold 2^-17
            eh = 1.1 * ea * b.abs() + (s.abs() + 1.1 * ea) * eb + (8 * U + 2.0 ** -17) * h.abs()
            y[t] += p * (h @ W2[e].t())[0]
            e_y[t] += abs(p) * (eh @ W2[e].abs().t() + w4_product_bound(h, W2[e]))[0]
    return y, e_y + (k + 2) * U * y.abs()


def assert_within(name, got, ref, bound, dtype=None):
    """|got - ref| <= bound + half a step of dtype (and, for values below the
    type's normal range, its smallest step)."""
    got, ref = got.detach().double(), ref.double()
    tol = bound.double()
    if dtype is not None:
        tol = tol + half(dtype) * (ref.abs() + tol) + torch.finfo(dtype).tiny
    off = (got - ref).abs() - tol
    bad = ~(off <= 0)
    assert not bad.any(), "%s: %d of %d out of bounds, worst %.3g over at %s" % (
        name, int(bad.sum()), bad.numel(), float(off[bad].max()),
        torch.nonzero(bad)[0].tolist())
