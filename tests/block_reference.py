"""64-bit references of the transformer-block operators and the error bounds the tests hold the
kernels to.

Bounds.  A result that sums terms t_k is off by at most a few ulps of sum |t_k| (call it A) from
its fp32 arithmetic, half an ulp of its type at the store, and, where the kernel rounds the
factors of a product to its 16-bit type before the tensor cores (the softmax weights and their
gradients), half an ulp of that type of A more.  With u the spacing of the type at 1 (2^-7 bf16,
2^-10 fp16, 2^-23 fp32):

    |err| <= u / 2 * (|ref| + A) * 1.05 + C * 2^-24 * A + tiny

C covers the fp32 part: the score of D products (its error enters the weight as a factor), the
exponential, and the sums; scores here stay below 32 in absolute terms, a score is off by less
than 32 * 4 * 2^-24 and a weight relatively by as much, so C = 256 covers score, shift and sums.
"""
import math

import torch

U = {"float32": 2.0 ** -23, "float16": 2.0 ** -10, "bfloat16": 2.0 ** -7}
TINY = {"float32": 1e-30, "float16": 2.0 ** -24, "bfloat16": 1e-30}
DT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def bound(ref, A, dtype, C=256.0):
    return U[dtype] / 2 * (ref.abs() + A) * 1.05 + C * 2.0 ** -24 * A + TINY[dtype]


def check(got, ref, A, dtype, what="", C=256.0):
    got = got.to(torch.float64).cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    err = (got - ref).abs()
    lim = bound(ref, A, dtype, C)
    bad = fine & ~(err <= lim)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, err / lim, torch.zeros_like(err))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at flat {i}: "
                             f"got {got.flatten()[i]!r}, ref {ref.flatten()[i]!r}, "
                             f"bound {lim.flatten()[i]!r}")


# ------------------------------------------------------------------ layer norm

def layer_norm(x, scale, b, eps):
    mean = x.mean(1, keepdim=True)
    inv = 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    xh = (x - mean) * inv
    y = xh * scale + (b if b is not None else 0.0)
    return y, mean, inv


def layer_norm_backward(dy, x, scale, mean, inv):
    """Gradients and the sums of absolute terms that bound their errors."""
    xh, g = (x - mean) * inv, dy * scale
    a, c = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = inv * (g - a - xh * c)
    adx = inv * (g.abs() + g.abs().mean(1, keepdim=True)
                 + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    return (dx, (dy * xh).sum(0), dy.sum(0)), (adx, (dy * xh).abs().sum(0), dy.abs().sum(0))


# ------------------------------------------------------------------ dropout

def philox_words(n, seed, offset):
    """n words of Philox4x32-10 in Python integers (a few thousand at most)."""
    out = []
    for i in range((n + 3) // 4):
        c = [i & 0xFFFFFFFF, i >> 32, offset & 0xFFFFFFFF, offset >> 32]
        k = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF,
                 (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        out += c
    return out[:n]


# ------------------------------------------------------------------ attention

def pair_bias(table, buckets, q_extent, k_extent):
    """(H, Lq, Lk) bias in 64 bits, -inf where a bucket lies outside the table, and the buckets."""
    (hq, wq), (hk, wk) = q_extent, k_extent
    i, j = torch.arange(hq * wq), torch.arange(hk * wk)
    dy = (i // wq)[:, None] - (j // wk)[None, :] + hk - 1
    dx = (i % wq)[:, None] - (j % wk)[None, :] + wk - 1
    b = buckets.cpu().reshape(hq + hk - 1, wq + wk - 1)[dy, dx].long()
    out = (b < 0) | (b >= table.shape[0])
    bias = table.cpu().to(torch.float64)[b.clamp(0, table.shape[0] - 1)].permute(2, 0, 1).clone()
    bias[:, out] = -math.inf
    return bias, torch.where(out, -1, b)


def _heads(t):
    return t.detach().cpu().to(torch.float64).permute(0, 2, 1, 3)


def scores(Q, K, scale, bias, k_len):
    q, k = _heads(Q), _heads(K)
    Lk = k.shape[2]
    dead = (torch.arange(Lk)[None, :] >= k_len.cpu()[:, None].clamp(0, Lk) if k_len is not None
            else torch.zeros((q.shape[0], Lk), dtype=torch.bool))
    k = torch.where(dead[:, None, :, None], 0.0, k)   # masked keys are never used
    s = q @ k.transpose(2, 3) * scale
    if bias is not None:
        s = s + bias
    return s.masked_fill(dead[:, None, None, :], -math.inf), dead


def attention(Q, K, V, scale, bias=None, k_len=None):
    """O (N, Lq, H, D), LSE and the sum of absolute terms of O."""
    s, dead = scores(Q, K, scale, bias, k_len)
    v = torch.where(dead[:, None, :, None], 0.0, _heads(V))
    if s.shape[3] == 0:
        z = torch.zeros((s.shape[0], s.shape[2], s.shape[1], v.shape[3]), dtype=torch.float64)
        return z, torch.full(s.shape[:3], -math.inf, dtype=torch.float64), z
    top = s.amax(3, keepdim=True)
    p = torch.where(s == -math.inf, 0.0, torch.exp(s - torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(3, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf).squeeze(3)
    p = torch.where(total > 0, p / total, torch.where(torch.isnan(total), total, 0.0))
    return (p @ v).permute(0, 2, 1, 3), lse, (p @ v.abs()).permute(0, 2, 1, 3)


def attention_backward(dO, Q, K, V, O, LSE, scale, bias=None, k_len=None, which=None, nb=0):
    """(dQ, dK, dV, dTable) and the sums of absolute terms that bound their errors."""
    s, dead = scores(Q, K, scale, bias, k_len)
    blank = dead[:, None, :, None]
    k, v = (torch.where(blank, 0.0, _heads(t)) for t in (K, V))
    q, do, o = _heads(Q), _heads(dO), _heads(O)
    lse = LSE.detach().cpu().to(torch.float64).unsqueeze(3)
    live = (s != -math.inf) & (lse != -math.inf)
    p = torch.where(live, torch.exp(s - lse), 0.0)
    ds = torch.where(live, p * (do @ v.transpose(2, 3) - (do * o).sum(3, keepdim=True)), 0.0)
    ads = p * (do.abs() @ v.abs().transpose(2, 3) + (do * o).abs().sum(3, keepdim=True))
    back = lambda t: t.permute(0, 2, 1, 3)
    grads = [back(ds @ k) * scale, back(ds.transpose(2, 3) @ q) * scale, back(p.transpose(2, 3) @ do)]
    sums = [back(ads @ k.abs()) * scale, back(ads.transpose(2, 3) @ q.abs()) * scale,
            back(p.transpose(2, 3) @ do.abs())]
    if which is not None:
        rows = which.reshape(-1)
        for t, into in ((ds, grads), (ads, sums)):
            per = t.sum(0).permute(1, 2, 0).reshape(-1, t.shape[1])
            z = torch.zeros((nb + 1, t.shape[1]), dtype=torch.float64)
            into.append(z.index_add_(0, torch.where(rows < 0, nb, rows), per)[:nb])
    return grads, sums
