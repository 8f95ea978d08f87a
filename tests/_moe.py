"""64-bit definitions of the few-token and mixture-of-experts operators for the tests.

Error bounds used with them:
  * FP32 sums of n products: at most n roundings (or truncations), each within 2^-23 of
    the partial sum, so within n * 2^-23 * sum |a b| of the exact sum; n counts the K
    products and three more roundings per 128-block (scale product, scaling, addition).
  * One rounding to BF16: within 2^-8 of the value (half of eps = 2^-7).
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -23
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def values(codes):
    """E4M3 codes (uint8) as float64: sign, exponent (bias 7), 3 bits of mantissa."""
    c = torch.arange(256, device=codes.device)
    exp, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(exp > 0, (1 + man / 8) * torch.exp2((exp - 7).double()), man * 2.0 ** -9)
    return torch.where(c > 127, -mag, mag)[codes.long()]


def nearest(v):
    """float64 onto E4M3: nearest, ties to even, saturating."""
    _, ex = torch.frexp(v)
    step = torch.exp2((ex.clamp(min=-5) - 4).double())
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def groups(x):
    """1x128 groups of the rows of float64 x: (quotients [M][K/128][128], scales [M][K/128][1]),
    the scale and the quotients rounded to binary32."""
    m, k = x.shape
    v = x.view(m, k // 128, 128)
    s = (v.abs().amax(-1, keepdim=True) / 448).float().double()
    return (v / torch.where(s > 0, s, torch.ones_like(s))).float().double(), s


def dequant_rows(x):
    """The values that quantizing the rows of x (any float) keeps, in float64."""
    q, s = groups(x.double())
    return (nearest(q) * s).view(x.shape)


def rows64(codes, s):
    """Codes [M][K] with scales [K/128][M]."""
    return values(codes) * s.t().double().repeat_interleave(128, 1)


def blocks64(codes, s):
    """Codes [N][K] with scales [N/128][K/128]."""
    return values(codes) * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def sum_bound(k):
    return (k + 3 * (k // 128)) * U32


def check(y, ref, slack, what=""):
    """|y - ref| <= slack elementwise (NaN fails)."""
    err = (y.double() - ref).abs()
    bad = ~(err <= slack)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; first at {i}: "
                             f"{y[i].item()!r}, expected {ref[i].item()!r} within {slack[i].item()!r}")


def check_bf16(y, ref, asum, k, what=""):
    """A BF16 result of FP32 sums over k products whose magnitudes sum to asum."""
    acc = sum_bound(k) * asum
    # the rounding is of the FP32 sum; a result in BF16's subnormals is off by 2^-134 at most
    check(y, ref, acc + BF16_HALF * (ref.abs() + acc) + 2.0 ** -134, what)


def acts(gen, m, k, std=1.0):
    x = torch.randn(m, k, generator=gen, device=gen.device) * std
    x[:, :: max(1, k // 7)] *= 20.0
    return x.bfloat16()


def weights(gen, e, n, k):
    """E quantized weights: codes [E][N][K], scales [E][N/128][K/128] (fp8_quant_weight)."""
    import blockwise_fp8_linear_b200 as fb
    w = (torch.randn(e * n, k, generator=gen, device="cuda") * 0.02).bfloat16()
    q, s, _ = fb.fp8_quant_weight(w)
    return q.view(e, n, k), s.view(e, n // 128, k // 128)


def route(logits, k, renorm):
    """ids (-1 where nothing is left) and float64 weights, by comparing every pair."""
    v = logits.double()
    v = torch.where(v > -torch.inf, v.clamp(max=torch.finfo(logits.dtype).max), -torch.inf)
    e = v.shape[1]
    at = torch.arange(e, device=v.device)
    ahead = (v.unsqueeze(1) > v.unsqueeze(2)) | \
        ((v.unsqueeze(1) == v.unsqueeze(2)) & (at.view(1, 1, e) < at.view(1, e, 1)))
    rank = ahead.sum(2)  # [T][E]: experts before this one
    ids = torch.full((v.shape[0], k), -1, dtype=torch.long, device=v.device)
    some = (rank < k) & (v > -torch.inf)
    t, x = torch.nonzero(some, as_tuple=True)
    ids[t, rank[t, x]] = x
    high = v.amax(1, keepdim=True)
    p = torch.exp(v - torch.where(high > -torch.inf, high, torch.zeros_like(high)))
    den = (p * some if renorm else p).sum(1, keepdim=True)
    p = p / torch.where(den > 0, den, torch.ones_like(den))
    w = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), torch.zeros(1, dtype=p.dtype, device=p.device))
    return ids, w, p * some if renorm else p


def plan(ids, e, rows):
    """seg, row, src by going through the pairs one by one (host lists)."""
    flat = ids.reshape(-1).tolist()
    mine = [[p for p, x in enumerate(flat) if x == y] for y in range(e)]
    seg, row, src = [0], [-1] * len(flat), [-1] * rows
    for y in range(e):
        for i, p in enumerate(mine[y]):
            row[p] = 128 * seg[-1] + i
            src[row[p]] = p
        seg.append(seg[-1] + (len(mine[y]) + 127) // 128)
    return seg, row, src


def layer(x, w1, s1, w2, s2, ids, wt):
    """The few-token layer: (y, slack), slack bounding every allowed rounding: FP32 sums,
    the codes of h that an error of h within its own bound can move, and the BF16 result."""
    t, h = x.shape
    e, _, i = w2.shape
    xd = dequant_rows(x)
    y = torch.zeros(t, h, dtype=torch.float64, device=x.device)
    acc = torch.zeros_like(y)
    for n in range(e):
        tok = torch.nonzero((ids == n).any(1)).view(-1)
        if not tok.numel():
            continue
        w = torch.where(ids[tok] == n, wt[tok].double(), torch.zeros(1, dtype=torch.float64, device=x.device)).sum(1)
        a1, a2 = blocks64(w1[n], s1[n]), blocks64(w2[n], s2[n])
        gu, mag = xd[tok] @ a1.t(), xd[tok].abs() @ a1.abs().t()
        eg, eu = (sum_bound(h) * mag).chunk(2, 1)
        g, u = gu.chunk(2, 1)
        sg = g * torch.sigmoid(g)
        act = sg * u
        # |d silu| <= 1.1 |dg|; exp, its division and the products are good to 2^-20
        ea = 1.1 * eg * (u.abs() + eu) + sg.abs() * eu + 2.0 ** -20 * act.abs() + 2.0 ** -149
        q, s = groups(act)
        es = ea.view(s.shape[0], -1, 128).amax(-1, keepdim=True) / 448 + 2.0 ** -23 * s + 2.0 ** -149
        safe = torch.where(s > 0, s, torch.ones_like(s))
        eq = ea.view(q.shape) / safe + q.abs() * (es / safe) + 2.0 ** -22 * q.abs()
        c = nearest(q)
        ec = torch.maximum((nearest(q + eq) - c).abs(), (nearest(q - eq) - c).abs())
        hd = (c * s).view(act.shape)
        eh = (ec * (s + es) + c.abs() * es).view(act.shape)
        part, pm = hd @ a2.t(), hd.abs() @ a2.abs().t()
        ep = eh @ a2.abs().t() * (1 + 2.0 ** -10) + sum_bound(i) * pm
        y[tok] += w.view(-1, 1) * part
        # the weighted sum of up to k products: k + 1 more roundings of what is summed
        acc[tok] += w.abs().view(-1, 1) * (ep + (ids.shape[1] + 2) * U32 * pm)
    return y, acc + BF16_HALF * (y.abs() + acc) + 2.0 ** -134
