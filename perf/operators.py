"""Workloads of the mixture-of-experts and few-token operators.

Four operators around the blockwise-FP8 linear layer (E4M3 codes, activations scaled per
1x128 group along the reduction, weights per 128x128 block, scale = amax / 448):

  few      y = x W^T for 1 to 64 tokens, activations quantized inside the call
  route    softmax router: top-k choices and weights; for training also the plan that
           lays the (token, choice) pairs out by expert and the gradient of the logits
  grouped  the experts' fprop, dgrad and wgrad products over that layout
  layer    all experts of a SwiGLU mixture-of-experts layer for 1 to 64 tokens

`run` computes them in plain torch operations, or, with `own` set, by the package's calls.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
MODES = {"fprop": 0, "dgrad": 1, "wgrad": 2}
DEV = "cuda"


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # One decoded token through an attention output projection: pure latency.
        {"name": "few-1x2048x2048", "op": "few", "m": 1, "n": 2048, "k": 2048},
        # A few decoded sequences through a down projection with a long reduction.
        {"name": "few-7x2048x6144", "op": "few", "m": 7, "n": 2048, "k": 6144},
        # A full small batch through the gate/up projection: the widest linear.
        {"name": "few-61x12288x2048", "op": "few", "m": 61, "n": 12288, "k": 2048},
        # Router of a decode step: BF16 logits, so ties occur; two experts are disabled.
        {"name": "route-5x64", "op": "route", "t": 5, "e": 64, "k": 6, "bf16": True,
         "renorm": True, "train": False, "off": 2, "gone": 0.0},
        # Router of a training step at the repository's 8192 tokens, with its plan and
        # gradient; some rows are padding that no expert may take.
        {"name": "route-8192x128-train", "op": "route", "t": 8192, "e": 128, "k": 8, "bf16": False,
         "renorm": True, "train": True, "off": 0, "gone": 0.01},
        # Many experts, an odd token count, weights that keep the full softmax's denominator.
        {"name": "route-65521x256-train", "op": "route", "t": 65521, "e": 256, "k": 8, "bf16": True,
         "renorm": False, "train": True, "off": 3, "gone": 0.0},
        # Experts' forward product of a short micro-batch: less than one row tile each.
        {"name": "grouped-fprop-1000", "op": "grouped", "mode": "fprop", "rows": 1000, "e": 16,
         "n": 1024, "k": 1024, "skew": 0.5, "idle": 2, "acc32": False},
        # The gate/up product of a training step: 8192 tokens, 8 choices each, 128 experts.
        {"name": "grouped-fprop-65536", "op": "grouped", "mode": "fprop", "rows": 65536, "e": 128,
         "n": 1536, "k": 2048, "skew": 0.3, "idle": 0, "acc32": False},
        # Input gradient of the down product, uneven experts.
        {"name": "grouped-dgrad-16384", "op": "grouped", "mode": "dgrad", "rows": 16384, "e": 32,
         "n": 1024, "k": 2048, "skew": 0.6, "idle": 1, "acc32": False},
        # Weight gradient into FP32 main gradients that the step has just cleared.
        {"name": "grouped-wgrad-32768", "op": "grouped", "mode": "wgrad", "rows": 32768, "e": 32,
         "n": 2048, "k": 1536, "skew": 0.4, "idle": 1, "acc32": True},
        # One decoded token through a whole layer of 128 experts.
        {"name": "layer-1x2048", "op": "layer", "t": 1, "e": 128, "k": 8, "h": 2048, "i": 768,
         "gone": 0.0},
        # A decode batch with padding rows: most experts have a token or two.
        {"name": "layer-40x2048", "op": "layer", "t": 40, "e": 128, "k": 8, "h": 2048, "i": 768,
         "gone": 0.05},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999 * step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("few", "route", "grouped", "layer"))
    if op == "few":
        return {"op": op, "m": _log(rng, 1, 64), "n": _log(rng, 256, 12288, 128),
                "k": _log(rng, 256, 12288, 128)}
    if op == "route":
        e = _log(rng, 4, 256)
        return {"op": op, "t": _log(rng, 1, 65536), "e": e, "k": rng.randint(1, min(8, e)),
                "bf16": rng.random() < 0.5, "renorm": rng.random() < 0.6,
                "train": rng.random() < 0.6, "off": rng.choice((0, 0, 1, e // 2)),
                "gone": rng.choice((0.0, 0.02))}
    if op == "grouped":
        mode = rng.choice(tuple(MODES))
        e = _log(rng, 2, 64)
        return {"op": op, "mode": mode, "rows": _log(rng, 16, 32768), "e": e,
                "n": _log(rng, 256, 2048, 128), "k": _log(rng, 256, 2048, 128),
                "skew": round(rng.uniform(0.0, 1.0), 2), "idle": rng.choice((0, 1)),
                "acc32": mode == "wgrad" and rng.random() < 0.5}
    e = _log(rng, 8, 128)
    return {"op": op, "t": _log(rng, 1, 64), "e": e, "k": rng.randint(1, 8),
            "h": _log(rng, 512, 2048, 128), "i": _log(rng, 256, 1024, 128),
            "gone": rng.choice((0.0, 0.1))}


def _capacity(pairs, e):
    """Rows of the padded layout that hold any split of `pairs` over `e` experts."""
    return 128 * ((pairs + 127 * min(e, pairs)) // 128)


def work(case):
    op = case["op"]
    if op == "few":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k + 4 * n * k // 16384 + 2 * m * (n + k), "flops": 2 * m * n * k}
    if op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        size = 2 if case["bf16"] else 4
        b, f = t * e * size + 8 * t * k, 4 * t * e
        if case["train"]:
            # dlogits written, dweights read; seg, row and src written
            b += t * e * size + 4 * t * k + 4 * (e + 1) + 4 * t * k + 4 * _capacity(t * k, e)
            f += 4 * t * e
        return {"bytes": b, "flops": f}
    if op == "grouped":
        p, e, n, k = case["rows"], case["e"], case["n"], case["k"]
        live = max(1, e - case["idle"])
        if case["mode"] == "wgrad":
            return {"bytes": p * (n + k) * (1 + 4 / 128) + (4 if case["acc32"] else 2) * e * n * k,
                    "flops": 2 * p * n * k}
        return {"bytes": p * k * (1 + 4 / 128) + live * n * k + 2 * p * n, "flops": 2 * p * n * k}
    t, e, k, h, i = case["t"], case["e"], case["k"], case["h"], case["i"]
    hit = e * (1.0 - (1.0 - min(1.0, k / e)) ** t)
    return {"bytes": hit * 3 * i * h + 4 * t * h + 8 * t * k, "flops": 6 * t * k * i * h}


# -------------------------------------------------------------- inputs (made on the GPU)

def _div(a, c):
    # by a tensor: division by a Python scalar multiplies by its reciprocal
    return a / torch.full_like(a, c)


def _codes(v, s):
    q = torch.where(s > 0, v / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(v))
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quant_rows(x):
    """x[M][K] -> codes uint8 [M][K], scales float32 [K/128][M]."""
    m, k = x.shape
    v = x.float().view(m, k // 128, 128)
    s = _div(v.abs().amax(-1, keepdim=True), E4M3_MAX)
    return _codes(v, s).view(torch.uint8).view(m, k), s.view(m, k // 128).t().contiguous()


def _quant_blocks(w):
    """w[N][K] -> codes uint8 [N][K], scales float32 [N/128][K/128]."""
    n, k = w.shape
    v = w.float().view(n // 128, 128, k // 128, 128)
    s = _div(v.abs().amax(dim=(1, 3), keepdim=True), E4M3_MAX)
    return _codes(v, s).view(torch.uint8).view(n, k), s.view(n // 128, k // 128)


def _weights(gen, e, n, k):
    w = torch.randn(e * n, k, generator=gen, device=DEV).mul_(0.02).bfloat16()
    q, s = _quant_blocks(w)
    return q.view(e, n, k), s.view(e, n // 128, k // 128)


def _acts(gen, m, k, std):
    # one channel in a hundred is an outlier, as in Transformer activations
    x = torch.randn(m, k, generator=gen, device=DEV).mul_(std)
    big = torch.rand(k, generator=gen, device=DEV) < 0.01
    return torch.where(big, 20.0 * x, x).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "few":
        st["x"] = _acts(gen, case["m"], case["k"], 1.0)
        q, s = _weights(gen, 1, case["n"], case["k"])
        st["qw"], st["sw"] = q[0], s[0].contiguous()
    elif op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        logits = 2.0 * torch.randn(t, e, generator=gen, device=DEV)
        logits += torch.randn(e, generator=gen, device=DEV)
        if case["off"]:
            dead = torch.randperm(e, generator=gen, device=DEV)[:case["off"]]
            logits[:, dead] = -math.inf
        gone = torch.rand(t, generator=gen, device=DEV) < case["gone"]
        logits[gone] = -math.inf
        st["logits"] = logits.bfloat16() if case["bf16"] else logits
        st["dweights"] = torch.randn(t, k, generator=gen, device=DEV)
    elif op == "grouped":
        p, e, n, k = case["rows"], case["e"], case["n"], case["k"]
        odds = torch.exp(case["skew"] * torch.randn(e, generator=gen, device=DEV))
        if case["idle"] < e:
            odds[:case["idle"]] = 0.0
        ids = torch.multinomial(odds, p, replacement=True, generator=gen).view(p, 1).int()
        seg, _, src = _plan(ids, e)
        real = (src >= 0).view(-1, 1)
        rows = src.numel()
        st["seg"] = seg
        if case["mode"] == "wgrad":
            dy = _acts(gen, rows, n, 1e-3) * real
            x = _acts(gen, rows, k, 1.0) * real
            st["a"], st["sa"] = _quant_rows(dy.t().contiguous())
            st["b"], st["sb"] = _quant_rows(x.t().contiguous())
            if not case["acc32"]:
                st["out"] = torch.zeros(e, n, k, dtype=torch.bfloat16, device=DEV)
        else:
            fprop = case["mode"] == "fprop"
            st["a"], st["sa"] = _quant_rows(_acts(gen, rows, k, 1.0 if fprop else 1e-3) * real)
            st["b"], st["sb"] = _weights(gen, e, n, k) if fprop else _weights(gen, e, k, n)
            # rows behind the last expert's are left as they were: a cleared buffer
            st["out"] = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    else:
        t, e, k, h, i = case["t"], case["e"], case["k"], case["h"], case["i"]
        st["x"] = _acts(gen, t, h, 1.0)
        st["w1"], st["s1"] = _weights(gen, e, 2 * i, h)
        st["w2"], st["s2"] = _weights(gen, e, h, i)
        logits = torch.randn(t, e, generator=gen, device=DEV)
        logits[torch.rand(t, generator=gen, device=DEV) < case["gone"]] = -math.inf
        st["weights"], st["ids"] = _route(logits, min(k, e), True)
    return st


# ------------------------------------------------------------------------ plain forms

def _f32(q):
    return q.view(torch.float8_e4m3fn).float()


def _rows32(q, s):
    """Codes [M][K] with scales [K/128][M] as float32 values."""
    m, k = q.shape
    return (_f32(q).view(m, k // 128, 128) * s.t().unsqueeze(-1)).view(m, k)


def _blocks32(q, s):
    """Codes [..., N, K] with scales [..., N/128, K/128] as float32 values."""
    *b, n, k = q.shape
    v = _f32(q).view(*b, n // 128, 128, k // 128, 128) * s.view(*b, n // 128, 1, k // 128, 1)
    return v.view(*b, n, k)


def _few(x, qw, sw):
    q, s = _quant_rows(x)
    return (_rows32(q, s) @ _blocks32(qw, sw).t()).bfloat16()


def _route(logits, k, renorm):
    v = logits.float()
    top, ids = torch.sort(v, dim=1, descending=True, stable=True)  # ties: lowest index first
    top, ids = top[:, :k], ids[:, :k]
    some = top > -math.inf
    high = torch.where(some[:, :1], top[:, :1], torch.zeros_like(top[:, :1]))
    p = torch.exp(top - high)
    den = (p if renorm else torch.exp(v - high)).sum(1, keepdim=True)
    w = torch.where(some, p / torch.where(den > 0, den, torch.ones_like(den)), torch.zeros_like(p))
    return w, torch.where(some, ids, torch.full_like(ids, -1)).int()


def _route_bwd(dw, w, ids, logits, renorm):
    t, e = logits.shape
    some = ids >= 0
    at = torch.where(some, ids, torch.zeros_like(ids)).long()
    g = torch.where(some, w * dw, torch.zeros_like(w))
    total = g.sum(1, keepdim=True)
    if renorm:
        return torch.zeros(t, e, device=DEV).scatter_add_(1, at, g - w * total).to(logits.dtype)
    v = logits.float()
    high = v.amax(1, keepdim=True)
    p = torch.exp(v - torch.where(high > -math.inf, high, torch.zeros_like(high)))
    den = p.sum(1, keepdim=True)
    p = p / torch.where(den > 0, den, torch.ones_like(den))
    return (-p * total).scatter_add_(1, at, g).to(logits.dtype)


def _plan(ids, e):
    t, k = ids.shape
    flat = ids.reshape(-1).long()
    pairs = flat.numel()
    ok = (flat >= 0) & (flat < e)
    key = torch.where(ok, flat, torch.full_like(flat, e))
    count = torch.zeros(e + 1, dtype=torch.long, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(count, 0) - count
    blocks = (count[:e] + 127) // 128
    seg = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(blocks, 0)])
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(pairs, device=DEV) - first[key[order]]
    row = torch.where(ok, 128 * seg[key] + place, torch.full_like(flat, -1))
    rows = _capacity(pairs, e)
    src = torch.full((rows + 1,), -1, dtype=torch.long, device=DEV)
    src[torch.where(ok, row, torch.full_like(row, rows))] = torch.arange(pairs, device=DEV)
    return seg.int(), row.view(t, k).int(), src[:rows].int()


def _block_expert(seg, blocks):
    """Which expert each block of 128 rows belongs to, and whether it belongs to one."""
    at = torch.arange(blocks, device=DEV)
    e = (at.unsqueeze(1) >= seg[1:].long().unsqueeze(0)).sum(1)
    live = e < seg.numel() - 1
    return torch.where(live, e, torch.zeros_like(e)), live


def _grouped(st):
    c, seg = st["case"], st["seg"]
    if c["mode"] == "wgrad":
        blocks = st["a"].shape[1] // 128
        e, live = _block_expert(seg, blocks)
        a = _rows32(st["a"], st["sa"]).view(-1, blocks, 128).transpose(0, 1)
        b = _rows32(st["b"], st["sb"]).view(-1, blocks, 128).transpose(0, 1)
        part = torch.bmm(a, b.transpose(1, 2)).view(blocks, -1)
        pick = (e.unsqueeze(0) == torch.arange(c["e"], device=DEV).unsqueeze(1)) & live
        d = (pick.float() @ part).view(c["e"], a.shape[1], b.shape[1])
        return torch.zeros_like(d) + d if c["acc32"] else d.bfloat16()
    rows, k = st["a"].shape
    e, live = _block_expert(seg, rows // 128)
    a = _rows32(st["a"], st["sa"]).view(rows // 128, 128, k)
    w = _blocks32(st["b"], st["sb"])[e]
    y = torch.bmm(a, w.transpose(1, 2) if c["mode"] == "fprop" else w)
    return torch.where(live.view(-1, 1, 1), y, torch.zeros_like(y)).view(rows, -1).bfloat16()


def _layer(st):
    x, ids, wt = st["x"], st["ids"], st["weights"]
    t, k = ids.shape
    e, h, i = st["w2"].shape
    q, s = _quant_rows(x)
    xd = _rows32(q, s)
    some = ids >= 0
    at = torch.where(some, ids, torch.zeros_like(ids)).long()
    if t * k < e:  # few pairs: their experts' weights alone
        pair = at.view(-1)
        gu = torch.bmm(_blocks32(st["w1"][pair], st["s1"][pair]),
                       xd.repeat_interleave(k, 0).unsqueeze(-1)).view(t * k, 2 * i)
    else:
        every = (xd @ _blocks32(st["w1"], st["s1"]).view(e * 2 * i, h).t()).view(t, e, 2 * i)
        gu = every[torch.arange(t, device=DEV).view(t, 1), at].view(t * k, 2 * i)
    g, u = gu[:, :i], gu[:, i:]
    act = g / (1.0 + torch.exp(-g)) * u
    hd = _rows32(*_quant_rows(act))
    if t * k < e:
        y = torch.bmm(_blocks32(st["w2"][pair], st["s2"][pair]), hd.unsqueeze(-1)).view(t, k, h)
    else:
        # rows laid out by (token, expert), so that one batched product serves every expert
        full = torch.zeros(e, t, i, device=DEV)
        live = some.view(-1, 1).float()
        tok = torch.arange(t, device=DEV).repeat_interleave(k)
        full.index_put_((at.view(-1), tok), hd * live, accumulate=True)
        every = torch.bmm(full, _blocks32(st["w2"], st["s2"]).transpose(1, 2))
        y = every[at, torch.arange(t, device=DEV).view(t, 1)]
    wt = torch.where(some, wt, torch.zeros_like(wt))
    return (y * wt.unsqueeze(-1)).sum(1).bfloat16()


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import blockwise_fp8_linear_b200 as fb
        if op == "few":
            return fb.fp8_linear_few(st["x"], st["qw"], st["sw"])
        if op == "route":
            w, ids = fb.fp8_moe_route(st["logits"], c["k"], renorm=c["renorm"])
            if not c["train"]:
                return {"weights": w, "ids": ids}
            seg, row, src = fb.fp8_moe_plan(ids, c["e"])
            dl = fb.fp8_moe_route_bwd(st["dweights"], w, ids, st["logits"], renorm=c["renorm"])
            return {"weights": w, "ids": ids, "seg": seg, "row": row, "src": src, "dlogits": dl}
        if op == "grouped":
            mode = MODES[c["mode"]]
            a, b = st["a"], st["b"]
            if c["mode"] == "wgrad":
                m, n, k = a.shape[0], b.shape[0], a.shape[1]
                if c["acc32"]:
                    dw = torch.zeros(c["e"], m, n, device=DEV)
                    return fb.fp8_gemm_grouped_wgrad_acc32(a, st["sa"], b, st["sb"], st["seg"],
                                                           m, n, k, dw)
            else:
                m, n, k = a.shape[0], c["n"], a.shape[1]
            return fb.fp8_gemm_grouped(mode, a, st["sa"], b, st["sb"], st["seg"], m, n, k,
                                       out=st["out"])
        return fb.fp8_moe_few(st["x"], st["w1"], st["s1"], st["w2"], st["s2"], st["ids"],
                              st["weights"])
    if op == "few":
        return _few(st["x"], st["qw"], st["sw"])
    if op == "route":
        w, ids = _route(st["logits"], c["k"], c["renorm"])
        if not c["train"]:
            return {"weights": w, "ids": ids}
        seg, row, src = _plan(ids, c["e"])
        dl = _route_bwd(st["dweights"], w, ids, st["logits"], c["renorm"])
        return {"weights": w, "ids": ids, "seg": seg, "row": row, "src": src, "dlogits": dl}
    return _grouped(st) if op == "grouped" else _layer(st)


# --------------------------------------------------- the definitions, in 64 bits

def _value(codes):
    """E4M3 codes as float64, from the format: sign, 4 exponent bits (bias 7), 3 of mantissa."""
    c = torch.arange(256, device=codes.device)
    exp, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(exp > 0, (1 + man / 8) * torch.exp2((exp - 7).double()), man * 2.0 ** -9)
    return torch.where(c > 127, -mag, mag)[codes.long()]


def _nearest(v):
    """float64 rounded onto E4M3: nearest, ties to even, saturating at 448."""
    _, ex = torch.frexp(v)
    step = torch.exp2((ex.clamp(min=-5) - 4).double())
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _dequant64(x):
    """The values that 1x128 quantization of the rows of x (float64) keeps. The scale and
    the quotients are rounded to binary32, as the scheme defines them."""
    m, k = x.shape
    v = x.view(m, k // 128, 128)
    s = (v.abs().amax(-1, keepdim=True) / 448).float().double()
    q = (v / torch.where(s > 0, s, torch.ones_like(s))).float().double()
    return (_nearest(q) * s).view(m, k)


def _spread64(q, s, along_rows):
    rows = 1 if along_rows else 128
    return _value(q) * s.double().repeat_interleave(rows, 0).repeat_interleave(128, 1)


def _exact_route(st, c):
    v = st["logits"].double()
    t, e = v.shape
    k, renorm = c["k"], c["renorm"]
    # rank of each expert: how many are larger, or equal with a lower index
    left, chosen, picked = v.clone(), [], torch.zeros(t, e, dtype=torch.bool, device=v.device)
    index = torch.arange(e, device=v.device)
    for _ in range(k):
        best = left.amax(1, keepdim=True)
        at = torch.where(left == best, index, e).amin(1)
        at = torch.where(best[:, 0] > -math.inf, at, -1)
        hit = index == at.view(-1, 1)
        left = left.masked_fill(hit, -math.inf)
        picked |= hit
        chosen.append(at)
    ids = torch.stack(chosen, 1)
    high = v.amax(1, keepdim=True)
    p = torch.exp(v - torch.where(high > -math.inf, high, 0.0))
    den = (p * picked if renorm else p).sum(1, keepdim=True)
    p = p / torch.where(den > 0, den, 1.0)
    w = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
    out = {"weights": w, "ids": ids.int()}
    if not c["train"]:
        return out
    flat = ids.reshape(-1)
    counts = (flat.view(-1, 1) == index).sum(0).tolist()
    seg, row = [0], torch.full_like(flat, -1)
    src = torch.full((_capacity(t * k, e),), -1, dtype=torch.long, device=v.device)
    for x in range(e):
        mine = torch.nonzero(flat == x).view(-1)
        at = 128 * seg[-1] + torch.arange(counts[x], device=v.device)
        row[mine], src[at] = at, mine
        seg.append(seg[-1] + -(-counts[x] // 128))
    # d w_j / d l_i = w_j ([i = j] - p_i), with p over the chosen experts alone or over all
    dw = torch.where(ids >= 0, st["dweights"].double(), 0.0)
    direct = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), w * dw)
    dl = direct - (p * picked if renorm else p) * (w * dw).sum(1, keepdim=True)
    out.update(seg=torch.tensor(seg, dtype=torch.int32), row=row.view(t, k).int(), src=src.int(),
               dlogits=dl)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "few":
        return _dequant64(st["x"].double()) @ _spread64(st["qw"], st["sw"], False).t()
    if op == "route":
        return _exact_route(st, case)
    if op == "grouped":
        seg = st["seg"].tolist()
        n = case["n"]
        if case["mode"] == "wgrad":
            d = torch.zeros(case["e"], n, case["k"], dtype=torch.float64, device=DEV)
        else:
            d = torch.zeros(st["a"].shape[0], n, dtype=torch.float64, device=DEV)
        for x in range(case["e"]):
            lo, hi = seg[x], seg[x + 1]
            cut = slice(128 * lo, 128 * hi)
            if case["mode"] == "wgrad":
                a = _spread64(st["a"][:, cut], st["sa"][lo:hi].t(), True)
                d[x] = a @ _spread64(st["b"][:, cut], st["sb"][lo:hi].t(), True).t()
            else:
                a = _spread64(st["a"][cut], st["sa"][:, cut].t(), True)
                w = _spread64(st["b"][x], st["sb"][x], False)
                d[cut] = a @ (w.t() if case["mode"] == "fprop" else w)
        return d
    x = _dequant64(st["x"].double())
    ids, i = st["ids"], case["i"]
    y = torch.zeros(case["t"], case["h"], dtype=torch.float64, device=DEV)
    for e in range(case["e"]):
        tok, j = torch.nonzero(ids == e, as_tuple=True)
        if tok.numel():
            gu = x[tok] @ _spread64(st["w1"][e], st["s1"][e], False).t()
            act = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
            part = _dequant64(act) @ _spread64(st["w2"][e], st["s2"][e], False).t()
            y[tok] += part * st["weights"][tok, j].double().view(-1, 1)
    return y
