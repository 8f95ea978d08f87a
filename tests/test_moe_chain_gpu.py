"""The mixture-of-experts calls as a program uses them: a training step of a SwiGLU expert
layer, decode steps on streams, and captured graphs."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import acts, check, layer, weights

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def gather(x, src, k):
    """Rows of x in the layout by expert, zero where no pair stands."""
    tok = (src.clamp(min=0) // k).long()
    return torch.where((src >= 0).view(-1, 1), x[tok], torch.zeros((), dtype=x.dtype, device=x.device))


def swiglu(gu):
    g, u = gu.float().chunk(2, 1)
    return g * torch.sigmoid(g) * u


def train_step(x, w1, s1, w2, s2, logits, k, dy):
    """Forward and backward of the layer; returns y, dx, dlogits, dw1, dw2."""
    t, h = x.shape
    e, _, i = w2.shape
    wt, ids = fb.fp8_moe_route(logits, k)
    seg, row, src = fb.fp8_moe_plan(ids, e)
    rows = src.numel()
    live = (src >= 0).view(-1, 1)
    xp = gather(x, src, k)
    qx, sx, qxt, sxt = fb.fp8_quant_act_dual(xp)
    zeros = lambda n: torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    gu = fb.fp8_gemm_grouped(fb.FPROP, qx, sx, w1, s1, seg, rows, 2 * i, h, out=zeros(2 * i))
    act = swiglu(gu).bfloat16()
    qh, sh, qht, sht = fb.fp8_quant_act_dual(act)
    yp = fb.fp8_gemm_grouped(fb.FPROP, qh, sh, w2, s2, seg, rows, h, i, out=zeros(h))
    pair_y = yp[row.long().clamp(min=0)].float()                     # [t][k][h]
    y = (pair_y * wt.unsqueeze(-1)).sum(1)
    # backward
    dwt = (pair_y * dy.float().unsqueeze(1)).sum(-1)
    dlogits = fb.fp8_moe_route_bwd(dwt, wt, ids, logits)
    scale = wt.reshape(-1)[src.clamp(min=0).long()].view(-1, 1)
    dyp = torch.where(live, gather(dy, src, k).float() * scale, torch.zeros((), device="cuda")).bfloat16()
    qd, sd, qdt, sdt = fb.fp8_quant_act_dual(dyp)
    dact = fb.fp8_gemm_grouped(fb.DGRAD, qd, sd, w2, s2, seg, rows, i, h, out=zeros(i)).float()
    dw2 = torch.zeros(e, h, i, device="cuda")
    fb.fp8_gemm_grouped_wgrad_acc32(qdt, sdt, qht, sht, seg, h, i, rows, dw2)
    g, u = gu.float().chunk(2, 1)
    sg = torch.sigmoid(g)
    dgu = torch.cat([dact * u * sg * (1 + g * (1 - sg)), dact * g * sg], 1).bfloat16()
    qg, sgs, qgt, sgt = fb.fp8_quant_act_dual(dgu)
    dxp = fb.fp8_gemm_grouped(fb.DGRAD, qg, sgs, w1, s1, seg, rows, h, 2 * i, out=zeros(h))
    dw1 = fb.fp8_gemm_grouped(fb.WGRAD, qgt, sgt, qxt, sxt, seg, 2 * i, h, rows)
    dx = dxp[row.long().clamp(min=0)].float().sum(1)
    return y, dx, dlogits, dw1, dw2


def autograd(x, w1, w2, logits, k, dy):
    """The same layer on float64 values with dequantized weights."""
    x, w1, w2, lg = (v.double().detach().clone().requires_grad_() for v in (x, w1, w2, logits))
    top, ids = torch.topk(lg, k, dim=1)
    wt = torch.softmax(top, 1)
    y = torch.zeros_like(x)
    for e in range(w2.shape[0]):
        tok, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[tok] @ w1[e].t()
        g, u = gu.chunk(2, 1)
        y = y.index_add(0, tok, (g * torch.sigmoid(g) * u @ w2[e].t()) * wt[tok, j].unsqueeze(1))
    y.backward(dy.double())
    return y.detach(), x.grad, lg.grad, w1.grad, w2.grad


def dequant(q, s):
    from _moe import blocks64
    return torch.stack([blocks64(a, b) for a, b in zip(q, s)])


@pytest.mark.parametrize("t,e,k,h,i", [(300, 6, 2, 256, 128), (64, 16, 4, 128, 256)])
def test_training_step(t, e, k, h, i):
    g = gen(t)
    x = torch.randn(t, h, generator=g, device="cuda").bfloat16()
    w1, s1 = weights(g, e, 2 * i, h)
    w2, s2 = weights(g, e, h, i)
    logits = torch.randn(t, e, generator=g, device="cuda")
    logits[:, 1] -= 100.0                                            # an expert without tokens
    dy = torch.randn(t, h, generator=g, device="cuda").bfloat16()
    got = train_step(x, w1, s1, w2, s2, logits, k, dy)
    ref = autograd(x, dequant(w1, s1), dequant(w2, s2), logits, k, dy)
    # Each quantized operand carries E4M3's rounding, at most 2^-4 and about 2^-4 / sqrt(3)
    # of a value in the mean square; no result passes through more than four quantized
    # operands (x, h, dy and dgu), whose errors, were they all aligned, add to 4 * 2^-4.
    for name, a, b in zip(("y", "dx", "dlogits", "dw1", "dw2"), got, ref):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel <= 0.25, f"{name}: {rel}"
    assert (got[3][1] == 0).all() and (got[4][1] == 0).all()
    # few tokens: the decode layer is the same function
    if t <= fb.FEW_TOKENS:
        wt, ids = fb.fp8_moe_route(logits, k)
        y = fb.fp8_moe_few(x, w1, s1, w2, s2, ids, wt)
        want, slack = layer(x, w1, s1, w2, s2, ids, wt)
        check(y, want, slack, "decode")


def decode(a, ws, out):
    """Router, expert layer and a following linear of one decode step."""
    x, lg, w1, s1, w2, s2, qw, sw = a
    wt, ids = fb.fp8_moe_route(lg, 2, weights=out[0], ids=out[1])
    fb.fp8_moe_few(x, w1, s1, w2, s2, ids, wt, out=out[2], workspace=ws)
    fb.fp8_linear_few(out[2], qw, sw, out=out[3])
    return out


def decode_state(seed, t=9, e=8, h=256, i=256):
    g = gen(seed)
    w1, s1 = weights(g, e, 2 * i, h)
    w2, s2 = weights(g, e, h, i)
    qw, sw = weights(g, 1, 384, h)
    a = [acts(g, t, h), torch.randn(t, e, generator=g, device="cuda"), w1, s1, w2, s2, qw[0], sw[0]]
    ws = torch.empty(fb.fp8_moe_few_workspace(t, 2, h, i), dtype=torch.uint8, device="cuda")
    out = [torch.empty(t, 2, device="cuda"), torch.empty(t, 2, dtype=torch.int32, device="cuda"),
           torch.empty(t, h, dtype=torch.bfloat16, device="cuda"),
           torch.empty(t, 384, dtype=torch.bfloat16, device="cuda")]
    return a, ws, out


def test_decode_chain_back_to_back():
    # dependent launches: no synchronization between steps, inputs change from step to step
    a, ws, out = decode_state(1)
    xs = [acts(gen(50 + n), 9, 256) for n in range(8)]
    want = []
    for x in xs:
        a[0].copy_(x)
        torch.cuda.synchronize()
        want.append([o.clone() for o in decode(a, ws, out)])
        torch.cuda.synchronize()
    got = []
    for x in xs:
        a[0].copy_(x)
        got.append([o.clone() for o in decode(a, ws, out)])
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(p, q))
    assert fb.fp8bw_last_device_error() == 0


def test_decode_on_two_streams():
    states = [decode_state(n) for n in (2, 3)]
    want = []
    for s in states:
        want.append([o.clone() for o in decode(*s)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(20):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                decode(*s)
    torch.cuda.synchronize()
    for w, s in zip(want, states):
        assert all(torch.equal(u, v) for u, v in zip(w, s[2]))


def test_stream_argument_and_own_workspace():
    # the workspace that the call allocates for itself belongs to the stream it runs on
    (x, lg, w1, s1, w2, s2, _, _), _, _ = decode_state(4)
    wt, ids = fb.fp8_moe_route(lg, 2)
    want = fb.fp8_moe_few(x, w1, s1, w2, s2, ids, wt)
    seg = fb.fp8_moe_plan(ids, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.empty_like(want) for _ in range(10)]
    for o in outs:
        fb.fp8_moe_few(x, w1, s1, w2, s2, ids, wt, out=o, stream=side)
        plan = fb.fp8_moe_plan(ids, 8, seg=torch.empty_like(seg[0]), row=torch.empty_like(seg[1]),
                               src=torch.empty_like(seg[2]), stream=side)
        torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")  # reuses freed memory, if any
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert all(torch.equal(u, v) for u, v in zip(seg, plan))


def test_decode_graphs():
    """Two captured decode steps, each with its own workspace, replayed side by side on
    inputs that change between replays."""
    states = [decode_state(n) for n in (5, 6)]
    for s in states:
        decode(*s)          # eager first: sets the kernels' shared-memory limits
    torch.cuda.synchronize()
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode(*s)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in states]
    for n in range(4):
        for m, s in enumerate(states):
            s[0][0].copy_(acts(gen(100 + 10 * n + m), 9, 256))
            s[0][1].copy_(torch.randn(9, 8, generator=gen(7 * n + m), device="cuda"))
        want = [[o.clone() for o in decode(*s)] for s in states]
        for s in states:
            for o in s[2]:
                o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for w, s in zip(want, states):
            assert all(torch.equal(u, v) for u, v in zip(w, s[2]))


def test_training_graph():
    t, e, k, h, i = 200, 4, 2, 128, 128
    g = gen(8)
    w1, s1 = weights(g, e, 2 * i, h)
    w2, s2 = weights(g, e, h, i)
    x = torch.randn(t, h, generator=g, device="cuda").bfloat16()
    logits = torch.randn(t, e, generator=g, device="cuda")
    dy = torch.randn(t, h, generator=g, device="cuda").bfloat16()
    args = (x, w1, s1, w2, s2, logits, k, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train_step(*args)
    for n in range(3):
        x.copy_(torch.randn(t, h, generator=g, device="cuda"))
        logits.copy_(torch.randn(t, e, generator=g, device="cuda"))
        want = train_step(*args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(("y", "dx", "dlogits", "dw1", "dw2"), out, want):
            assert torch.equal(a, b), name
