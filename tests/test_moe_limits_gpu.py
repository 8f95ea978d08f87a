"""Few-token and mixture-of-experts calls at the ends of their ranges: the largest sizes of
one dimension, the most choices, offsets past 32 bits, two calls at once."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import U32, acts, blocks64, check, check_bf16, dequant_rows, layer, rows64, route, sum_bound, weights

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("m,n,k", [(3, 128, 1 << 20), (33, 128, 1 << 20), (64, 1 << 20, 128), (2, 1 << 20, 256)])
def test_linear_longest_sides(m, n, k):
    g = gen(m)
    x = acts(g, m, k)
    qw, sw = weights(g, 1, n, k)
    y = fb.fp8_linear_few(x, qw[0], sw[0])
    a = dequant_rows(x)
    step = 1 << 14 if n > 128 else 128
    for lo in range(0, n, step):
        cut = slice(lo, lo + step)
        w = blocks64(qw[0][cut], sw[0][lo // 128:(lo + step) // 128])
        check_bf16(y[:, cut], a @ w.t(), a.abs() @ w.abs().t(), k, f"columns from {lo}")


def make(g, t, e, k, h, i):
    x = acts(g, t, h)
    # the gate and the up rows quantized apart: one call takes no more than fb.MAX_DIM rows
    halves = [weights(g, e, i, h) for _ in range(2)]
    w1, s1 = (torch.cat(t, 1) for t in zip(*halves))
    w2, s2 = weights(g, e, h, i)
    wt, ids = fb.fp8_moe_route(torch.randn(t, e, generator=g, device="cuda"), k)
    return [x, w1, s1, w2, s2, ids, wt]


@pytest.mark.parametrize("t,e,k,h,i", [
    (64, 32, 32, 128, 128),      # every token chooses every expert: two units of rows each
    (16, 1024, 32, 128, 128),    # the most experts that 16 tokens can hit
    (64, 1024, 32, 128, 128),
    (2, 1, 1, 1 << 20, 128), (33, 2, 2, 1 << 19, 128), (2, 1, 1, 128, 1 << 19), (2, 1, 1, 128, 1 << 20), (20, 2, 1, 128, 1 << 18)])
def test_layer_ends_of_the_ranges(t, e, k, h, i):
    a = make(gen(t + e), t, e, k, h, i)
    y = fb.fp8_moe_few(*a)
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
    ref, slack = layer(*a)
    check(y, ref, slack, "layer")


def last_expert(g, e, n, k):
    """E experts' weights of more than 4 GB, all zero but the last one's."""
    w, s = torch.zeros(e, n, k, dtype=torch.uint8, device="cuda"), torch.zeros(e, n // 128, k // 128, device="cuda")
    q, sc = weights(g, 1, n, k)
    w[-1], s[-1] = q[0], sc[0]
    return w, s


def test_layer_weights_past_4_gb():
    g = gen(2)
    t, e, h, i = 5, 1024, 2048, 1152
    w1, s1 = last_expert(g, e, 2 * i, h)
    w2, s2 = last_expert(g, e, h, i)
    assert w1.numel() > 1 << 32
    x = acts(g, t, h)
    ids = torch.tensor([[e - 1, 0]] * t, dtype=torch.int32, device="cuda")
    wt = torch.rand(t, 2, generator=g, device="cuda")
    y = fb.fp8_moe_few(x, w1, s1, w2, s2, ids, wt)
    # expert 0 is all zero: the last one alone counts
    ref, slack = layer(x, w1[-1:], s1[-1:], w2[-1:], s2[-1:], torch.zeros_like(ids[:, :1]), wt[:, :1])
    check(y, ref, slack, "layer")


@pytest.mark.parametrize("mode", [fb.FPROP, fb.DGRAD])
def test_grouped_weights_past_4_gb(mode):
    g = gen(3)
    e, n, k, blocks = 600, 2048, 4096, 3
    b, sb = last_expert(g, e, n, k) if mode == fb.FPROP else last_expert(g, e, k, n)
    assert b.numel() > 1 << 32
    a, sa = fb.fp8_quant_act(acts(g, 128 * blocks, k))
    seg = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    seg[1:] = 1
    seg[-1] = blocks             # one block for expert 0, the rest for the last
    d = fb.fp8_gemm_grouped(mode, a, sa, b, sb, seg, 128 * blocks, n, k)
    assert (d[:128] == 0).all()
    a64 = rows64(a, sa)[128:]
    w = blocks64(b[-1], sb[-1])
    w = w.t() if mode == fb.FPROP else w
    check_bf16(d[128:], a64 @ w, a64.abs() @ w.abs(), k, "last expert")


@pytest.mark.parametrize("acc32", [False, True])
def test_grouped_wgrad_output_past_4_gb(acc32):
    g = gen(4)
    e, m, n, blocks = 600, 2048, 4096, 3
    a, sa = fb.fp8_quant_act_t(acts(g, 128 * blocks, m, 1e-3))
    b, sb = fb.fp8_quant_act_t(acts(g, 128 * blocks, n))
    seg = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    seg[-1] = blocks             # all for the last expert
    if acc32:
        d = torch.ones(e, m, n, device="cuda")
        fb.fp8_gemm_grouped_wgrad_acc32(a, sa, b, sb, seg, m, n, 128 * blocks, d)
        assert all(bool((x == 1).all()) for x in d[:-1].split(50))
    else:
        d = torch.ones(e, m, n, dtype=torch.bfloat16, device="cuda")
        fb.fp8_gemm_grouped(fb.WGRAD, a, sa, b, sb, seg, m, n, 128 * blocks, out=d)
        assert all(bool((x == 0).all()) for x in d[:-1].split(50))
    a64, b64 = rows64(a, sa), rows64(b, sb)
    ref, mag = a64 @ b64.t(), a64.abs() @ b64.abs().t()
    if acc32:
        # 1 + sum: the sum's own error, and one rounding of the total
        check(d[-1], 1 + ref, sum_bound(128 * blocks) * mag + 2.0 ** -24 * (1 + ref.abs() + mag), "last expert")
    else:
        check_bf16(d[-1], ref, mag, 128 * blocks, "last expert")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_rows_past_2_gb(dtype):
    t, e, k = 1 << 20, 1024 if dtype == torch.float32 else 1023, 2
    x = torch.zeros(t, e, dtype=dtype, device="cuda")
    rows = torch.tensor([0, 1, t // 2 + 1, t - 2, t - 1], device="cuda")
    x[rows] = torch.randn(5, e, generator=gen(5), device="cuda").to(dtype)
    w, ids = fb.fp8_moe_route(x, k, renorm=False)
    few_w, few_ids = fb.fp8_moe_route(x[rows], k, renorm=False)
    assert torch.equal(w[rows], few_w) and torch.equal(ids[rows], few_ids)
    assert ids[2:t // 2].eq(torch.tensor([0, 1], device="cuda")).all() and w[2:t // 2].eq(1 / torch.tensor(float(e), device="cuda")).all()
    dw = torch.ones(t, k, device="cuda")
    dw[rows] = torch.randn(5, k, generator=gen(6), device="cuda")
    dl = fb.fp8_moe_route_bwd(dw, w, ids, x, renorm=False)
    few = fb.fp8_moe_route_bwd(dw[rows], few_w, few_ids, x[rows], renorm=False)
    assert torch.equal(dl[rows], few)


@pytest.mark.parametrize("t,e,k,out", [
    (130000, 16, 8, False),   # nearly 2^20 pairs: every step of the warps' runs
    (300, 1024, 8, True), (1021, 1000, 16, True), (2341, 7, 7, True), (1 << 15, 1, 1, False),
    (4096, 64, 8, True), (4097, 64, 8, True),
    (8192, 128, 8, True), (8193, 128, 8, True), (2048, 1024, 32, True)])   # 2^16 pairs and a token more
def test_plan_of_many_pairs(t, e, k, out):
    g = gen(7)
    _, ids = fb.fp8_moe_route(torch.randn(t, e, generator=g, device="cuda"), k)
    if out:
        ids[torch.rand(t, k, generator=g, device="cuda") < 0.1] = -1
        ids[3] = e
    seg, row, src = (x.long() for x in fb.fp8_moe_plan(ids, e))
    flat, r = ids.reshape(-1).long(), row.reshape(-1)
    pairs = torch.nonzero((flat >= 0) & (flat < e)).view(-1)
    flat = flat[pairs]
    count = torch.bincount(flat, minlength=e)
    assert int(seg[0]) == 0 and torch.equal(seg[1:] - seg[:-1], (count + 127) // 128)
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device="cuda") - (torch.cumsum(count, 0) - count)[flat[order]]
    assert torch.equal(r[pairs], 128 * seg[flat] + place) and int((r >= 0).sum()) == len(pairs)
    assert torch.equal(src[r[pairs]], pairs) and int((src >= 0).sum()) == len(pairs)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(65, 7, 7), (130, 64, 8), (130, 256, 32), (67, 1000, 5), (65, 1024, 32)])
def test_route_among_few_values(t, e, k, dtype):
    # equal logits within a lane, across lanes, and around the last choice
    g = gen(e)
    levels = torch.randint(1, 2 * e, (t, 1), generator=g, device="cuda")
    x = (torch.randint(0, 1 << 20, (t, e), generator=g, device="cuda") % levels / 64).to(dtype)
    x[torch.rand(t, e, generator=g, device="cuda") < 0.2] = -torch.inf
    w, ids = fb.fp8_moe_route(x, k)
    ref_ids, ref_w, _ = route(x, k, True)
    assert torch.equal(ids.long(), ref_ids)
    # exp to 2 ulp, its argument within |d| 2^-24, |d| <= 32; k + 1 sums and a division
    check(w, ref_w, (64 + k) * U32 * ref_w + 2.0 ** -126, "weights")


def test_two_layers_of_many_tokens_at_once():
    # kernels with one CTA per SM on two streams
    states = [make(gen(20 + n), 40, 24, 4, 512, 384) for n in range(2)]
    outs = [torch.empty_like(s[0]) for s in states]
    ws = [torch.empty(fb.fp8_moe_few_workspace(40, 4, 512, 384), dtype=torch.uint8, device="cuda") for _ in states]
    want = [fb.fp8_moe_few(*s).clone() for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(30):
        for s, o, w, st in zip(states, outs, ws, streams):
            with torch.cuda.stream(st):
                fb.fp8_moe_few(*s, out=o, workspace=w)
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_overlapping_arguments_are_refused():
    # CTAs of one launch would read what others have stored
    a = make(gen(30), 4, 8, 2, 256, 256)
    x, w1, s1, w2, s2, ids, wt = a
    square, scales = w2[0], s2[0]
    logits = torch.randn(4, 8, generator=gen(31), device="cuda")
    dw = torch.ones(4, 2, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    many = x.repeat(16, 1)
    codes, sc = fb.fp8_quant_act(acts(gen(32), 256, 256))
    seg = torch.tensor([0, 1, 2] + [2] * 6, dtype=torch.int32, device="cuda")
    q, qs = fb.fp8_quant_act_t(acts(gen(33), 256, 256))
    main = torch.zeros(1 << 21, device="cuda")
    inside = main[:8 * 256 * 256].view(8, 256, 256)
    for call in (
            lambda: fb.fp8_linear_few(x, square, scales, out=x),
            lambda: fb.fp8_linear_few(many, square, scales, out=ws[:64 * 256 * 2].view(torch.bfloat16).view(64, 256),
                                      workspace=ws),
            lambda: fb.fp8_moe_route(logits, 8, weights=logits),
            lambda: fb.fp8_moe_route(logits, 2, weights=dw, ids=dw.view(torch.int32)),
            lambda: fb.fp8_moe_route_bwd(dw, wt, ids, logits, dlogits=logits),
            lambda: fb.fp8_moe_plan(ids, 8, row=ids),
            lambda: fb.fp8_moe_plan(ids, 8, seg=ws[:36].view(torch.int32), workspace=ws),
            lambda: fb.fp8_gemm_grouped(fb.FPROP, codes, sc, w2, s2, seg, 256, 256, 256,
                                        out=w2.view(-1)[:256 * 256 * 2].view(torch.bfloat16).view(256, 256)),
            lambda: fb.fp8_gemm_grouped_wgrad_acc32(q, qs, inside[0].view(torch.uint8).view(-1)[:65536].view(256, 256),
                                                    qs, seg, 256, 256, 256, inside),
            lambda: fb.fp8_moe_few(*a, out=x),
            lambda: fb.fp8_moe_few(*a, workspace=w1.view(-1))):
        with pytest.raises(fb.Fp8bwError) as e:
            call()
        assert e.value.status == 1
    # neighbours in one buffer are apart
    both = torch.empty(2, 4, 256, dtype=torch.bfloat16, device="cuda")
    both[0] = x
    y = fb.fp8_linear_few(both[0], square, scales, out=both[1])
    assert torch.equal(y, fb.fp8_linear_few(x, square, scales))


def test_outputs_on_another_stream_take_no_block_of_the_current_one():
    # work queued on the current stream may still read a block that Python has freed
    x, w1, s1, w2, s2, ids, wt = a = make(gen(40), 64, 8, 2, 1024, 256)
    logits = torch.randn(64, 1024, generator=gen(41), device="cuda")
    lw, lids = fb.fp8_moe_route(logits, 32)
    codes, sc = fb.fp8_quant_act(acts(gen(42), 256, 1024))
    b, sb = fb.fp8_quant_act(acts(gen(43), 8 * 512, 1024))[0].view(8, 512, 1024), torch.ones(8, 4, 8, device="cuda")
    seg = torch.tensor([0, 1, 2] + [2] * 6, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda **kw: fb.fp8_linear_few(x, w1[0], s1[0], **kw),
                 lambda **kw: fb.fp8_moe_route(logits, 32, **kw),
                 lambda **kw: fb.fp8_moe_route_bwd(lw, lw, lids, logits, **kw),
                 lambda **kw: fb.fp8_moe_plan(lids, 1024, **kw),
                 lambda **kw: fb.fp8_gemm_grouped(fb.FPROP, codes, sc, b, sb, seg, 256, 512, 1024, **kw),
                 lambda **kw: fb.fp8_moe_few(*a, **kw)):
        here = call()
        here = here if isinstance(here, tuple) else (here,)
        freed = {t.untyped_storage().data_ptr() for t in here}
        want = [t.clone() for t in here]
        torch.cuda.synchronize()
        del here
        there = call(stream=side)
        there = there if isinstance(there, tuple) else (there,)
        assert not freed & {t.untyped_storage().data_ptr() for t in there}
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(there, want))


@pytest.mark.parametrize("t", [2, 5, 12, 40, 64])
def test_a_token_without_finite_values_stays_alone(t):
    # (its own results are unspecified)
    a = make(gen(50 + t), t, 12, 3, 512, 384)
    x, w1, s1 = a[:3]
    a[5][t - 1] = -1                  # one that chooses nothing: zero whatever its values are
    clean, layer_clean = fb.fp8_linear_few(x, w1[0], s1[0]), fb.fp8_moe_few(*a)
    for value in (float("nan"), float("inf")):
        for row in {0, t // 2, t - 1}:
            bad = x.clone()
            bad[row, 100:300] = value
            rest = torch.arange(t, device="cuda") != row
            assert torch.equal(fb.fp8_linear_few(bad, w1[0], s1[0])[rest], clean[rest])
            y = fb.fp8_moe_few(bad, *a[1:])
            assert torch.equal(y[rest], layer_clean[rest]) and (y[t - 1] == 0).all()
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
