"""Router, its gradient and the plan against 64-bit definitions."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import BF16_HALF, U32, check, plan, route

pytestmark = pytest.mark.gpu
INF = float("inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def logits_of(t, e, dtype, seed):
    return (torch.randn(t, e, generator=gen(seed), device="cuda") * 2).to(dtype)


def check_route(logits, k, renorm):
    t, e = logits.shape
    w, ids = fb.fp8_moe_route(logits, k, renorm=renorm)
    ref_ids, ref_w, _ = route(logits, k, renorm)
    assert ids.dtype == torch.int32 and torch.equal(ids.long(), ref_ids)
    # p = exp(l - top) / den: the difference is rounded once (relative to it), expf is good
    # to 1 ulp, den sums at most e / 32 + 5 terms in a row, one division
    span = (logits.double().clamp(-1e30, 1e30).amax(1, keepdim=True) -
            logits.double().gather(1, ref_ids.clamp(min=0)).clamp(-1e30, 1e30))
    span = torch.where(ref_ids >= 0, span, torch.zeros_like(span)).clamp(max=200.0)
    check(w, ref_w, (span + e / 32 + 10 + span.amax(1, keepdim=True)) * U32 * ref_w + 2.0 ** -126, "weights")
    return w, ids


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 2, 2), (3, 5, 4), (9, 31, 8), (8, 32, 8), (17, 33, 3),
                                   (5, 64, 6), (40, 127, 8), (33, 128, 32), (7, 129, 8), (100, 256, 8),
                                   (6, 260, 5), (5, 511, 7), (4, 512, 8), (4, 1000, 9), (3, 1023, 4),
                                   (3, 1024, 32)])
def test_route(t, e, k, renorm, dtype):
    check_route(logits_of(t, e, dtype, 1000 * e + t), k, renorm)


def test_route_many_rows():
    # more rows than the grid has warps
    check_route(logits_of(30011, 16, torch.float32, 3), 2, True)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_ties_and_masks(dtype, renorm):
    x = logits_of(12, 48, dtype, 5)
    x[0] = 0.0                       # all equal: the first experts
    x[1, ::2], x[1, 1::2] = 0.0, -0.0   # zeros of both signs are equal
    x[2] = -INF                      # nothing to choose
    x[3, 3:] = -INF                  # fewer than k
    x[4] = torch.finfo(dtype).min    # masks of the type's lowest value are values
    x[5] = torch.finfo(dtype).max
    x[6, 7] = INF
    x[7, 7], x[7, 9] = INF, INF
    x[8, 1:] = torch.finfo(dtype).min
    x[9, 0], x[9, 1:] = -INF, 1.0
    x[10, 3], x[10, 5] = torch.finfo(dtype).max, INF   # equal: the lower comes first
    x[11] = -x[11].abs() - 1         # all negative
    w, ids = check_route(x, 6, renorm)
    assert ids[0].tolist() == list(range(6)) and ids[1].tolist() == list(range(6))
    assert ids[2].tolist() == [-1] * 6 and w[2].tolist() == [0.0] * 6
    assert ids[3].tolist()[3:] == [-1] * 3
    # NaN counts as -inf
    y = x.clone()
    y[3, 3:] = float("nan")
    y[2] = float("nan")
    w2, ids2 = fb.fp8_moe_route(y, 6, renorm=renorm)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (5, 7, 3), (20, 64, 8), (9, 130, 8), (33, 256, 4),
                                   (3, 1024, 32), (2, 1001, 5)])
def test_route_bwd(t, e, k, renorm, dtype):
    x = logits_of(t, e, dtype, 7 * e + t)
    if t > 3:
        x[1] = -INF
        x[2, k - 1:] = -INF
    w, ids = fb.fp8_moe_route(x, k, renorm=renorm)
    dw = torch.randn(t, k, generator=gen(t), device="cuda")
    dl = fb.fp8_moe_route_bwd(dw, w, ids, x, renorm=renorm)
    assert dl.dtype == dtype and dl.shape == (t, e)
    rid, rw, p = route(x, k, renorm)
    g = torch.where(rid >= 0, rw * dw.double(), torch.zeros_like(rw))
    direct = torch.zeros_like(p).scatter_add_(1, rid.clamp(min=0), g)
    ref = direct - p * g.sum(1, keepdim=True)
    # weights and probabilities as in test_route (span <= 20 here), sums of k terms
    rel = (2 * 20 + e / 32 + 10 + k + 6) * U32
    slack = rel * (direct.abs() + p * g.abs().sum(1, keepdim=True)) + 2.0 ** -126
    check(dl, ref, slack + (BF16_HALF * (ref.abs() + slack) if dtype == torch.bfloat16 else 0), "dlogits")


@pytest.mark.parametrize("renorm", [True, False])
def test_route_bwd_against_differences(renorm):
    t, e, k = 4, 12, 3
    x = logits_of(t, e, torch.float32, 11)
    dw = torch.randn(t, k, generator=gen(2), device="cuda")
    w, ids = fb.fp8_moe_route(x, k, renorm=renorm)
    dl = fb.fp8_moe_route_bwd(dw, w, ids, x, renorm=renorm)

    def loss(v):  # the chosen experts stay the same under a small step
        p = torch.softmax(v, 1).gather(1, ids.long())
        return ((p / p.sum(1, keepdim=True) if renorm else p) * dw.double()).sum(1)

    step = 1e-4
    for c in range(e):
        d = torch.zeros(t, e, dtype=torch.float64, device="cuda")
        d[:, c] = step
        diff = (loss(x.double() + d) - loss(x.double() - d)) / (2 * step)
        # third derivative of a softmax is below 1 in size: step^2 / 6 * sum |dw|, and FP32
        assert ((dl[:, c].double() - diff).abs() <= 1e-8 * dw.abs().sum(1) + 1e-5).all()


def test_route_bwd_left_out_and_repeated_choices():
    # ids outside the range take no part; an expert named twice collects both gradients
    x = logits_of(1, 6, torch.float32, 4)
    w = torch.tensor([[0.25, 0.5, 0.25, 9.0]], device="cuda")
    ids = torch.tensor([[2, 4, 2, 6]], dtype=torch.int32, device="cuda")
    dw = torch.tensor([[1.0, 2.0, 4.0, 7.0]], device="cuda")
    dl = fb.fp8_moe_route_bwd(dw, w, ids, x, renorm=True)
    total = 0.25 + 1.0 + 1.0
    want = [0, 0, 0.25 + 1.0 - 0.5 * total, 0, 1.0 - 0.5 * total, 0]
    assert dl[0].tolist() == want


def check_plan(ids, e):
    seg, row, src = fb.fp8_moe_plan(ids, e)
    rows = fb.fp8_moe_plan_rows(ids.shape[0], e, ids.shape[1])
    rs, rr, rc = plan(ids, e, rows)
    assert seg.tolist() == rs and row.reshape(-1).tolist() == rr and src.tolist() == rc


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 3), (127, 3, 1), (128, 2, 1), (129, 2, 1), (64, 64, 8),
                                   (300, 5, 4), (1000, 33, 3), (2048, 4, 1), (2049, 4, 1), (5000, 128, 8),
                                   (513, 1024, 8), (700, 1000, 32)])
def test_plan(t, e, k):
    g = gen(t + e)
    logits = torch.randn(t, e, generator=g, device="cuda") + 2 * torch.randn(e, generator=g, device="cuda")
    _, ids = fb.fp8_moe_route(logits, k)
    check_plan(ids, e)


def test_plan_special_ids():
    t, k, e = 700, 4, 9
    ids = torch.randint(-2, e + 3, (t, k), generator=gen(8), device="cuda", dtype=torch.int32)
    check_plan(ids, e)                                   # some outside the range
    check_plan(torch.full_like(ids, -1), e)              # none at all
    check_plan(torch.full_like(ids, e - 1), e)           # one expert takes everything, repeatedly
    ids[:, 0] = 2 ** 31 - 1
    ids[:, 1] = -2 ** 31
    check_plan(ids, e)


def test_plan_large_is_consistent():
    # 128 chunks: the placement checked by its own inverse and order
    t, e, k = 60000, 200, 8
    _, ids = fb.fp8_moe_route(logits_of(t, e, torch.bfloat16, 9), k)
    seg, row, src = (x.long() for x in fb.fp8_moe_plan(ids, e))
    flat, r = ids.reshape(-1).long(), row.reshape(-1)
    pairs = torch.arange(t * k, device="cuda")
    assert torch.equal(src[r], pairs) and int((src >= 0).sum()) == t * k
    count = torch.bincount(flat, minlength=e)
    assert torch.equal(seg[1:] - seg[:-1], (count + 127) // 128) and int(seg[0]) == 0
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = pairs - (torch.cumsum(count, 0) - count)[flat[order]]
    assert torch.equal(r, 128 * seg[flat] + place)


def test_plan_caller_buffers():
    ids = torch.randint(0, 6, (4000, 3), generator=gen(1), device="cuda", dtype=torch.int32)
    need = fb.lib().fp8_moe_plan_workspace(4000, 6, 3)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a = fb.fp8_moe_plan(ids, 6)
    b = fb.fp8_moe_plan(ids, 6, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(ValueError):
        fb.fp8_moe_plan(ids, 6, workspace=ws[:-16])
