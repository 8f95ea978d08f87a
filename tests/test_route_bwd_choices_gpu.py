"""Gradient of the logits where the caller has left choices out since the forward call, the
first among them, or lists them in another order."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import BF16_HALF, U32, check, route

pytestmark = pytest.mark.gpu
INF = float("inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inputs(t, e, k, renorm, dtype):
    """Logits within 20 of each other, but for some of -inf and one row with +inf."""
    x = (torch.randn(t, e, generator=gen(e + t), device="cuda") * 2).clamp(-10, 10).to(dtype)
    if e > k + 2:
        x[::3, k + 1] = -INF
        x[t - 1, 1] = INF
    w, ids = fb.fp8_moe_route(x, k, renorm=renorm)
    return x, w, ids, torch.randn(t, k, generator=gen(k), device="cuda")


def check_bwd(x, w, ids, dw, p, renorm):
    """Against g - p G of the choices that are there, p in 64 bits."""
    t, e = x.shape
    k = ids.shape[1]
    dl = fb.fp8_moe_route_bwd(dw, w, ids, x, renorm=renorm)
    some = (ids >= 0) & (ids < e)
    g = torch.where(some, w.double() * dw.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    direct = torch.zeros_like(p).scatter_add_(1, torch.where(some, ids, 0).long(), g)
    ref = direct - p * g.sum(1, keepdim=True)
    # p: exp of a difference d, |d| <= 20, is off by (|d| + 2) 2^-23, so are the sum's terms or
    # the weight that stands for them; the sum has e / 32 + 5 roundings, G at most k + 6, the
    # quotient and the products four
    rel = (2 * (20 + 2) + e / 32 + 5 + k + 6 + 4) * U32
    slack = rel * (direct.abs() + p * g.abs().sum(1, keepdim=True)) + 2.0 ** -126
    check(dl, ref, slack + (BF16_HALF * (ref.abs() + slack) if dl.dtype == torch.bfloat16 else 0), "dlogits")
    return dl


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(5, 2, 2), (7, 7, 3), (20, 64, 8), (9, 130, 8), (33, 256, 4), (12, 512, 6),
                                   (9, 1001, 5), (9, 1024, 32)])
def test_over_all_with_choices_left_out(t, e, k, dtype):
    x, w, ids, dw = inputs(t, e, k, False, dtype)
    ref_ids, _, p = route(x, k, False)
    assert torch.equal(ids.long(), ref_ids)
    first = ids.clone()
    first[:, 0] = -1
    dl = check_bwd(x, w, first, dw, p, False)
    if k > 1:
        assert bool((dl.abs().sum(1) > 0).any())     # the total is not zero
    first[:, 0] = e                                  # above the range: the same
    assert torch.equal(fb.fp8_moe_route_bwd(dw, w, first, x, renorm=False), dl)
    some = ids.clone()
    some[torch.rand(t, k, generator=gen(9), device="cuda") < 0.5] = -1
    check_bwd(x, w, some, dw, p, False)
    none = check_bwd(x, w, torch.full_like(ids, -1), dw, p, False)
    assert bool((none == 0).all())


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k", [(7, 7, 3), (20, 64, 8), (9, 130, 8), (33, 256, 4), (9, 1024, 32)])
def test_choices_in_another_order(t, e, k, dtype, renorm):
    x, w, ids, dw = inputs(t, e, k, renorm, dtype)
    x, w, ids, dw = (v[:t - 1].contiguous() for v in (x, w, ids, dw))   # (without +inf)
    _, _, p = route(x, k, renorm)
    order = torch.randperm(k, generator=torch.Generator().manual_seed(t)).cuda()
    check_bwd(x, w[:, order].contiguous(), ids[:, order].contiguous(), dw[:, order].contiguous(), p, renorm)
    back = list(range(k - 1, -1, -1))
    check_bwd(x, w[:, back].contiguous(), ids[:, back].contiguous(), dw[:, back].contiguous(), p, renorm)


def test_dropping_a_renormalized_choice_by_its_gradient():
    # a choice that is to count no more keeps its id and gets dweights 0
    x, w, ids, dw = inputs(20, 64, 8, True, torch.float32)
    _, _, p = route(x, 8, True)
    dw[::2, 0] = 0
    dw[1::3, 5] = 0
    check_bwd(x, w, ids, dw, p, True)
