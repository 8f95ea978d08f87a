"""Router rows with fewer distinct logits than choices, among them rows whose experts fill
every register of the kernel's warp (E = 128, 256, 1024) and that have no -inf."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import U32, check, plan, route

pytestmark = pytest.mark.gpu


def rows_of_levels(e, k, dtype, seed):
    """Rows of 1 to 5 values, all finite.  The levels above the lowest hold k logits
    together, one fewer, one more, or any number; the lowest holds the rest."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for levels in (1, 2, 3, 4, 5):
        for upper in (k - 1, k, k + 1, int(torch.randint(1, e, (1,), generator=g))):
            x = torch.zeros(e)
            n = min(max(upper, 0), e) if levels > 1 else 0
            x[:n] = torch.arange(n).remainder(max(levels - 1, 1)).float() + 1.0
            rows.append(x[torch.randperm(e, generator=g)])
    x = torch.stack(rows)
    # the same rows with the lowest level as a mask: the type's lowest value
    masked = torch.where(x > 0, x, torch.tensor(torch.finfo(dtype).min))
    return torch.cat([x, masked, x - 2.0]).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 7, 8, 31, 32])
@pytest.mark.parametrize("e", [64, 100, 128, 256, 512, 1000, 1024])
def test_fewer_values_than_choices(e, k, dtype):
    x = rows_of_levels(e, k, dtype, 100 * e + k)
    ids, _, _ = route(x, k, True)
    for renorm in (True, False):
        w, got = fb.fp8_moe_route(x, k, renorm=renorm)
        ref_ids, ref_w, _ = route(x, k, renorm)
        assert torch.equal(got.long(), ref_ids)
        # exp(d), |d| <= 5 or d below the underflow: the product with log2(e) is off by
        # |d| 2^-23, the exponential by 2^-22, in the term and in the sum; the sum has at most
        # e / 32 + 5 roundings, the division one
        check(w, ref_w, (2 * (5 + 2) + e / 32 + 6) * U32 * ref_w + 2.0 ** -126, "weights")
    seg, row, src = fb.fp8_moe_plan(got, e)
    rs, rr, rc = plan(ids, e, fb.fp8_moe_plan_rows(len(x), e, k))
    assert seg.tolist() == rs and row.reshape(-1).tolist() == rr and src.tolist() == rc


@pytest.mark.parametrize("e,k,high", [(128, 3, 3), (128, 7, 7), (256, 5, 5), (1024, 3, 3)])
def test_k_equal_logits_over_equal_others(e, k, high):
    x = torch.zeros(1, e, device="cuda")
    at = torch.arange(high, device="cuda") * (e // high - 1)
    x[0, at] = 1.0
    w, ids = fb.fp8_moe_route(x, k)
    assert ids[0].tolist() == at.tolist()
    # exp(0) = 1 exactly: each weight is 1 / k, rounded once
    assert w[0].tolist() == [float(torch.tensor(1.0) / k)] * k
