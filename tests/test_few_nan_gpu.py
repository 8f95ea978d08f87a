"""Few-token expert layer: a NaN that arises in an expert's hidden values reaches the token's
output, whatever stands beside it."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import check, layer
from test_few_gpu import gen, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cause", ["code", "overflow"])
@pytest.mark.parametrize("t,e,k,h,i", [(1, 4, 2, 256, 256), (6, 8, 2, 256, 384), (16, 4, 3, 512, 128),
                                       (40, 8, 2, 256, 256), (64, 16, 4, 384, 256)])
def test_nan_among_zeros(t, e, k, h, i, cause):
    # one expert's hidden values are all zero but for one column, which is NaN
    a = make_layer(gen(t + h), t, e, k, h, i)
    x, w1, s1, w2, s2, ids, wt = a
    x.copy_(x.abs() + 1)
    bad = int(ids[0, 0])
    clean = fb.fp8_moe_few(*a)
    col = i - 3
    w1[bad] = 0
    if cause == "code":
        w1[bad, i + col, 5] = 0x7F              # E4M3's NaN among the up rows
    else:
        # the gate row gives 0, the up row infinity (its block's scale is near the largest float)
        w1[bad, i + col] = 0x7E
        s1[bad, (i + col) // 128] = 3e38
    assert bool((w1[bad, :i] == 0).all())
    y = fb.fp8_moe_few(*a)
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
    hit = (ids == bad).any(1)
    assert bool(hit[0]) and bool(y[hit].isnan().all())
    assert torch.equal(y[~hit], clean[~hit])


def test_groups_without_nan_keep_their_codes():
    # zero groups, subnormal and large hidden values beside each other
    a = make_layer(gen(3), 9, 4, 2, 256, 512)
    x, w1, s1 = a[:3]
    w1[:, :128] = 0                             # the first group of every expert's h is zero
    s1[:, 1] *= 2.0 ** -60
    s1[:, 2] *= 2.0 ** 20
    y = fb.fp8_moe_few(*a)
    ref, slack = layer(*a)
    check(y, ref, slack, "layer")
