"""Grouped GEMMs (one weight per expert) against 64-bit products of the same codes."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import acts, blocks64, check, check_bf16, rows64, sum_bound, weights

pytestmark = pytest.mark.gpu
MARK = 1.5  # what an output buffer holds before the call


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def seg_of(counts, first=0):
    s = [first]
    for c in counts:
        s.append(s[-1] + c)
    return s


def run_rows(mode, seg, blocks, n, k, seed=1):
    """FPROP / DGRAD over `blocks` blocks of 128 rows laid out by seg."""
    g = gen(seed)
    e, m = len(seg) - 1, 128 * blocks
    a, sa = fb.fp8_quant_act(acts(g, m, k))
    b, sb = weights(g, e, n, k) if mode == fb.FPROP else weights(g, e, k, n)
    out = torch.full((m, n), MARK, dtype=torch.bfloat16, device="cuda")
    st = torch.tensor(seg, dtype=torch.int32, device="cuda")
    d = fb.fp8_gemm_grouped(mode, a, sa, b, sb, st, m, n, k, out=out)
    assert d is out
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
    a64 = rows64(a, sa)
    owner = torch.full((blocks,), -1)
    for x in range(e):
        owner[seg[x]:seg[x + 1]] = x
    for blk in range(blocks):
        cut, x = slice(128 * blk, 128 * blk + 128), int(owner[blk])
        if x < 0:
            assert (d[cut] == MARK).all(), f"block {blk} belongs to no expert"
            continue
        w = blocks64(b[x], sb[x])
        w = w.t() if mode == fb.FPROP else w
        check_bf16(d[cut], a64[cut] @ w, a64[cut].abs() @ w.abs(), k, f"block {blk} of expert {x}")
    return d


ROWS = [  # blocks per expert, blocks in all, n, k
    ([1], 1, 128, 128),
    ([1, 1], 2, 128, 256),
    ([2, 0, 1], 3, 256, 128),
    ([0, 0, 3, 0], 4, 384, 384),
    ([3, 1, 2, 5], 13, 256, 512),
    ([0, 0], 2, 256, 256),
    ([1] * 9, 9, 512, 640),
    ([7, 2, 0, 4, 1], 14, 1280, 256),
    ([17, 3], 20, 2048, 384),
    ([1, 4, 1, 9, 0, 2, 6, 3], 30, 1024, 1024),
]


@pytest.mark.parametrize("mode", [fb.FPROP, fb.DGRAD])
@pytest.mark.parametrize("counts,blocks,n,k", ROWS)
def test_rows(mode, counts, blocks, n, k):
    run_rows(mode, seg_of(counts), blocks, n, k)


@pytest.mark.parametrize("mode", [fb.FPROP, fb.DGRAD])
def test_rows_before_the_first_expert(mode):
    run_rows(mode, seg_of([2, 1], first=1), 6, 256, 256)


def test_many_experts():
    # the most there may be, one block each in a hundred of them
    counts = [0] * 1024
    for i in range(100):
        counts[(i * 37) % 1024] = 1
    run_rows(fb.FPROP, seg_of(counts), 101, 128, 128)
    run_rows(fb.DGRAD, seg_of(counts), 100, 256, 128)


@pytest.mark.parametrize("mode", [fb.FPROP, fb.DGRAD])
@pytest.mark.parametrize("m,n,k", [(256, 256, 256), (1280, 2048, 512), (384, 384, 128)])
def test_one_expert_is_the_plain_gemm(mode, m, n, k):
    g = gen(m + n)
    a, sa = fb.fp8_quant_act(acts(g, m, k))
    b, sb = weights(g, 1, n, k) if mode == fb.FPROP else weights(g, 1, k, n)
    st = torch.tensor([0, m // 128], dtype=torch.int32, device="cuda")
    d = fb.fp8_gemm_grouped(mode, a, sa, b, sb, st, m, n, k)
    assert torch.equal(d, fb.fp8_gemm_blockwise(mode, a, sa, b[0], sb[0], m, n, k))


def run_wgrad(seg, blocks, m, n, acc32, seed=2):
    g = gen(seed)
    e, k = len(seg) - 1, 128 * blocks
    a, sa = fb.fp8_quant_act_t(acts(g, k, m, 1e-3))
    b, sb = fb.fp8_quant_act_t(acts(g, k, n))
    st = torch.tensor(seg, dtype=torch.int32, device="cuda")
    if acc32:
        d0 = torch.randn(e, m, n, generator=g, device="cuda")
        d = d0.clone()
        assert fb.fp8_gemm_grouped_wgrad_acc32(a, sa, b, sb, st, m, n, k, d) is d
    else:
        d = torch.full((e, m, n), MARK, dtype=torch.bfloat16, device="cuda")
        fb.fp8_gemm_grouped(fb.WGRAD, a, sa, b, sb, st, m, n, k, out=d)
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
    a64, b64 = rows64(a, sa), rows64(b, sb)
    for x in range(e):
        cut = slice(128 * seg[x], 128 * seg[x + 1])
        kx = 128 * (seg[x + 1] - seg[x])
        ref, mag = a64[:, cut] @ b64[:, cut].t(), a64[:, cut].abs() @ b64[:, cut].abs().t()
        if not acc32:
            check_bf16(d[x], ref, mag, kx, f"expert {x}")
        elif kx == 0:
            assert torch.equal(d[x], d0[x]), f"expert {x} has no tokens"
        else:
            want = d0[x].double() + ref
            check(d[x], want, sum_bound(kx) * mag + 2.0 ** -24 * (want.abs() + sum_bound(kx) * mag),
                  f"expert {x}")


@pytest.mark.parametrize("acc32", [False, True])
@pytest.mark.parametrize("counts,blocks,m,n", [
    ([1], 1, 128, 128), ([0], 1, 128, 128), ([2, 0, 1], 3, 128, 256), ([0, 3, 0, 2], 7, 256, 128),
    ([5, 1, 2], 8, 384, 384), ([0, 0, 0], 2, 256, 256), ([3, 9, 0, 4, 1], 17, 512, 768),
    ([1, 0, 2, 7, 1, 0, 0, 3], 14, 1024, 512)])
def test_wgrad(counts, blocks, m, n, acc32):
    run_wgrad(seg_of(counts), blocks, m, n, acc32)


@pytest.mark.parametrize("acc32", [False, True])
def test_wgrad_blocks_of_nobody(acc32):
    run_wgrad(seg_of([2, 1], first=2), 7, 256, 512, acc32)


def test_table_is_clamped():
    """Entries outside [0, blocks], or below their predecessor, count as the nearest value
    that is not: nothing outside the operands is touched."""
    g = gen(3)
    blocks, n, k = 5, 256, 128
    m = 128 * blocks
    a, sa = fb.fp8_quant_act(acts(g, m, k))
    b, sb = weights(g, 4, n, k)

    def out(seg):
        d = torch.full((m, n), MARK, dtype=torch.bfloat16, device="cuda")
        st = torch.tensor(seg, dtype=torch.int32, device="cuda")
        return fb.fp8_gemm_grouped(fb.FPROP, a, sa, b, sb, st, m, n, k, out=d)

    assert torch.equal(out([-7, 2, 1, 4, 99]), out([0, 2, 2, 4, 5]))
    assert torch.equal(out([3, 2, 1, 0, -1]), out([3, 3, 3, 3, 3]))
    assert torch.equal(out([-2 ** 31, 2 ** 31 - 1, 0, 0, 0]), out([0, 5, 5, 5, 5]))


def test_rows_on_a_side_stream_and_repeated():
    seg = seg_of([3, 0, 5, 2])
    first = run_rows(fb.FPROP, seg, 11, 512, 512, seed=5).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run_rows(fb.FPROP, seg, 11, 512, 512, seed=5)
    assert torch.equal(first, again)
