"""Few-token linear and few-token expert layer against 64-bit definitions."""
import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from _moe import acts, blocks64, check, check_bf16, dequant_rows, layer, weights

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check_linear(x, qw, sw):
    y = fb.fp8_linear_few(x, qw, sw)
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
    a, w = dequant_rows(x), blocks64(qw, sw)
    check_bf16(y, a @ w.t(), a.abs() @ w.abs().t(), x.shape[1], "few")
    return y


@pytest.mark.parametrize("m", [1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("n,k", [(128, 128), (256, 512), (384, 1408)])
def test_linear_tokens(m, n, k):
    g = gen(m)
    qw, sw = weights(g, 1, n, k)
    check_linear(acts(g, m, k), qw[0], sw[0])


@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (3, 128, 12288), (64, 128, 6144), (5, 4096, 256),
                                   (20, 12288, 128), (40, 6144, 2048), (1, 128, 128 * 129), (64, 20480, 384),
                                   (8, 8192, 4096), (9, 8192, 4096), (16, 8192, 4096), (13, 12288, 12288)])
def test_linear_shapes(m, n, k):
    g = gen(n + k)
    qw, sw = weights(g, 1, n, k)
    check_linear(acts(g, m, k), qw[0], sw[0])


@pytest.mark.parametrize("m", [9, 12, 16])
@pytest.mark.parametrize("n,k", [(4096, 4096), (4224, 4096), (12288, 2048), (2048, 12288)])
def test_linear_where_the_codes_change_hands(m, n, k):
    # weights about the size from which the quantizer's kernel makes the codes
    g = gen(m + n)
    qw, sw = weights(g, 1, n, k)
    x = acts(g, m, k)
    y = check_linear(x, qw[0], sw[0])
    # fewer tokens are quantized in the kernel at every size: the same codes, other sums
    a, w = dequant_rows(x[:8]), blocks64(qw[0], sw[0])
    check_bf16(fb.fp8_linear_few(x[:8].contiguous(), qw[0], sw[0]), a @ w.t(), a.abs() @ w.abs().t(), k, "8 tokens")
    assert y.shape == (m, n)


def test_linear_values():
    """Zero rows and groups, scales at both ends of the range, outliers."""
    g = gen(4)
    m, n, k = 24, 256, 512
    x = acts(g, m, k)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 2.0 ** 100
    x[3] *= 2.0 ** -100       # a scale below 2^-90: plain division
    x[4] = 2.0 ** -80
    x[5, 3] = 3.0e38
    qw, sw = weights(g, 1, n, k)
    # 2^100 * 0.02 * K stays finite, 3e38 * 0.1 as well
    y = check_linear(x, qw[0], sw[0])
    assert (y[0] == 0).all()
    zero = torch.zeros_like(qw[0])
    assert (fb.fp8_linear_few(x, zero, torch.zeros_like(sw[0])) == 0).all()


def test_linear_codes_are_those_of_the_quantizer():
    # with an identity weight the result is the quantized activation itself
    g = gen(6)
    m, k = 48, 384
    x = acts(g, m, k)
    eye = torch.eye(k, device="cuda").bfloat16()
    qw, sw, _ = fb.fp8_quant_weight(eye)
    q, s = fb.fp8_quant_act(x)
    want = fb.fp8_gemm_blockwise(fb.FPROP, q, s, qw, sw, m, k, k)
    assert torch.equal(fb.fp8_linear_few(x, qw, sw), want)


def test_linear_rows_do_not_mix():
    # a row's result does not depend on the others, NaN and infinities among them
    g = gen(7)
    x = acts(g, 33, 1024)
    qw, sw = weights(g, 1, 512, 1024)
    y = check_linear(x, qw[0], sw[0])
    bad = x.clone()
    bad[5], bad[6, 100], bad[32] = float("nan"), float("inf"), -float("inf")
    z = fb.fp8_linear_few(bad, qw[0], sw[0])
    keep = [r for r in range(33) if r not in (5, 6, 32)]
    assert torch.equal(z[keep], y[keep])


def make_layer(g, t, e, k, h, i, seed=0):
    x = acts(g, t, h)
    w1, s1 = weights(g, e, 2 * i, h)
    w2, s2 = weights(g, e, h, i)
    wt, ids = fb.fp8_moe_route(torch.randn(t, e, generator=g, device="cuda"), k)
    return [x, w1, s1, w2, s2, ids, wt]


def check_layer(args):
    y = fb.fp8_moe_few(*args)
    torch.cuda.synchronize()
    assert fb.fp8bw_last_device_error() == 0
    ref, slack = layer(*args)
    check(y, ref, slack, "layer")
    # the bound is far below the values, so that it can fail
    if float(ref.norm()) > 0:
        assert float((y.double() - ref).norm()) <= 0.02 * float(ref.norm())
    return y


@pytest.mark.parametrize("t,e,k,h,i", [
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (2, 4, 4, 128, 256), (3, 16, 8, 512, 384), (16, 8, 2, 256, 256),
    (17, 8, 3, 384, 128), (32, 64, 8, 256, 256), (33, 5, 2, 128, 640), (64, 4, 2, 512, 256), (64, 64, 32, 128, 128),
    (63, 130, 8, 256, 128), (5, 1024, 8, 128, 128), (1, 128, 8, 2048, 768), (64, 1, 1, 1024, 512)])
def test_layer(t, e, k, h, i):
    check_layer(make_layer(gen(t + e + k), t, e, k, h, i))


def test_layer_choices_left_out():
    g = gen(9)
    t, e, k = 20, 6, 3
    a = make_layer(g, t, e, k, 256, 256)
    ids, wt = a[5], a[6]
    ids[0] = -1                                   # a padding row
    ids[1, 1:] = -1
    ids[2] = torch.tensor([e, 2 ** 31 - 1, -2 ** 31])   # outside the range: left out too
    ids[3] = torch.tensor([4, 4, 4])              # one expert three times
    ids[4] = torch.tensor([1, 5, 1])
    wt[5] = 0.0
    wt[6] *= -3.0
    wt[0] = float("nan")                          # weights of choices that are left out
    wt[1, 1:] = float("inf")
    wt[2] = float("nan")
    y = fb.fp8_moe_few(*a)
    torch.cuda.synchronize()
    ref, slack = layer(*a)
    check(y, ref, slack, "layer")
    assert (y[0] == 0).all() and (y[2] == 0).all() and (y[5] == 0).all()


def test_layer_nothing_chosen():
    a = make_layer(gen(10), 9, 4, 2, 256, 128)
    a[5].fill_(-1)
    y = torch.full((9, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    assert fb.fp8_moe_few(*a, out=y) is y and (y == 0).all()


def test_layer_one_expert_takes_all():
    a = make_layer(gen(11), 64, 12, 1, 256, 384)
    a[5].fill_(7)
    check_layer(a)


def test_layer_small_and_large_values():
    g = gen(12)
    a = make_layer(g, 12, 4, 2, 256, 256)
    a[0][0] = 0
    a[0][1] *= 2.0 ** -60
    a[0][2] *= 30.0        # saturates the sigmoid on both sides
    a[0][3, ::2] = 0
    check_layer(a)


def test_layer_is_deterministic():
    a = make_layer(gen(13), 48, 32, 8, 512, 256)
    y = fb.fp8_moe_few(*a)
    for _ in range(5):
        assert torch.equal(y, fb.fp8_moe_few(*a))


def test_layer_workspace():
    a = make_layer(gen(14), 7, 8, 2, 256, 128)
    need = fb.fp8_moe_few_workspace(7, 2, 256, 128)
    want = fb.fp8_moe_few(*a)
    ws = torch.full((need + 512,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes
    for _ in range(2):
        assert torch.equal(want, fb.fp8_moe_few(*a, workspace=ws[:need]))
        assert (ws[need:] == 0x7F).all()
    with pytest.raises(ValueError):
        fb.fp8_moe_few(*a, workspace=ws[:need - 16])
    with pytest.raises(TypeError):
        fb.fp8_moe_few(*a, workspace=ws.view(torch.int32))


def test_misaligned_and_strided_arguments():
    g = gen(15)
    qw, sw = weights(g, 1, 256, 256)
    buf = acts(g, 9, 256).view(-1)
    with pytest.raises(fb.Fp8bwError) as e:
        fb.fp8_linear_few(buf[4:4 + 8 * 256].view(8, 256), qw[0], sw[0])   # 8 bytes off
    assert e.value.status == 2
    wide = acts(g, 8, 512)
    with pytest.raises(ValueError):
        fb.fp8_linear_few(wide[:, :256], qw[0], sw[0])                     # rows with a gap
    assert torch.equal(fb.fp8_linear_few(wide[:, :256].contiguous(), qw[0], sw[0]),
                       fb.fp8_linear_few(wide[:, :256].contiguous(), qw[0], sw[0],
                                         stream=torch.cuda.current_stream()))
    # a Parameter is a tensor like any other
    x = torch.nn.Parameter(wide[:, :256].contiguous())
    assert torch.equal(fb.fp8_linear_few(x, qw[0], sw[0]),
                       fb.fp8_linear_few(x.detach(), qw[0], sw[0]))


def test_compiled_calls_and_python_agree():
    """The compiled form of each call and the Python one (taken for an explicit stream)."""
    a = make_layer(gen(16), 21, 6, 3, 256, 256)
    st = torch.cuda.current_stream()
    qw, sw = a[1][0], a[2][0]
    assert torch.equal(fb.fp8_linear_few(a[0], qw, sw), fb.fp8_linear_few(a[0], qw, sw, stream=st))
    assert torch.equal(fb.fp8_moe_few(*a), fb.fp8_moe_few(*a, stream=st))
    lg = torch.randn(21, 6, generator=gen(1), device="cuda")
    one, two = fb.fp8_moe_route(lg, 2, False), fb.fp8_moe_route(lg, 2, False, stream=st)
    assert all(torch.equal(u, v) for u, v in zip(one, two))
    dw = torch.randn(21, 2, generator=gen(2), device="cuda")
    assert torch.equal(fb.fp8_moe_route_bwd(dw, *one, lg, False), fb.fp8_moe_route_bwd(dw, *one, lg, False, stream=st))
    p1, p2 = fb.fp8_moe_plan(one[1], 6), fb.fp8_moe_plan(one[1], 6, stream=st)
    assert all(torch.equal(u, v) for u, v in zip(p1, p2))
    rows = p1[2].numel()
    q, s = fb.fp8_quant_act(acts(gen(3), rows, 256))
    g1 = fb.fp8_gemm_grouped(fb.FPROP, q, s, a[1], a[2], p1[0], rows, 512, 256, out=torch.zeros(rows, 512, dtype=torch.bfloat16, device="cuda"))
    g2 = fb.fp8_gemm_grouped(fb.FPROP, q, s, a[1], a[2], p1[0], rows, 512, 256, stream=st, out=torch.zeros_like(g1))
    assert torch.equal(g1, g2)
    # numpy integers and the like are taken by the Python form
    import numpy as np
    assert torch.equal(fb.fp8_moe_route(lg, np.int64(2), False)[1], one[1])
