"""Refusals of the few-token and mixture-of-experts calls: the C ABI reports bad arguments
before it touches a device, and the binding raises before it reaches the C ABI."""
import ctypes as C

import pytest
import torch

import blockwise_fp8_linear_b200 as fb
from blockwise_fp8_linear_b200 import build as fbuild

bf16, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fb.lib()


def z(*shape, dtype=u8):
    return torch.zeros(*shape, dtype=dtype)


P, ODD, NUL, S = C.c_void_p(0x10000), C.c_void_p(0x10008), C.c_void_p(0), C.c_void_p(0)


def test_linear_few_arguments(L):
    f = L.fp8_linear_few
    assert f(NUL, P, P, P, 1, 128, 128, P, S) == 1
    assert f(P, P, P, NUL, 1, 128, 128, P, S) == 1
    assert f(P, P, P, P, 64, 128, 128, NUL, S) == 1   # 64 tokens need a workspace
    for m, n, k in ((0, 128, 128), (65, 128, 128), (-1, 128, 128), (1, 100, 128), (1, 128, 0),
                    (1, (1 << 20) + 128, 128)):
        assert f(P, P, P, P, m, n, k, P, S) == 3
    assert f(ODD, P, P, P, 1, 128, 128, P, S) == 2
    assert f(P, P, P, P, 64, 128, 128, ODD, S) == 2
    w = L.fp8_linear_few_workspace
    assert w(0, 128) == 0 and w(65, 128) == 0 and w(64, 100) == 0
    assert w(1, 128) == 0 and w(64, 256) >= 64 * 256 + 2 * 64 * 4


def test_route_arguments(L):
    f = L.fp8_moe_route
    assert f(NUL, 0, 1, 8, 2, 1, P, P, S) == 1
    assert f(P, 0, 1, 8, 2, 1, P, NUL, S) == 1
    for t, e, k in ((0, 8, 2), (1, 0, 1), (1, 1025, 2), (1, 8, 0), (1, 8, 9), (1, 64, 33),
                    ((1 << 20) + 1, 8, 2)):
        assert f(P, 0, t, e, k, 1, P, P, S) == 3
        assert L.fp8_moe_route_bwd(P, P, P, P, 0, t, e, k, 1, P, S) == 3
    assert f(P, 1, 1, 8, 2, 1, ODD, P, S) == 2
    assert L.fp8_moe_route_bwd(P, P, NUL, P, 0, 1, 8, 2, 1, P, S) == 1
    assert L.fp8_moe_route_bwd(P, P, P, P, 0, 1, 8, 2, 1, ODD, S) == 2


def test_plan_arguments(L):
    f = L.fp8_moe_plan
    assert f(P, 4, 8, 2, P, P, P, NUL, S) == 1
    assert f(P, 0, 8, 2, P, P, P, P, S) == 3
    assert f(P, 4, 8, 2, P, P, ODD, P, S) == 2
    # 2^20 pairs leave no room for the padding
    assert f(P, 1 << 17, 8, 8, P, P, P, P, S) == 3
    assert L.fp8_moe_plan_rows(1 << 17, 8, 8) == 0 and L.fp8_moe_plan_workspace(1 << 17, 8, 8) == 0
    assert L.fp8_moe_plan_rows(0, 8, 2) == 0
    # rows: any split fits -- all pairs in one expert, or one pair in each
    for t, e, k in ((1, 1, 1), (3, 8, 2), (100, 8, 2), (1000, 5, 5), (64, 1024, 32)):
        pairs, rows = t * k, L.fp8_moe_plan_rows(t, e, k)
        hit = min(pairs, e)
        assert rows % 128 == 0 and rows >= (pairs + 127) // 128 * 128
        assert rows >= 128 * (hit - 1) + (pairs - hit + 1 + 127) // 128 * 128
        assert L.fp8_moe_plan_workspace(t, e, k) > 0


def test_grouped_arguments(L):
    f, g = L.fp8_gemm_grouped, L.fp8_gemm_grouped_wgrad_acc32
    assert f(3, P, P, P, P, P, 2, P, 128, 128, 128, S) == 1
    assert f(0, P, P, P, P, NUL, 2, P, 128, 128, 128, S) == 1
    assert f(0, P, P, P, P, P, 0, P, 128, 128, 128, S) == 3
    assert f(0, P, P, P, P, P, 1025, P, 128, 128, 128, S) == 3
    assert f(0, P, P, P, P, P, 2, P, 144, 128, 128, S) == 3   # the layout has whole blocks
    assert f(2, P, P, P, P, P, 2, P, 128, 128, 144, S) == 3
    assert f(0, P, P, P, P, P, 1024, P, 128, 1 << 20, 128, S) in (4, 6)   # 2^30 rows are the most
    assert f(0, P, P, P, P, ODD, 2, P, 128, 128, 128, S) == 2
    assert g(P, P, P, P, P, 2, NUL, 128, 128, 128, S) == 1
    assert g(P, P, P, P, P, 2, P, 128, 64, 128, S) == 3
    assert g(P, P, P, P, P, 2, ODD, 128, 128, 128, S) == 2


def test_moe_few_arguments(L):
    f = L.fp8_moe_few
    ok = [P] * 8 + [4, 8, 2, 128, 128, P, S]

    def at(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for i in (0, 1, 2, 3, 4, 5, 6, 7, 13):
        assert at(**{f"a{i}": NUL}) == 1
        assert at(**{f"a{i}": ODD}) == 2
    assert at(a8=0) == 3 and at(a8=65) == 3
    assert at(a9=0) == 3 and at(a9=1025) == 3
    assert at(a10=0) == 3 and at(a10=9) == 3
    assert at(a11=64) == 3 and at(a12=130) == 3
    assert L.fp8_moe_few_workspace(65, 2, 128, 128) == 0
    assert L.fp8_moe_few_workspace(1, 33, 128, 128) == 0
    # codes and scales of h, the pairs' products and the counters
    assert L.fp8_moe_few_workspace(4, 2, 256, 128) >= 8 * 128 + 8 * 4 + 8 * 256 * 4 + 4 * 2 * 4


X = z(5, 256, dtype=bf16)
LOGITS = z(6, 8, dtype=f32)
IDS, WT = z(6, 2, dtype=i32), z(6, 2, dtype=f32)
SEG = z(4, dtype=i32)


def grouped(mode, **kw):
    m, n, k = 256, 384, 512
    e, a, sa, b, sb, d = fb._grouped_shapes(mode, m, n, k, SEG)
    t = {"a": z(*a), "sa": z(*sa, dtype=f32), "b": z(*b), "sb": z(*sb, dtype=f32), "seg": SEG,
         "out": z(*d, dtype=bf16)}
    t.update(kw)
    return fb.fp8_gemm_grouped(mode, t["a"], t["sa"], t["b"], t["sb"], t["seg"], m, n, k, out=t["out"])


def layer(**kw):
    t = {"x": X, "w1": z(3, 512, 256), "s1": z(3, 4, 2, dtype=f32), "w2": z(3, 256, 256),
         "s2": z(3, 2, 2, dtype=f32), "ids": z(5, 2, dtype=i32), "weights": z(5, 2, dtype=f32)}
    t.update(kw)
    return fb.fp8_moe_few(**t)


@pytest.mark.parametrize("call", [
    lambda: fb.fp8_linear_few(z(0, 256, dtype=bf16), z(128, 256), z(1, 2, dtype=f32)),
    lambda: fb.fp8_linear_few(z(65, 256, dtype=bf16), z(128, 256), z(1, 2, dtype=f32)),
    lambda: fb.fp8_linear_few(z(256, dtype=bf16), z(128, 256), z(1, 2, dtype=f32)),
    lambda: fb.fp8_linear_few(X, z(100, 256), z(1, 2, dtype=f32)),
    lambda: fb.fp8_linear_few(X, z(128, 384), z(1, 3, dtype=f32)),
    lambda: fb.fp8_linear_few(X, z(128, 256), z(2, 1, dtype=f32)),
    lambda: fb.fp8_linear_few(X, z(128, 256), z(1, 2, dtype=f32), out=z(5, 256, dtype=bf16)),
    lambda: fb.fp8_moe_route(z(0, 8, dtype=f32), 2),
    lambda: fb.fp8_moe_route(z(6, 1025, dtype=f32), 2),
    lambda: fb.fp8_moe_route(LOGITS, 9),
    lambda: fb.fp8_moe_route(LOGITS, 0),
    lambda: fb.fp8_moe_route(z(6, 64, dtype=f32), 33),
    lambda: fb.fp8_moe_route(LOGITS, 2, ids=z(6, 3, dtype=i32)),
    lambda: fb.fp8_moe_route_bwd(z(6, 3, dtype=f32), WT, IDS, LOGITS),
    lambda: fb.fp8_moe_route_bwd(WT, WT, IDS, z(5, 8, dtype=f32)),
    lambda: fb.fp8_moe_route_bwd(WT, WT, IDS, LOGITS, dlogits=z(6, 9, dtype=f32)),
    lambda: fb.fp8_moe_plan(IDS, 1),
    lambda: fb.fp8_moe_plan(IDS, 8, seg=z(8, dtype=i32)),
    lambda: fb.fp8_moe_plan(IDS, 8, src=z(128, dtype=i32)),
    lambda: fb.fp8_moe_plan_rows(1 << 17, 8, 8),
    lambda: grouped(3),
    lambda: grouped(fb.FPROP, seg=z(1, dtype=i32)),
    lambda: grouped(fb.FPROP, seg=z(5, dtype=i32)),      # another number of experts than b has
    lambda: grouped(fb.FPROP, b=z(3, 512, 384)),
    lambda: grouped(fb.DGRAD, b=z(3, 384, 512)),
    lambda: grouped(fb.DGRAD, sb=z(3, 3, 4, dtype=f32)),
    lambda: grouped(fb.WGRAD, out=z(256, 384, dtype=bf16)),
    lambda: layer(x=z(65, 256, dtype=bf16)),
    lambda: layer(w1=z(3, 256, 256)),
    lambda: layer(w2=z(3, 256, 128)),
    lambda: layer(s2=z(3, 1, 2, dtype=f32)),
    lambda: layer(ids=z(4, 2, dtype=i32)),
    lambda: layer(weights=z(5, 3, dtype=f32)),
    lambda: fb.fp8_moe_few_workspace(65, 2, 128, 128),
    lambda: fb.fp8_linear_few_workspace(65, 128),
], ids=lambda c: "")
def test_sizes_are_refused(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: fb.fp8_linear_few(z(5, 256, dtype=f32), z(128, 256), z(1, 2, dtype=f32)),
    lambda: fb.fp8_linear_few(X, z(128, 256), z(1, 2, dtype=f32)),       # CPU tensors
    lambda: fb.fp8_moe_route(z(6, 8, dtype=torch.float16), 2),
    lambda: fb.fp8_moe_route(LOGITS, 2),
    lambda: fb.fp8_moe_route_bwd(WT, WT, IDS.long(), LOGITS),
    lambda: fb.fp8_moe_plan(IDS.long(), 8),
    lambda: grouped(fb.FPROP, seg=SEG.long()),
    lambda: grouped(fb.WGRAD),
    lambda: fb.fp8_gemm_grouped_wgrad_acc32(z(128, 128), z(1, 128, dtype=f32), z(128, 128),
                                            z(1, 128, dtype=f32), SEG, 128, 128, 128, None),
    lambda: layer(ids=z(5, 2, dtype=torch.int64)),
    lambda: layer(),
], ids=lambda c: "")
def test_kinds_are_refused(call):
    with pytest.raises(TypeError):
        call()


def test_layout_must_be_contiguous():
    with pytest.raises(ValueError):
        fb.fp8_moe_route(z(8, 6, dtype=f32).t(), 2)
