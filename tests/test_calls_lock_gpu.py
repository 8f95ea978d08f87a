"""The compiled calls release the interpreter lock around allocation and launch, as the calls
through ctypes do: entry points of a stand-in library see whether the lock is held, and a
host function in the stream that needs the lock finishes while calls queue up behind it."""
import ctypes as C
import importlib.util
import os
import shutil
import subprocess
import threading
import time

import pytest
import torch

import blockwise_fp8_linear_b200 as fb

pytestmark = pytest.mark.gpu
bf16, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32

STAND_IN = """
#include <stdint.h>
int PyGILState_Check(void);
int seen[16], status;
int64_t size(void) { return 256; }
int call(void) { seen[0] += 1; seen[1] += PyGILState_Check(); return status; }
"""


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    """(a second instance of the compiled calls, bound to the stand-in; the stand-in)"""
    d = tmp_path_factory.mktemp("calls")
    (d / "stand_in.c").write_text(STAND_IN)
    subprocess.run(["gcc", "-shared", "-fPIC", str(d / "stand_in.c"), "-o", str(d / "stand_in.so")], check=True)
    lib = C.PyDLL(str(d / "stand_in.so"))
    shutil.copy(os.path.join(os.path.dirname(fb.library_path), "_calls.so"), d / "_calls.so")
    spec = importlib.util.spec_from_file_location("_calls", str(d / "_calls.so"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    size, call = (C.cast(f, C.c_void_p).value for f in (lib.size, lib.call))
    m.open(fb.Fp8bwError, size, call, call, call, size, size, call, call, call, size, call)
    return m, lib


def z(*shape, dtype=u8):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def arguments():
    x, q, s = z(16, 256, dtype=bf16), z(256, 256), z(2, 2, dtype=f32)
    w1, s1, w2, s2 = z(3, 512, 256), z(3, 4, 2, dtype=f32), z(3, 256, 256), z(3, 2, 2, dtype=f32)
    lg, wt, ids, seg = z(16, 3, dtype=f32), z(16, 2, dtype=f32), z(16, 2, dtype=i32), z(4, dtype=i32)
    a, sa = z(256, 256), z(2, 256, dtype=f32)
    return {"linear_few": (x, q, s, None, None, None),
            "moe_route": (lg, 2, True, None, None, None),
            "moe_route_bwd": (wt, wt, ids, lg, True, None, None),
            "moe_plan": (ids, 3, None, None, None, None, None),
            "gemm_grouped": (fb.FPROP, a, sa, w2, s2, seg, 256, 256, 256, None, None),
            "gemm_grouped_wgrad_acc32": (a, sa, a, sa, seg, 256, 256, 256, z(3, 256, 256, dtype=f32), None),
            "moe_few": (x, w1, s1, w2, s2, ids, wt, None, None, None)}


def test_lock_is_released_around_each_call(stand_in):
    m, lib = stand_in
    seen, status = (C.c_int * 16).in_dll(lib, "seen"), C.c_int.in_dll(lib, "status")
    for name, args in arguments().items():
        seen[0] = seen[1] = status.value = 0
        assert getattr(m, name)(*args) is not NotImplemented, name
        assert (seen[0], seen[1]) == (1, 0), f"{name}: lock held in {seen[1]} of {seen[0]} calls"
        status.value = 3            # an error is still raised, with the lock
        with pytest.raises(fb.Fp8bwError) as e:
            getattr(m, name)(*args)
        assert e.value.status == 3


def test_arguments_and_results_are_released(stand_in):
    import sys
    m, lib = stand_in
    C.c_int.in_dll(lib, "status").value = 0
    for name, args in arguments().items():
        for _ in range(3):
            getattr(m, name)(*args)
        before = [sys.getrefcount(a) for a in args]
        r = getattr(m, name)(*args)
        del r
        assert [sys.getrefcount(a) for a in args] == before, name


def test_calls_from_several_threads():
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = [torch.randn(32, 64, generator=g, device="cuda") for _ in range(4)]
    want = [fb.fp8_moe_route(x, 8) for x in logits]
    torch.cuda.synchronize()
    got = [[] for _ in logits]

    def work(n):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(200):
                got[n].append(fb.fp8_moe_route(logits[n], 8))
        st.synchronize()

    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(logits))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, rs in zip(want, got):
        assert len(rs) == 200 and all(torch.equal(w[0], r[0]) and torch.equal(w[1], r[1]) for r in rs)


def test_host_function_that_needs_the_lock():
    # more calls than a launch queue holds, behind a host function that runs Python code
    rt = C.CDLL("libcudart.so.12")
    ran = []

    @C.CFUNCTYPE(None, C.c_void_p)
    def host(_):
        time.sleep(0.05)
        ran.append(1)

    x = torch.randn(4, 16, device="cuda")
    w, ids = fb.fp8_moe_route(x, 2)
    out = [torch.empty_like(w), torch.empty_like(ids)]
    torch.cuda.synchronize()
    st = torch.cuda.current_stream()
    assert rt.cudaLaunchHostFunc(C.c_void_p(st.cuda_stream), host, None) == 0
    for _ in range(4000):
        fb.fp8_moe_route(x, 2, weights=out[0], ids=out[1])
    torch.cuda.synchronize()
    assert ran == [1] and torch.equal(out[0], w) and torch.equal(out[1], ids)
