"""Blockwise-FP8 Transformer linear layer for NVIDIA B200 (sm_100a).

A thin ctypes binding over the C ABI of ``libfp8bw.so`` (declared in
``include/fp8bw.h``).  Every function here only marshals arguments: it allocates
outputs with torch, checks dtypes and devices, and calls the C entry point of the
same name on the current CUDA stream.  All arithmetic runs in the CUDA kernels.
There is no CPU fallback: if the library is missing or the device is not sm_100,
the calls raise.

Method (Puro-2B, part 3/7, section 3.2 "FP8 Mixed-Precision Training"): E4M3
operands; activations and their gradients scaled per 128 neighbouring elements in
the summed (K) direction, weights per 128x128 tile; FP32
scales amax/448, and fprop / dgrad / wgrad GEMMs in FP8 with a BF16 result.
"""
from __future__ import annotations

import ctypes as C
import os

__all__ = [
    "FPROP", "DGRAD", "WGRAD", "Fp8bwError", "lib", "library_path",
    "fp8_quant_act", "fp8_quant_act_t", "fp8_quant_act_dual", "fp8_quant_weight",
    "fp8_gemm_blockwise", "fp8_gemm_wgrad_acc32",
    "fp8_quant_act_e8m0", "fp8_quant_act_t_e8m0", "fp8_quant_act_dual_e8m0",
    "fp8_quant_weight_e8m0", "fp8_gemm_blockwise_e8m0",
    "fp8bw_status_string", "fp8bw_last_device_error", "fp8bw_version",
    "fp8bw_selftest_wait_timeout",
    "linear_fprop", "linear_dgrad", "linear_wgrad",
    "MAX_DIM", "FEW_TOKENS", "MAX_EXPERTS", "MAX_CHOICES",
    "fp8_linear_few", "fp8_linear_few_workspace", "fp8_moe_route", "fp8_moe_route_bwd", "fp8_moe_plan_rows", "fp8_moe_plan",
    "fp8_gemm_grouped", "fp8_gemm_grouped_wgrad_acc32", "fp8_moe_few", "fp8_moe_few_workspace",
]

FPROP, DGRAD, WGRAD = 0, 1, 2
# the limits of include/fp8bw.h
MAX_DIM, FEW_TOKENS, MAX_EXPERTS, MAX_CHOICES = 1 << 20, 64, 1024, 32

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libfp8bw.so")
_lib = None


class Fp8bwError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {fp8bw_status_string(status)} (status {status})")


def lib():
    """Load libfp8bw.so (built in-tree by ``python -m blockwise_fp8_linear_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"{library_path} is missing: build it with "
                "`python -m blockwise_fp8_linear_b200.build` (no CPU fallback exists)")
        L = C.CDLL(library_path)
        vp, i64, i32 = C.c_void_p, C.c_int64, C.c_int
        L.fp8_quant_act.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8_quant_act_t.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8_quant_act_dual.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.fp8_quant_weight.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.fp8_gemm_blockwise.argtypes = [i32, vp, vp, vp, vp, vp, i64, i64, i64, vp]
        L.fp8_gemm_wgrad_acc32.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        L.fp8_quant_act_e8m0.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8_quant_act_t_e8m0.argtypes = [vp, i64, i64, vp, vp, vp]
        L.fp8_quant_act_dual_e8m0.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
        L.fp8_quant_weight_e8m0.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.fp8_gemm_blockwise_e8m0.argtypes = [i32, vp, vp, vp, vp, vp, i64, i64, i64, vp]
        L.fp8_linear_few.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
        L.fp8_linear_few_workspace.argtypes = [i64, i64]
        L.fp8_linear_few_workspace.restype = i64
        L.fp8_moe_route.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, vp]
        L.fp8_moe_route_bwd.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i32, vp, vp]
        L.fp8_moe_plan.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
        L.fp8_gemm_grouped.argtypes = [i32, vp, vp, vp, vp, vp, i64, vp, i64, i64, i64, vp]
        L.fp8_gemm_grouped_wgrad_acc32.argtypes = [vp, vp, vp, vp, vp, i64, vp, i64, i64, i64, vp]
        L.fp8_moe_few.argtypes = [vp] * 8 + [i64] * 5 + [vp, vp]
        for f in (L.fp8_moe_plan_rows, L.fp8_moe_plan_workspace):
            f.argtypes = [i64, i64, i64]
            f.restype = i64
        L.fp8_moe_few_workspace.argtypes = [i64, i64, i64, i64]
        L.fp8_moe_few_workspace.restype = i64
        for f in (L.fp8_linear_few, L.fp8_moe_route, L.fp8_moe_route_bwd, L.fp8_moe_plan,
                  L.fp8_gemm_grouped, L.fp8_gemm_grouped_wgrad_acc32, L.fp8_moe_few):
            f.restype = i32
        for f in (L.fp8_quant_act, L.fp8_quant_act_t, L.fp8_quant_act_dual, L.fp8_quant_weight,
                  L.fp8_gemm_blockwise, L.fp8_gemm_wgrad_acc32, L.fp8_quant_act_e8m0,
                  L.fp8_quant_act_t_e8m0, L.fp8_quant_act_dual_e8m0, L.fp8_quant_weight_e8m0,
                  L.fp8_gemm_blockwise_e8m0):
            f.restype = i32
        L.fp8bw_status_string.argtypes = [i32]
        L.fp8bw_status_string.restype = C.c_char_p
        L.fp8bw_last_device_error.argtypes = [vp]
        L.fp8bw_last_device_error.restype = i32
        L.fp8bw_selftest_wait_timeout.argtypes = [i64, vp]
        L.fp8bw_selftest_wait_timeout.restype = i32
        L.fp8bw_version.argtypes = []
        L.fp8bw_version.restype = C.c_char_p
        _lib = L
    return _lib


# The compiled calls (csrc/calls.cpp): each takes the arguments of the function that it
# stands in for and makes the plain call, or returns NotImplemented.
_calls = None


def _open_calls():
    """Load _calls.so and hand it the library's entry points."""
    global _calls
    import torch  # noqa: F401  (its libraries have to be there)
    L = lib()
    path = os.path.join(_HERE, "_calls.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m blockwise_fp8_linear_b200.build`")
    import importlib.util
    spec = importlib.util.spec_from_file_location("_calls", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.open(Fp8bwError, *[C.cast(getattr(L, n), C.c_void_p).value for n in (
        "fp8_linear_few_workspace", "fp8_linear_few", "fp8_moe_route", "fp8_moe_route_bwd",
        "fp8_moe_plan_rows", "fp8_moe_plan_workspace", "fp8_moe_plan", "fp8_gemm_grouped",
        "fp8_gemm_grouped_wgrad_acc32", "fp8_moe_few_workspace", "fp8_moe_few")])
    _calls = m
    return m


def fp8bw_status_string(status: int) -> str:
    return lib().fp8bw_status_string(int(status)).decode()


def fp8bw_version() -> str:
    return lib().fp8bw_version().decode()


def _stream(stream):
    """The cudaStream_t of a call: of the given stream, or of the current device's current
    one (asked for as a plain number: making a Stream object costs more than a launch)."""
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != 0:
        raise Fp8bwError(status, what)


def _validate(items):
    """Check the tensor arguments of one call before anything reaches the C ABI.
    items: (tensor or None, dtype, shape, name); None marks an output to allocate.
    A size that disagreed with the M, N, K handed to the C call would let a kernel read or
    write past an allocation, so every mismatch raises here (ValueError for shapes and
    devices, TypeError for kinds).  Returns the index of their device."""
    dev = None
    try:
        for t, dt, shp, _ in items:
            if t is None:
                continue
            if t.shape != shp or t.dtype is not dt or not t.is_contiguous():
                break
            d = t.get_device()
            if d != dev:
                if d < 0 or dev is not None:
                    break
                dev = d
        else:
            return dev
    except AttributeError:  # not a tensor
        pass
    return _refuse(items)


def _refuse(items):
    """Raise for the first fault of _validate's items: shapes come first, for every tensor,
    then dtype, contiguity and that all are CUDA tensors of one device."""
    import torch
    given = [i for i in items if i[0] is not None]
    for t, _, shp, name in given:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if tuple(t.shape) != tuple(int(d) for d in shp):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shp)}")
    for t, dt, _, name in given:
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
    dev = given[0][0].device
    for t, _, _, name in given:
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev} (one device per call)")
    return dev.index


def _alloc(t, shape, dtype, device, stream=None):
    """t, or a new tensor.  With a stream it comes from the allocator's pool of that stream:
    a block of the current stream's may still be read there by work queued before."""
    import torch
    if t is not None:
        return t
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _dims(M, N=None, K=None):
    """Sizes must be positive multiples of 128 (the ABI rejects others; checked here
    so that buffer shapes derived from them are whole)."""
    for d in (M, N, K):
        if d is not None and (d <= 0 or d % 128):
            raise ValueError(f"size {d} is not a positive multiple of 128")


class _Current:
    """The context of a call whose device is current already."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_current = _Current()


def _on(device):
    """Context that makes the device of this index current, so the call's stream and the
    current device match its buffers (the ABI rejects buffers of another device)."""
    import torch
    if torch._C._cuda_getDevice() == device:
        return _current
    return torch.cuda.device(device)


def _tokens(M):
    """A token count (the M of the activation quantizers and of FPROP/DGRAD, the
    reduction K of WGRAD) may end in a partial group of 128: a positive multiple of
    16 (the 16-byte row stride of the token-major codes)."""
    if int(M) <= 0 or int(M) % 16:
        raise ValueError(f"token count {M} is not a positive multiple of 16")


def _x2(x, name, tokens=False):
    """Rows and columns of a 2-D input; with tokens=True the rows are a token count
    (a multiple of 16), else both are multiples of 128."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    M, K = x.shape
    if tokens:
        _tokens(M)
        _dims(K)
    else:
        _dims(M, K)
    return int(M), int(K)


def _groups(M):
    return (int(M) + 127) // 128


def fp8bw_last_device_error(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device error word status."""
    return int(lib().fp8bw_last_device_error(_stream(stream)))


def fp8bw_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Run the bounded-wait self-test kernel (a wait that nothing satisfies)."""
    _check(lib().fp8bw_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "fp8bw_selftest_wait_timeout")


def fp8_quant_act(x, q=None, s=None, stream=None):
    """X[M][K] bf16 -> (Q[M][K] uint8 E4M3 codes, S[K/128][M] float32); M any
    multiple of 16 tokens."""
    import torch
    M, K = _x2(x, "x", tokens=True)
    dev = _validate([(x, torch.bfloat16, (M, K), "x"), (q, torch.uint8, (M, K), "q"),
                     (s, torch.float32, (K // 128, M), "s")])
    q = _alloc(q, (M, K), torch.uint8, dev)
    s = _alloc(s, (K // 128, M), torch.float32, dev)
    with _on(dev):
        _check(lib().fp8_quant_act(x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
                                   _stream(stream)), "fp8_quant_act")
    return q, s


def fp8_quant_act_t(x, qt=None, st=None, stream=None):
    """X[M][K] bf16 -> (Q^T[K][M] uint8, S^T[ceil(M/128)][K] float32), groups along M
    (the last group holds the M mod 128 tokens present)."""
    import torch
    M, K = _x2(x, "x", tokens=True)
    dev = _validate([(x, torch.bfloat16, (M, K), "x"), (qt, torch.uint8, (K, M), "qt"),
                     (st, torch.float32, (_groups(M), K), "st")])
    qt = _alloc(qt, (K, M), torch.uint8, dev)
    st = _alloc(st, (_groups(M), K), torch.float32, dev)
    with _on(dev):
        _check(lib().fp8_quant_act_t(x.data_ptr(), M, K, qt.data_ptr(), st.data_ptr(),
                                     _stream(stream)), "fp8_quant_act_t")
    return qt, st


def fp8_quant_act_dual(x, q=None, s=None, qt=None, st=None, stream=None):
    """X[M][K] bf16 -> (Q, S, Q^T, S^T): both layouts from one read of X."""
    import torch
    M, K = _x2(x, "x", tokens=True)
    dev = _validate([(x, torch.bfloat16, (M, K), "x"), (q, torch.uint8, (M, K), "q"),
                     (s, torch.float32, (K // 128, M), "s"), (qt, torch.uint8, (K, M), "qt"),
                     (st, torch.float32, (_groups(M), K), "st")])
    q = _alloc(q, (M, K), torch.uint8, dev)
    s = _alloc(s, (K // 128, M), torch.float32, dev)
    qt = _alloc(qt, (K, M), torch.uint8, dev)
    st = _alloc(st, (_groups(M), K), torch.float32, dev)
    with _on(dev):
        _check(lib().fp8_quant_act_dual(x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
                                        qt.data_ptr(), st.data_ptr(), _stream(stream)),
               "fp8_quant_act_dual")
    return q, s, qt, st


def fp8_quant_weight(w, want_t: bool = False, q=None, s=None, qt=None, stream=None):
    """W[N][K] bf16 -> (Q[N][K] uint8, S[N/128][K/128] float32, Q^T[K][N] or None)."""
    import torch
    N, K = _x2(w, "w")
    dev = _validate([(w, torch.bfloat16, (N, K), "w"), (q, torch.uint8, (N, K), "q"),
                     (s, torch.float32, (N // 128, K // 128), "s"),
                     (qt, torch.uint8, (K, N), "qt")])
    q = _alloc(q, (N, K), torch.uint8, dev)
    s = _alloc(s, (N // 128, K // 128), torch.float32, dev)
    if want_t:
        qt = _alloc(qt, (K, N), torch.uint8, dev)
    with _on(dev):
        _check(lib().fp8_quant_weight(w.data_ptr(), N, K, q.data_ptr(), s.data_ptr(),
                                      qt.data_ptr() if qt is not None else None,
                                      _stream(stream)), "fp8_quant_weight")
    return q, s, qt


def _gemm_shapes(mode: int, M: int, N: int, K: int, e8m0: bool = False):
    """Operand shapes of each GEMM mode (include/fp8bw.h): a, sa, b, sb."""
    if mode not in (FPROP, DGRAD, WGRAD):
        raise ValueError(f"mode must be FPROP, DGRAD or WGRAD, got {mode}")
    if e8m0:
        _dims(M, N, K)
    elif mode == WGRAD:   # the reduction runs over tokens
        _dims(M, N)
        _tokens(K)
    else:                 # M is the token count
        _tokens(M)
        _dims(N, K)
    a = (M, K)
    b = (K, N) if mode == DGRAD else (N, K)
    if not e8m0:
        sa = (_groups(K), M)
        sb = {FPROP: (N // 128, K // 128), DGRAD: (K // 128, N // 128), WGRAD: (_groups(K), N)}[mode]
    else:  # 512-byte scale blocks, one per 128 rows x 128-deep reduction block
        sa = (M // 128, (K // 128) * 512)
        sb = (K // 128, (N // 128) * 512) if mode == DGRAD else (N // 128, (K // 128) * 512)
    return a, sa, b, sb


def fp8_gemm_blockwise(mode: int, a, sa, b, sb, M: int, N: int, K: int, out=None, stream=None):
    """D[M][N] bf16 from FP8 operands and blockwise scales; see include/fp8bw.h for the
    operand layouts of FPROP, DGRAD and WGRAD."""
    import torch
    M, N, K = int(M), int(N), int(K)
    sh_a, sh_sa, sh_b, sh_sb = _gemm_shapes(mode, M, N, K)
    dev = _validate([(a, torch.uint8, sh_a, "a"), (sa, torch.float32, sh_sa, "sa"),
                     (b, torch.uint8, sh_b, "b"), (sb, torch.float32, sh_sb, "sb"),
                     (out, torch.bfloat16, (M, N), "out")])
    out = _alloc(out, (M, N), torch.bfloat16, dev)
    with _on(dev):
        _check(lib().fp8_gemm_blockwise(int(mode), a.data_ptr(), sa.data_ptr(), b.data_ptr(),
                                        sb.data_ptr(), out.data_ptr(), M, N, K, _stream(stream)),
               "fp8_gemm_blockwise")
    return out


def fp8_gemm_wgrad_acc32(a, sa, b, sb, M: int, N: int, K: int, dw32, stream=None):
    """dw32[M][N] (float32, caller-owned) += the wgrad sum, kept in FP32 (no BF16
    rounding); a, sa, b, sb as for fp8_gemm_blockwise(WGRAD, ...)."""
    import torch
    M, N, K = int(M), int(N), int(K)
    sh_a, sh_sa, sh_b, sh_sb = _gemm_shapes(WGRAD, M, N, K)
    if dw32 is None:
        raise TypeError("dw32 must be a caller-owned float32 tensor")
    dev = _validate([(a, torch.uint8, sh_a, "a"), (sa, torch.float32, sh_sa, "sa"),
                     (b, torch.uint8, sh_b, "b"), (sb, torch.float32, sh_sb, "sb"),
                     (dw32, torch.float32, (M, N), "dw32")])
    with _on(dev):
        _check(lib().fp8_gemm_wgrad_acc32(a.data_ptr(), sa.data_ptr(), b.data_ptr(),
                                          sb.data_ptr(), dw32.data_ptr(), M, N, K,
                                          _stream(stream)), "fp8_gemm_wgrad_acc32")
    return dw32


# -- power-of-two (E8M0) scales: the MXFP8 form of the recipe --------------------

def fp8_quant_act_e8m0(x, q=None, s=None, stream=None):
    """X[M][K] bf16 -> (Q[M][K] uint8, S: E8M0 scale blocks [M/128][(K/128)*512] uint8,
    the tensor-core layout described in include/fp8bw.h)."""
    import torch
    M, K = _x2(x, "x")
    ssh = (M // 128, (K // 128) * 512)
    dev = _validate([(x, torch.bfloat16, (M, K), "x"), (q, torch.uint8, (M, K), "q"),
                     (s, torch.uint8, ssh, "s")])
    q = _alloc(q, (M, K), torch.uint8, dev)
    s = _alloc(s, ssh, torch.uint8, dev)
    with _on(dev):
        _check(lib().fp8_quant_act_e8m0(x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
                                        _stream(stream)), "fp8_quant_act_e8m0")
    return q, s


def fp8_quant_act_t_e8m0(x, qt=None, st=None, stream=None):
    """X[M][K] bf16 -> (Q^T[K][M] uint8, S^T: E8M0 scale blocks [K/128][(M/128)*512])."""
    import torch
    M, K = _x2(x, "x")
    tsh = (K // 128, (M // 128) * 512)
    dev = _validate([(x, torch.bfloat16, (M, K), "x"), (qt, torch.uint8, (K, M), "qt"),
                     (st, torch.uint8, tsh, "st")])
    qt = _alloc(qt, (K, M), torch.uint8, dev)
    st = _alloc(st, tsh, torch.uint8, dev)
    with _on(dev):
        _check(lib().fp8_quant_act_t_e8m0(x.data_ptr(), M, K, qt.data_ptr(), st.data_ptr(),
                                          _stream(stream)), "fp8_quant_act_t_e8m0")
    return qt, st


def fp8_quant_act_dual_e8m0(x, q=None, s=None, qt=None, st=None, stream=None):
    """X[M][K] bf16 -> (Q, S, Q^T, S^T) with E8M0 scale codes, from one read of X."""
    import torch
    M, K = _x2(x, "x")
    ssh, tsh = (M // 128, (K // 128) * 512), (K // 128, (M // 128) * 512)
    dev = _validate([(x, torch.bfloat16, (M, K), "x"), (q, torch.uint8, (M, K), "q"),
                     (s, torch.uint8, ssh, "s"), (qt, torch.uint8, (K, M), "qt"),
                     (st, torch.uint8, tsh, "st")])
    q = _alloc(q, (M, K), torch.uint8, dev)
    s = _alloc(s, ssh, torch.uint8, dev)
    qt = _alloc(qt, (K, M), torch.uint8, dev)
    st = _alloc(st, tsh, torch.uint8, dev)
    with _on(dev):
        _check(lib().fp8_quant_act_dual_e8m0(x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
                                             qt.data_ptr(), st.data_ptr(), _stream(stream)),
               "fp8_quant_act_dual_e8m0")
    return q, s, qt, st


def fp8_quant_weight_e8m0(w, want_t: bool = False, q=None, s=None, qt=None, stream=None):
    """W[N][K] bf16 -> (Q[N][K], S: E8M0 scale blocks [N/128][(K/128)*512], Q^T or None)."""
    import torch
    N, K = _x2(w, "w")
    ssh = (N // 128, (K // 128) * 512)
    dev = _validate([(w, torch.bfloat16, (N, K), "w"), (q, torch.uint8, (N, K), "q"),
                     (s, torch.uint8, ssh, "s"), (qt, torch.uint8, (K, N), "qt")])
    q = _alloc(q, (N, K), torch.uint8, dev)
    s = _alloc(s, ssh, torch.uint8, dev)
    if want_t:
        qt = _alloc(qt, (K, N), torch.uint8, dev)
    with _on(dev):
        _check(lib().fp8_quant_weight_e8m0(w.data_ptr(), N, K, q.data_ptr(), s.data_ptr(),
                                           qt.data_ptr() if qt is not None else None,
                                           _stream(stream)), "fp8_quant_weight_e8m0")
    return q, s, qt


def fp8_gemm_blockwise_e8m0(mode: int, a, sa, b, sb, M: int, N: int, K: int, out=None,
                            stream=None):
    """fp8_gemm_blockwise with E8M0 scale blocks (from the *_e8m0 quantizers), applied by
    the block-scaled MMA."""
    import torch
    M, N, K = int(M), int(N), int(K)
    sh_a, sh_sa, sh_b, sh_sb = _gemm_shapes(mode, M, N, K, e8m0=True)
    dev = _validate([(a, torch.uint8, sh_a, "a"), (sa, torch.uint8, sh_sa, "sa"),
                     (b, torch.uint8, sh_b, "b"), (sb, torch.uint8, sh_sb, "sb"),
                     (out, torch.bfloat16, (M, N), "out")])
    out = _alloc(out, (M, N), torch.bfloat16, dev)
    with _on(dev):
        _check(lib().fp8_gemm_blockwise_e8m0(int(mode), a.data_ptr(), sa.data_ptr(),
                                             b.data_ptr(), sb.data_ptr(), out.data_ptr(), M, N, K,
                                             _stream(stream)), "fp8_gemm_blockwise_e8m0")
    return out


# -- the three GEMMs of the linear layer, composed from the entry points above ----

def linear_fprop(x, w, stream=None):
    """Y = X W^T with X[T][Din], W[Dout][Din] (bf16).  Returns (Y, saved) where saved
    holds the quantized weight for dgrad."""
    T, Din = x.shape
    Dout = w.shape[0]
    qx, sx = fp8_quant_act(x, stream=stream)
    qw, sw, _ = fp8_quant_weight(w, stream=stream)
    y = fp8_gemm_blockwise(FPROP, qx, sx, qw, sw, T, Dout, Din, stream=stream)
    return y, (qw, sw)


def linear_dgrad(dy, qw, sw, stream=None):
    """dX = dY W with dY[T][Dout] and the weight quantized by fp8_quant_weight."""
    T, Dout = dy.shape
    Din = qw.shape[1]
    qdy, sdy = fp8_quant_act(dy, stream=stream)
    return fp8_gemm_blockwise(DGRAD, qdy, sdy, qw, sw, T, Din, Dout, stream=stream)


def linear_wgrad(dy, x, stream=None):
    """dW = dY^T X with both operands quantized along the token dimension."""
    T, Dout = dy.shape
    Din = x.shape[1]
    qdyt, sdyt = fp8_quant_act_t(dy, stream=stream)
    qxt, sxt = fp8_quant_act_t(x, stream=stream)
    return fp8_gemm_blockwise(WGRAD, qdyt, sdyt, qxt, sxt, Dout, Din, T, stream=stream)


# -- few tokens: the linear of a decode step --------------------------------------

def fp8_linear_few(x, qw, sw, out=None, workspace=None, stream=None):
    """Y[M][N] bf16 = X W^T for X[M][K] bf16 with 1 <= M <= FEW_TOKENS tokens and a weight
    quantized by fp8_quant_weight; X is quantized inside the call as by fp8_quant_act.
    workspace: uint8, fp8_linear_few_workspace(M, K) bytes or more, one for each call (or
    captured graph) that may run at the same time."""
    r = (_calls or _open_calls()).linear_few(x, qw, sw, out, workspace, stream)
    if r is not NotImplemented:
        return r
    import torch
    M, K = _few_rows(x, "x")
    if not isinstance(qw, torch.Tensor) or qw.dim() != 2:
        raise ValueError("qw must be a 2-D tensor")
    N = qw.shape[0]
    _dims(N, K)
    dev = _validate([(x, torch.bfloat16, (M, K), "x"), (qw, torch.uint8, (N, K), "qw"),
                     (sw, torch.float32, (N // 128, K // 128), "sw"),
                     (out, torch.bfloat16, (M, N), "out")])
    L = lib()
    need = L.fp8_linear_few_workspace(M, K)
    with _on(dev):
        out = _alloc(out, (M, N), torch.bfloat16, dev, stream)
        if need:
            workspace = _workspace(workspace, need, dev, stream)
        _check(L.fp8_linear_few(x.data_ptr(), qw.data_ptr(), sw.data_ptr(), out.data_ptr(),
                                    M, N, K, workspace.data_ptr() if need else None,
                                    _stream(stream)), "fp8_linear_few")
    return out


def fp8_linear_few_workspace(M: int, K: int) -> int:
    """Bytes of workspace that fp8_linear_few needs (0 for the smallest token counts)."""
    if not 1 <= int(M) <= FEW_TOKENS:
        raise ValueError(f"{M} tokens, expected 1 to {FEW_TOKENS}")
    _dims(K)
    return int(lib().fp8_linear_few_workspace(int(M), int(K)))


def _few_rows(x, name):
    """Rows and columns of a few-token activation."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    M, K = x.shape
    if not 1 <= M <= FEW_TOKENS:
        raise ValueError(f"{name} has {M} tokens, expected 1 to {FEW_TOKENS}")
    return M, K


# -- mixture of experts -----------------------------------------------------------

def _experts(T, E, k):
    if T < 1:
        raise ValueError(f"token count {T} is not positive")
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"{E} experts, expected 1 to {MAX_EXPERTS}")
    if not 1 <= k <= min(E, MAX_CHOICES):
        raise ValueError(f"{k} choices per token, expected 1 to {min(E, MAX_CHOICES)}")


def _logits(logits, k):
    """Sizes of a router call: (T, E, k, whether the logits are bf16)."""
    import torch
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a 2-D tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    (T, E), k = logits.shape, int(k)
    _experts(T, E, k)
    return T, E, k, logits.dtype == torch.bfloat16


def fp8_moe_route(logits, k: int, renorm: bool = True, weights=None, ids=None, stream=None):
    """logits[T][E] (float32 or bf16) -> (weights[T][k] float32, ids[T][k] int32): the k
    largest, ties to the lowest expert, with softmax weights over the chosen experts
    (renorm) or over all.  -inf and NaN are never chosen (id -1, weight 0)."""
    r = (_calls or _open_calls()).moe_route(logits, k, renorm, weights, ids, stream)
    if r is not NotImplemented:
        return r
    import torch
    T, E, k, bf16 = _logits(logits, k)
    dev = _validate([(logits, logits.dtype, (T, E), "logits"),
                     (weights, torch.float32, (T, k), "weights"), (ids, torch.int32, (T, k), "ids")])
    with _on(dev):
        weights = _alloc(weights, (T, k), torch.float32, dev, stream)
        ids = _alloc(ids, (T, k), torch.int32, dev, stream)
        _check(lib().fp8_moe_route(logits.data_ptr(), int(bf16), T, E, k, int(bool(renorm)),
                                   weights.data_ptr(), ids.data_ptr(), _stream(stream)),
               "fp8_moe_route")
    return weights, ids


def fp8_moe_route_bwd(dweights, weights, ids, logits, renorm: bool = True, dlogits=None,
                      stream=None):
    """Gradient of the logits (of their type) from that of the weights; weights, ids,
    logits and renorm as in the forward call."""
    r = (_calls or _open_calls()).moe_route_bwd(dweights, weights, ids, logits, renorm, dlogits, stream)
    if r is not NotImplemented:
        return r
    import torch
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a 2-D tensor")
    T, E, k, bf16 = _logits(logits, ids.shape[1])
    dev = _validate([(dweights, torch.float32, (T, k), "dweights"),
                     (weights, torch.float32, (T, k), "weights"), (ids, torch.int32, (T, k), "ids"),
                     (logits, logits.dtype, (T, E), "logits"),
                     (dlogits, logits.dtype, (T, E), "dlogits")])
    with _on(dev):
        dlogits = _alloc(dlogits, (T, E), logits.dtype, dev, stream)
        _check(lib().fp8_moe_route_bwd(dweights.data_ptr(), weights.data_ptr(), ids.data_ptr(),
                                       logits.data_ptr(), int(bf16), T, E, k, int(bool(renorm)),
                                       dlogits.data_ptr(), _stream(stream)), "fp8_moe_route_bwd")
    return dlogits


def fp8_moe_plan_rows(T: int, E: int, k: int) -> int:
    """Rows of the layout by expert that hold any split of T * k pairs over E experts."""
    T, E, k = int(T), int(E), int(k)
    _experts(T, E, k)
    rows = (T * k + 127 * min(E, T * k)) // 128 * 128  # as the library has it
    if rows > MAX_DIM:
        raise ValueError(f"{T} tokens with {k} choices exceed the largest layout")
    return rows


def fp8_moe_plan(ids, E: int, seg=None, row=None, src=None, workspace=None, stream=None):
    """ids[T][k] int32 -> (seg[E + 1], row[T][k], src[rows]) int32: expert e owns the blocks of
    128 rows seg[e] .. seg[e + 1] - 1; row is each pair's row (-1: left out), src each row's
    pair t * k + j (-1: none).  workspace: uint8, at least what the header asks for."""
    r = (_calls or _open_calls()).moe_plan(ids, E, seg, row, src, workspace, stream)
    if r is not NotImplemented:
        return r
    import torch
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a 2-D tensor")
    T, k, E = int(ids.shape[0]), int(ids.shape[1]), int(E)
    rows = fp8_moe_plan_rows(T, E, k)
    dev = _validate([(ids, torch.int32, (T, k), "ids"), (seg, torch.int32, (E + 1,), "seg"),
                     (row, torch.int32, (T, k), "row"), (src, torch.int32, (rows,), "src")])
    need = int(lib().fp8_moe_plan_workspace(T, E, k))
    with _on(dev):
        seg = _alloc(seg, (E + 1,), torch.int32, dev, stream)
        row = _alloc(row, (T, k), torch.int32, dev, stream)
        src = _alloc(src, (rows,), torch.int32, dev, stream)
        workspace = _workspace(workspace, need, dev, stream)
        _check(lib().fp8_moe_plan(ids.data_ptr(), T, E, k, seg.data_ptr(), row.data_ptr(),
                                  src.data_ptr(), workspace.data_ptr(), _stream(stream)),
               "fp8_moe_plan")
    return seg, row, src


def _workspace(ws, need, dev, stream):
    """The caller's workspace, checked, or one of this call's own.  It is freed when the
    call returns, so it has to come from the allocator's pool of the stream that uses it."""
    import torch
    if ws is None:
        return _alloc(None, (need,), torch.uint8, dev, stream)
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    if ws.dim() != 1 or ws.numel() < need:
        raise ValueError(f"workspace has shape {tuple(ws.shape)}, expected ({need},) or longer")
    if _validate([(ws, torch.uint8, ws.shape, "workspace")]) != dev:
        raise ValueError(f"workspace is on {ws.device}, expected cuda:{dev} (one device per call)")
    return ws


def _grouped_shapes(mode, M, N, K, seg):
    """Operand shapes of a grouped GEMM (include/fp8bw.h): E, a, sa, b, sb, d."""
    import torch
    if mode not in (FPROP, DGRAD, WGRAD):
        raise ValueError(f"mode must be FPROP, DGRAD or WGRAD, got {mode}")
    if not isinstance(seg, torch.Tensor) or seg.dim() != 1 or seg.numel() < 2:
        raise ValueError("seg must be a 1-D tensor of E + 1 block offsets")
    E = int(seg.numel()) - 1
    if E > MAX_EXPERTS:
        raise ValueError(f"{E} experts, expected 1 to {MAX_EXPERTS}")
    _dims(M, N, K)
    a, sa = (M, K), (K // 128, M)
    if mode == WGRAD:
        return E, a, sa, (N, K), (K // 128, N), (E, M, N)
    r, c = (N, K) if mode == FPROP else (K, N)
    return E, a, sa, (E, r, c), (E, r // 128, c // 128), (M, N)


def fp8_gemm_grouped(mode: int, a, sa, b, sb, seg, M: int, N: int, K: int, out=None, stream=None):
    """fp8_gemm_blockwise with one weight per expert: expert e owns the 128-token blocks
    seg[e] .. seg[e + 1] - 1 (see fp8_moe_plan and include/fp8bw.h).  FPROP and DGRAD give
    [M][N] and leave the rows of blocks that no expert owns as they were; WGRAD gives
    [E][M][N]."""
    r = (_calls or _open_calls()).gemm_grouped(mode, a, sa, b, sb, seg, M, N, K, out, stream)
    if r is not NotImplemented:
        return r
    import torch
    M, N, K = int(M), int(N), int(K)
    E, sh_a, sh_sa, sh_b, sh_sb, sh_d = _grouped_shapes(mode, M, N, K, seg)
    dev = _validate([(a, torch.uint8, sh_a, "a"), (sa, torch.float32, sh_sa, "sa"),
                     (b, torch.uint8, sh_b, "b"), (sb, torch.float32, sh_sb, "sb"),
                     (seg, torch.int32, (E + 1,), "seg"), (out, torch.bfloat16, sh_d, "out")])
    with _on(dev):
        out = _alloc(out, sh_d, torch.bfloat16, dev, stream)
        _check(lib().fp8_gemm_grouped(int(mode), a.data_ptr(), sa.data_ptr(), b.data_ptr(),
                                      sb.data_ptr(), seg.data_ptr(), E, out.data_ptr(), M, N, K,
                                      _stream(stream)), "fp8_gemm_grouped")
    return out


def fp8_gemm_grouped_wgrad_acc32(a, sa, b, sb, seg, M: int, N: int, K: int, dw32, stream=None):
    """dw32[E][M][N] (float32, caller-owned) += the grouped WGRAD, kept in FP32."""
    r = (_calls or _open_calls()).gemm_grouped_wgrad_acc32(a, sa, b, sb, seg, M, N, K, dw32, stream)
    if r is not NotImplemented:
        return r
    import torch
    M, N, K = int(M), int(N), int(K)
    E, sh_a, sh_sa, sh_b, sh_sb, sh_d = _grouped_shapes(WGRAD, M, N, K, seg)
    if dw32 is None:
        raise TypeError("dw32 must be a caller-owned float32 tensor")
    dev = _validate([(a, torch.uint8, sh_a, "a"), (sa, torch.float32, sh_sa, "sa"),
                     (b, torch.uint8, sh_b, "b"), (sb, torch.float32, sh_sb, "sb"),
                     (seg, torch.int32, (E + 1,), "seg"), (dw32, torch.float32, sh_d, "dw32")])
    with _on(dev):
        _check(lib().fp8_gemm_grouped_wgrad_acc32(a.data_ptr(), sa.data_ptr(), b.data_ptr(),
                                                  sb.data_ptr(), seg.data_ptr(), E,
                                                  dw32.data_ptr(), M, N, K, _stream(stream)),
               "fp8_gemm_grouped_wgrad_acc32")
    return dw32


def fp8_moe_few_workspace(T: int, k: int, H: int, I: int) -> int:
    """Bytes of workspace that fp8_moe_few needs."""
    need = int(lib().fp8_moe_few_workspace(int(T), int(k), int(H), int(I)))
    if need == 0:
        raise ValueError(f"no few-token layer of {T} tokens, {k} choices, sizes {H} and {I}")
    return need


def fp8_moe_few(x, w1, s1, w2, s2, ids, weights, out=None, workspace=None, stream=None):
    """Y[T][H] bf16: all experts of a SwiGLU layer for X[T][H] bf16, 1 <= T <= FEW_TOKENS.
    w1[E][2I][H] (gate rows, then up rows) with s1[E][2I/128][H/128] and w2[E][H][I] with
    s2[E][H/128][I/128] as fp8_quant_weight gives them; ids, weights[T][k] as from
    fp8_moe_route.  workspace: uint8, fp8_moe_few_workspace(T, k, H, I) bytes or more, one
    for each call (or captured graph) that may run at the same time."""
    r = (_calls or _open_calls()).moe_few(x, w1, s1, w2, s2, ids, weights, out, workspace, stream)
    if r is not NotImplemented:
        return r
    import torch
    T, H = _few_rows(x, "x")
    for t, name in ((w1, "w1"), (w2, "w2")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name} must be a 3-D tensor")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a 2-D tensor")
    (E, _, I), k = w2.shape, ids.shape[1]
    _dims(H, I)
    _experts(T, E, k)
    dev = _validate([(x, torch.bfloat16, (T, H), "x"),
                     (w1, torch.uint8, (E, 2 * I, H), "w1"),
                     (s1, torch.float32, (E, 2 * I // 128, H // 128), "s1"),
                     (w2, torch.uint8, (E, H, I), "w2"),
                     (s2, torch.float32, (E, H // 128, I // 128), "s2"),
                     (ids, torch.int32, (T, k), "ids"),
                     (weights, torch.float32, (T, k), "weights"),
                     (out, torch.bfloat16, (T, H), "out")])
    with _on(dev):
        out = _alloc(out, (T, H), torch.bfloat16, dev, stream)
        workspace = _workspace(workspace, fp8_moe_few_workspace(T, k, H, I), dev, stream)
        _check(lib().fp8_moe_few(x.data_ptr(), w1.data_ptr(), s1.data_ptr(), w2.data_ptr(),
                                 s2.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                                 out.data_ptr(), T, E, k, H, I, workspace.data_ptr(),
                                 _stream(stream)), "fp8_moe_few")
    return out
