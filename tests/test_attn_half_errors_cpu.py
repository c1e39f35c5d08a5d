"""Argument checks of the attention-half entry points, without a GPU: every call below is
invalid (or has no work) and returns before any CUDA call."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="argument checks with fake pointers: CPU only")

OK, EINVAL, EALIGN, EUNSUPPORTED = 0, -1, -2, -3
A = ctypes.c_void_p(1 << 20)          # a 16-byte aligned fake device address (never read)
MIS = ctypes.c_void_p((1 << 20) + 4)  # a misaligned one


@pytest.fixture(scope="module")
def L():
    from mxfp4_block_scaled_moe_b200 import binding, build
    lib = ctypes.CDLL(build.build())
    for name, args in binding._SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "mxmoe_last_error" else ctypes.c_int
    return lib


def err(L):
    return L.mxmoe_last_error().decode()


def _f(v):
    return ctypes.cast(ctypes.pointer(ctypes.c_float(v)), ctypes.c_void_p)


def _norm(L, T=4, H=64, x=A, ldx=None, res=A, ldr=None, w=A, eps=1e-5, so=A, y=A, q=None, qs=None, s=None):
    return L.rmsnorm_residual(x, H if ldx is None else ldx, res, H if ldr is None else ldr, w, eps, T, H, so, y, q, qs,
                              s, None)


def test_norm_argument_checks(L):
    assert _norm(L, T=0) == OK and _norm(L, T=0, x=None) == OK
    assert _norm(L, T=-1) == EINVAL and _norm(L, H=0) == EINVAL
    assert _norm(L, H=60) == EALIGN and "multiple of 8" in err(L)
    assert _norm(L, H=32776) == EUNSUPPORTED
    assert _norm(L, ldx=56) == EINVAL and _norm(L, ldx=68) == EINVAL and _norm(L, ldr=0) == EINVAL
    for eps in (0.0, -1.0, 2.0, float("nan"), float("inf")):
        assert _norm(L, eps=eps) == EINVAL and "eps" in err(L)
    assert _norm(L, so=None) == EINVAL and _norm(L, res=None) == EINVAL
    assert _norm(L, y=None) == EINVAL
    assert _norm(L, q=A) == EINVAL and _norm(L, q=A, qs=A, s=_f(1.0)) == EINVAL and _norm(L, qs=A) == EINVAL
    for s in (0.0, -1.0, float("nan"), float("inf"), 1e-38):
        assert _norm(L, q=A, s=_f(s)) == EINVAL and "act_scale" in err(L)
    assert _norm(L, x=None) == EINVAL and _norm(L, w=None) == EINVAL
    for k in ("x", "res", "w", "so", "y"):
        assert _norm(L, **{k: MIS}) == EINVAL and "aligned" in err(L)
    assert _norm(L, q=A, qs=MIS) == EINVAL
