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


def _append(L, k=A, ldk=128, v=A, ldv=128, slots=A, T=4, Hkv=2, D=64, kb=A, ks=A, vb=A, vs=A, pages=3, page=16):
    return L.mxfp4_kv_append(k, ldk, v, ldv, slots, T, Hkv, D, kb, ks, vb, vs, pages, page, None)


def test_kv_append_argument_checks(L):
    assert _append(L, T=0) == OK and _append(L, T=0, k=None, slots=None) == OK
    assert _append(L, T=-1) == EINVAL and _append(L, Hkv=0) == EINVAL and _append(L, D=0) == EINVAL
    assert _append(L, D=48) == EALIGN and "multiple of 32" in err(L)
    for page in (0, 8, 24, 512, -16):
        assert _append(L, page=page) == EUNSUPPORTED and "page_size" in err(L)
    assert _append(L, ldk=120) == EINVAL and _append(L, ldv=132) == EINVAL
    for n in ("k", "v", "slots", "kb", "ks", "vb", "vs"):
        assert _append(L, **{n: None}) == EINVAL
        assert _append(L, **{n: MIS}) == EINVAL and "aligned" in err(L)
    assert _append(L, pages=-1) == EINVAL and _append(L, pages=1 << 31) == EUNSUPPORTED


def _attend(L, q=A, ldq=512, kb=A, ks=A, vb=A, vs=A, pages=3, page=16, table=A, width=2, lens=A, sinks=None, B=2, Lq=1,
            Hq=8, Hkv=2, D=64, scale=0.125, window=0, out=A, ws=A, nbytes=0):
    return L.mxfp4_kv_attention(q, ldq, kb, ks, vb, vs, pages, page, table, width, lens, sinks, B, Lq, Hq, Hkv, D, scale,
                                window, out, ws, nbytes, None)


def test_kv_attention_argument_checks(L):
    assert _attend(L, B=0) == OK and _attend(L, B=0, q=None, lens=None, out=None, ws=None) == OK
    assert _attend(L, B=-1) == EINVAL and _attend(L, Lq=0) == EINVAL and _attend(L, Hkv=0) == EINVAL
    assert _attend(L, Hq=9) == EINVAL and "multiple of Hkv" in err(L)
    for D in (32, 96, 256):
        assert _attend(L, D=D) == EUNSUPPORTED
    assert _attend(L, Lq=129) == EUNSUPPORTED and _attend(L, Hq=2048) == EUNSUPPORTED and _attend(L, B=65537) == EUNSUPPORTED
    assert _attend(L, page=48) == EUNSUPPORTED and _attend(L, window=-1) == EINVAL
    assert _attend(L, window=(1 << 30) + 1) == EUNSUPPORTED
    assert _attend(L, scale=float("nan")) == EINVAL and _attend(L, scale=float("inf")) == EINVAL
    assert _attend(L, ldq=504) == EINVAL and _attend(L, ldq=516) == EINVAL
    for n in ("q", "kb", "ks", "vb", "vs", "table", "lens", "out", "ws"):
        assert _attend(L, **{n: None}) == EINVAL
        assert _attend(L, **{n: MIS}) == EINVAL and "aligned" in err(L)
    assert _attend(L, sinks=MIS) == EINVAL
    n = ctypes.c_int64(0)
    assert L.mxfp4_kv_attention_workspace(2, 1, 8, 2, 96, ctypes.byref(n)) == EUNSUPPORTED
    assert L.mxfp4_kv_attention_workspace(2, 1, 8, 2, 64, None) == EINVAL


def _linear(L, xq=A, T=4, K=64, wq=A, N=16, sx=None, sxa=1.0, sw=None, swa=1.0, bias=None, act=0, res=None, out=A):
    return L.fp8_linear_fused(xq, T, K, wq, N, sx, sxa, sw, swa, bias, act, res, out, None)


def test_linear_fused_argument_checks(L):
    assert _linear(L, T=0) == OK and _linear(L, T=0, xq=None, out=None) == OK
    assert _linear(L, T=-1) == EINVAL and _linear(L, K=0) == EINVAL and _linear(L, N=0) == EINVAL
    assert _linear(L, K=48) == EALIGN and "multiple of 32" in err(L)
    assert _linear(L, N=12) == EALIGN and "multiple of 8" in err(L)
    assert _linear(L, T=1 << 24) == EUNSUPPORTED and _linear(L, act=3) == EUNSUPPORTED and _linear(L, act=-1) == EUNSUPPORTED
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _linear(L, sxa=s) == EINVAL and _linear(L, swa=s) == EINVAL
    for n in ("xq", "wq", "out"):
        assert _linear(L, **{n: None}) == EINVAL
    for n in ("xq", "wq", "out", "sx", "sw", "bias", "res"):
        assert _linear(L, **{n: MIS}) == EINVAL and "aligned" in err(L)


def test_linear_fused_columns_argument_checks(L):
    n = ctypes.c_int(7)
    for T, K, N in ((0, 64, 64), (64, 0, 64), (64, 64, 0), (-1, 64, 64)):
        assert L.fp8_linear_fused_columns(T, K, N, ctypes.byref(n)) == EINVAL and n.value == 7
    assert L.fp8_linear_fused_columns(64, 64, 64, None) == EINVAL
