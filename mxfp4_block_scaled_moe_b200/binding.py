"""Thin Python binding of libmxfp4moe (include/mxfp4_moe.h), same names as the C ABI.

Argument marshalling only: torch tensors give their device pointers and the current
CUDA stream; every step of the computation runs in the library's kernels. There is no
CPU path: without a CUDA device, or without the built library, every call raises.
bf16 tensors are passed as their bit patterns (torch.bfloat16 storage).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxfp4moe.so")

OK, EINVAL, EALIGN, EUNSUPPORTED, ECUDA, ETIMEOUT, ENOMEM, EDEVICE = 0, -1, -2, -3, -4, -5, -6, -7
OUT_F32, OUT_BF16 = 0, 1

_lib = None
_lock = threading.Lock()

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_SIGS = {
    "mxfp4_quantize": [_vp, _i64, _i64, _vp, _vp, _vp],
    "mxfp4_dequantize": [_vp, _vp, _i64, _i64, _vp, _i32, _vp],
    "mxfp4_quantize_axis": [_vp, _i64, _i64, _i64, _vp, _vp, _vp],
    "mxfp4_dequantize_axis": [_vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp],
    "mxfp4_linear": [_vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp],
    "fp8_linear": [_vp, _i32, _i32, _vp, _i32, _f32, _f32, _vp, _vp, _vp],
    "moe_route_topk": [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp],
    "moe_topk_from_logits": [_vp, _i32, _i32, _i32, _vp, _vp, _vp],
    "moe_permute": [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp],
    "moe_permute_noalloc": [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp],
    "moe_fp8_quantize": [_vp, _i64, _f32, _vp, _vp],
    "moe_mxfp4_forward": [_vp] * 9 + [_i32] * 5 + [_vp, _vp, _vp],
    "moe_mxfp4_forward_dense": [_vp] * 9 + [_i32] * 5 + [_vp, _vp, _vp],
    "moe_mxfp4_calibrate": [_vp] * 9 + [_i32] * 5 + [_vp, _vp],
    "moe_mxfp4_experts": [_vp, _vp, _i32, _i32, _i32, _i32] + [_vp] * 9,
    "moe_combine": [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp],
    "rmsnorm_residual": [_vp, _i64, _vp, _i64, _vp, _f32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp],
    "fp8_linear_fused": [_vp, _i32, _i32, _vp, _i32, _vp, _f32, _vp, _f32, _vp, _i32, _vp, _vp, _vp],
    "mxfp4_kv_append": [_vp, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _i32, _vp],
    "mxfp4_kv_attention_workspace": [_i32, _i32, _i32, _i32, _i32, _vp],
    "mxfp4_kv_attention": [_vp, _i64, _vp, _vp, _vp, _vp, _i64, _i32, _vp, _i32, _vp, _vp] + [_i32] * 5
                          + [_f32, _i32, _vp, _vp, _i64, _vp],
    "mxmoe_check": [_vp],
    "mxmoe_last_error": [],
    "mxmoe_last_launch_count": [],
    "mxmoe_release": [],
    "mxmoe_selftest_wait_timeout": [_vp],
    "mxmoe_tc_rate_probe": [_i32, _i32, _i32, _i32, _i32, _vp, _vp],
    "mxmoe_profile_enable": [_i32],
    "mxmoe_profile_read": [_vp, _vp, _vp, _i32],
}


class MxmoeError(RuntimeError):
    def __init__(self, rc: int, fn: str, msg: str):
        super().__init__(f"{fn} failed ({rc}): {msg}")
        self.rc = rc


def lib() -> ctypes.CDLL:
    """Load the library (once). Raises if it is missing or no CUDA device is visible."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not torch.cuda.is_available():
                    raise RuntimeError("libmxfp4moe needs a CUDA device; there is no CPU path")
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is missing: run mxfp4_block_scaled_moe_b200/build.py")
                L = ctypes.CDLL(LIB_PATH)
                for name, args in _SIGS.items():
                    fn = getattr(L, name)
                    fn.argtypes = args
                    fn.restype = ctypes.c_char_p if name == "mxmoe_last_error" else ctypes.c_int
                _lib = L
    return _lib


def _call(name, *args):
    L = lib()
    rc = getattr(L, name)(*args)
    if rc != OK:
        msg = L.mxmoe_last_error().decode(errors="replace")
        raise MxmoeError(rc, name, msg)
    return rc


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dev(t, dtype, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# ----------------------------------------------------------------------- codec -----

def mxfp4_quantize(w: torch.Tensor, blocks=None, scales=None, stream=None):
    """fp32 (..., K) -> (blocks (..., K/2) uint8, scales (..., K/32) uint8)."""
    _dev(w, torch.float32, "w")
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    if blocks is None:
        blocks = torch.empty(*w.shape[:-1], K // 2, dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(*w.shape[:-1], max(K // 32, 0), dtype=torch.uint8, device=w.device)
    _call("mxfp4_quantize", _ptr(w), rows, K, _ptr(blocks), _ptr(scales), _stream(stream))
    return blocks, scales


def mxfp4_dequantize(blocks: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32,
                     out=None, stream=None):
    """(..., K/2) uint8 + (..., K/32) uint8 -> (..., K) fp32 or bf16."""
    _dev(blocks, torch.uint8, "blocks")
    _dev(scales, torch.uint8, "scales")
    K = blocks.shape[-1] * 2
    rows = blocks.numel() // blocks.shape[-1] if blocks.shape[-1] else 0
    code = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    if out is None:
        out = torch.empty(*blocks.shape[:-1], K, dtype=out_dtype, device=blocks.device)
    _call("mxfp4_dequantize", _ptr(blocks), _ptr(scales), rows, K, _ptr(out), code, _stream(stream))
    return out


# --------------------------------------------------------------------- routing -----

def moe_route_topk(x, router_w, router_b, k, with_logits=False, stream=None):
    """Returns (topk_idx int32 (T,k), topk_w fp32 (T,k)[, logits fp32 (T,E)])."""
    _dev(x, torch.bfloat16, "x")
    _dev(router_w, torch.bfloat16, "router_w")
    _dev(router_b, torch.bfloat16, "router_b")
    T, H = x.shape
    E = router_w.shape[0]
    idx = torch.empty(T, k, dtype=torch.int32, device=x.device)
    w = torch.empty(T, k, dtype=torch.float32, device=x.device)
    logits = torch.empty(T, E, dtype=torch.float32, device=x.device) if with_logits else None
    _call("moe_route_topk", _ptr(x), _ptr(router_w), _ptr(router_b), T, H, E, k, _ptr(logits),
          _ptr(idx), _ptr(w), _stream(stream))
    return (idx, w, logits) if with_logits else (idx, w)


def moe_topk_from_logits(logits, k, stream=None):
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    _call("moe_topk_from_logits", _ptr(logits), T, E, k, _ptr(idx), _ptr(w), _stream(stream))
    return idx, w


def moe_permute(topk_idx, E, stream=None):
    """Returns (offsets (E+1), perm_token (T*k), perm_slot (T*k)), all int32."""
    _dev(topk_idx, torch.int32, "topk_idx")
    T, k = topk_idx.shape
    dev = topk_idx.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    pt = torch.empty(T * k, dtype=torch.int32, device=dev)
    ps = torch.empty(T * k, dtype=torch.int32, device=dev)
    _call("moe_permute", _ptr(topk_idx), T, E, k, _ptr(offsets), _ptr(pt), _ptr(ps), _stream(stream))
    return offsets, pt, ps


def moe_permute_noalloc(topk_idx, E, offsets, perm_token, perm_slot, stream=None):
    """moe_permute into caller-provided outputs without any device allocation by the
    library (its scratch is a fixed array; T*k <= 262144, E <= 256)."""
    _dev(topk_idx, torch.int32, "topk_idx")
    T, k = topk_idx.shape
    _call("moe_permute_noalloc", _ptr(topk_idx), T, E, k, _ptr(offsets), _ptr(perm_token),
          _ptr(perm_slot), _stream(stream))
    return offsets, perm_token, perm_slot


def moe_fp8_quantize(x, s, stream=None):
    """bf16 tensor -> uint8 E4M3 codes of x / s."""
    _dev(x, torch.bfloat16, "x")
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _call("moe_fp8_quantize", _ptr(x), x.numel(), float(s), _ptr(q), _stream(stream))
    return q


def _axis_view(shape, axis):
    axis = axis % len(shape)
    K = int(shape[axis])
    outer = 1
    for d in shape[:axis]:
        outer *= int(d)
    inner = 1
    for d in shape[axis + 1:]:
        inner *= int(d)
    return axis, outer, K, inner


def mxfp4_quantize_axis(w: torch.Tensor, axis: int, stream=None):
    """fp32 tensor -> (blocks, scales) along `axis`, moved to the end: blocks have the
    shape of w with that axis last and K/2 long, scales K/32 long."""
    _dev(w, torch.float32, "w")
    axis, outer, K, inner = _axis_view(w.shape, axis)
    moved = tuple(w.shape[:axis]) + tuple(w.shape[axis + 1:])
    blocks = torch.empty(*moved, K // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(*moved, max(K // 32, 0), dtype=torch.uint8, device=w.device)
    _call("mxfp4_quantize_axis", _ptr(w), outer, K, inner, _ptr(blocks), _ptr(scales), _stream(stream))
    return blocks, scales


def mxfp4_dequantize_axis(blocks: torch.Tensor, scales: torch.Tensor, axis: int, out_dtype=torch.float32,
                          out=None, stream=None):
    """Inverse of mxfp4_quantize_axis: the packed (last) axis goes back to position `axis`."""
    _dev(blocks, torch.uint8, "blocks")
    _dev(scales, torch.uint8, "scales")
    K = blocks.shape[-1] * 2
    moved = tuple(blocks.shape[:-1])
    nd = len(moved) + 1
    axis = axis % nd
    shape = moved[:axis] + (K,) + moved[axis:]
    _, outer, _, inner = _axis_view(shape, axis)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=blocks.device)
    code = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    _call("mxfp4_dequantize_axis", _ptr(blocks), _ptr(scales), outer, K, inner, _ptr(out), code, _stream(stream))
    return out


def mxfp4_linear(x, blocks, scales, bias=None, act_scale=None, out=None, stream=None):
    """out (T, N) bf16 = x (T, K) bf16 . W^T + bias with W MXFP4 (blocks (N, K/2), scales
    (N, K/32)); act_scale (one float) casts the input to FP8 E4M3 first."""
    _dev(x, torch.bfloat16, "x")
    _dev(blocks, torch.uint8, "blocks")
    _dev(scales, torch.uint8, "scales")
    _dev(bias, torch.float32, "bias")
    T, K = x.shape
    N = blocks.shape[0]
    if out is None:
        out = torch.empty(T, N, dtype=torch.bfloat16, device=x.device)
    s = None if act_scale is None else ctypes.byref(ctypes.c_float(float(act_scale)))
    _call("mxfp4_linear", _ptr(x), T, K, _ptr(blocks), _ptr(scales), N, _ptr(bias), s, _ptr(out), _stream(stream))
    return out


def fp8_linear(x, wq, s_x, s_w, bias=None, out=None, stream=None):
    """out (T, N) bf16 = bf16(s_x s_w e4m3(x / s_x) . wq^T + bias); wq: (N, K) uint8 E4M3 codes."""
    _dev(x, torch.bfloat16, "x")
    _dev(wq, torch.uint8, "wq")
    _dev(bias, torch.float32, "bias")
    T, K = x.shape
    N = wq.shape[0]
    if out is None:
        out = torch.empty(T, N, dtype=torch.bfloat16, device=x.device)
    _call("fp8_linear", _ptr(x), T, K, _ptr(wq), N, float(s_x), float(s_w), _ptr(bias), _ptr(out), _stream(stream))
    return out


# ----------------------------------------------------------------------- layer -----

def _layer_ptrs(x, router_w, router_b, gu_blocks, gu_scales, gu_bias, d_blocks, d_scales, d_bias):
    _dev(x, torch.bfloat16, "x")
    _dev(router_w, torch.bfloat16, "router_w")
    _dev(router_b, torch.bfloat16, "router_b")
    for n, t in (("gu_blocks", gu_blocks), ("gu_scales", gu_scales), ("d_blocks", d_blocks),
                 ("d_scales", d_scales)):
        _dev(t, torch.uint8, n)
    _dev(gu_bias, torch.float32, "gu_bias")
    _dev(d_bias, torch.float32, "d_bias")
    T, H = x.shape
    E = router_w.shape[0]
    I = d_blocks.shape[-1] * 2
    ptrs = [_ptr(t) for t in (x, router_w, router_b, gu_blocks, gu_scales, gu_bias, d_blocks,
                              d_scales, d_bias)]
    return ptrs, E, T, H, I


def _forward(name, x, router_w, router_b, gu_blocks, gu_scales, gu_bias, d_blocks, d_scales,
             d_bias, k, act_scale, out, stream):
    ptrs, E, T, H, I = _layer_ptrs(x, router_w, router_b, gu_blocks, gu_scales, gu_bias,
                                   d_blocks, d_scales, d_bias)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    _dev(out, torch.bfloat16, "out")
    acts = None
    if act_scale is not None:
        s = [float(v) for v in act_scale]
        acts = (ctypes.c_float * 2)(s[0], s[1])
    _call(name, *ptrs, E, k, T, H, I,
          ctypes.cast(acts, ctypes.c_void_p) if acts is not None else None, _ptr(out),
          _stream(stream))
    return out


def moe_mxfp4_forward(x, router_w, router_b, gu_blocks, gu_scales, gu_bias, d_blocks, d_scales,
                      d_bias, k, act_scale=None, out=None, stream=None):
    """The MoE expert layer; act_scale = None (bf16 activations) or two floats {s0, s1}."""
    return _forward("moe_mxfp4_forward", x, router_w, router_b, gu_blocks, gu_scales, gu_bias,
                    d_blocks, d_scales, d_bias, k, act_scale, out, stream)


def moe_mxfp4_forward_dense(x, router_w, router_b, gu_blocks, gu_scales, gu_bias, d_blocks,
                            d_scales, d_bias, k, act_scale=None, out=None, stream=None):
    """The same layer by the dense all-experts path (every token through all E experts,
    zero gates off the top-k)."""
    return _forward("moe_mxfp4_forward_dense", x, router_w, router_b, gu_blocks, gu_scales,
                    gu_bias, d_blocks, d_scales, d_bias, k, act_scale, out, stream)


def moe_mxfp4_calibrate(x, router_w, router_b, gu_blocks, gu_scales, gu_bias, d_blocks, d_scales,
                        d_bias, k, stream=None):
    """Static FP8 scales {s0, s1} (device fp32 (2,)) from a calibration batch x."""
    ptrs, E, T, H, I = _layer_ptrs(x, router_w, router_b, gu_blocks, gu_scales, gu_bias,
                                   d_blocks, d_scales, d_bias)
    out = torch.empty(2, dtype=torch.float32, device=x.device)
    _call("moe_mxfp4_calibrate", *ptrs, E, k, T, H, I, _ptr(out), _stream(stream))
    return out


def moe_mxfp4_experts(x_rows, offsets, gu_blocks, gu_scales, gu_bias, d_blocks, d_scales, d_bias,
                      act_scale=None, y=None, stream=None):
    """fp32 (P, H) expert outputs of rows grouped by expert (offsets: int32 (E+1))."""
    _dev(x_rows, torch.bfloat16, "x_rows")
    _dev(offsets, torch.int32, "offsets")
    P, H = x_rows.shape
    E = gu_blocks.shape[0]
    I = d_blocks.shape[-1] * 2
    if y is None:
        y = torch.empty(P, H, dtype=torch.float32, device=x_rows.device)
    acts = None
    if act_scale is not None:
        s = [float(v) for v in act_scale]
        acts = (ctypes.c_float * 2)(s[0], s[1])
    _call("moe_mxfp4_experts", _ptr(x_rows), _ptr(offsets), E, P, H, I, _ptr(gu_blocks), _ptr(gu_scales),
          _ptr(gu_bias), _ptr(d_blocks), _ptr(d_scales), _ptr(d_bias),
          ctypes.cast(acts, ctypes.c_void_p) if acts is not None else None, _ptr(y), _stream(stream))
    return y


def moe_combine(y, topk_idx, topk_w, inv, out=None, stream=None):
    """bf16 (T, H): each token's k expert outputs y[inv] weighted and summed in ascending expert id."""
    _dev(y, torch.float32, "y")
    T, k = topk_idx.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    _call("moe_combine", _ptr(y), _ptr(topk_idx), _ptr(topk_w), _ptr(inv), T, H, k, _ptr(out), _stream(stream))
    return out


# -------------------------------------------------------------- attention half -----

# These operators take a few microseconds on the GPU, so their host side is kept short: flat
# checks whose messages are formed only on failure, no checks of tensors made here, raw
# device and stream handles.

def _device(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _refuse(t, dtype, shape, dev, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the other tensors on cuda:{dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, dtype, shape, dev, name):
    """Device pointer of a dense tensor of that type, shape and device (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(t, dtype, shape, dev, name)
    return t.data_ptr()


def _rows(t, H, dev, name):
    """(device pointer, row stride) of a bf16 tensor (..., H) as rows: a dense tensor of any
    rank, or two-dimensional rows cut from wider ones."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev:
        _refuse(t, torch.bfloat16, None, dev, name)
    if t.is_contiguous():
        return t.data_ptr(), H
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous, or two-dimensional with contiguous rows")
    return t.data_ptr(), t.stride(0)


def _run_on(dev, name, *args):
    """_call with the tensors' device current; that device's current stream goes last. (An
    operator given `stream` calls itself with that stream current first, so that the
    outputs and workspaces it makes belong to the stream that uses them.)"""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _run_on(dev, name, *args)
    L = _lib or lib()
    rc = getattr(L, name)(*args, torch._C._cuda_getCurrentRawStream(dev))
    if rc != OK:
        raise MxmoeError(rc, name, L.mxmoe_last_error().decode(errors="replace"))


def _norm(x, weight, residual, eps, sum_out, y, q, fp8, act_scale):
    """Shared by the two norms: makes the outputs that were not given, checks the rest."""
    dev = _device(x, "x")
    shape = x.shape
    H = shape[-1]
    px, ldx = _rows(x, H, dev, "x")
    pr = ps = py = pq = pt = s = scale = None
    ldr = H
    if residual is not None:
        if residual.shape != shape:
            raise ValueError(f"residual must have x's shape {tuple(shape)}, got {tuple(residual.shape)}")
        pr, ldr = _rows(residual, H, dev, "residual")
        if sum_out is None:
            sum_out = torch.empty_like(x, memory_format=torch.contiguous_format)
            ps = sum_out.data_ptr()
        else:
            ps = _arg(sum_out, torch.bfloat16, shape, dev, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    if y is not None:
        py = _arg(y, torch.bfloat16, shape, dev, "y")
    elif not fp8:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        py = y.data_ptr()
    if fp8:
        if q is None:
            q = torch.empty_like(x, dtype=torch.uint8, memory_format=torch.contiguous_format)
            pq = q.data_ptr()
        else:
            pq = _arg(q, torch.uint8, shape, dev, "q")
        if act_scale is None:
            scale = x.new_empty(shape[:-1], dtype=torch.float32)
            pt = scale.data_ptr()
        else:
            s = ctypes.byref(_f32(act_scale))
    _run_on(dev, "rmsnorm_residual", px, ldx, pr, ldr, _arg(weight, torch.bfloat16, (H,), dev, "weight"), eps,
            x.numel() // H if H else 0, H, ps, py, pq, pt, s)
    return y, q, scale, sum_out


def rmsnorm_residual(x, weight, residual=None, eps=1e-5, sum_out=None, y=None, stream=None):
    """(y, sum): h = bf16(x + residual) (x without one; sum is then None) and y = bf16(h *
    weight / sqrt(mean(h^2) + eps)) over the last axis. sum_out may be `residual` (the
    stream updated in place). Strided rows of a 2-D x or residual are taken as they are."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm_residual(x, weight, residual, eps, sum_out, y)
    y, _, _, sum_out = _norm(x, weight, residual, eps, sum_out, y, None, False, None)
    return y, sum_out


def rmsnorm_residual_fp8(x, weight, residual=None, eps=1e-5, act_scale=None, sum_out=None, q=None, y=None,
                         stream=None):
    """(q, scale, sum): as rmsnorm_residual with E4M3 codes (uint8) of the norm: divided by the
    static act_scale (scale is then None), or by one scale per token, max|n| / 448 (scale:
    fp32 of x's leading shape). y, if given, receives the bf16 norm too."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm_residual_fp8(x, weight, residual, eps, act_scale, sum_out, q, y)
    return _norm(x, weight, residual, eps, sum_out, y, q, True, act_scale)[1:]


ACTS = {None: 0, "silu": 1, "gelu": 2}


def fp8_linear_fused(xq, wq, s_x, s_w, bias=None, act=None, residual=None, out=None, stream=None):
    """bf16 (T, N) = act(s_x s_w xq . wq^T + bias) + residual, of E4M3 codes (uint8) xq (T, K)
    and wq (N, K). s_x: a float, or fp32 (T), one scale per token; s_w: a float, or fp32 (N),
    one per output channel; act: None, "silu" or "gelu" (by erf); bias fp32 (N); residual
    bf16 (T, N). out may be `residual` (the stream updated in place)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return fp8_linear_fused(xq, wq, s_x, s_w, bias, act, residual, out)
    dev = _device(xq, "xq")
    T, K = xq.shape
    N = wq.shape[0]
    if act not in ACTS:
        raise ValueError(f"act must be one of {list(ACTS)}, got {act!r}")
    px = pw = None
    if isinstance(s_x, torch.Tensor):
        px, s_x = _arg(s_x, torch.float32, (T,), dev, "s_x"), 1.0
    if isinstance(s_w, torch.Tensor):
        pw, s_w = _arg(s_w, torch.float32, (N,), dev, "s_w"), 1.0
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=xq.device)
        po = out.data_ptr()
    else:
        po = _arg(out, torch.bfloat16, (T, N), dev, "out")
    _run_on(dev, "fp8_linear_fused", _arg(xq, torch.uint8, (T, K), dev, "xq"), T, K,
            _arg(wq, torch.uint8, (N, K), dev, "wq"), N, px, s_x, pw, s_w, _arg(bias, torch.float32, (N,), dev, "bias"),
            ACTS[act], _arg(residual, torch.bfloat16, (T, N), dev, "residual"), po)
    return out


def _cache(k_blocks, k_scales, v_blocks, v_scales, dev):
    """(pointers, num_pages, Hkv, page_size, D) of a paged cache's four arrays."""
    shape = k_blocks.shape
    if len(shape) != 4:
        raise ValueError(f"k_blocks must be (num_pages, Hkv, page_size, D/2), got {tuple(shape)}")
    pages, Hkv, page_size, half = shape
    sc = (pages, Hkv, page_size, half // 16)
    ptrs = (_arg(k_blocks, torch.uint8, shape, dev, "k_blocks"), _arg(k_scales, torch.uint8, sc, dev, "k_scales"),
            _arg(v_blocks, torch.uint8, shape, dev, "v_blocks"), _arg(v_scales, torch.uint8, sc, dev, "v_scales"))
    return ptrs, pages, Hkv, page_size, 2 * half


def _tokens(t, dev, name):
    """(device pointer, token stride) of a bf16 tensor (..., heads, D) whose heads are dense and
    whose tokens are one stride apart."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev:
        _refuse(t, torch.bfloat16, None, dev, name)
    shape = t.shape
    if t.is_contiguous():
        return t.data_ptr(), shape[-2] * shape[-1]
    stride = t.stride()
    if stride[-1] != 1 or stride[-2] != shape[-1]:
        raise ValueError(f"{name}: each token's heads must be dense")
    if len(shape) == 3 and shape[0] > 1:
        return t.data_ptr(), stride[0]
    step = n = None
    for size, st in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if size == 1:
            continue
        if step is None:
            step, n = st, size
        elif st != step * n:
            raise ValueError(f"{name}: the tokens must be one stride apart")
        else:
            n *= size
    return t.data_ptr(), shape[-2] * shape[-1] if step is None else step


def mxfp4_kv_append(k, v, slots, k_blocks, k_scales, v_blocks, v_scales, stream=None):
    """Quantize the rows of k and v, bf16 (T, Hkv, D), to MXFP4 along D and write them to the
    paged cache: blocks (num_pages, Hkv, page_size, D/2) and scales (num_pages, Hkv, page_size,
    D/32), uint8. slots: int64 (T), page * page_size + offset; negative skips the token. k and
    v may be slices of a fused projection's rows."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mxfp4_kv_append(k, v, slots, k_blocks, k_scales, v_blocks, v_scales)
    dev = _device(k, "k")
    ptrs, pages, Hkv, page_size, D = _cache(k_blocks, k_scales, v_blocks, v_scales, dev)
    T = k.shape[0]
    if k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D):
        raise ValueError(f"k and v must be (T, {Hkv}, {D}), got {tuple(k.shape)} and {tuple(v.shape)}")
    pk, ldk = _tokens(k, dev, "k")
    pv, ldv = _tokens(v, dev, "v")
    _run_on(dev, "mxfp4_kv_append", pk, ldk, pv, ldv, _arg(slots, torch.int64, (T,), dev, "slots"), T, Hkv, D, *ptrs,
            pages, page_size)


_attention_bytes: dict = {}


def mxfp4_kv_attention_workspace(B, Lq, Hq, Hkv, D, device=None) -> int:
    """Bytes of workspace that mxfp4_kv_attention needs for these sizes."""
    dev = torch.device("cuda" if device is None else device).index
    dev = torch.cuda.current_device() if dev is None else dev
    key = (dev, B, Lq, Hq, Hkv, D)
    if key not in _attention_bytes:
        n = ctypes.c_int64(0)
        with torch.cuda.device(dev):
            _call("mxfp4_kv_attention_workspace", B, Lq, Hq, Hkv, D, ctypes.byref(n))
        _attention_bytes[key] = n.value
    return _attention_bytes[key]


def mxfp4_kv_attention(q, k_blocks, k_scales, v_blocks, v_scales, block_table, seq_lens, scale=None, window=0, sinks=None,
                       out=None, workspace=None, stream=None):
    """Attention of q, bf16 (B, Lq, Hq, D) or (B, Hq, D), the last Lq tokens of B sequences, over
    the paged MXFP4 cache; returns bf16 of q's shape. block_table: int32 (B, max_pages);
    seq_lens: int32 (B), the new tokens included; scale: 1 / sqrt(D) unless given; window: the
    keys a query sees, itself included (0: all); sinks: fp32 (Hq) logits joining each softmax.
    q's tokens may be slices of a fused projection's rows. workspace: uint8 of at least
    mxfp4_kv_attention_workspace's size, made by the call unless given."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mxfp4_kv_attention(q, k_blocks, k_scales, v_blocks, v_scales, block_table, seq_lens, scale, window,
                                      sinks, out, workspace)
    dev = _device(q, "q")
    ptrs, pages, Hkv, page_size, D = _cache(k_blocks, k_scales, v_blocks, v_scales, dev)
    shape = q.shape
    if len(shape) not in (3, 4) or shape[-1] != D:
        raise ValueError(f"q must be (B, Lq, Hq, {D}) or (B, Hq, {D}), got {tuple(shape)}")
    B, Hq = shape[0], shape[-2]
    Lq = shape[1] if len(shape) == 4 else 1
    pq, ldq = _tokens(q, dev, "q")
    if block_table.dim() != 2:
        raise ValueError(f"block_table must be (B, max_pages), got {tuple(block_table.shape)}")
    max_pages = block_table.shape[1]
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        po = out.data_ptr()
    else:
        po = _arg(out, torch.bfloat16, shape, dev, "out")
    if workspace is None:
        nbytes = _attention_bytes.get((dev, B, Lq, Hq, Hkv, D))
        if nbytes is None:
            nbytes = mxfp4_kv_attention_workspace(B, Lq, Hq, Hkv, D, q.device)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        pw = workspace.data_ptr()
    else:
        nbytes, pw = workspace.numel(), _arg(workspace, torch.uint8, workspace.shape, dev, "workspace")
    _run_on(dev, "mxfp4_kv_attention", pq, ldq, *ptrs, pages, page_size,
            _arg(block_table, torch.int32, (B, max_pages), dev, "block_table"), max_pages,
            _arg(seq_lens, torch.int32, (B,), dev, "seq_lens"), _arg(sinks, torch.float32, (Hq,), dev, "sinks"), B, Lq,
            Hq, Hkv, D, D ** -0.5 if scale is None else scale, window, po, pw, nbytes)
    return out


def mxmoe_check(stream=None):
    _call("mxmoe_check", _stream(stream))


def mxmoe_last_launch_count() -> int:
    return lib().mxmoe_last_launch_count()


def mxmoe_release():
    _call("mxmoe_release")


def mxmoe_tc_rate_probe(n=256, with_scale_copy=False, iters=20000, ctas=None, stream=None,
                        random_operands=True) -> float:
    """Launch the tensor-pipe rate probe (kind::mxf8f6f4 MMAs, M = 128, N = n) on `ctas`
    CTAs (default: one per SM), on pseudo-random operands (or zeros); returns the FLOPs the
    launch performs. Time it with CUDA events on `stream`."""
    if ctas is None:
        ctas = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    f = ctypes.c_double(0.0)
    _call("mxmoe_tc_rate_probe", int(n), 1 if with_scale_copy else 0, 1 if random_operands else 0, int(iters),
          int(ctas), ctypes.byref(f), _stream(stream))
    return f.value


def mxmoe_selftest_wait_timeout(stream=None):
    """Launch a bounded device wait that expires (about a second); the next
    mxmoe_check raises MxmoeError with MXMOE_ETIMEOUT."""
    _call("mxmoe_selftest_wait_timeout", _stream(stream))


def mxmoe_profile_enable(on: bool = True):
    _call("mxmoe_profile_enable", 1 if on else 0)


def mxmoe_profile_read(max_entries: int = 32):
    """{stage: (total_ms, calls)} recorded since profiling was enabled or last read."""
    L = lib()
    names = ctypes.create_string_buffer(32 * max_entries)
    ms = (ctypes.c_float * max_entries)()
    calls = (ctypes.c_int * max_entries)()
    n = L.mxmoe_profile_read(names, ms, calls, max_entries)
    if n < 0:
        raise MxmoeError(n, "mxmoe_profile_read", L.mxmoe_last_error().decode(errors="replace"))
    out = {}
    for i in range(min(n, max_entries)):
        nm = names.raw[32 * i:32 * (i + 1)].split(b"\0", 1)[0].decode()
        out[nm] = (float(ms[i]), int(calls[i]))
    return out
