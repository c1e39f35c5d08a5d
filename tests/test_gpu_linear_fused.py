"""fp8_linear_fused against the formula in 64 bits.

Bar. Products of two E4M3 values are exact in fp32; a sum of K of them is taken in K / 32
steps, each with an error below 2^-22 of A = s_x s_w sum |xq wq| (alignment and rounding of a
step, of the partials' joining, and of the scale products: 8 more). SiLU and GELU have slopes
below 1.13 and an error of a few fp32 roundings of their value. Then one bf16 rounding, 2^-8.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mxfp4_block_scaled_moe_b200 import binding
    return binding


def _codes(g, rows, cols):
    """E4M3 codes of normal values with the largest near 448."""
    v = torch.randn(rows, cols, generator=g, device="cuda") * 110
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


class Case:
    def __init__(self, T, K, N, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + T + K + N)
        self.xq, self.wq = _codes(g, T, K), _codes(g, N, K)
        self.sx = 0.01 * (0.5 + torch.rand(T, generator=g, device="cuda")) / math.sqrt(K)
        self.sw = 0.01 * (0.5 + torch.rand(N, generator=g, device="cuda"))
        self.bias = torch.randn(N, generator=g, device="cuda")
        self.res = torch.randn(T, N, generator=g, device="cuda").bfloat16()

    def check(self, out, s_x, s_w, bias=None, act=None, residual=None):
        x, w = (t.view(torch.float8_e4m3fn).double() for t in (self.xq, self.wq))
        s = torch.as_tensor(s_x, device="cuda").double().reshape(-1, 1) * torch.as_tensor(s_w, device="cuda").double()
        y, mag = (x @ w.t()) * s, (x.abs() @ w.abs().t()) * s
        if bias is not None:
            y = y + bias.double()
            mag = mag + bias.double().abs()
        if act == "silu":
            y = y * torch.sigmoid(y)
        elif act == "gelu":
            y = 0.5 * y * torch.special.erfc(-y / math.sqrt(2))
        if residual is not None:
            y = y + residual.double()
            mag = mag + residual.double().abs()
        tol = y.abs() * 2.0 ** -8 + 1.13 * mag * (x.shape[1] / 32 + 8) * 2.0 ** -22
        assert out.dtype == torch.bfloat16 and out.shape == y.shape
        err = (out.double() - y).abs()
        assert bool((err <= tol).all()), (float((err - tol).max()), float(y.abs().max()))


SHAPES = [(1, 32, 8), (1, 2880, 5120), (3, 96, 136), (16, 4096, 2880), (17, 256, 64), (32, 160, 1000), (33, 1024, 256),
          (64, 4096, 2880), (65, 512, 384), (128, 2880, 640), (129, 128, 128), (200, 2880, 5120), (777, 1024, 4096),
          (1000, 352, 2048), (513, 64, 8200), (3000, 288, 1544), (4100, 2880, 264), (300, 8192, 4096)]


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_linear_fused(B, T, K, N):
    c = Case(T, K, N)
    sx, sw = float(c.sx[0]), float(c.sw[0])
    kw = [dict(s_x=c.sx, s_w=c.sw, bias=c.bias, residual=c.res), dict(s_x=sx, s_w=sw),
          dict(s_x=c.sx, s_w=sw, act="silu", bias=c.bias), dict(s_x=sx, s_w=c.sw, act="gelu", residual=c.res)]
    for k in kw:
        out = B.fp8_linear_fused(c.xq, c.wq, **k)
        B.mxmoe_check()
        c.check(out, **k)
        assert torch.equal(B.fp8_linear_fused(c.xq, c.wq, **k), out)


@pytest.mark.parametrize("T,K,N", [(66, 96, 40), (100, 32, 136), (250, 480, 8104), (700, 512, 4680), (2300, 64, 1160),
                                   (1300, 64, 2104), (520, 160, 5000), (260, 512, 13992), (9000, 64, 264), (1100, 96, 3848),
                                   (5000, 1024, 488), (6000, 1024, 200), (2300, 2048, 904)])
def test_linear_fused_tile_widths(B, T, K, N):
    """Sizes whose tiles are 64 to 256 columns wide, the last ones cut, one round of them and several."""
    c = Case(T, K, N)
    for k in (dict(s_x=c.sx, s_w=c.sw, bias=c.bias, residual=c.res), dict(s_x=float(c.sx[0]), s_w=c.sw, act="gelu")):
        out = B.fp8_linear_fused(c.xq, c.wq, **k)
        B.mxmoe_check()
        c.check(out, **k)
        assert torch.equal(B.fp8_linear_fused(c.xq, c.wq, **k), out)


@pytest.mark.parametrize("T", [5, 600])
def test_in_place_residual_and_given_output(B, T):
    c = Case(T, 512, 4096)
    want = B.fp8_linear_fused(c.xq, c.wq, c.sx, c.sw, c.bias, residual=c.res)
    out = torch.full_like(want, float("nan"))
    assert B.fp8_linear_fused(c.xq, c.wq, c.sx, c.sw, c.bias, residual=c.res, out=out) is out
    assert torch.equal(out, want)
    B.fp8_linear_fused(c.xq, c.wq, c.sx, c.sw, c.bias, residual=c.res, out=c.res)
    assert torch.equal(c.res, want)


@pytest.mark.parametrize("T,N", [(9, 264), (515, 4104)])
def test_nothing_beside_the_output_is_written(B, T, N):
    c = Case(T, 256, N)
    guard = torch.full((T + 16, N), 7.0, device="cuda", dtype=torch.bfloat16)
    B.fp8_linear_fused(c.xq, c.wq, c.sx, c.sw, out=guard[8:8 + T])
    B.mxmoe_check()
    assert bool((guard[:8] == 7).all()) and bool((guard[8 + T:] == 7).all())
    c.check(guard[8:8 + T], c.sx, c.sw)


def test_activation_tails(B):
    """Pre-activations from -30 to 30: the tails keep their relative precision."""
    xq = torch.full((1, 32), 0, dtype=torch.uint8, device="cuda")
    wq = torch.zeros(1024, 32, dtype=torch.uint8, device="cuda")
    bias = torch.linspace(-30, 30, 1024, device="cuda")
    for act, f in (("silu", lambda v: v * torch.sigmoid(v)), ("gelu", lambda v: 0.5 * v * torch.special.erfc(-v / math.sqrt(2)))):
        out = B.fp8_linear_fused(xq, wq, 1.0, 1.0, bias=bias, act=act).double()[0]
        ref = f(bias.double())
        # erfc's argument carries two fp32 roundings: 2 v^2 2^-24 of its value at the tail
        assert bool(((out - ref).abs() <= ref.abs() * (2.0 ** -8 + bias.double() ** 2 * 2.0 ** -20) + 2.0 ** -126).all())


def test_streams_and_graph(B):
    for T in (4, 700):
        c = Case(T, 2880, 4096)
        want = B.fp8_linear_fused(c.xq, c.wq, c.sx, c.sw, c.bias)
        s = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        got = [B.fp8_linear_fused(c.xq, c.wq, c.sx, c.sw, c.bias, stream=s[i % 2]) for i in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in got)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = B.fp8_linear_fused(c.xq, c.wq, c.sx, c.sw, c.bias)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    B.mxmoe_check()


def test_refusals(B):
    c = Case(4, 64, 32)
    for bad in (lambda: B.fp8_linear_fused(c.xq.float(), c.wq, 1.0, 1.0), lambda: B.fp8_linear_fused(c.xq, c.wq[:, :32], 1.0, 1.0),
                lambda: B.fp8_linear_fused(c.xq, c.wq, c.sx[:3], 1.0), lambda: B.fp8_linear_fused(c.xq, c.wq, 1.0, c.sw.double()),
                lambda: B.fp8_linear_fused(c.xq, c.wq, 1.0, 1.0, act="relu"),
                lambda: B.fp8_linear_fused(c.xq, c.wq, 1.0, 1.0, residual=c.res[:, :16]),
                lambda: B.fp8_linear_fused(c.xq, c.wq, 1.0, 1.0, bias=c.bias.cpu()),
                lambda: B.fp8_linear_fused(c.xq.t(), c.wq, 1.0, 1.0)):
        with pytest.raises(ValueError):
            bad()
    for rc, bad in ((B.EINVAL, lambda: B.fp8_linear_fused(c.xq, c.wq, 0.0, 1.0)),
                    (B.EALIGN, lambda: B.fp8_linear_fused(c.xq[:, :48].contiguous(), c.wq[:, :48].contiguous(), 1.0, 1.0)),
                    (B.EALIGN, lambda: B.fp8_linear_fused(c.xq, c.wq[:12], 1.0, 1.0))):
        with pytest.raises(B.MxmoeError) as ei:
            bad()
        assert ei.value.rc == rc
    assert B.fp8_linear_fused(c.xq[:0], c.wq, 1.0, 1.0).shape == (0, 32)


@pytest.mark.parametrize("T,N", [(1, 4096), (40, 4096), (300, 4096)])   # either kernel
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_linear_fused_activation_range(B, T, N, act):
    """The activations over their whole range, given by the bias over codes of zero. A bf16 rounding
    (2^-8), and 2^-14 for the functions: their exponent is at most 2^7 and is rounded to 2^-23 of it
    by two steps, the fit adds 2^-19. Below 87.4 2^-126 the reciprocal of 1 + e^-v is flushed."""
    v = torch.cat((torch.linspace(-16, 16, 3001), torch.linspace(-200, 200, 1001),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 1e4, -1e4, 1e30, -1e30, 3e38, -3e38]))).float()
    v = torch.cat((v, torch.zeros(N - v.numel()))).cuda()
    xq, wq = (torch.zeros(n, 64, dtype=torch.uint8, device="cuda") for n in (T, N))
    out = B.fp8_linear_fused(xq, wq, 1.0, 1.0, bias=v, act=act).double()
    d = v.double()
    y = d * torch.sigmoid(d) if act == "silu" else d * 0.5 * torch.special.erfc(-d / 2 ** 0.5)
    assert bool(((out - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -14) + 87.4 * 2.0 ** -126).all())
    big = torch.full((N,), float("inf"), device="cuda")
    assert bool(B.fp8_linear_fused(xq, wq, 1.0, 1.0, bias=big, act=act).isinf().all())
    assert bool(B.fp8_linear_fused(xq, wq, 1.0, 1.0, bias=big * 0, act=act).isnan().all())
    B.mxmoe_check()


@pytest.mark.parametrize("T,N", [(3, 64), (70, 4096), (300, 4096)])   # either kernel
def test_scales_whose_product_leaves_fp32(B, T, N):
    """Scales far from 1: only the scaled sums have to lie in range, not the product of the scales."""
    c = Case(T, 1024, N)
    one = torch.ones_like
    for a, b in ((1e-22, 1e-22), (1e-36, 1e-5), (3e-40, 1e-3), (1e20, 1e-25), (1e25, 1e-20)):
        for s_x, s_w in ((a, b), (a * one(c.sx), b), (a, b * one(c.sw)), (a * one(c.sx), b * one(c.sw))):
            out = B.fp8_linear_fused(c.xq, c.wq, s_x, s_w)
            x, w = (t.view(torch.float8_e4m3fn).double() for t in (c.xq, c.wq))
            s = float(torch.tensor(a, dtype=torch.float32)) * float(torch.tensor(b, dtype=torch.float32))
            y, mag = (x @ w.t()) * s, (x.abs() @ w.abs().t()) * s
            # the bar above, and half a least step of bf16's and fp32's subnormals; a step of sum * s_x that is subnormal
            tol = y.abs() * 2.0 ** -8 + mag * (1024 / 32 + 8) * 2.0 ** -22 + 2.0 ** -134 + 2.0 ** -149 * max(1.0, b)
            assert bool(((out.double() - y).abs() <= tol).all()), (a, b, type(s_x), type(s_w))
    zero = torch.zeros_like(c.xq)
    out = B.fp8_linear_fused(zero, c.wq, 1e30, 1e30, bias=c.bias)
    assert torch.equal(out, c.bias.bfloat16().expand(T, N))
    B.mxmoe_check()


# sizes that take tiles of each width, in one round of them and in several, and split products
EACH = [(140, 1600, 3608), (5465, 2304, 152), (1165, 1184, 1096), (550, 128, 4624), (250, 480, 8104), (4774, 320, 776),
        (4204, 1664, 624), (1024, 2880, 5120), (4427, 288, 1128), (5000, 352, 488), (1784, 448, 8056), (297, 1632, 7152),
        (4096, 352, 5120), (777, 1024, 4096), (3000, 352, 4104), (2154, 2880, 8176), (300, 8192, 1024), (128, 1024, 8192)]


def test_each_width_is_tested(B):
    widths = [B.fp8_linear_fused_columns(*s) for s in EACH]
    assert set(widths) == {0, 64, 96, 128, 160, 192, 224, 256}, widths
    assert B.fp8_linear_fused_columns(64, 1024, 4096) == 0
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    several = {w for w, (T, K, N) in zip(widths, EACH) if w and -(-T // 256) * -(-N // w) > pairs}
    one = {w for w, (T, K, N) in zip(widths, EACH) if w and -(-T // 256) * -(-N // w) <= pairs}
    assert several >= {96, 128, 160, 192, 224, 256} and one >= {64, 96, 128, 160, 192, 224, 256}, widths


@pytest.mark.parametrize("T,K,N", EACH)
def test_linear_fused_each_width(B, T, K, N):
    c = Case(T, K, N)
    for k in (dict(s_x=c.sx, s_w=c.sw, bias=c.bias, residual=c.res), dict(s_x=c.sx, s_w=float(c.sw[0]), act="silu")):
        out = B.fp8_linear_fused(c.xq, c.wq, **k)
        B.mxmoe_check()
        c.check(out, **k)
        assert torch.equal(B.fp8_linear_fused(c.xq, c.wq, **k), out)
