"""rmsnorm_residual and rmsnorm_residual_fp8 against the formula in 64 bits.

Bars. The stored sum is one fp32 addition rounded to bf16: bit-equal. The row factor is
fp32: the sum of H squares has a relative error below (H/32 + 12) 2^-24 < 2^-13.9 at the
longest row if every rounding went one way, the factor half of that; REL = 2^-14 covers it
with the products' roundings. A bf16 output adds half a step, 2^-8 of the value; an E4M3
code 2^-4 of it, or 2^-10 below the least normal value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

REL = 2.0 ** -14
EPS = 1e-5


@pytest.fixture(scope="module")
def B():
    from mxfp4_block_scaled_moe_b200 import binding
    return binding


def _inputs(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    res = (3 * torch.randn(T, H, generator=g, device="cuda")).bfloat16()
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    return x, res, w


def _norm64(h, w, eps=EPS):
    h = h.double()
    return h * w.double() / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)


def _check_y(y, n):
    assert y.dtype == torch.bfloat16
    assert bool(((y.double() - n).abs() <= n.abs() * (2.0 ** -8 + REL) + 2.0 ** -133).all())


def _check_q(q, v):
    """codes q of values v (64 bits, already divided by the scale)"""
    got = q.view(torch.float8_e4m3fn).double()
    want = v.clamp(-448, 448)
    assert bool(((got - want).abs() <= want.abs() * (2.0 ** -4 + REL) + 2.0 ** -10).all())


SHAPES = [(1, 8), (1, 2880), (3, 64), (2, 4088), (5, 4104), (3, 8192), (2, 16376), (2, 32768), (593, 8), (601, 264),
          (700, 520), (600, 1024), (597, 2040), (700, 2880), (640, 4096)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_outputs(B, T, H, residual):
    x, res, w = _inputs(T, H, T + H)
    h = (x.float() + res.float()).bfloat16() if residual else x
    n = _norm64(h, w)
    y, s = B.rmsnorm_residual(x, w, res if residual else None, EPS)
    _check_y(y, n)
    q, scale, s2 = B.rmsnorm_residual_fp8(x, w, res if residual else None, EPS, act_scale=0.02)
    assert scale is None
    _check_q(q, n / 0.02)
    y3 = torch.empty_like(x)
    qt, st, s3 = B.rmsnorm_residual_fp8(x, w, res if residual else None, EPS, y=y3)
    _check_y(y3, n)
    want = n.abs().amax(1) / 448
    assert st.shape == (T,) and bool(((st.double() - want).abs() <= want * REL).all())
    _check_q(qt, n / st.double()[:, None])
    for got in (s, s2, s3):
        assert torch.equal(got, h) if residual else got is None


def test_strided_rows_in_place_and_leading_shapes(B):
    T, H = 70, 512
    wide, _, w = _inputs(T, 3 * H, 5)
    res = wide[:, 2 * H:].clone()
    x = wide[:, H:2 * H]
    h = (x.float() + res.float()).bfloat16()
    before = wide.clone()
    y, s = B.rmsnorm_residual(x, w[:H].contiguous(), res, EPS, sum_out=res)
    assert s is res and torch.equal(res, h) and torch.equal(wide, before)
    _check_y(y, _norm64(h, w[:H]))
    y2, _ = B.rmsnorm_residual(h, w[:H].contiguous(), y=h)          # y over x
    assert torch.equal(y2, y)
    x3 = x.contiguous().view(7, 10, H)
    q, sc, _ = B.rmsnorm_residual_fp8(x3, w[:H].contiguous())
    assert q.shape == (7, 10, H) and sc.shape == (7, 10)
    _check_q(q, _norm64(x3, w[:H]) / sc.double()[..., None])


@pytest.mark.parametrize("T", [3, 700])
def test_extreme_rows(B, T):
    """Zero rows, rows whose squares leave fp32, rows and weights near the least values."""
    H = 320
    x, _, w = _inputs(T, H, 9)
    for row, f in ((0, 0.0), (1, 2.0 ** 100), (2, 2.0 ** -100)):
        x[row] = (x[row].float() * f).bfloat16()
    n = _norm64(x, w)
    y, _ = B.rmsnorm_residual(x, w)
    _check_y(y, n)
    q, sc, _ = B.rmsnorm_residual_fp8(x, w)
    assert float(sc[0]) == 1.0 and not bool(q[0].bitwise_and(0x7F).any())
    _check_q(q, n / sc.double()[:, None])
    want = n.abs().amax(1)[1:] / 448
    assert bool(((sc[1:].double() - want).abs() <= want * REL).all())
    tiny = (w.float() * 2.0 ** -110).bfloat16()
    q, sc, _ = B.rmsnorm_residual_fp8(x[3 if T > 3 else 1:], tiny)
    n = _norm64(x[3 if T > 3 else 1:], tiny)
    ok = n.abs().amax(1) / 448 > 2.0 ** -125      # scales that fp32 holds to its full precision
    assert bool(ok.any())
    _check_q(q[ok], (n / sc.double()[:, None])[ok])


def test_saturation_and_nonfinite(B):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = 5.0
    x[1, 3], x[2, 3] = float("nan"), float("inf")
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    q, _, _ = B.rmsnorm_residual_fp8(x, w, act_scale=1e-3)
    assert float(q.view(torch.float8_e4m3fn).float()[0, 0]) == 448.0
    y, _ = B.rmsnorm_residual(x, w)
    assert bool(y[1].isnan().all()) and torch.equal(y[0], y[3])
    B.rmsnorm_residual_fp8(x, w)
    B.mxmoe_check()


def test_streams_graph_and_empty(B):
    x, res, w = _inputs(33, 2880, 3)
    want, _ = B.rmsnorm_residual(x, w, res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, h = B.rmsnorm_residual(x, w, res)
    s.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, h = B.rmsnorm_residual(x, w, res)
    x.neg_()
    res.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, -want)
    one = x[0].clone()                                    # a single row without a token axis
    q, sc, _ = B.rmsnorm_residual_fp8(one, w)
    assert q.shape == one.shape and sc.shape == ()
    _check_q(q, _norm64(one, w) / sc.double())
    e = torch.empty(0, 2880, device="cuda", dtype=torch.bfloat16)
    assert B.rmsnorm_residual(e, w, e)[0].shape == (0, 2880)
    assert B.rmsnorm_residual_fp8(e, w)[1].shape == (0,)


def test_refusals(B):
    x, res, w = _inputs(4, 64, 1)
    for bad in (lambda: B.rmsnorm_residual(x.float(), w), lambda: B.rmsnorm_residual(x, w[:32]),
                lambda: B.rmsnorm_residual(x, w, res[:3]), lambda: B.rmsnorm_residual(x.t(), w),
                lambda: B.rmsnorm_residual(x, w.cpu()), lambda: B.rmsnorm_residual(x, w, sum_out=res),
                lambda: B.rmsnorm_residual(x, w, y=res[:2])):
        with pytest.raises(ValueError):
            bad()
    for rc, bad in ((B.EINVAL, lambda: B.rmsnorm_residual(x, w, eps=0.0)),
                    (B.EINVAL, lambda: B.rmsnorm_residual_fp8(x, w, act_scale=0.0)),
                    (B.EINVAL, lambda: B.rmsnorm_residual(x[:1].expand(4, 64), w)),
                    (B.EALIGN, lambda: B.rmsnorm_residual(x[:, :60].contiguous(), w[:60].contiguous()))):
        with pytest.raises(B.MxmoeError) as ei:
            bad()
        assert ei.value.rc == rc


@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("power", [31, 32, 40, 100, 127, -40, -120])
def test_token_scales_with_weights_far_from_one(B, T, power):
    """Rows of zeros, with zeros and with the least values, next to weights from 2^-120 to 2^127, some of
    them infinite products' halves: zeros stay zeros, and the rest keeps the norm's precision."""
    H = 320
    x, _, _ = _inputs(T, H, 11)
    w = torch.full((H,), 2.0 ** power, device="cuda").bfloat16()
    w[::3] = 1.0
    w[1::7] = -(2.0 ** min(power, 126))
    x[0] = 0
    x[1] = 0
    x[1, 0], x[1, 5] = 2.0 ** -133, -(2.0 ** -130)
    x[2, ::2] = 0
    q, sc, _ = B.rmsnorm_residual_fp8(x, w)
    y, _ = B.rmsnorm_residual(x, w)
    assert float(sc[0]) == 1.0 and not bool(q[0].bitwise_and(0x7F).any()) and not bool(y[0].any())
    n = _norm64(x, w)
    want = n.abs().amax(1) / 448
    fits = (want > 2.0 ** -125) & (want < 2.0 ** 127)      # scales that fp32 holds to its full precision
    fits[0] = False
    # products h w in range: h is below 8
    fits &= (x.double() * w.double()).abs().amax(1) < 2.0 ** 127.9
    assert bool(fits[1:].any()) or power == 127
    assert bool(((sc[fits].double() - want[fits]).abs() <= want[fits] * REL).all())
    _check_q(q[fits], n[fits] / sc[fits].double()[:, None])
    tiny = torch.isfinite(n[1]) & (n[1].abs() < 3e38)
    assert bool((y[1].double() - n[1]).abs()[tiny].le(n[1].abs()[tiny] * (2.0 ** -8 + REL) + 2.0 ** -133).all())
