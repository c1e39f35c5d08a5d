"""mxfp4_kv_append and mxfp4_kv_attention: the append bit for bit against the codec, the
attention against the formula in 64 bits over the decoded cache.

Bar of the attention. With A = sum_j p_j |v_j| / l (what the output would be if no value
cancelled): each weight is rounded to f16 once (2^-11) and carries the score's fp32 error
(at most 100 in sum_d |q_d k_d| scale here: 100 * 2^-21 < 2^-14) and ex2's (2^-22); weights
below 2^-40 of a block's largest value scale count as zero; then one bf16 rounding, 2^-8.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def B():
    from mxfp4_block_scaled_moe_b200 import binding
    return binding


def _decode(blocks, scales):
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device=blocks.device)
    v = torch.stack((grid[(blocks & 15).long()], grid[(blocks >> 4).long()]), -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _fresh(pages, Hkv, page, D):
    """A cache full of bytes that are no data: every scale byte 255, every code -6."""
    return [torch.full((pages, Hkv, page, d), 255, dtype=torch.uint8, device="cuda") for d in (D // 2, D // 32) * 2]


# -------------------------------------------------------------------------- append -----

@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 32, 16), (3, 8, 64, 16), (64, 8, 64, 64), (5, 2, 96, 32), (17, 3, 128, 256),
                                          (1000, 1, 64, 128), (7, 40, 256, 16)])
def test_append_matches_the_codec(B, T, Hkv, D, page):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    rows = torch.randn(T, 2 * Hkv * D + 8, generator=g, device="cuda")
    rows *= torch.exp2(torch.randint(-20, 20, (T, 1), generator=g, device="cuda").float())
    rows = rows.bfloat16()
    k, v = rows[:, :Hkv * D].view(T, Hkv, D), rows[:, Hkv * D:2 * Hkv * D].view(T, Hkv, D)
    pages = -(-T // page) + 2
    cache = _fresh(pages, Hkv, page, D)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    slots[T // 2] = -1
    B.mxfp4_kv_append(k, v, slots, *cache)
    B.mxmoe_check()
    want = _fresh(pages, Hkv, page, D)
    live = slots >= 0
    for i, x in ((0, k), (2, v)):
        blocks, scales = B.mxfp4_quantize(x.float().contiguous())
        want[i][slots[live] // page, :, slots[live] % page] = blocks[live]
        want[i + 1][slots[live] // page, :, slots[live] % page] = scales[live]
    for got, w in zip(cache, want):
        assert torch.equal(got, w)


def test_append_extreme_values(B):
    """Zeros of both signs, the least and largest bf16 values, ties between grid points."""
    D = 64
    x = torch.zeros(6, 1, D, device="cuda")
    x[0, 0, ::2] = -0.0
    x[1, 0] = 2.0 ** -133
    x[1, 0, 40:] = 2.0 ** -126
    x[2, 0] = 3.3895313892515355e38
    x[2, 0, 1] = -1.0
    x[3, 0] = torch.arange(D, device="cuda") / 8 - 4
    x[4, 0] = torch.arange(D, device="cuda") * 0.25 * 2.0 ** -60
    x[5, 0, 3] = -5.0
    x = x.bfloat16()
    cache = _fresh(1, 1, 16, D)
    B.mxfp4_kv_append(x, x, torch.arange(6, device="cuda"), *cache)
    blocks, scales = B.mxfp4_quantize(x.float().contiguous())
    for i in (0, 2):
        assert torch.equal(cache[i][0, 0, :6], blocks[:, 0]) and torch.equal(cache[i + 1][0, 0, :6], scales[:, 0])


def test_append_bad_slots_and_refusals(B):
    k = torch.ones(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    cache = _fresh(2, 2, 16, 64)
    before = [c.clone() for c in cache]
    B.mxfp4_kv_append(k, k, torch.tensor([32, 1 << 40, -5], device="cuda"), *cache)
    with pytest.raises(B.MxmoeError) as ei:
        B.mxmoe_check()
    assert ei.value.rc == B.EDEVICE
    B.mxmoe_check()
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: B.mxfp4_kv_append(k, k[:2], s, *cache), lambda: B.mxfp4_kv_append(k, k, s.int(), *cache),
                lambda: B.mxfp4_kv_append(k.float(), k, s, *cache), lambda: B.mxfp4_kv_append(k.transpose(1, 2), k, s, *cache),
                lambda: B.mxfp4_kv_append(k, k, s, cache[0], cache[1][:1], *cache[2:]),
                lambda: B.mxfp4_kv_append(k, k, s.cpu(), *cache)):
        with pytest.raises(ValueError):
            bad()
    odd = [torch.zeros(2, 2, 24, d, dtype=torch.uint8, device="cuda") for d in (32, 2, 32, 2)]
    with pytest.raises(B.MxmoeError) as ei:
        B.mxfp4_kv_append(k, k, s, *odd)
    assert ei.value.rc == B.EUNSUPPORTED
    B.mxfp4_kv_append(k[:0], k[:0], s[:0], *cache)


# ----------------------------------------------------------------------- attention -----

class Case:
    """A cache of garbage into which only the sequences' keys are appended."""

    def __init__(self, B, lens, Lq, Hq, Hkv, D, page, window=0, sinks=False, seed=0, kscale=1.0, vspread=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * D + page)
        self.n, self.Lq, self.Hq, self.Hkv, self.D, self.page, self.window = len(lens), Lq, Hq, Hkv, D, page, window
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        self.cache = _fresh(pages, Hkv, page, D)
        order = torch.randperm(pages, generator=g, device="cuda").cpu()
        table = torch.full((self.n, max(need + [1])), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
        self.table = table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            if n:
                pos = torch.arange(n, device="cuda")
                slots = self.table[b].long()[pos // page] * page + pos % page
                k = (kscale * torch.randn(n, Hkv, D, generator=g, device="cuda")).bfloat16()
                v = torch.randn(n, Hkv, D, generator=g, device="cuda")
                v = (v * torch.exp2(vspread * torch.randn(n, Hkv, 1, generator=g, device="cuda"))).bfloat16()
                B.mxfp4_kv_append(k, v, slots, *self.cache)
        self.q = torch.randn(self.n, Lq, Hq, D, generator=g, device="cuda").bfloat16()
        self.sinks = torch.randn(Hq, generator=g, device="cuda") if sinks else None
        B.mxmoe_check()

    def run(self, B, **kw):
        return B.mxfp4_kv_attention(self.q, *self.cache, self.table, self.lens, window=self.window, sinks=self.sinks, **kw)

    def check(self, out, scale=None, hide=()):
        """hide: (sequence, page number) pairs that count as unseen."""
        lens, table = self.lens.tolist(), self.table.long()
        G = self.Hq // self.Hkv
        scale = self.D ** -0.5 if scale is None else scale
        for b, n in enumerate(lens):
            n = max(0, min(n, table.shape[1] * self.page))
            used = table[b, :-(-n // self.page)].clamp(0, self.cache[0].shape[0] - 1)
            k = _decode(self.cache[0][used], self.cache[1][used]).transpose(1, 2).flatten(0, 1)[:n]   # (n, Hkv, D)
            v = _decode(self.cache[2][used], self.cache[3][used]).transpose(1, 2).flatten(0, 1)[:n]
            pos = torch.arange(n, device="cuda")
            gone = torch.zeros(n, dtype=torch.bool, device="cuda")
            for hb, hp in hide:
                if hb == b:
                    gone |= pos // self.page == hp
            for i in range(self.Lq):
                p = n - self.Lq + i
                seen = (pos <= p) & ~gone
                if self.window:
                    seen &= pos > p - self.window
                kk, vv = k[seen], v[seen]
                q = self.q[b, i].double().view(self.Hkv, G, self.D)
                z = torch.einsum("hgd,nhd->hgn", q, kk) * scale
                if self.sinks is not None:
                    z = torch.cat((z, self.sinks.double().view(self.Hkv, G, 1)), -1)
                w = torch.softmax(z, -1)[..., :kk.shape[0]] if z.shape[-1] else z
                ref = torch.einsum("hgn,nhd->hgd", w, vv).reshape(self.Hq, self.D)
                mag = torch.einsum("hgn,nhd->hgd", w, vv.abs()).reshape(self.Hq, self.D)
                err = (out.view(self.n, self.Lq, self.Hq, self.D)[b, i].double() - ref).abs()
                floor = 2.0 ** -36 * (float(vv.abs().max()) if vv.numel() else 0.0)
                ok = err <= ref.abs() * 2.0 ** -8 + mag * (2.0 ** -11 + 2.0 ** -13) + floor
                assert bool(ok.all()), (b, i, n, float((err - ref.abs() * 2.0 ** -8).max()), float(mag.max()))


CASES = [
    dict(lens=[1], Lq=1, Hq=8, Hkv=1, D=64, page=16),
    dict(lens=[0], Lq=1, Hq=1, Hkv=1, D=64, page=16),
    dict(lens=[31, 32, 33, 16, 17, 0, 5], Lq=1, Hq=8, Hkv=1, D=64, page=16),
    dict(lens=[2000], Lq=1, Hq=64, Hkv=8, D=64, page=16, sinks=True),
    dict(lens=[5000, 3, 700, 0, 1], Lq=1, Hq=64, Hkv=8, D=64, page=64, sinks=True),
    dict(lens=[777, 1200], Lq=1, Hq=16, Hkv=4, D=128, page=128),
    dict(lens=[777, 1200], Lq=1, Hq=4, Hkv=4, D=128, page=32, sinks=True),
    dict(lens=[300, 90], Lq=1, Hq=20, Hkv=4, D=64, page=32),
    dict(lens=[300, 90], Lq=1, Hq=48, Hkv=3, D=64, page=32),                 # 16 rows
    dict(lens=[411, 90], Lq=1, Hq=40, Hkv=2, D=128, page=256),               # 20 rows, two row tiles
    dict(lens=[300, 2, 4, 0, 1], Lq=4, Hq=16, Hkv=2, D=64, page=16, sinks=True),
    dict(lens=[300, 2, 4, 0, 1], Lq=4, Hq=6, Hkv=2, D=128, page=16),
    dict(lens=[130, 50], Lq=33, Hq=8, Hkv=4, D=64, page=64),
    dict(lens=[1000, 128, 129, 127, 1], Lq=1, Hq=64, Hkv=8, D=64, page=16, window=128, sinks=True),
    dict(lens=[1000, 40, 3], Lq=3, Hq=8, Hkv=2, D=128, page=32, window=37),
    dict(lens=[500, 33], Lq=2, Hq=8, Hkv=1, D=64, page=16, window=1),
    dict(lens=[150 + i % 90 for i in range(120)], Lq=1, Hq=16, Hkv=8, D=64, page=16, window=128, sinks=True),
    dict(lens=[150 + i % 90 for i in range(400)], Lq=1, Hq=16, Hkv=8, D=64, page=16, window=128),
    dict(lens=[90, 0, 64, 5], Lq=1, Hq=8, Hkv=1, D=128, page=32, sinks=True),             # a short table
    dict(lens=[90, 0, 64, 5] * 90, Lq=1, Hq=16, Hkv=8, D=128, page=32),
    dict(lens=[20000], Lq=1, Hq=8, Hkv=1, D=64, page=256),
    dict(lens=[9] * 700, Lq=1, Hq=2, Hkv=2, D=64, page=16),
    dict(lens=[40000, 11], Lq=2, Hq=8, Hkv=2, D=128, page=64),
    dict(lens=[600, 35], Lq=1, Hq=8, Hkv=2, D=64, page=16, kscale=3.0, vspread=6.0),
    dict(lens=[600, 35], Lq=1, Hq=8, Hkv=2, D=128, page=16, kscale=3.0, vspread=6.0),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(B, case):
    c = Case(B, **case)
    out = c.run(B)
    B.mxmoe_check()
    assert out.shape == c.q.shape and out.dtype == torch.bfloat16
    c.check(out)
    assert torch.equal(c.run(B), out)


@pytest.mark.parametrize("n", [31, 32, 33, 64, 65, 127, 128, 129, 256, 385])
@pytest.mark.parametrize("Hq,Hkv,D,Lq", [(5, 1, 64, 1), (14, 2, 128, 1), (6, 2, 64, 7)])
def test_attention_many_sequences(B, n, Hq, Hkv, D, Lq):
    """Long runs over many uneven sequences, empty ones and stretches of them among them, so that a
    warp's first unit can lie in any sequence; groups and row counts that are no power of two."""
    lens = [0 if i % 7 == 3 or 40 <= i < 75 else 1 + (i * i * 37) % (900 if i % 5 else 40) for i in range(n)]
    c = Case(B, lens, Lq, Hq, Hkv, D, 16, sinks=True)
    out = c.run(B)
    B.mxmoe_check()
    c.check(out)
    assert torch.equal(c.run(B), out)


def test_attention_scale_strides_and_three_dims(B):
    c = Case(B, [70, 200], 1, 16, 2, 64, 32)
    wide = torch.randn(2, 16 * 64 + 256, device="cuda").bfloat16()
    q3 = wide[:, 128:128 + 16 * 64].view(2, 16, 64)
    assert not q3.is_contiguous()
    c.q = q3[:, None]
    out = B.mxfp4_kv_attention(q3, *c.cache, c.table, c.lens, scale=0.3)
    assert out.shape == (2, 16, 64)
    c.check(out, scale=0.3)
    ws = torch.empty(B.mxfp4_kv_attention_workspace(2, 1, 16, 2, 64), dtype=torch.uint8, device="cuda")
    buf = torch.empty_like(out)
    assert torch.equal(B.mxfp4_kv_attention(q3, *c.cache, c.table, c.lens, scale=0.3, out=buf, workspace=ws), out)


def test_attention_query_magnitudes(B):
    """Rows of very different size, and blocks within a row: the scores are still fp32."""
    c = Case(B, [500], 1, 8, 1, 64, 16)
    f = torch.tensor([1.0, 2.0 ** 40, 2.0 ** -40, 0.0, 2.0 ** -126, 1.0, 1.0, 1.0], device="cuda")
    q = c.q.float() * f[:, None]
    q[0, 0, 5, :32] *= 2.0 ** -30
    c.q = q.bfloat16()
    out = c.run(B)
    # a score of 2^40 picks one key: the bar on weights holds as long as no two scores tie
    c.check(out)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30])
def test_attention_unusual_scales(B, scale):
    c = Case(B, [70, 33, 500], 1, 8, 2, 64, 16, window=40, sinks=True)
    c.check(c.run(B, scale=scale), scale=scale)


def test_attention_sinks_alone_and_extreme_sinks(B):
    c = Case(B, [0, 40], 1, 8, 1, 64, 16, sinks=True)
    c.sinks = torch.tensor([-math.inf, -1e30, -200.0, 0.0, 200.0, 1e30, 3.0, -3.0], device="cuda")
    out = c.run(B)
    assert not bool(out[0].any())
    c.check(out)


def test_nan_stays_in_its_row(B):
    c = Case(B, [100], 1, 8, 1, 64, 16)
    want = c.run(B)
    c.q[0, 0, 3, 5] = float("nan")
    out = c.run(B)
    assert bool(out[0, 0, 3].isnan().all())
    keep = [i for i in range(8) if i != 3]
    assert torch.equal(out[0, 0, keep], want[0, 0, keep])


def test_offsets_past_32_bits(B):
    """Codes of more than 4 GiB each for keys and values: the last pages are reached."""
    page, Hkv, D, n = 256, 8, 64, 700
    pages = (1 << 32) // (Hkv * page * D // 2) + 5
    cache = [torch.empty(pages, Hkv, page, d, dtype=torch.uint8, device="cuda") for d in (D // 2, D // 32) * 2]
    assert cache[0].numel() > 1 << 32
    c = Case(B, [n], 1, 64, Hkv, D, page)
    table = torch.tensor([[pages - 1, 2, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = table[0].long()[pos // page] * page + pos % page
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(n, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    B.mxfp4_kv_append(k, v, slots, *cache)
    small = [torch.empty(3, Hkv, page, d, dtype=torch.uint8, device="cuda") for d in (D // 2, D // 32) * 2]
    B.mxfp4_kv_append(k, v, pos, *small)
    for big, s in zip(cache, small):
        for i, p in enumerate(table[0].tolist()):
            m = min(page, n - i * page)
            assert torch.equal(big[p, :, :m], s[i, :, :m])
    want = B.mxfp4_kv_attention(c.q, *small, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), c.lens)
    assert torch.equal(B.mxfp4_kv_attention(c.q, *cache, table, c.lens), want)
    B.mxmoe_check()


def test_attention_pages_that_are_gone(B):
    c = Case(B, [900, 64], 2, 16, 2, 64, 16, window=100)
    keep = c.table.clone()
    c.table[0, :(900 - 2 + 1 - 100) // 16] = -1           # wholly before the first query's window
    out = c.run(B)
    B.mxmoe_check()
    c.table = keep
    c.check(out)
    c.table = keep.clone()
    c.table[0, 54] = c.cache[0].shape[0]                   # a page that is needed, past the cache
    c.table[1, 3] = -7
    out = c.run(B)
    with pytest.raises(B.MxmoeError) as ei:
        B.mxmoe_check()
    assert ei.value.rc == B.EDEVICE
    c.check(out, hide=((0, 54), (1, 3)))


def test_attention_lengths_out_of_range(B):
    c = Case(B, [128, 60], 1, 8, 1, 64, 32)
    c.lens = torch.tensor([1000, -3], dtype=torch.int32, device="cuda")    # past the table; negative
    out = c.run(B)
    with pytest.raises(B.MxmoeError) as ei:
        B.mxmoe_check()
    assert ei.value.rc == B.EDEVICE
    assert not bool(out[1].any())
    c.check(out)


def test_attention_captured_follows_lengths(B):
    c = Case(B, [3000, 2500], 1, 64, 8, 64, 64, sinks=True)
    c.run(B)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.run(B)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        out2 = c.run(B, scale=0.05)
    for lens in ([3000, 2500], [5, 2100], [0, 33], [2999, 1]):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        c.check(out)
        c.check(out2, scale=0.05)
    B.mxmoe_check()


def test_attention_on_two_streams_at_once(B):
    c = [Case(B, [4000, 3000, 17], 1, 64, 8, 64, 64, seed=i) for i in range(2)]
    want = [x.run(B) for x in c]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(c[i].run(B, stream=s[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_attention_refusals(B):
    c = Case(B, [40], 1, 8, 2, 64, 16)
    args = lambda **k: B.mxfp4_kv_attention(*[k.get(n, d) for n, d in zip(
        ("q", "kb", "ks", "vb", "vs", "table", "lens"), (c.q, *c.cache, c.table, c.lens))])
    for bad in (dict(q=c.q.float()), dict(q=c.q[..., :32]), dict(table=c.table.long()), dict(lens=c.lens[:0]),
                dict(table=c.table[0]), dict(q=c.q.transpose(2, 3)), dict(ks=c.cache[0]), dict(lens=c.lens.cpu())):
        with pytest.raises(ValueError):
            args(**bad)
    for rc, kw in ((B.EINVAL, dict(window=-1)), (B.EINVAL, dict(scale=math.inf)),
                   (B.EINVAL, dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(B.MxmoeError) as ei:
            B.mxfp4_kv_attention(c.q, *c.cache, c.table, c.lens, **kw)
        assert ei.value.rc == rc
    with pytest.raises(B.MxmoeError) as ei:
        B.mxfp4_kv_attention(c.q[:, :, :7].contiguous(), *c.cache, c.table, c.lens)
    assert ei.value.rc == B.EINVAL
    wide = [torch.zeros(1, 2, 16, d, dtype=torch.uint8, device="cuda") for d in (48, 3, 48, 3)]
    with pytest.raises(B.MxmoeError) as ei:
        B.mxfp4_kv_attention(torch.zeros(1, 8, 96, dtype=torch.bfloat16, device="cuda"), *wide, c.table, c.lens)
    assert ei.value.rc == B.EUNSUPPORTED
    e = c.q[:0]
    assert B.mxfp4_kv_attention(e, *c.cache, c.table[:0], c.lens[:0]).shape == e.shape


@pytest.mark.parametrize("D", [64, 96])
def test_append_nonfinite_values_match_the_codec(B, D):
    """NaN of either sign and infinities, alone in a block, with numbers, and blocks of nothing else."""
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn(40, 3, D, generator=g, device="cuda").bfloat16()
    bits = x.view(torch.int16)
    nan = torch.tensor([0x7FC0, -0x40, 0x7F81, -0x7F, 0x7FFF, -1], dtype=torch.int16, device="cuda")
    bits[:6, 0, 5] = nan
    bits[6:12, 1, 32:] = nan[:, None]
    bits[12:18, :, ::3] = nan[:, None, None]
    x[18:20, 0, 1], x[20:22, 2, 33] = math.inf, -math.inf
    x[22, 1, 0], x[22, 1, 1] = math.inf, math.nan
    x[23, 0, :] = 0.0
    x[23, 0, 2] = math.nan
    cache = _fresh(3, 3, 16, D)
    B.mxfp4_kv_append(x, x, torch.arange(40, device="cuda"), *cache)
    B.mxmoe_check()
    blocks, scales = B.mxfp4_quantize(x.float().contiguous())
    for i in (0, 2):
        for got, want in ((cache[i], blocks), (cache[i + 1], scales)):
            assert torch.equal(got.transpose(1, 2).flatten(0, 1)[:40], want)


def test_one_head_cut_from_wider_rows(B):
    """A single key/value head (or query head): the stride of an axis of one element has no meaning."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(2, 20, 320, generator=g, device="cuda").bfloat16()
    k, v, q = (rows[0, :, a:a + 64].unsqueeze(0).transpose(0, 1) for a in (0, 64, 128))       # (20, 1, 64)
    assert k.stride(1) != 64 and not k.is_contiguous()
    cache, want = _fresh(2, 1, 16, 64), _fresh(2, 1, 16, 64)
    slots = torch.arange(20, device="cuda")
    B.mxfp4_kv_append(k, v, slots, *cache)
    B.mxfp4_kv_append(k.contiguous(), v.contiguous(), slots, *want)
    assert all(torch.equal(a, b) for a, b in zip(cache, want))
    table, lens = torch.tensor([[0, 1]] * 20, dtype=torch.int32, device="cuda"), 1 + slots.int()
    assert torch.equal(B.mxfp4_kv_attention(q, *cache, table, lens), B.mxfp4_kv_attention(q.contiguous(), *cache, table, lens))
    B.mxmoe_check()


@pytest.mark.parametrize("n", [31, 129, 256, 257, 385, 600])
@pytest.mark.parametrize("Hq,Hkv,Lq", [(20, 2, 1), (6, 2, 3)])
def test_attention_many_sequences_in_eight_warps(B, n, Hq, Hkv, Lq):
    """As above for 9 to 16 rows of 128 columns, whose CTAs have 256 threads: their search over the sequences
    takes one chunk of them, or several."""
    lens = [0 if i % 7 == 3 or 40 <= i < 75 else 1 + (i * i * 37) % (700 if i % 5 else 40) for i in range(n)]
    c = Case(B, lens, Lq, Hq, Hkv, 128, 16, sinks=True)
    out = c.run(B)
    B.mxmoe_check()
    c.check(out)
    assert torch.equal(c.run(B), out)


@pytest.mark.parametrize("case", [dict(lens=[150, 40], Lq=128, Hq=8, Hkv=2, D=64, page=32),
                                  dict(lens=[260], Lq=128, Hq=1, Hkv=1, D=128, page=16, window=50, sinks=True),
                                  dict(lens=[70], Lq=3, Hq=1024, Hkv=1, D=64, page=16),
                                  dict(lens=[70, 33], Lq=1, Hq=1024, Hkv=1024, D=64, page=16, sinks=True)])
def test_attention_most_queries_and_heads(B, case):
    c = Case(B, **case)
    out = c.run(B)
    B.mxmoe_check()
    c.check(out)


@pytest.mark.parametrize("width", [1, 40])
def test_attention_most_sequences(B, width):
    """65,536 sequences of up to 16 keys, over a table of one page each (items stay in a CTA) and a wide one
    (a line of units); every one against the same keys read from another place of the batch."""
    n, page = 65536, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = _fresh(64, 1, page, 64)
    k, v = (torch.randn(64 * page, 1, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    B.mxfp4_kv_append(k, v, torch.arange(64 * page, device="cuda"), *cache)
    seq = torch.arange(n, device="cuda")
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = seq % 64
    lens = ((seq // 64) % 17).int()
    q = torch.randn(64, 17, 2, 64, generator=g, device="cuda").bfloat16()[seq % 64, (seq // 64) % 17]
    out = B.mxfp4_kv_attention(q, *cache, table, lens)
    B.mxmoe_check()
    some = 64 * 17
    want = B.mxfp4_kv_attention(q[:some], *cache, table[:some, :1].contiguous(), lens[:some])
    assert torch.equal(out[:some // 64 * 64], want) or float((out[:some] - want).abs().max()) < 2.0 ** -6
    for i in range(0, n, some):
        assert torch.equal(out[i:i + some].view(torch.int16), out[:min(some, n - i)].view(torch.int16))
    assert not bool(out[lens == 0].any())
