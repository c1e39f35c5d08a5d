"""mxfp4_kv_attention at the ends of its ranges: the least values a cache holds, keys that only some of
a call's queries see, lengths near the largest.

Bar: that of test_gpu_kv_cache.py (a bf16 rounding, 2^-8; 11-bit weights and the scores' error,
2^-11 + 2^-13 of the sum of magnitudes; 2^-36 of the largest value that the query sees), and half of
bf16's least step, 2^-134, with as much again for the fp32 sums' own least step.
"""
import pytest
import torch

from test_gpu_kv_cache import Case, _decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mxfp4_block_scaled_moe_b200 import binding
    return binding


def check(c, out, queries=None):
    """Every query of the case (or those (sequence, query) given) against the formula in 64 bits, a
    32-column block of a key/value head at a time for the values' size."""
    lens, G = c.lens.tolist(), c.Hq // c.Hkv
    for b, n in enumerate(lens):
        used = c.table[b, :-(-n // c.page)].long()
        k, v = (_decode(c.cache[i][used], c.cache[i + 1][used]).transpose(1, 2).flatten(0, 1)[:n] for i in (0, 2))
        pos = torch.arange(n, device="cuda")
        for i in range(c.Lq):
            if queries is not None and (b, i) not in queries:
                continue
            p = n - c.Lq + i
            seen = (pos <= p) & (pos > p - c.window) if c.window else pos <= p
            kk, vv = k[seen], v[seen]
            z = torch.einsum("hgd,nhd->hgn", c.q[b, i].double().view(c.Hkv, G, c.D), kk) * c.D ** -0.5
            if c.sinks is not None:
                z = torch.cat((z, c.sinks.double().view(c.Hkv, G, 1)), -1)
            w = torch.softmax(z, -1)[..., :kk.shape[0]]
            ref = torch.einsum("hgn,nhd->hgd", w, vv)
            mag = torch.einsum("hgn,nhd->hgd", w, vv.abs())
            top = vv.abs().amax(0).unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)[:, None] if kk.shape[0] else 0.0
            err = (out.view(c.n, c.Lq, c.Hkv, G, c.D)[b, i].double() - ref).abs()
            ok = err <= ref.abs() * 2.0 ** -8 + mag * (2.0 ** -11 + 2.0 ** -13) + top * 2.0 ** -36 + 2.0 ** -133
            assert bool(ok.all()), (b, i, n, float(err.max()), float(ref.abs().max()))


@pytest.mark.parametrize("less", [90, 105, 112, 118, 124, 127])
@pytest.mark.parametrize("D,lens,Hq,window", [(64, [90, 700], 16, 0), (128, [5000, 40], 8, 0), (64, [2000], 16, 100),
                                              (64, [300], 48, 0)])
def test_small_values(B, D, lens, Hq, window, less):
    """Value scale bytes down to 0, by each way an output is written (by the warp that holds its item, by
    the joining kernel, by warps that share an item)."""
    c = Case(B, lens, 1, Hq, 2, D, 16, window=window, sinks=True, vspread=1.0)
    s = c.cache[3]
    c.cache[3] = torch.where(s == 255, s.int(), (s.int() - less).clamp(min=0)).to(torch.uint8)
    out = c.run(B)
    B.mxmoe_check()
    assert bool(out.any())
    check(c, out)


def _slots(c, b, pos):
    return c.table[b].long()[pos // c.page] * c.page + pos % c.page


HIDDEN = [dict(Lq=2, Hq=16, Hkv=2, D=64, page=64, window=0), dict(Lq=2, Hq=8, Hkv=2, D=128, page=16, window=0),
          dict(Lq=3, Hq=8, Hkv=2, D=64, page=16, window=100), dict(Lq=4, Hq=8, Hkv=2, D=128, page=32, window=37),
          dict(Lq=2, Hq=48, Hkv=2, D=64, page=32, window=0), dict(Lq=5, Hq=6, Hkv=2, D=128, page=16, window=600),
          dict(Lq=17, Hq=4, Hkv=2, D=64, page=64, window=0), dict(Lq=2, Hq=8, Hkv=1, D=64, page=16, window=1)]


@pytest.mark.parametrize("case", HIDDEN, ids=[str(i) for i in range(len(HIDDEN))])
@pytest.mark.parametrize("what", ["inf", "nan", "3e38", "1e6"])
@pytest.mark.parametrize("lens", [[1000, 33, 300], [4, 64, 9000, 65], [128] * 40])
def test_a_key_that_is_hidden_from_a_query_leaves_it_alone(B, case, what, lens):
    """The last token's key and value are no numbers, or huge, in some elements: queries before it do not see
    it, whatever the later ones of the same call make of it. The same of the first token in the first
    query's window, which the later ones no longer see."""
    c = Case(B, lens, sinks=True, seed=5, **case)
    bad = torch.full((1, c.Hkv, c.D), float(what), device="cuda").bfloat16()
    bad[:, :, 5:].mul_(0.0 if what == "1e6" else 1.0)        # an outlier in one block only, or all of them
    if what in ("inf", "nan"):
        bad[:, :, 40:] = 1.0
    for place in ("last", "first"):
        c = Case(B, lens, sinks=True, seed=5, **case)
        for b, n in enumerate(lens):
            at = n - 1 if place == "last" else n - c.Lq + 1 - c.window
            if at >= 0 and (place == "last" or c.window):
                B.mxfp4_kv_append(bad, bad, _slots(c, b, torch.tensor([at], device="cuda")), *c.cache)
        out = c.run(B)
        B.mxmoe_check()
        first, last = (0, c.Lq - 1) if place == "last" else (1, c.Lq)
        check(c, out, {(b, i) for b in range(len(lens)) for i in range(first, last)})
        assert torch.equal(c.run(B).view(torch.int16), out.view(torch.int16))


def test_queries_on_both_sides_of_a_huge_value(B):
    """Queries that see a value 2^60 above the rest beside queries that do not: both are right."""
    for D in (64, 128):
        c = Case(B, [500, 70, 2000], 4, 8, 2, D, 16, sinks=True, seed=2)
        for b, n in enumerate([500, 70, 2000]):
            v = torch.full((1, 2, D), 2.0 ** 60, device="cuda").bfloat16()
            k = torch.zeros_like(v)
            B.mxfp4_kv_append(k, v, _slots(c, b, torch.tensor([n - 2], device="cuda")), *c.cache)
        out = c.run(B)
        B.mxmoe_check()
        check(c, out)


@pytest.mark.parametrize("n", [(1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 31) - 600, (1 << 31) - 1])
@pytest.mark.parametrize("Lq,G", [(1, 8), (2, 4)])
def test_longest_sequences(B, n, Lq, G):
    """Lengths up to the largest int32 over a table that holds as many (its pages repeat, a window keeps the
    work small): 2^30 keys are taken, a longer length is cut to them and reported."""
    page, window, keep = 256, 40, min(n, 1 << 30)
    c = Case(B, [3 * page], Lq, G, 1, 64, page, window=window)
    table = c.table[0, torch.arange(-(-n // page), device="cuda") % 3][None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = B.mxfp4_kv_attention(c.q, *c.cache, table, lens, window=window)
    if n > 1 << 30:
        with pytest.raises(B.MxmoeError) as ei:
            B.mxmoe_check()
        assert ei.value.rc == B.EDEVICE
    B.mxmoe_check()
    # the same keys of a short sequence: the window's pages in their order
    last = (keep - 1) // page
    short = torch.tensor([[table[0, last - 1], table[0, last]]], dtype=torch.int32, device="cuda")
    want = B.mxfp4_kv_attention(c.q, *c.cache, short, torch.tensor([keep - (last - 1) * page], dtype=torch.int32, device="cuda"),
                                window=window)
    B.mxmoe_check()
    assert torch.equal(out, want)


@pytest.mark.parametrize("seed", range(40))
def test_random_calls_with_outliers(B, seed):
    """Shapes, windows and lengths at random, some keys' values 2^-20 to 2^50 of the rest, most of them where
    the queries of a call begin or end to differ in what they see."""
    import random
    r = random.Random(seed)
    D, Hkv, G, Lq = r.choice((64, 128)), r.choice((1, 2, 3)), r.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 20)), r.choice((1, 2, 2, 3, 5, 17))
    page, window = r.choice((16, 32, 64, 128, 256)), r.choice((0, 0, 1, 5, 37, 64, 100, 700))
    n = r.choice((1, 2, 5, 40, 130))
    top = r.choice((3, 40, 130, 700, 3000)) // (4 if n > 5 else 1) + 1
    lens = [r.choice((0, 1, Lq, Lq + 1, top, r.randint(0, top))) for _ in range(n)]
    c = Case(B, lens, Lq, Hkv * G, Hkv, D, page, window=window, sinks=r.random() < 0.5, seed=seed, vspread=float(r.choice((0, 1, 3))))
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b in range(min(n, 8)):
        for _ in range(r.choice((0, 1, 2, 4)) if lens[b] else 0):
            at = r.choice((lens[b] - 1, lens[b] - 2, lens[b] - Lq - window, lens[b] - Lq - window + 1, r.randint(0, lens[b] - 1)))
            v = torch.randn(1, Hkv, D // 32, 32, generator=g, device="cuda")
            v[:, :, r.randrange(D // 32):] *= 2.0 ** r.choice((-20, 5, 6, 20, 50))
            k = torch.randn(1, Hkv, D, generator=g, device="cuda").bfloat16()
            place = torch.tensor([min(max(at, 0), lens[b] - 1)], device="cuda")
            B.mxfp4_kv_append(k, v.flatten(2).bfloat16(), _slots(c, b, place), *c.cache)
    out = c.run(B)
    B.mxmoe_check()
    check(c, out, {(b, i) for b in range(min(n, 10)) for i in range(Lq)})
    assert torch.equal(c.run(B), out)
