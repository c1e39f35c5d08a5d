"""The operators together, as a decoder layer uses them: norm -> FP8 Q/K/V product -> cache
append -> attention over the 4-bit cache -> FP8 cast -> O product with the residual -> norm ->
expert layer; a prefill chunk, then decode steps, the last of them captured.

The reference is the same chain in 64 bits, rounded where the operators round (bf16 stream,
E4M3 codes, MXFP4 cache). The two differ where a value lies within an fp32 rounding (about
2^-22) of a rounding border: for a step of 2^-8 (bf16) that is one element in 2^13, of 2^-4
(E4M3) one in 2^17, and such an element is off by one step; an MXFP4 element by up to a third.
In 2-norm that is below sqrt(2^-13) 2^-8 + sqrt(2^-17) 2^-3 (E4M3 and MXFP4 steps on the
bf16 flips before them: sqrt(2^-13) again) < 2^-9 a stage; six stages, the attention's
11-bit weights (2^-11) and the outputs' own bf16 flips stay below 2^-6.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, PAGE, EPS = 512, 16, 2, 64, 16, 1e-5
QKV = (HQ + 2 * HKV) * D
BAR = 2.0 ** -6


@pytest.fixture(scope="module")
def B():
    from mxfp4_block_scaled_moe_b200 import binding
    return binding


def _bf16(v):
    return v.to(torch.bfloat16).double()


def _e4m3(v):
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _mxfp4(v):
    v = v.unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 2, -127.0).clamp(-127, 127))
    r = (v / s).abs()
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).double()
    return (torch.copysign((torch.round(r / step) * step).clamp(max=6), v) * s).flatten(-2)


def _norm(h, w):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w.double()


class Layer:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.n1, self.n2 = (1 + 0.1 * rnd(H)).bfloat16(), (1 + 0.1 * rnd(H)).bfloat16()
        w, o = 0.05 * rnd(QKV, H), 0.03 * rnd(H, HQ * D)
        self.ws, self.os = w.abs().amax(1) / 448, float(o.abs().max()) / 448
        self.w = (w / self.ws[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.o = (o / self.os).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.wb, self.ob = 0.1 * rnd(QKV), 0.1 * rnd(H)
        self.sinks = rnd(HQ)
        self.as_ = 0.01

    def run(self, B, x, res, cache, table, lens, slots, Lq):
        """x, res (tokens, H) bf16 -> (the stream after attention, the expert layer's input)"""
        q, s, res = B.rmsnorm_residual_fp8(x, self.n1, res, EPS)
        qkv = B.fp8_linear_fused(q, self.w, s, self.ws, bias=self.wb).view(-1, HQ + 2 * HKV, D)
        B.mxfp4_kv_append(qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], slots, *cache)
        a = B.mxfp4_kv_attention(qkv[:, :HQ].unflatten(0, (-1, Lq)), *cache, table, lens, window=48, sinks=self.sinks)
        aq = B.moe_fp8_quantize(a.view(-1, HQ * D), self.as_)
        return B.fp8_linear_fused(aq, self.o, self.as_, self.os, bias=self.ob, residual=res, out=res), \
            B.rmsnorm_residual(res, self.n2, eps=EPS)[0]

    def ref(self, x, res, past, Lq):
        """past: one (k, v) of decoded (tokens, HKV, D) per sequence, extended in place"""
        h = _bf16(x + res)
        n = _norm(h, self.n1)
        s = n.abs().amax(1, keepdim=True) / 448
        w = self.w.view(torch.float8_e4m3fn).double() * self.ws.double()[:, None]
        qkv = _bf16(_e4m3(n / s) * s @ w.t() + self.wb.double()).view(-1, HQ + 2 * HKV, D)
        out = []
        for b in range(len(past)):
            rows = qkv[b * Lq:(b + 1) * Lq]
            k, v = (torch.cat((p, _mxfp4(c))) for p, c in zip(past[b], (rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:])))
            past[b] = (k, v)
            at = torch.arange(k.shape[0], device="cuda")
            for i in range(Lq):
                p = k.shape[0] - Lq + i
                seen = (at <= p) & (at > p - 48)
                z = torch.einsum("hgd,nhd->hgn", rows[i, :HQ].view(HKV, HQ // HKV, D), k[seen]) / math.sqrt(D)
                z = torch.cat((z, self.sinks.double().view(HKV, -1, 1)), -1)
                out.append(torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1)[..., :-1], v[seen]).reshape(-1))
        a = _e4m3(_bf16(torch.stack(out)) / self.as_) * self.as_
        o = self.o.view(torch.float8_e4m3fn).double() * self.os
        h = _bf16(a @ o.t() + self.ob.double() + h)
        return h, _bf16(_norm(h, self.n2))


def _near(got, want):
    return float((got.double() - want).norm() / want.norm()) < BAR


def test_a_layer_over_prefill_and_decode(B):
    L, nseq, chunk, steps = Layer(), 3, 37, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    pages = -(-(chunk + steps) // PAGE)
    cache = [torch.full((nseq * pages, HKV, PAGE, d), 255, dtype=torch.uint8, device="cuda") for d in (D // 2, D // 32) * 2]
    table = torch.randperm(nseq * pages, generator=g, device="cuda").view(nseq, pages).int()
    lens = torch.zeros(nseq, dtype=torch.int32, device="cuda")
    past = [(torch.zeros(0, HKV, D, dtype=torch.float64, device="cuda"),) * 2 for _ in range(nseq)]

    def slots(first, n):
        pos = first + torch.arange(n, device="cuda")
        return (table[:, pos // PAGE].long() * PAGE + pos % PAGE).reshape(-1)

    def stream(n):
        return [torch.randn(nseq * n, H, generator=g, device="cuda").bfloat16() for _ in range(2)]

    x, res = stream(chunk)
    lens += chunk
    want = L.ref(x.double(), res.double(), past, chunk)
    got = L.run(B, x, res, cache, table, lens, slots(0, chunk), chunk)
    assert _near(got[0], want[0]) and _near(got[1], want[1])

    x, res = stream(1)
    sl = slots(chunk, 1)
    for step in range(steps):
        if step == 2:                      # from here on by replays: lengths and slots are read on the device
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = L.run(B, x, res, cache, table, lens, sl, 1)
        for t, new in zip((x, res), stream(1)):
            t.copy_(new)
        sl.copy_(slots(chunk + step, 1))
        lens += 1
        want = L.ref(x.double(), res.double(), past, 1)
        if step < 2:
            got = L.run(B, x, res, cache, table, lens, sl, 1)
        else:
            graph.replay()
        assert _near(got[0], want[0]) and _near(got[1], want[1]), step
    B.mxmoe_check()


def test_the_norm_feeds_the_expert_layer(B):
    """The norm's bf16 output into moe_mxfp4_forward, its FP8 codes next to it: one launch makes
    both, and the layer's A-FP8 input is those codes."""
    from mxfp4_block_scaled_moe_b200 import inputs
    lay = inputs.tiny_layer(seed=0)
    h = lay.H
    g = torch.Generator(device="cuda").manual_seed(4)
    x, res = (torch.randn(lay.T, h, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(h, device="cuda", dtype=torch.bfloat16)
    y = torch.empty_like(x)
    q, _, s = B.rmsnorm_residual_fp8(x, w, res, act_scale=0.02, y=y)
    y2, s2 = B.rmsnorm_residual(x, w, res)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    gu = [B.mxfp4_quantize(lay.gate_up(e).cuda().contiguous()) for e in range(lay.E)]
    dn = [B.mxfp4_quantize(lay.down(e).cuda().contiguous()) for e in range(lay.E)]
    pack = lambda ws, i: torch.stack([p[i] for p in ws]).contiguous()
    out = B.moe_mxfp4_forward(y, lay.router_w.cuda(), lay.router_b.cuda(), pack(gu, 0), pack(gu, 1), lay.gu_bias.cuda(),
                              pack(dn, 0), pack(dn, 1), lay.d_bias.cuda(), lay.k)
    B.mxmoe_check()
    assert out.shape == x.shape and bool(out.isfinite().all())
    # the codes are those of the norm itself: one E4M3 step of the cast of its bf16 rounding at most
    a, b = q.view(torch.float8_e4m3fn).float(), B.moe_fp8_quantize(y, 0.02).view(torch.float8_e4m3fn).float()
    assert bool(((a - b).abs() <= 2.0 ** -3 * b.abs() + 2.0 ** -9).all())


@pytest.mark.parametrize("T,E,H,I", [(1, 8, 320, 192), (8, 4, 256, 256), (16, 4, 256, 256), (40, 8, 320, 192), (77, 8, 320, 192),
                                     (77, 8, 352, 224)])
def test_the_norm_and_the_expert_layer_against_the_oracle(B, T, E, H, I):
    """Norm -> expert layer -> norm with the layer's output added to the stream, eager and replayed with new
    inputs: the norm lets its successor start early, and each path of the layer reads what it wrote. The
    layer's output is checked against the oracle on the norm's output."""
    import numpy as np
    import test_gpu_layer as TL
    from mxfp4_block_scaled_moe_b200 import inputs
    p = TL.pack(inputs.small_layer(E=E, k=2, T=T, H=H, I=I, seed=3, router_bias=True))
    d = TL.to_device(p)
    g = torch.Generator(device="cuda").manual_seed(T)
    w1, w2 = ((1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16() for _ in range(2))
    x, res = (torch.empty(T, H, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    y, out, s1 = (torch.empty_like(x) for _ in range(3))

    def layer():
        B.rmsnorm_residual(x, w1, res, sum_out=s1, y=y)
        B.moe_mxfp4_forward(y, d["router_w"], d["router_b"], d["gu_blocks"], d["gu_scales"], d["gu_bias"], d["d_blocks"],
                            d["d_scales"], d["d_bias"], p.lay.k, out=out)
        return B.rmsnorm_residual(out, w2, s1)

    def fill(n):
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        res.copy_(n * torch.randn(T, H, generator=g, device="cuda"))
        for t in (y, out, s1):
            t.fill_(float("nan"))

    def check(got):
        B.mxmoe_check()
        h = (x.float() + res.float()).bfloat16()
        assert torch.equal(s1, h)
        n = _norm(h.double(), w1)
        assert bool(((y.double() - n).abs() <= n.abs() * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -133).all())
        p.x = inputs.bits(y)
        d["x"] = y
        TL.check_rows(B, p, d, np.arange(T), out=out)
        h2 = (out.float() + s1.float()).bfloat16()
        n2 = _norm(h2.double(), w2)
        assert torch.equal(got[1], h2)
        assert bool(((got[0].double() - n2).abs() <= n2.abs() * (2.0 ** -8 + 2.0 ** -14) + 2.0 ** -133).all())

    fill(1)
    check(layer())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for n in (2, 0.5):
        fill(n)
        graph.replay()
        check(got)


def test_two_threads_on_two_streams(B):
    """Calls from two host threads at once, each on its own stream with its own buffers: the results are
    those of one thread alone."""
    import threading
    g = torch.Generator(device="cuda").manual_seed(8)
    L = Layer(seed=2)
    n = 5

    def make():
        cache = [torch.full((2 * n, HKV, PAGE, d), 255, dtype=torch.uint8, device="cuda") for d in (D // 2, D // 32) * 2]
        table = torch.randperm(2 * n, generator=g, device="cuda").view(n, 2).int()
        lens = torch.tensor([1, 16, 17, 30, 32], dtype=torch.int32, device="cuda")
        fill = torch.randn(2 * n * PAGE, 2 * HKV, D, generator=g, device="cuda").bfloat16()
        B.mxfp4_kv_append(fill[:, :HKV], fill[:, HKV:], torch.arange(2 * n * PAGE, device="cuda"), *cache)
        last = lens.long() - 1
        slots = table[torch.arange(n, device="cuda"), last // PAGE].long() * PAGE + last % PAGE
        x, res = (torch.randn(n, H, generator=g, device="cuda").bfloat16() for _ in range(2))
        return x, res, cache, table, lens, slots

    def run(s, out, times):
        for _ in range(times):
            x, res, *rest = s
            out.append(L.run(B, x, res.clone(), *rest, 1))

    states, want = [make(), make()], [[], []]
    for s, w in zip(states, want):
        run(s, w, 1)
    B.mxmoe_check()
    got, streams, errors = [[], []], [torch.cuda.Stream(), torch.cuda.Stream()], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                run(states[i], got[i], 60)
                streams[i].synchronize()
        except Exception as e:      # a thread's failure is the test's
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and not any(t.is_alive() for t in threads)
    for i in range(2):
        assert len(got[i]) == 60 and all(torch.equal(a, b) for o in got[i] for a, b in zip(o, want[i][0]))
    B.mxmoe_check()
