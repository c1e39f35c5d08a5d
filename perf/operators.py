"""What is measured of the operators around the expert layer's attention half.

 norm       rmsnorm_residual / rmsnorm_residual_fp8: residual addition, root-mean-square
            norm, output in bf16 or in FP8 E4M3 (a static scale, or one scale per token)
 linear     fp8_linear_fused: FP8 E4M3 matrix product with per-token / per-channel scales,
            bias, activation and residual in its epilogue
 append     mxfp4_kv_append: new keys and values into a paged MXFP4 cache (read back as
            bf16 by mxfp4_dequantize, the values that the cache stands for)
 attention  mxfp4_kv_attention: attention of a few queries per sequence over that cache

Sizes: hidden 2880, 64 query heads and 8 key/value heads of 64, fused Q/K/V 2880 -> 5120
and O 4096 -> 2880 are this repository's attention-projection workload; the others are
generic. `run` computes either the plain form (elementary torch, 32 bits, one rounding at
the end) or, with `own`, makes the framework's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0


# --------------------------------------------------------------------------- cases -----

def listed():
    return [
        # one decoded token: the norm before the FP8 Q/K/V projection, static input scale
        dict(name="norm_decode1", op="norm", T=1, H=2880, out="static", residual=True),
        # a prefill batch, one scale per token
        dict(name="norm_prefill", op="norm", T=4096, H=2880, out="token", residual=True),
        # the norm before the expert layer (bf16 output), ragged token count, no residual
        dict(name="norm_bf16_ragged", op="norm", T=9973, H=4096, out="bf16", residual=False),
        # fused Q/K/V of one decoded token
        dict(name="qkv_decode1", op="linear", T=1, K=2880, N=5120, sx="token", sw="channel", bias=True, act="", residual=False),
        # O projection of a decode batch, residual added
        dict(name="o_decode64", op="linear", T=64, K=4096, N=2880, sx="static", sw="tensor", bias=True, act="", residual=True),
        # an MLP projection with its activation, ragged tokens
        dict(name="mlp_gelu", op="linear", T=777, K=1024, N=4096, sx="token", sw="tensor", bias=True, act="gelu", residual=False),
        # fused Q/K/V of a prefill batch
        dict(name="qkv_prefill", op="linear", T=4096, K=2880, N=5120, sx="token", sw="channel", bias=True, act="", residual=False),
        # one new token of each of 64 sequences
        dict(name="append_decode64", op="append", T=64, Hkv=8, D=64, page=16),
        # a prefill batch written to the cache
        dict(name="append_prefill", op="append", T=16384, Hkv=8, D=64, page=64),
        # one sequence, one query, a sliding window's worth of keys, sinks
        dict(name="attn_window1", op="attention", B=1, Lq=1, Hq=64, Hkv=8, D=64, page=16, lo=4001, hi=4001, window=128, sinks=True),
        # a decode batch of ragged lengths, sinks
        dict(name="attn_decode64", op="attention", B=64, Lq=1, Hq=64, Hkv=8, D=64, page=64, lo=500, hi=8192, window=0, sinks=True),
        # few sequences, long context, two queries each (a drafted token), heads of 128
        dict(name="attn_long", op="attention", B=3, Lq=2, Hq=32, Hkv=8, D=128, page=128, lo=30011, hi=131072, window=0, sinks=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "append", "attention"))
    if op == "norm":
        H = 8 * _log(rng, 8, 1024)
        T = min(_log(rng, 1, 16384), 40_000_000 // H)
        return dict(op=op, T=max(1, T), H=H, out=rng.choice(("static", "token", "bf16")), residual=rng.random() < 0.7)
    if op == "linear":
        K, N = 32 * _log(rng, 8, 256), 8 * _log(rng, 8, 1024)
        T = min(_log(rng, 1, 8192), 60_000_000_000 // (K * N))
        return dict(op=op, T=max(1, T), K=K, N=N, sx=rng.choice(("token", "static")), sw=rng.choice(("channel", "tensor")),
                    bias=rng.random() < 0.7, act=rng.choice(("", "", "silu", "gelu")), residual=rng.random() < 0.5)
    if op == "append":
        Hkv, D = rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((64, 128))
        return dict(op=op, T=max(1, min(_log(rng, 1, 16384), 8_388_608 // (Hkv * D))), Hkv=Hkv, D=D, page=rng.choice((16, 32, 64, 128)))
    Hkv, D, G = rng.choice((1, 2, 4, 8)), rng.choice((64, 128)), rng.choice((1, 2, 4, 5, 8, 16))
    B, Lq = _log(rng, 1, 96), rng.choice((1, 1, 1, 2, 3, 4))
    hi = max(Lq, min(_log(rng, 1, 131072), 130_000_000 // (B * Hkv * D)))
    return dict(op=op, B=B, Lq=Lq, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice((16, 32, 64, 128)), lo=max(Lq, hi // rng.choice((1, 2, 16))), hi=hi,
                window=rng.choice((0, 0, 128, 1000)), sinks=rng.random() < 0.5)


def _lens(case):
    """The sequences' lengths: spread over [lo, hi], the longest not first."""
    r, B = random.Random(case["B"] * 1009 + case["hi"]), case["B"]
    lens = [case["lo"] + (case["hi"] - case["lo"]) * (i + 1) // B for i in range(B)]
    r.shuffle(lens)
    return lens


def _seen(case, n, i):
    """Keys [from, to) that query i of a sequence of n keys sees: the queries are its last Lq tokens."""
    to = n - case["Lq"] + i + 1
    return (max(0, to - case["window"]) if case["window"] else 0), max(0, to)


# ------------------------------------------------------------------------- prepare -----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _e4m3_codes(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # a residual stream: a few channels carry values well above the rest
        gain = 1 + 9 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        s["x"] = (torch.randn(T, H, generator=g, device="cuda") * gain).to(torch.bfloat16)
        s["res"] = (2 * torch.randn(T, H, generator=g, device="cuda") * gain).to(torch.bfloat16) if case["residual"] else None
        s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s["s"] = 0.05 if case["out"] == "static" else None
    elif case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        # activations and weights as their quantizers leave them: the largest value at 448
        x, w = torch.randn(T, K, generator=g, device="cuda"), 0.02 * torch.randn(N, K, generator=g, device="cuda")
        ax, aw = x.abs().amax(1) / E4M3_MAX, w.abs().amax(1) / E4M3_MAX
        s["sx"] = ax if case["sx"] == "token" else float(ax.max())
        s["sw"] = aw if case["sw"] == "channel" else float(aw.max())
        s["xq"] = _e4m3_codes(x / (ax[:, None] if case["sx"] == "token" else ax.max()))
        s["wq"] = _e4m3_codes(w / (aw[:, None] if case["sw"] == "channel" else aw.max()))
        s["b"] = 0.1 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["res"] = _bf16(g, T, N) if case["residual"] else None
    elif case["op"] == "append":
        T, Hkv, D, page = case["T"], case["Hkv"], case["D"], case["page"]
        # k and v as slices of a fused projection's rows; slots in the order of a shuffled page list
        s["kv"] = _bf16(g, T, 2 * Hkv * D)
        pages = -(-T // page)
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        s["slots"] = order[t // page] * page + t % page
        for n in "kv":
            s[n + "b"] = torch.zeros(pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
            s[n + "s"] = torch.zeros(pages, Hkv, page, D // 32, dtype=torch.uint8, device="cuda")
    else:
        B, Lq, Hq, Hkv, D, page = (case[n] for n in ("B", "Lq", "Hq", "Hkv", "D", "page"))
        lens = _lens(case)
        need = [-(-n // page) for n in lens]
        table = torch.zeros(B, max(need), dtype=torch.int32)
        order, at = torch.randperm(sum(need) + 1, generator=g, device="cuda").cpu().to(torch.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"], s["lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _bf16(g, B, Lq, Hq, D)
        s["sinks"] = torch.randn(Hq, generator=g, device="cuda") if case["sinks"] else None
        # keys with a common direction (scores that are not flat), values of uneven size
        lean = torch.randn(Hkv, 1, D, generator=g, device="cuda")
        for n in "kv":
            b = torch.empty(sum(need) + 1, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
            c = torch.empty(sum(need) + 1, Hkv, page, D // 32, dtype=torch.uint8, device="cuda")
            step = max(1, (1 << 24) // (Hkv * page * D))
            for i in range(0, b.shape[0], step):
                x = torch.randn(min(step, b.shape[0] - i), Hkv, page, D, generator=g, device="cuda")
                x = x + lean if n == "k" else x * torch.exp(torch.randn(x.shape[:3] + (1,), generator=g, device="cuda"))
                b[i:i + step], c[i:i + step] = _pack(x)
            s[n + "b"], s[n + "s"] = b, c
    return s


# --------------------------------------------------------------------- plain forms -----

def _pack(x):
    """MXFP4 of fp32 rows: blocks of 32 along the last axis, exponent floor(log2 amax) - 2, ties to the even code."""
    v = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    _, e = torch.frexp(v.abs().amax(-1, keepdim=True))
    e = torch.where(v.abs().amax(-1, keepdim=True) > 0, e - 3, -127).clamp(-127, 127)
    m = torch.ldexp(v.abs(), -e)
    c = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte() + (m > 2.5).byte() + (m >= 3.5).byte() + (m > 5).byte()
         + 8 * torch.signbit(v).byte()).reshape(x.shape[:-1] + (x.shape[-1] // 2, 2))
    return c[..., 0] | (c[..., 1] << 4), (e[..., 0] + 127).to(torch.uint8)


def _unpack(blocks, scales):
    """fp32 values of MXFP4 rows."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=blocks.device)
    c = torch.stack((blocks & 15, blocks >> 4), -1).flatten(-2)
    v = grid[c.int()].unflatten(-1, (scales.shape[-1], 32))
    return torch.ldexp(v, scales.int()[..., None] - 127).flatten(-2)


def _act(y, act):
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    return y


def _norm(s):
    h = s["x"].float()
    out = {}
    if s["res"] is not None:
        out["sum"] = (h + s["res"].float()).to(torch.bfloat16)
        h = out["sum"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    if s["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
        return out
    if s["out"] == "token":
        a = y.abs().amax(1)
        scale = out["scale"] = torch.where(a > 0, a / E4M3_MAX, torch.ones_like(a))
        y = y / scale[:, None]
    else:
        y = y / s["s"]
    out["q"] = y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return out


def _linear(s):
    y = s["xq"].view(torch.float8_e4m3fn).float() @ s["wq"].view(torch.float8_e4m3fn).float().t()
    y = y * (s["sx"][:, None] if torch.is_tensor(s["sx"]) else s["sx"]) * (s["sw"] if torch.is_tensor(s["sw"]) else s["sw"])
    if s["b"] is not None:
        y = y + s["b"]
    y = _act(y, s["act"])
    return (y if s["res"] is None else y + s["res"].float()).to(torch.bfloat16)


def _kv_rows(s):
    T, Hkv, D = s["T"], s["Hkv"], s["D"]
    return s["kv"][:, :Hkv * D].view(T, Hkv, D), s["kv"][:, Hkv * D:].view(T, Hkv, D)


def _append(s):
    out = []
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    for n, rows in zip("kv", _kv_rows(s)):
        s[n + "b"][page, :, at], s[n + "s"][page, :, at] = _pack(rows.float())
        out.append(_unpack(s[n + "b"], s[n + "s"]).to(torch.bfloat16))
    return out


def _attention(s):
    B, Lq, Hq, Hkv, D = (s[n] for n in ("B", "Lq", "Hq", "Hkv", "D"))
    # a group of sequences at a time: the cache in 32 bits is eight times its packed size
    n = s["table"].shape[1] * s["page"]
    some = max(1, (1 << 29) // (n * Hkv * D))
    return torch.cat([_attend(s, slice(b, b + some)) for b in range(0, B, some)]).to(torch.bfloat16)


def _attend(s, part):
    Lq, Hq, Hkv, D = (s[n] for n in ("Lq", "Hq", "Hkv", "D"))
    table, lens = s["table"][part].long(), s["lens"][part]
    k = _unpack(s["kb"][table], s["ks"][table]).transpose(1, 2).flatten(2, 3)      # (B, Hkv, keys, D)
    v = _unpack(s["vb"][table], s["vs"][table]).transpose(1, 2).flatten(2, 3)
    B, keys = k.shape[0], k.shape[2]
    at = torch.arange(keys, device=k.device)
    to = (lens[:, None] - Lq + 1 + torch.arange(Lq, device=k.device))[..., None]   # (B, Lq, 1)
    seen = at < to
    if s["window"]:
        seen = seen & (at >= to - s["window"])
    q = s["q"][part].float().view(B, Lq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)  # (B, Hkv, G, Lq, D)
    z = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (Hq // Hkv, Lq)) / math.sqrt(D)
    z = torch.where(seen[:, None, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, Hq // Hkv, 1, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        l = l + torch.exp(sink - m)
    v = torch.where((at < lens[:, None])[:, None, :, None], v, 0.0)
    o = (p.flatten(2, 3) @ v).unflatten(2, (Hq // Hkv, Lq)) / torch.where(l > 0, l, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, D)


# ----------------------------------------------------------------------------- run -----

def run(state):
    s = state
    if own:
        from mxfp4_block_scaled_moe_b200 import binding as B
        if s["op"] == "norm":
            if s["out"] == "bf16":
                y, h = B.rmsnorm_residual(s["x"], s["w"], s["res"], EPS)
                return {"y": y} if h is None else {"y": y, "sum": h}
            q, scale, h = B.rmsnorm_residual_fp8(s["x"], s["w"], s["res"], EPS, act_scale=s["s"])
            out = {"q": q.view(torch.float8_e4m3fn), "scale": scale, "sum": h}
            return {n: t for n, t in out.items() if t is not None}
        if s["op"] == "linear":
            return B.fp8_linear_fused(s["xq"], s["wq"], s["sx"], s["sw"], bias=s["b"], act=s["act"] or None, residual=s["res"])
        if s["op"] == "append":
            k, v = _kv_rows(s)
            B.mxfp4_kv_append(k, v, s["slots"], s["kb"], s["ks"], s["vb"], s["vs"])
            return [B.mxfp4_dequantize(s[n + "b"], s[n + "s"], torch.bfloat16) for n in "kv"]
        return B.mxfp4_kv_attention(s["q"], s["kb"], s["ks"], s["vb"], s["vs"], s["table"], s["lens"], window=s["window"], sinks=s["sinks"])
    return {"norm": _norm, "linear": _linear, "append": _append, "attention": _attention}[s["op"]](s)


# ---------------------------------------------------------------------------- work -----

def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        each = 2 + (4 if case["residual"] else 0) + (2 if case["out"] == "bf16" else 1)
        return {"bytes": n * each + 2 * case["H"] + (4 * case["T"] if case["out"] == "token" else 0), "flops": 6 * n}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        b = T * K + N * K + 2 * T * N * (2 if case["residual"] else 1) + (4 * T if case["sx"] == "token" else 0)
        return {"bytes": b + 4 * N * ((case["sw"] == "channel") + case["bias"]), "flops": 2 * T * K * N}
    if case["op"] == "append":
        # the new rows in, their packed form out, and the read-back of every page as bf16
        rows, D, page = 2 * case["T"] * case["Hkv"], case["D"], case["page"]
        pool = 2 * -(-case["T"] // page) * page * case["Hkv"]
        return {"bytes": rows * (2 * D + D // 2 + D // 32) + pool * 2 * D + 8 * case["T"], "flops": 8 * rows * D}
    D, pairs, keys = case["D"], 0, 0
    for n in _lens(case):
        seen = [_seen(case, n, i) for i in range(case["Lq"])]
        pairs += sum(b - a for a, b in seen)
        keys += seen[-1][1] - seen[0][0]
    b = 2 * keys * case["Hkv"] * (D // 2 + D // 32) + 4 * case["B"] * case["Lq"] * case["Hq"] * D
    return {"bytes": b, "flops": 4 * pairs * case["Hq"] * D}


# --------------------------------------------------------------------------- exact -----

_CODE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest_e4m3(v):
    """E4M3's nearest value (three mantissa bits, least exponent -6), ties to even, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _decode64(blocks, scales):
    codes = torch.tensor(_CODE + [-c for c in _CODE], dtype=torch.float64, device=blocks.device)
    pairs = torch.empty(blocks.shape + (2,), dtype=torch.float64, device=blocks.device)
    pairs[..., 0], pairs[..., 1] = codes[(blocks % 16).long()], codes[(blocks // 16).long()]
    return pairs.flatten(-2) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _nearest_mxfp4(x):
    """The value that MXFP4 holds for each of x's along its last axis, in 64 bits."""
    v = x.double().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 2, torch.full_like(top, -127.0)).clamp(-127, 127)
    r = (v / torch.exp2(e)).abs()
    # the grid's steps are 0.5 up to 2, 1 up to 4, 2 up to 6; halves of a step go to the even code
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).double()
    return (torch.copysign((torch.round(r / step) * step).clamp(max=6.0), v) * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h, out = s["x"].double(), {}
        if s["res"] is not None:
            out["sum"] = h + s["res"].double()
            h = out["sum"].to(torch.bfloat16).double()  # the norm is of the stream as it is stored
        n = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["H"] + EPS) * s["w"].double()
        if case["out"] == "bf16":
            return {**out, "y": n}
        unit = torch.full((case["T"],), float(s["s"] or 0), dtype=torch.float64, device="cuda")
        if case["out"] == "token":
            top = n.abs().max(1).values
            unit = out["scale"] = torch.where(top > 0, top / E4M3_MAX, 1.0)
        return {**out, "q": _nearest_e4m3(n / unit[:, None])}
    if case["op"] == "linear":
        a, w = (s[n].view(torch.float8_e4m3fn).double() for n in ("xq", "wq"))
        y = torch.einsum("tk,nk->tn", a, w) * torch.as_tensor(s["sw"], device="cuda").double()
        y *= torch.as_tensor(s["sx"], device="cuda").double().reshape(-1, 1)
        if s["b"] is not None:
            y += s["b"].double()
        if case["act"]:
            y = y / (1 + torch.exp(-y)) if case["act"] == "silu" else y * torch.special.erfc(-y / math.sqrt(2)) / 2
        return y if s["res"] is None else y + s["res"].double()
    if case["op"] == "append":
        got, W = [], case["Hkv"] * case["D"]
        for i in range(2):
            flat = torch.zeros(s["kb"].shape[0] * case["page"], case["Hkv"], case["D"], dtype=torch.float64, device="cuda")
            flat[s["slots"]] = _nearest_mxfp4(s["kv"][:, i * W:(i + 1) * W].reshape(case["T"], case["Hkv"], case["D"]))
            got.append(flat.unflatten(0, (-1, case["page"])).transpose(1, 2))
        return got
    out = torch.zeros(case["B"], case["Lq"], case["Hq"], case["D"], dtype=torch.float64, device="cuda")
    G = case["Hq"] // case["Hkv"]
    for b, n in enumerate(_lens(case)):
        used = s["table"][b, :-(-n // case["page"])].long()
        for h in range(case["Hkv"]):
            k, v = (_decode64(s[c + "b"][used, h], s[c + "s"][used, h]).flatten(0, 1) for c in "kv")
            for i in range(case["Lq"]):
                first, last = _seen(case, n, i)
                if last <= first:
                    continue
                z = s["q"][b, i, h * G:(h + 1) * G].double() @ k[first:last].t() / case["D"] ** 0.5
                if s["sinks"] is not None:
                    z = torch.cat((z, s["sinks"][h * G:(h + 1) * G, None].double()), 1)
                p = torch.softmax(z, 1)[:, :last - first]
                out[b, i, h * G:(h + 1) * G] = p @ v[first:last]
    return out
