"""Operators between a model's projections and the attention over them: their cases, plain forms and calls.

  table    cos and sin of the rotary angles of each token's position: one axis, or several (t, y, x of a video)
  rotate   q and k rotated by them, after a norm over each head if there is one, from the projection's layout to the
           one that the attention reads; its transpose (the gradient, or a rotation taken back)
  append   a serving step's k rotated on its way into the 4-bit paged cache, its v stored, its q rotated
  cross    attention of queries over an encoder's states of another length

An angle is 2 pi times the fraction of position * turns / 2^64: turns (int64) is the frequency in 2^-64 turns a
position, so that positions of any size keep their angles.  The rotation's products and sums are rounded to float32
one by one, which makes the codes of the cache a definition rather than a matter of the order of operations.

The cache is uint8 [pages, H, P / 16, 18 D]; a strip of 16 tokens of a KV head holds
  K codes   [16 tokens][D / 2]            byte c / 2 of a token: channel c, low nibble when c is even
  V codes   [D / 16 groups][16 tokens][8] byte c / 2 of a token in group g: channel 16 g + c
  K scales  [16 tokens][D / 16]           E4M3
  V scales  [D / 16][16 tokens]           E4M3
and an element's value is code * scale * (its head's float32 scale).
"""

import math

import torch

own = False

STEPS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of E2M1, by code
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _table(name, T, P, axes, far, base, stretch):
    return {"name": name, "op": "table", "T": T, "P": P, "axes": axes, "far": far, "base": base, "stretch": stretch}


def _rotate(name, B, T, HQ, H, D, P, interleaved, norm, transpose, heads_first, dtype):
    return {"name": name, "op": "rotate", "B": B, "T": T, "HQ": HQ, "H": H, "D": D, "P": P, "interleaved": interleaved,
            "norm": norm, "transpose": transpose, "heads_first": heads_first, "dtype": dtype}


def _append(name, T, HQ, H, D, P, interleaved, page, pages, dtype):
    return {"name": name, "op": "append", "T": T, "HQ": HQ, "H": H, "D": D, "P": P, "interleaved": interleaved,
            "page": page, "pages": pages, "dtype": dtype}


def _cross(name, B, nlo, nhi, mlo, mhi, HQ, H, D, packed, heads_first, dtype):
    return {"name": name, "op": "cross", "B": B, "nlo": nlo, "nhi": nhi, "mlo": mlo, "mhi": mhi, "HQ": HQ, "H": H, "D": D,
            "packed": packed, "heads_first": heads_first, "dtype": dtype}


def listed():
    return [
        # the positions of one decode step in long contexts, stretched past the trained length
        _table("table decode 64", 64, 64, 1, 131072, 500000.0, 8.0),
        # the (t, y, x) grid of the video workload, a third of the head to each axis
        _table("table video 115200", 115200, 64, 3, 0, 10000.0, 1.0),
        # q and k of the video workload: norm, rotation and the move to heads-first rows in one pass
        _rotate("rotate video 115200", 1, 115200, 24, 24, 128, 64, True, True, False, True, "bf16"),
        # float32 rows, part of a small head, an odd count; the transposed rotation
        _rotate("rotate f32 part odd", 1, 1021, 12, 3, 64, 20, False, False, True, False, "f32"),
        # one decode step of a running batch (the NSA heads): latency
        _append("append decode 64", 64, 64, 4, 128, 64, False, 64, 512, "bf16"),
        # a long prompt (the MSA prefill's length and heads)
        _append("append prefill 32768", 32768, 64, 4, 128, 64, False, 64, 640, "bf16"),
        # the video workload's tokens over a caption of 512 tokens
        _cross("cross video 512", 1, 115200, 115200, 512, 512, 24, 24, 128, False, False, "bf16"),
        # a batch whose captions have other lengths, one of them empty; small heads, heads-first rows
        _cross("cross ragged D64", 6, 4001, 4001, 0, 1024, 16, 16, 64, False, True, "bf16"),
        # prompts of a serving step, packed, over their encoder states; grouped heads
        _cross("cross packed 16", 16, 1, 511, 64, 4096, 64, 4, 128, True, False, "bf16"),
        # single tokens over long states: the states are read once
        _cross("cross decode long 8", 8, 1, 1, 1024, 32768, 32, 8, 128, True, False, "bf16"),
        # single tokens over short states: latency
        _cross("cross decode short 8", 8, 1, 1, 100, 600, 8, 8, 128, False, False, "bf16"),
        # float32, odd sizes
        _cross("cross f32 odd", 3, 77, 333, 5, 517, 12, 3, 64, True, False, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("table", "rotate", "append", "cross", "cross", "cross"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "table":
        axes = rng.randint(1, 3)
        case = _table("", _log(rng, 1, 115200), rng.randint(max(4, axes), 64), axes, _log(rng, 16, 1 << 24),
                      rng.choice((10000.0, 500000.0, 1e6)), rng.choice((1.0, 1.0, 4.0, 32.0)))
    elif op == "rotate":
        H, D = rng.randint(1, 8), rng.choice((64, 80, 128, 128))
        HQ, norm = H * rng.choice((1, 1, 2, 4, 8)), rng.random() < 0.5
        P = rng.choice((D // 2, D // 2, D // 4, rng.randint(1, D // 2)))
        B, T = rng.choice((1, 1, 2, 3)), _log(rng, 1, 32768)
        T = max(1, min(T, (1 << 27) // (B * (HQ + H) * D)))
        case = _rotate("", B, T, HQ, H, D, P, rng.random() < 0.5, norm, not norm and rng.random() < 0.3,
                       rng.random() < 0.5, dtype)
    elif op == "append":
        H, D, page = rng.randint(1, 8), rng.choice((64, 128, 128)), rng.choice((16, 32, 64, 128))
        HQ, T = H * rng.choice((1, 2, 4, 8, 16)), _log(rng, 1, 32768)
        T = max(1, min(T, (1 << 27) // ((HQ + 2 * H) * D)))
        case = _append("", T, HQ, H, D, rng.choice((D // 2, D // 4)), rng.random() < 0.5, page,
                       T // page + 1 + rng.randint(1, 64), dtype)
    else:
        H, D = rng.randint(1, 12), rng.choice((64, 64, 80, 128, 128, 128))
        HQ, B = H * rng.choice((1, 1, 2, 3, 4, 8, 16)), _log(rng, 1, 32)
        nhi, mhi = rng.choice((1, rng.randint(1, 16), _log(rng, 16, 16384))), _log(rng, 1, 32768)
        mhi = max(1, min(mhi, (1 << 29) // (B * HQ * nhi), (1 << 28) // (B * H * D)))
        case = _cross("", B, rng.randint(1, nhi), nhi, rng.randint(0, mhi), mhi, HQ, H, D, rng.random() < 0.4,
                      rng.random() < 0.4, dtype)
        if not case["packed"]:
            case["nlo"] = nhi
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _ramp(R, lo, hi):
    return [lo + (hi - lo) * i // max(1, R - 1) for i in range(R)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _turns(P, base, stretch, axes):
    """Frequencies in 2^-64 turns a position and their axes: each axis has its own ladder base^(-i / n).  A context
    that is `stretch` times the trained one slows down the low ones, those with less than a turn in 2048 positions."""
    turns, axis = [], []
    for a in range(axes):
        n = P // axes + (a < P % axes)
        for i in range(n):
            f = base ** (-i / n) / (2 * math.pi)
            turns.append(round((f / stretch if f * 2048 < 1 else f) * 2.0 ** 64))
            axis.append(a)
    return (torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device="cuda"),
            torch.tensor(axis, dtype=torch.int32, device="cuda"))


def _prepare_table(c, seed):
    g = _gen(seed)
    turns, axis = _turns(c["P"], c["base"], c["stretch"], c["axes"])
    T, far = c["T"], c["far"]
    if far:
        pos = torch.randint(0, far, (T, c["axes"]), generator=g, device="cuda")
    else:  # a (30, 48, 80) grid that starts somewhere in a longer video
        i = torch.arange(T, device="cuda")
        first = torch.randint(0, 4096, (1,), generator=g, device="cuda")
        pos = torch.stack([first + i // 3840, i // 80 % 48, i % 80], 1)
    return dict(pos=pos.int().contiguous(), turns=turns, axis=axis, factor=0.1 * math.log(c["stretch"]) + 1.0)


def _tables(g, shape, P, far):
    """cos and sin [..., P] of random positions."""
    turns, _ = _turns(P, 10000.0, 1.0, 1)
    pos = torch.randint(0, far, shape + (1,), generator=g, device="cuda")
    angle = pos * (turns.double() * (2 * math.pi * 2.0 ** -64))
    return angle.cos().float(), angle.sin().float()


def _prepare_rotate(c, seed):
    g = _gen(seed)
    B, T, HQ, H, D = (c[x] for x in ("B", "T", "HQ", "H", "D"))
    rows = torch.randn((B, T, HQ + 2 * H, D), generator=g, device="cuda")
    rows *= 1 + 3 * torch.rand((1, 1, 1, D), generator=g, device="cuda").pow(4)  # a few strong channels
    rows = rows.to(_dtype(c))  # q, k and v of a token side by side, as one projection gives them
    cos, sin = _tables(g, (T,), c["P"], 32768)
    s = dict(case=c, q=rows[:, :, :HQ], k=rows[:, :, HQ:HQ + H], cos=cos, sin=sin, qw=None, kw=None)
    if c["norm"]:
        s["qw"], s["kw"] = 1 + 0.2 * torch.randn((2, D), generator=g, device="cuda")
    return s


def _prepare_append(c, seed):
    g = _gen(seed)
    T, HQ, H, D, page = c["T"], c["HQ"], c["H"], c["D"], c["page"]
    rows = torch.randn((T, HQ + 2 * H, D), generator=g, device="cuda")
    rows[:, HQ:HQ + H] *= 1 + 3 * torch.rand((1, 1, D), generator=g, device="cuda").pow(4)
    rows[:, HQ + H:] *= 0.25
    rows = rows.to(_dtype(c))
    pages = torch.randperm(c["pages"], generator=g, device="cuda")[: -(-(T + 5) // page)]
    pos = torch.arange(T, device="cuda") + 5  # the first page is partly filled already
    slots = (pages[pos // page] * page + pos % page).contiguous()
    cos, sin = _tables(g, (T,), c["P"], 131072)
    kv = torch.rand((2, H), generator=g, device="cuda") * 0.2 + 0.05
    new = lambda n: torch.zeros((T, n, D), dtype=rows.dtype, device="cuda")  # noqa: E731
    return dict(case=c, q=rows[:, :HQ], k=rows[:, HQ:HQ + H], v=rows[:, HQ + H:], cos=cos, sin=sin, slots=slots,
                cache=torch.zeros((c["pages"], H, page // 16, 18 * D), dtype=torch.uint8, device="cuda"),
                k_scale=kv[0].contiguous(), v_scale=(kv[1] * 0.1).contiguous(), q_out=new(HQ), k_val=new(H), v_val=new(H))


def _starts(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(lens, 0)]).int()


def _prepare_cross(c, seed):
    g = _gen(seed)
    B, HQ, H, D = c["B"], c["HQ"], c["H"], c["D"]
    order = torch.randperm(B, generator=g, device="cuda")
    n, m = (torch.tensor(_ramp(B, c[lo], c[hi]), device="cuda")[order] for lo, hi in (("nlo", "nhi"), ("mlo", "mhi")))
    m = m.flip(0) if B > 1 and c["nlo"] != c["nhi"] else m
    s = dict(case=c, n=n, m=m, query_start=None, key_start=None, key_lens=None)
    if c["packed"]:
        q = torch.randn((int(sum(_ramp(B, c["nlo"], c["nhi"]))), HQ, D), generator=g, device="cuda")
        kv = torch.randn((int(sum(_ramp(B, c["mlo"], c["mhi"]))), 2, H, D), generator=g, device="cuda").to(_dtype(c))
        s.update(query_start=_starts(n), key_start=_starts(m), k=kv[:, 0], v=kv[:, 1])
    else:
        q = torch.randn((B, HQ, c["nhi"], D) if c["heads_first"] else (B, c["nhi"], HQ, D), generator=g, device="cuda")
        kv = torch.randn((B, c["mhi"], 2, H, D), generator=g, device="cuda").to(_dtype(c))
        if c["heads_first"]:
            q, kv = q.transpose(1, 2), kv.permute(2, 0, 3, 1, 4).contiguous().permute(1, 3, 0, 2, 4)
        s.update(key_lens=m.int(), k=kv[:, :, 0], v=kv[:, :, 1])
    s["q"] = (1.5 * q).to(_dtype(c))
    return s


def prepare(case, seed):
    return {"table": _prepare_table, "rotate": _prepare_rotate, "append": _prepare_append,
            "cross": _prepare_cross}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms

def _plain_table(s):
    turn = s["pos"].long()[:, s["axis"].long()] * s["turns"]  # wraps at 2^64, a whole turn
    angle = turn.double() * (2 * math.pi * 2.0 ** -64)
    return {"cos": (angle.cos() * s["factor"]).float(), "sin": (angle.sin() * s["factor"]).float()}


def _rotated(x, cos, sin, interleaved):
    """Float32 rows [..., heads, D] rotated by tables [..., P], every product and sum rounded by itself."""
    P = cos.shape[-1]
    cos, sin = cos[..., None, :], sin[..., None, :]
    a, b = (x[..., 0:2 * P:2], x[..., 1:2 * P:2]) if interleaved else (x[..., :P], x[..., P:2 * P])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., 2 * P:]], -1)


def _plain_rotate(s):
    c, out = s["case"], {}
    sin = -s["sin"] if c["transpose"] else s["sin"]
    for name in ("q", "k"):
        x = s[name].float()
        if s[name + "w"] is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s[name + "w"]
        y = _rotated(x, s["cos"], sin, c["interleaved"]).to(s[name].dtype)
        out[name] = y.transpose(1, 2).contiguous() if c["heads_first"] else y
    return out


def _quantise(x, head_scale):
    """E2M1 codes [..., D] uint8 and E4M3 scales [..., D / 16] of y = x * (1 / head_scale), a float32 product.  A
    group's scale is its largest magnitude / 6 rounded to E4M3; the codes are the magnitudes nearest to y / scale,
    ties to the even code."""
    y = (x * (1.0 / head_scale)).unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device="cuda")  # on the device: a division, not a product with a rounded 1 / 6
    scale = (y.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    a = torch.where(s > 0, y.abs() / s, 0.0).clamp(max=6.0)
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = torch.where(y.signbit(), code + 8, code)
    return code.to(torch.uint8).flatten(-2), scale


def _plain_append(s):
    c, cache, slots = s["case"], s["cache"], s["slots"]
    D, page_size = c["D"], c["page"]
    page, strip, t = slots // page_size, slots % page_size // 16, slots % 16
    out = {"q": _rotated(s["q"].float(), s["cos"], s["sin"], c["interleaved"]).to(s["q"].dtype)}
    rows = {"k": _rotated(s["k"].float(), s["cos"], s["sin"], c["interleaved"]), "v": s["v"].float()}
    for name, base in (("k", 0), ("v", 8 * D)):
        codes, scales = _quantise(rows[name], s[name + "_scale"][:, None])
        codes_at, scales_at = cache[..., base:base + 8 * D], cache[..., 16 * D + base // 8:][..., :D]
        groups = (D // 16, 16) if name == "v" else (16, D // 16)
        codes_at, scales_at = codes_at.unflatten(3, groups + (8,)), scales_at.unflatten(3, groups)
        if name == "v":
            codes_at, scales_at = codes_at.transpose(3, 4), scales_at.transpose(3, 4)
        codes_at[page, :, strip, t] = (codes[..., 0::2] | (codes[..., 1::2] << 4)).unflatten(2, (-1, 8))
        scales_at[page, :, strip, t] = scales.view(torch.uint8)
        value = torch.tensor(STEPS + tuple(-x for x in STEPS), device="cuda")[codes.int()]
        value = (value.unflatten(2, (-1, 16)) * scales.float()[..., None]).flatten(2)
        out[name] = (value * s[name + "_scale"][:, None]).to(s[name].dtype)
    return out


def _padded(x, start, most):
    """Packed rows [total, ...] as [B, most, ...]; rows behind a sequence's last are some other row."""
    at = (start[:-1].long()[:, None] + torch.arange(most, device="cuda")).clamp(max=max(0, x.shape[0] - 1))
    return x[at]


def _plain_cross(s):
    c, q, k, v = s["case"], s["q"].float(), s["k"].float(), s["v"].float()
    HQ, H, D = c["HQ"], c["H"], c["D"]
    if c["packed"]:
        q = _padded(q, s["query_start"], c["nhi"])
        k, v = _padded(k, s["key_start"], c["mhi"]), _padded(v, s["key_start"], c["mhi"])
    B, N, M, G = q.shape[0], q.shape[1], k.shape[1], HQ // H
    q = q.view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5
    x.masked_fill_(torch.arange(M, device="cuda") >= s["m"][:, None, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(1, 2)) / total.clamp(min=torch.finfo(torch.float32).tiny)
    lse = (top + total.log()).view(B, HQ, N).transpose(1, 2)
    o = o.view(B, HQ, N, D).transpose(1, 2).to(s["q"].dtype)
    if c["packed"]:
        req = torch.repeat_interleave(torch.arange(B, device="cuda"), s["n"], output_size=s["q"].shape[0])
        at = torch.arange(s["q"].shape[0], device="cuda") - s["query_start"].long()[req]
        o, lse = o[req, at], lse[req, at]
    return {"out": o, "lse": lse}


# ---------------------------------------------------------------- calls

def run(state):
    s = state
    if own:
        from block_sparse_attention_tile_gb300 import pipeline
        if "pos" in s:
            cos, sin = pipeline.rotary_table(s["pos"], s["turns"], s["axis"], s["factor"])
            return {"cos": cos, "sin": sin}
        c = s["case"]
        if c["op"] == "rotate":
            q, k = pipeline.rotate(s["q"], s["k"], s["cos"], s["sin"], interleaved=c["interleaved"], q_weight=s["qw"],
                                   k_weight=s["kw"], eps=EPS, heads_first=c["heads_first"], transpose=c["transpose"])
            return {"q": q, "k": k}
        if c["op"] == "append":
            pipeline.cache_append_rotated(s["k"], s["v"], s["slots"], s["cache"], s["cos"], s["sin"], s["k_scale"],
                                          s["v_scale"], interleaved=c["interleaved"], values=(s["k_val"], s["v_val"]),
                                          q=s["q"], q_out=s["q_out"])
            return {"q": s["q_out"], "k": s["k_val"], "v": s["v_val"]}
        out, lse = pipeline.cross_attention(s["q"], s["k"], s["v"], key_lens=s["key_lens"], query_start=s["query_start"],
                                            key_start=s["key_start"])
        return {"out": out, "lse": lse}
    if "pos" in s:
        return _plain_table(s)
    return {"rotate": _plain_rotate, "append": _plain_append, "cross": _plain_cross}[s["case"]["op"]](s)


# ---------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "table":
        return {"bytes": 4 * c["T"] * c["axes"] + 12 * c["P"] + 8 * c["T"] * c["P"], "flops": 0}
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rotate":
        rows = c["B"] * c["T"] * (c["HQ"] + c["H"])
        return {"bytes": 2 * size * rows * c["D"] + 8 * c["T"] * c["P"], "flops": rows * (6 * c["P"] + 3 * c["D"] * c["norm"])}
    if c["op"] == "append":
        q, kv = c["T"] * c["HQ"] * c["D"], 2 * c["T"] * c["H"] * c["D"]
        return {"bytes": 2 * size * q + kv * (2 * size + 0.5 + 1 / 16) + 8 * c["T"] * (c["P"] + 1),
                "flops": 6 * c["P"] * c["T"] * (c["HQ"] + c["H"])}
    n, m = _ramp(c["B"], c["nlo"], c["nhi"]), _ramp(c["B"], c["mlo"], c["mhi"])
    if c["B"] > 1 and c["nlo"] != c["nhi"]:
        m = m[::-1]
    rows, pairs = sum(n), sum(x * y for x, y in zip(n, m)) if c["packed"] else c["nhi"] * sum(m)
    return {"bytes": rows * c["HQ"] * (2 * c["D"] * size + 4) + sum(m) * 2 * c["H"] * c["D"] * size,
            "flops": 4 * pairs * c["HQ"] * c["D"]}


# ---------------------------------------------------------------- 64 bits

def _exact_table(s):
    got, f = {}, (s["turns"].double() * 2.0 ** -64) % 1.0
    pos = s["pos"].double()[:, s["axis"].long()]
    high = torch.floor(pos / 4096)  # in two parts, so that no product has lost digits of its fraction
    part = ((high * ((f * 4096) % 1.0)) % 1.0 + ((pos - 4096 * high) * f) % 1.0) * (2 * math.pi)
    got["cos"], got["sin"] = s["factor"] * torch.cos(part), s["factor"] * torch.sin(part)
    return got


def _pairs(P, D, interleaved):
    """Partner channel of each channel, and the sign of the partner's part (0 for channels that stay)."""
    ch = torch.arange(D, device="cuda")
    first = ch % 2 == 0 if interleaved else ch < P
    other = torch.where(first, ch + 1, ch - 1) if interleaved else torch.where(first, ch + P, ch - P)
    live = ch < 2 * P
    pair = torch.where(live, ch // 2 if interleaved else ch % P, 0)
    return torch.where(live, other, ch), pair, torch.where(first, -1.0, 1.0).double() * live, live


def _exact_rotate(c, s):
    got = {}
    other, pair, sign, live = _pairs(c["P"], c["D"], c["interleaved"])
    cos = torch.where(live, s["cos"].double()[:, pair], 1.0)[:, None]
    sin = (s["sin"].double()[:, pair] * sign * (-1 if c["transpose"] else 1))[:, None]
    for name in ("q", "k"):
        x = s[name].double()
        if c["norm"]:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * s[name + "w"].double()
        y = x * cos + x[..., other] * sin
        got[name] = y.transpose(1, 2) if c["heads_first"] else y
    return got


def _nearest(x, grid):
    """Indices into the ascending grid of the nearest values to x >= 0, ties to the even index, the last for more."""
    up = torch.bucketize(x, grid).clamp(1, grid.numel() - 1)
    lo, hi = x - grid[up - 1], grid[up] - x
    return torch.where((hi < lo) | ((hi == lo) & (up % 2 == 0)), up, up - 1)


def _exact_append(c, s):
    steps = torch.tensor(STEPS, dtype=torch.float64, device="cuda")
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)]
                        + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device="cuda")
    other, pair, sign, live = _pairs(c["P"], c["D"], c["interleaved"])
    cos = torch.where(live, s["cos"].double()[:, pair], 1.0)[:, None]
    sin = (s["sin"].double()[:, pair] * sign)[:, None]
    got = {"q": s["q"].double() * cos + s["q"].double()[..., other] * sin}
    for name in ("k", "v"):
        x, h = s[name].double(), s[name + "_scale"].double()[:, None, None]
        if name == "k":  # float32 products and their float32 sum by definition, as y below; everything after is exact
            x = ((x * cos).float().double() + (x[..., other] * sin).float().double()).float().double()
        y = (x.unflatten(2, (-1, 16)) * (1 / h).float().double()).float().double()
        scale = grid[_nearest(y.abs().amax(3) / 6, grid)][..., None]
        code = _nearest((y.abs() / scale.clamp(min=1e-300)).clamp(max=6.0), steps)
        got[name] = (steps[code] * y.sign() * scale * h).flatten(2)
    return got


def _exact_cross(c, s):
    HQ, G, D, packed = c["HQ"], c["HQ"] // c["H"], c["D"], c["packed"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    n, m = s["n"].tolist(), s["m"].tolist()
    for b in range(c["B"]):
        if not m[b]:
            continue
        if packed:
            row, key = sum(n[:b]), sum(m[:b])
            q, o, z = s["q"][row:row + n[b]], out[row:row + n[b]], lse[row:row + n[b]]
            k, v = s["k"][key:key + m[b]], s["v"][key:key + m[b]]
        else:
            q, o, z, k, v = s["q"][b], out[b], lse[b], s["k"][b, :m[b]], s["v"][b, :m[b]]
        for h in range(HQ):
            x = torch.mm(q[:, h].double(), k[:, h // G].double().T) / math.sqrt(D)
            z[:, h] = torch.logsumexp(x, 1)
            o[:, h] = torch.mm(torch.softmax(x, 1), v[:, h // G].double())
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "table":
        return _exact_table(s)
    return {"rotate": _exact_rotate, "append": _exact_append, "cross": _exact_cross}[case["op"]](case, s)
