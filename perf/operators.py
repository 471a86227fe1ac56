"""Cases for the operators of a rotated, paged key/value cache: rotary positions (osm_rope,
osm_rope_bwd), appending keys and values with the rotation applied on the way (osm_kv_append),
reading the cache out (osm_kv_gather) and attention over it (fa_fwd_paged), the cache held in
bf16 or in 4 bits.

A 4-bit cache page holds, per key/value head, page * d / 2 bytes of codes (token after token,
value 2i in the low half of byte i) and then, per token and group of 64 values, a 16-bit word:
the upper ten bits of the step s (a float without sign, eight bits of exponent and two of
fraction) above a signed six-bit base b.  A value is s * (b + code), which bf16 holds exactly.
"""
import math
import random

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # Queries of a training step as the projection leaves them (token after token), rotated
        # into the [B, H, N, d] layout that attention reads.
        dict(name="rope-train-half", op="rope", B=2, H=32, N=8192, d=128, rot=128, layout="half",
             dtype="bf16", order="bnhd", start=0, scaling="none", factor=1.0),
        # The gradient of a rotation of half of each head, in fp32, an odd length.
        dict(name="rope-bwd-part", op="rope_bwd", B=3, H=16, N=2047, d=64, rot=32,
             layout="interleaved", dtype="fp32", order="bhnd", start=0, scaling="linear",
             factor=4.0),
        # One new token for each of 64 sequences at far positions of a stretched context.
        dict(name="rope-decode-far", op="rope", B=64, H=32, N=1, d=128, rot=128,
             layout="interleaved", dtype="bf16", order="bnhd", start=1000000, scaling="bands",
             factor=8.0),
        # A decoding step: one token of 64 sequences into bf16 pages, the queries rotated too.
        dict(name="append-decode-bf16", op="append", B=64, H=32, Hkv=8, N=1, d=128, past=4096,
             page=16, cache="bf16", rot=128, layout="half", ragged=True),
        # Prompts of different lengths, padded to the longest, into bf16 pages; half the head.
        dict(name="append-prompt-bf16", op="append", B=4, H=32, Hkv=8, N=4096, d=128, past=0,
             page=64, cache="bf16", rot=64, layout="interleaved", ragged=True),
        # A chunk of a long prompt into 4-bit pages, and the cache read out dense, as a dense
        # attention of the chunk takes it.
        dict(name="append-chunk-int4", op="append", B=4, H=32, Hkv=8, N=2048, d=128, past=1000,
             page=32, cache="int4", rot=128, layout="half", ragged=False),
        # The same for short odd prompts and small heads.
        dict(name="append-odd-int4-d64", op="append", B=16, H=16, Hkv=4, N=333, d=64, past=77,
             page=16, cache="int4", rot=64, layout="interleaved", ragged=True),
        # One sequence's next token over a short cache: latency.
        dict(name="attend-short-int4", op="attend", B=1, H=32, Hkv=8, Nq=1, d=128, len=1000,
             page=16, cache="int4", causal=True, ragged=False),
        # Decoding of 8 sequences over 32768 keys.
        dict(name="attend-long-int4", op="attend", B=8, H=32, Hkv=8, Nq=1, d=128, len=32768,
             page=64, cache="int4", causal=True, ragged=False),
        # Decoding of sequences of very different lengths over bf16 pages.
        dict(name="attend-ragged-bf16-d64", op="attend", B=24, H=32, Hkv=8, Nq=1, d=64, len=8191,
             page=16, cache="bf16", causal=True, ragged=True),
        # Checking up to 5 proposed tokens of each sequence, a shared head for 8 query heads.
        dict(name="attend-verify-int4", op="attend", B=16, H=32, Hkv=4, Nq=5, d=128, len=6001,
             page=32, cache="int4", causal=True, ragged=True),
        # A chunk of a prompt against a long cache.
        dict(name="attend-chunk-int4", op="attend", B=2, H=32, Hkv=8, Nq=1024, d=128, len=16384,
             page=64, cache="int4", causal=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "append", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    layout = rng.choice(["half", "interleaved"])
    if op in ("rope", "rope_bwd"):
        N = _log(rng, 1, 8192)
        H = rng.choice([1, 5, 8, 16, 32])
        B = max(1, min(64, _log(rng, 1, 64), 524288 // (N * H)))
        return dict(op=op, B=B, H=H, N=N, d=d, rot=rng.choice([d, d // 2, d // 4, 24]),
                    layout=layout, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    order=rng.choice(["bnhd", "bhnd"]), start=_log(rng, 1, 4000000),
                    scaling=rng.choice(["none", "linear", "ntk", "bands"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]))
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 7])
        N = _log(rng, 1, 2048)
        B = max(1, min(_log(rng, 1, 64), 8192 // N))
        return dict(op=op, B=B, H=H, Hkv=Hkv, N=N, d=d, past=_log(rng, 1, 1000) - 1,
                    page=rng.choice([16, 32, 48, 64, 128]), cache=rng.choice(["bf16", "int4"]),
                    rot=rng.choice([0, d, d // 2, 24]), layout=layout,
                    ragged=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 3, 4, 8, 16])
    Nq = rng.choice([1, 1, 1, 2, 7, _log(rng, 8, 512)])
    top = 65536 if Nq < 8 else 8192
    length = max(Nq, _log(rng, 1, top))
    room = min(262144 // length, (1 << 29) // (H * Nq * length))
    return dict(op=op, B=max(1, min(_log(rng, 1, 64), room)), H=H, Hkv=Hkv, Nq=Nq, d=d,
                len=length, page=rng.choice([16, 32, 48, 64, 128]),
                cache=rng.choice(["bf16", "int4", "int4"]), causal=rng.random() < 0.8,
                ragged=rng.random() < 0.5)


def _lens(case, most, least, salt):
    """Token counts of the case's sequences: all `most`, or, ragged, spread between."""
    if not case["ragged"]:
        return [most] * case["B"]
    r = random.Random("%d %d %d" % (case["B"], most, salt))
    out = [max(least, int(most * r.uniform(0.05, 1.0))) for _ in range(case["B"])]
    out[r.randrange(case["B"])] = most
    return out


def _inv_freq(rot, scaling="none", factor=1.0):
    """The rotation rates in radians a position, and the amplitude."""
    n, base, amp = rot // 2, 10000.0, 1.0
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(n)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "bands":
        # rates that turn more than 32 times within 4096 positions stay, those that turn less
        # than once are divided by the factor, and a ramp lies between
        w = [min(1.0, max(0.0, (4096.0 * x / (2 * math.pi) - 1.0) / 31.0)) for x in f]
        f = [x * (t + (1.0 - t) / factor) for x, t in zip(f, w)]
        amp = 0.1 * math.log(factor) + 1.0
    return f, amp


def _table(f, dev):
    """The rates in turns a position as 64-bit fractions (signed, modulo one turn)."""
    t = [int(x / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for x in f]
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in t], dtype=torch.int64,
                        device=dev)


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _randn(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _keys(shape, g, d):
    """Keys as projections make them: a few channels are much larger than the others."""
    w = torch.ones(d, device="cuda")
    w[torch.randperm(d, generator=g, device="cuda")[: d // 32]] = 4.0
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * w).to(
        torch.bfloat16)


def _quantise(x):
    """codes [..., d] (0..15) and the groups' words [..., d/64], from x [..., d]."""
    x = x.double().unflatten(-1, (-1, GROUP))
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    # the least step of three significant bits that spans the group and holds its base
    m, e = torch.frexp(torch.maximum((hi - lo) / 15, lo.abs() / 31))
    s = torch.ldexp(torch.ceil(m * 8) / 8, e)
    by = torch.where(s > 0, s, 1.0)
    b = torch.round(lo / by)
    codes = (torch.round(x / by) - b).clamp(0, 15).to(torch.uint8).flatten(-2)
    bits = s.to(torch.bfloat16).view(torch.int16).to(torch.int32) >> 5 << 6
    return codes, (bits | b.to(torch.int32) & 63).to(torch.int16).squeeze(-1)


def _pack(codes, words):
    """Page bytes [pages, heads, page * (d/2 + d/32)] of codes [pages, heads, page, d]."""
    c = codes.unflatten(-1, (-1, 2))
    b = (c[..., 0] | (c[..., 1] << 4)).flatten(-2)
    return torch.cat((b, words.flatten(-2).contiguous().view(torch.uint8)), -1)


def _pages(case, g, num_pages, keys):
    """Pages full of tokens written earlier."""
    shape = (num_pages, case["Hkv"], case["page"], case["d"])
    make = (lambda s: _keys(s, g, case["d"])) if keys else (lambda s: _randn(s, g))
    if case["cache"] == "bf16":
        return make(shape)
    parts = [_pack(*_quantise(make((min(512, num_pages - i),) + shape[1:])))
             for i in range(0, num_pages, 512)]
    return torch.cat(parts)


def _page_table(lens, page, g):
    """Each sequence's pages in order, scattered over the cache; -1 past its last one."""
    counts = [(n + page - 1) // page for n in lens]
    most, total = max(1, max(counts)), sum(counts)
    ids = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device="cuda")
    here = torch.arange(most, device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]
    table[here] = ids
    return table, total + 3


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    i32 = dict(dtype=torch.int32, device="cuda")
    if op in ("rope", "rope_bwd"):
        B, H, N, d = (case[k] for k in "BHNd")
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = _randn((B, N, H, d) if case["order"] == "bnhd" else (B, H, N, d), g, dt)
        s["x"] = x.transpose(1, 2) if case["order"] == "bnhd" else x
        start = torch.randint(0, case["start"] + 1, (B, 1), generator=g, **i32)
        s["positions"] = start + torch.arange(N, **i32)
        f, s["amplitude"] = _inv_freq(case["rot"], case["scaling"], case["factor"])
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["table"] = _table(f, "cuda")
        return s
    B, H, Hkv, d, page = (case[k] for k in ("B", "H", "Hkv", "d", "page"))
    if op == "append":
        N = case["N"]
        new = _lens(case, N, 1, 1)
        past = _lens(case, case["past"], 0, 2)
        total = [a + b for a, b in zip(past, new)]
        table, num_pages = _page_table(total, page, g)
        # the projections' output: queries, keys and values of a token side by side
        qkv = _randn((B, N, H + 2 * Hkv, d), g)
        s["q"], s["k"], s["v"] = (t.transpose(1, 2) for t in qkv.split([H, Hkv, Hkv], 2))
        s["cache_lens"] = torch.tensor(past, **i32)
        s["new_lens"] = torch.tensor(new, **i32)
        s["kv_lens"] = torch.tensor(total, **i32)
        s["most"] = max(total)
        # rows of padding tokens are not written: they keep what the buffer held
        s["q_out"] = torch.zeros((B, H, N, d), dtype=torch.bfloat16, device="cuda")
        s["page_table"] = table
        s["k_pages"], s["v_pages"] = (_pages(case, g, num_pages, k) for k in (True, False))
        f, s["amplitude"] = _inv_freq(case["rot"]) if case["rot"] else ([], 1.0)
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["table"] = _table(f, "cuda") if case["rot"] else None
        return s
    lens = _lens(case, case["len"], min(case["Nq"], case["len"]), 3)
    table, num_pages = _page_table(lens, page, g)
    s["q"] = _randn((B, H, case["Nq"], d), g)
    s["kv_lens"] = torch.tensor(lens, **i32)
    ql = _q_lens(case)
    s["q_lens"] = torch.tensor(ql, **i32) if ql else None
    s["most"] = max(lens)
    s["page_table"] = table
    s["k_pages"], s["v_pages"] = (_pages(case, g, num_pages, k) for k in (True, False))
    s["scale"] = 1.0 / math.sqrt(d)
    return s


def _q_lens(case):
    """Proposed tokens of each sequence where they differ, or None: all Nq."""
    if not case["ragged"] or case["Nq"] == 1:
        return None
    r = random.Random("%d %d" % (case["B"], case["Nq"]))
    return [r.randint(1, case["Nq"]) for _ in range(case["B"])]


# ------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------
def _angles(positions, inv_freq, amplitude):
    a = positions.double()[:, None, :, None] * inv_freq
    return a.cos() * amplitude, a.sin() * amplitude


def _rotate(x, c, s, rot, layout):
    """x [B, H, N, d] with its first `rot` values of each head rotated."""
    head, tail = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        return torch.cat((a * c - b * s, b * c + a * s, tail), -1)
    a, b = head[..., 0::2], head[..., 1::2]
    turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((turned, tail), -1)


def _plain_rope(s):
    case = s["case"]
    c, n = _angles(s["positions"], s["inv_freq"], s["amplitude"])
    n = -n if case["op"] == "rope_bwd" else n
    return _rotate(s["x"].float(), c.float(), n.float(), case["rot"], case["layout"]).to(
        s["x"].dtype)


def _slots(s, positions):
    """Page and place in it of positions [B, N]."""
    page = s["case"]["page"]
    p = s["page_table"].gather(1, (positions // page).clamp(max=s["page_table"].shape[1] - 1))
    return p.clamp(min=0).long(), (positions % page).long()


def _unpack(pages, case):
    """Values [pages, heads, page, d] in 32 bits of 4-bit pages."""
    P, d = case["page"], case["d"]
    b = pages[..., : P * d // 2].unflatten(-1, (P, d // 2))
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (d // GROUP, GROUP))
    w = pages[..., P * d // 2:].contiguous().view(torch.int16).unflatten(-1, (P, d // GROUP, 1))
    w = w.to(torch.int32)
    step = ((w & 0xffc0) << 15).view(torch.float32)
    base = ((w & 63) ^ 32) - 32
    return (step * (base + c)).flatten(-2)


def _dense(s, pages, n):
    """Tokens 0 .. n-1 of every sequence in 32 bits: [B, Hkv, n, d]."""
    case = s["case"]
    table = s["page_table"][:, : (n + case["page"] - 1) // case["page"]].clamp(min=0).long()
    x = pages[table]
    x = x.float() if case["cache"] == "bf16" else _unpack(x, case)
    return x.transpose(1, 2).flatten(2, 3)[:, :, :n]


def _plain_append(s):
    case = s["case"]
    N, rot = case["N"], case["rot"]
    n = torch.arange(N, device="cuda")
    pos = s["cache_lens"][:, None] + n
    real = n < s["new_lens"][:, None]
    k, q = s["k"].double(), s["q"].float()
    if rot:
        c, t = _angles(pos, s["inv_freq"], s["amplitude"])
        k = _rotate(k, c, t, rot, case["layout"])
        q = _rotate(q, c.float(), t.float(), rot, case["layout"])
    s["q_out"].copy_(torch.where(real[:, None, :, None], q.to(torch.bfloat16), s["q_out"]))
    page, place = _slots(s, pos)
    page, place = page[real], place[real]
    for pages, x in ((s["k_pages"], k), (s["v_pages"], s["v"])):
        x = x.transpose(1, 2)[real]  # [tokens, Hkv, d]
        if case["cache"] == "bf16":
            pages[page, :, place] = x.to(torch.bfloat16)
        else:
            codes, words = _quantise(x)
            codes = codes.unflatten(-1, (-1, 2))
            P, d = case["page"], case["d"]
            body = pages[..., : P * d // 2].unflatten(-1, (P, d // 2))
            body[page, :, place] = codes[..., 0] | (codes[..., 1] << 4)
            tail = pages[..., P * d // 2:].unflatten(-1, (P, d // 32))
            tail[page, :, place] = words.contiguous().view(torch.uint8)
    if case["cache"] == "bf16":
        return s["q_out"], s["k_pages"], s["v_pages"]
    here = torch.arange(s["most"], device="cuda") < s["kv_lens"][:, None]
    here = here[:, None, :, None]
    return (s["q_out"],
            torch.where(here, _dense(s, s["k_pages"], s["most"]), 0.0).to(torch.bfloat16),
            torch.where(here, _dense(s, s["v_pages"], s["most"]), 0.0).to(torch.bfloat16))


def _plain_attend(s):
    case = s["case"]
    B, H, Hkv, Nq, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "d"))
    k = _dense(s, s["k_pages"], s["most"])
    q = s["q"].float().view(B, Hkv, (H // Hkv) * Nq, d)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, H, Nq, s["most"])
    del k
    i, j = torch.arange(Nq, device="cuda"), torch.arange(s["most"], device="cuda")
    ql = s["q_lens"] if s["q_lens"] is not None else torch.full_like(s["kv_lens"], Nq)
    last = s["kv_lens"][:, None] - 1 + ((i - ql[:, None] + 1) if case["causal"] else 0 * i)
    last = torch.where(i < ql[:, None], last, -1)
    x.masked_fill_(j > last[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _dense(s, s["v_pages"], s["most"])
    o = (p.view(B, Hkv, -1, s["most"]) @ v).view(B, H, Nq, d)
    o = o / torch.where(total > 0, total, 1.0)
    return o.to(torch.bfloat16), (m + total.log()).squeeze(-1)


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def _own(s):
    from online_softmax_tiled_attn_gb300 import binding as osm

    case = s["case"]
    if case["op"] == "rope":
        return osm.osm_rope(s["x"], s["table"], positions=s["positions"], layout=case["layout"],
                            amplitude=s["amplitude"])
    if case["op"] == "rope_bwd":
        return osm.osm_rope_bwd(s["x"], s["table"], positions=s["positions"],
                                layout=case["layout"], amplitude=s["amplitude"])
    if case["op"] == "append":
        osm.osm_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"],
                          s["cache_lens"], new_lens=s["new_lens"], table=s["table"],
                          layout=case["layout"], amplitude=s["amplitude"], q=s["q"],
                          q_out=s["q_out"])
        if case["cache"] == "bf16":
            return s["q_out"], s["k_pages"], s["v_pages"]
        k, v = osm.osm_kv_gather(s["k_pages"], s["v_pages"], s["page_table"], s["kv_lens"],
                                 s["most"], case["d"])
        return s["q_out"], k, v
    return osm.fa_fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_lens"],
                            q_lens=s["q_lens"], scale=s["scale"], causal=case["causal"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return (_plain_attend if op == "attend" else _plain_append if op == "append"
            else _plain_rope)(state)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    d = case["d"]
    if case["op"] in ("rope", "rope_bwd"):
        n = case["B"] * case["H"] * case["N"]
        return {"bytes": 2 * n * d * (2 if case["dtype"] == "bf16" else 4), "flops": 3 * n * d}
    row = 2 * d if case["cache"] == "bf16" else d // 2 + d // 32  # a cached token's head
    if case["op"] == "append":
        new = sum(_lens(case, case["N"], 1, 1))
        total = new + sum(_lens(case, case["past"], 0, 2))
        n = new * (4 * d * case["H"] + 2 * case["Hkv"] * (2 * d + row))
        if case["cache"] == "int4":  # the read-out: every token once, and zeros behind it
            most = max(a + b for a, b in zip(_lens(case, case["N"], 1, 1),
                                             _lens(case, case["past"], 0, 2)))
            n += 2 * case["Hkv"] * (total * row + case["B"] * most * 2 * d)
        return {"bytes": n, "flops": 3 * new * d * (case["H"] + case["Hkv"])}
    lens = _lens(case, case["len"], min(case["Nq"], case["len"]), 3)
    ql = _q_lens(case) or [case["Nq"]] * case["B"]
    pairs = sum(sum(max(0, n - q + i + 1) for i in range(q)) if case["causal"] else n * q
                for n, q in zip(lens, ql))
    rows = case["B"] * case["H"] * case["Nq"]
    return {"bytes": 2 * sum(lens) * case["Hkv"] * row + rows * (4 * d + 4),
            "flops": 4 * pairs * case["H"] * d}


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------
def _turned(x, positions, f, amplitude, layout):
    """x [..., N, d] with the pairs of its first 2 len(f) values as complex numbers, each
    multiplied by amplitude * exp(i * position * rate)."""
    n = len(f)
    rate = torch.tensor(f, dtype=torch.float64, device=x.device)
    w = torch.polar(torch.full((), amplitude, dtype=torch.float64, device=x.device),
                    positions.double()[..., None] * rate)
    re = torch.arange(n, device=x.device) * (1 if layout == "half" else 2)
    im = re + (n if layout == "half" else 1)
    y = x.double().clone()
    t = torch.complex(y[..., re], y[..., im]) * w
    y[..., re], y[..., im] = t.real, t.imag
    return y


def _stored(x):
    """What a 4-bit cache gives back for x [..., d]."""
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], GROUP):
        v = x[..., a:a + GROUP]
        low = v.min(-1, keepdim=True).values
        need = torch.maximum((v.max(-1, keepdim=True).values - low) / 15, low.abs() / 31)
        unit = torch.exp2(torch.floor(torch.log2(need)) - 2)
        step = torch.ceil(need / unit) * unit
        base = (low / step).round()
        out[..., a:a + GROUP] = step * torch.minimum((v / step).round(), base + 15)
    return out


def _read(pages, ids, case):
    """Pages `ids` of one sequence as values [Hkv, tokens, d] in 64 bits."""
    P, d, H = case["page"], case["d"], case["Hkv"]
    raw = pages[ids.long()]
    if case["cache"] == "bf16":
        return raw.double().transpose(0, 1).reshape(H, -1, d)
    word = raw[:, :, P * d // 2:].contiguous().view(torch.int16).long() % 65536
    step = torch.exp2((word >> 8).double() - 127) * (1 + (word >> 6) % 4 / 4)
    base = (word + 32) % 64 - 32
    step, base = (t.view(len(ids), H, P, d // GROUP).repeat_interleave(GROUP, 3)
                  for t in (step, base))
    x = torch.empty((len(ids), H, P, d), dtype=torch.float64, device=raw.device)
    body = raw[:, :, : P * d // 2].reshape(len(ids), H, P, d // 2).double()
    x[..., 0::2], x[..., 1::2] = body % 16, body // 16
    return ((base + x) * step).transpose(0, 1).reshape(H, -1, d)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op in ("rope", "rope_bwd"):
        f, amp = _inv_freq(case["rot"], case["scaling"], case["factor"])
        sign = -1 if op == "rope_bwd" else 1
        return _turned(s["x"].contiguous(), sign * s["positions"][:, None], f, amp,
                       case["layout"])
    page, Hkv, B = case["page"], case["Hkv"], case["B"]
    if op == "append":
        f, amp = _inv_freq(case["rot"]) if case["rot"] else ([], 1.0)
        q_out = s["q_out"].double()
        most = s["most"]
        if case["cache"] == "bf16":
            dense = [s["k_pages"].double(), s["v_pages"].double()]
        else:
            dense = [torch.zeros((B, Hkv, most, d), dtype=torch.float64, device="cuda")
                     for _ in range(2)]
        for b, (past, new) in enumerate(zip(s["cache_lens"].tolist(), s["new_lens"].tolist())):
            pos = torch.arange(past, past + new, device="cuda")
            q_out[b, :, :new] = _turned(s["q"][b, :, :new], pos, f, amp, case["layout"])
            k = _turned(s["k"][b, :, :new], pos, f, amp, case["layout"])
            v = s["v"][b, :, :new].double()
            ids = s["page_table"][b].long()
            for x, to, pages in ((k, dense[0], s["k_pages"]), (v, dense[1], s["v_pages"])):
                if case["cache"] == "bf16":
                    to[ids[pos // page], :, pos % page] = x.transpose(0, 1)
                else:
                    n = (past + page - 1) // page
                    if past:
                        to[b, :, :past] = _read(pages, ids[:n], case)[:, :past]
                    to[b, :, past:past + new] = _stored(x)
        return q_out, dense[0], dense[1]
    H, Nq = case["H"], case["Nq"]
    o = torch.zeros((B, H, Nq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    queries = _q_lens(case) or [Nq] * B
    for b, (n, nq) in enumerate(zip(s["kv_lens"].tolist(), queries)):
        ids = s["page_table"][b, : (n + page - 1) // page]
        K, V = (_read(s[t], ids, case)[:, :n] for t in ("k_pages", "v_pages"))
        for h in range(H):
            g = h // (H // Hkv)
            x = s["q"][b, h, :nq].double() @ K[g].T * s["scale"]
            if case["causal"]:
                x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(n - nq + 1), -math.inf)
            lse[b, h, :nq] = torch.logsumexp(x, -1)
            o[b, h, :nq] = torch.softmax(x, -1).nan_to_num() @ V[g]
    return o, lse
