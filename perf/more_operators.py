"""Cases for the pages of a paged key/value cache that several sequences share: giving growing
sequences their pages (osm_kv_grow), forking sequences (osm_kv_fork), giving pages back
(osm_kv_free), closing the gaps of a cache (osm_kv_compact), and attention for groups of sequences
with a common prefix, which is read once for the group (fa_fwd_paged_shared).

The cache is a pool of pages for keys and one for values, a table of page numbers for each sequence
(a row), the rows' tokens (lens) and each page's uses (refs; a page without one is free).  A fork
shares all of its source's pages; a page that is not full is copied when one of its rows grows.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # A decoding step of 64 sequences: every sixteenth of them, or so, begins a page.
        dict(name="grow-decode-int4", op="grow", S=64, page=16, len=8191, new=1, most=8208, fan=1,
             spread=1.3, Hkv=8, d=128, cache="int4", ragged=True),
        # The first step of 8 prompts' samples, 8 drawn of each: a page that is not full is copied
        # before its sequences write on.
        dict(name="grow-samples-bf16", op="grow", S=64, page=64, len=4001, new=3, most=4224, fan=8,
             spread=1.5, Hkv=8, d=128, cache="bf16", ragged=True),
        # Eight prompts of about 4000 tokens, four samples drawn of each.
        dict(name="fork-samples", op="fork", S=40, page=64, len=4001, fan=1, spread=1.5, parents=8,
             ragged=True),
        # One long prompt in small pages for 64 branches.
        dict(name="fork-prompt", op="fork", S=80, page=16, len=32700, fan=1, spread=2.0, parents=1,
             ragged=False),
        # Proposed tokens that were refused: the ends of 64 rows.
        dict(name="free-refused", op="free", S=64, page=16, len=4099, fan=1, spread=1.2, rows=64,
             keep=0.998, ragged=True),
        # A finished half of 128 long rows, in families of 8 that share half of their pages.
        dict(name="free-finished", op="free", S=128, page=16, len=32768, fan=8, spread=1.1, rows=64,
             keep=0.0, ragged=True),
        # A pool with as many gaps as pages in use, closed.
        dict(name="compact-bf16", op="compact", S=64, page=64, len=8192, fan=1, spread=2.0, Hkv=8,
             d=128, cache="bf16", ragged=True),
        # The same for small 4-bit pages, some of them shared, fewer gaps.
        dict(name="compact-odd-int4", op="compact", S=31, page=48, len=3001, fan=3, spread=1.2,
             Hkv=3, d=64, cache="int4", ragged=True),
        # Eight samples of a short prompt: latency.
        dict(name="shared-samples-bf16-d64", op="shared", sizes="8", prefix=1000, own=40, H=16,
             Hkv=4, Nq=1, d=64, page=16, cache="bf16", causal=True),
        # 64 conversations behind one long set of instructions.
        dict(name="shared-instructions-bf16", op="shared", sizes="64", prefix=16384, own=1000, H=32,
             Hkv=8, Nq=1, d=128, page=64, cache="bf16", causal=True),
        # 32 branches of a long document, 3 proposed tokens each to check.
        dict(name="shared-document-int4", op="shared", sizes="32", prefix=32768, own=512, H=32,
             Hkv=8, Nq=3, d=128, page=32, cache="int4", causal=True),
        # Groups of several sizes, one sequence that shares nothing, odd lengths.
        dict(name="shared-groups-int4-d64", op="shared", sizes="3 12 1 7", prefix=7777, own=333,
             H=32, Hkv=4, Nq=1, d=64, page=48, cache="int4", causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grow", "fork", "free", "compact", "shared", "shared", "shared", "shared"])
    page = rng.choice([16, 32, 48, 64, 128])
    d = rng.choice([64, 128])
    if op == "shared":
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 3, 4, 8])
        Nq = rng.choice([1, 1, 2, 5])
        prefix = _log(rng, 100, 32768)
        B = max(2, min(_log(rng, 2, 64), 1048576 // prefix))
        sizes = []
        while B > 0:
            sizes.append(min(B, rng.choice([1, 2, 5, 16, 64])))
            B -= sizes[-1]
        return dict(op=op, sizes=" ".join(map(str, sizes)), prefix=prefix,
                    own=_log(rng, 8, 1000), H=H, Hkv=Hkv,
                    Nq=Nq, d=d, page=page, cache=rng.choice(["bf16", "int4"]),
                    causal=rng.random() < 0.8)
    S, length = _log(rng, 2, 128), _log(rng, 20, 16384)
    length = min(length, max(20, 262144 // S))
    base = dict(op=op, S=S, page=page, len=length, fan=rng.choice([1, 1, 3, 8]),
                spread=1.0 + _log(rng, 1, 400) / 100, ragged=rng.random() < 0.7)
    if op == "free":
        return dict(base, rows=rng.randint(1, S), keep=rng.choice([0.0, 0.5, 0.99]))
    if op == "fork":
        return dict(base, parents=rng.randint(1, max(1, S // 2)))
    base.update(Hkv=rng.choice([1, 2, 3, 8]), d=d, cache=rng.choice(["bf16", "int4"]))
    if op == "grow":
        new = _log(rng, 1, 2048)
        return dict(base, new=new, most=length + new + rng.randrange(1000))
    return base


def _lens(n, most, least, ragged, salt):
    """n token counts: all `most`, or, ragged, spread between."""
    if not ragged:
        return [most] * n
    r = random.Random("%d %d %d" % (n, most, salt))
    out = [max(least, int(most * r.uniform(0.05, 1.0))) for _ in range(n)]
    out[r.randrange(n)] = most
    return out


def _plan(case):
    """The case's numbers that do not depend on the seed: rows' tokens and what is done to them."""
    S, P, op = case["S"], case["page"], case["op"]
    live = case["parents"] if op == "fork" else S
    lens = _lens(live, case["len"], min(1, case["len"]), case["ragged"], 1) + [0] * (S - live)
    # A family shares the first half of its first row's full pages, where a row has as many; rows
    # about to grow are fresh forks of it and share all, a last page that is not full among them.
    shared = [0] * S
    for b in range(live):
        head = b - b % case["fan"]
        if b != head and op == "grow":
            lens[b] = lens[head]
            shared[b] = (lens[b] + P - 1) // P
        elif b != head:
            shared[b] = min(lens[head] // 2, lens[b]) // P
    out = {"lens": lens, "shared": shared}
    r = random.Random("%d %d %s" % (S, case["len"], op))
    if op == "grow":
        out["new"] = _lens(S, case["new"], 0, case["ragged"], 2)
        room = (case["most"] + P - 1) // P * P
        out["copies"] = [b for b in range(S) if case["fan"] > 1 and lens[b] % P and
                         min(out["new"][b], room - lens[b]) > 0 and
                         (shared[b] or b + 1 < S and shared[b + 1])]
    elif op == "fork":
        out["src"] = [r.randrange(live) for _ in range(S - live)]
        out["dst"] = list(range(live, S))
        r.shuffle(out["dst"])
    elif op == "free":
        out["rows"] = r.sample(range(S), case["rows"])
        out["keep"] = [int(lens[b] * case["keep"]) for b in out["rows"]]
    most = case.get("most", max(lens))
    out["max_pages"] = (most + P - 1) // P
    used = sum((n + P - 1) // P - s for n, s in zip(lens, shared))
    if op == "grow":  # room for the new tokens' pages and the copies
        used += sum((min(n + m, room) + P - 1) // P - n // P for n, m in zip(lens, out["new"]))
    out["num_pages"] = int(used * case["spread"]) + 3
    return out


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


def _quantised(x):
    """Bytes [pages, heads, page * (d/2 + d/32)] of 4-bit pages of values x [pages, heads, page, d]."""
    x = x.float().unflatten(-1, (-1, GROUP))
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    m, e = torch.frexp(torch.maximum((hi - lo) / 15, lo.abs() / 31))
    s = torch.ldexp(torch.ceil(m * 8) / 8, e)
    by = torch.where(s > 0, s, 1.0)
    b = torch.round(lo / by)
    codes = (torch.round(x / by) - b).clamp(0, 15).to(torch.uint8).flatten(-2)
    bits = s.to(torch.bfloat16).view(torch.int16).to(torch.int32) >> 5 << 6
    words = (bits | b.to(torch.int32) & 63).to(torch.int16).squeeze(-1)
    c = codes.unflatten(-1, (-1, 2))
    body = (c[..., 0] | (c[..., 1] << 4)).flatten(-2)
    return torch.cat((body, words.flatten(-2).contiguous().view(torch.uint8)), -1)


def _pages(case, g, num_pages, keys):
    """Pages full of tokens written earlier."""
    shape = (num_pages, case["Hkv"], case["page"], case["d"])
    make = (lambda s: _keys(s, g, case["d"])) if keys else (lambda s: _randn(s, g))
    parts = []
    for i in range(0, num_pages, 512):
        x = make((min(512, num_pages - i),) + shape[1:])
        parts.append(x if case["cache"] == "bf16" else _quantised(x))
    return torch.cat(parts)


def _table(lens, shared, heads, P, max_pages, num_pages, rng):
    """(table [S, max_pages], refs [num_pages]): row b's first shared[b] entries are those of row
    heads[b], the others its own, scattered over the pool; -1 past its last one."""
    ids = rng.permutation(num_pages).astype(np.int32)
    table = np.full((len(lens), max_pages), -1, dtype=np.int32)
    refs = np.zeros(num_pages, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        n = (n + P - 1) // P
        table[b, : shared[b]] = table[heads[b], : shared[b]]
        table[b, shared[b]:n] = ids[at:at + n - shared[b]]
        at += n - shared[b]
        refs[table[b, :n]] += 1
    return table, refs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 32))
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": case}
    P = case["page"]
    if case["op"] == "shared":
        H, Hkv, Nq, d = (case[k] for k in ("H", "Hkv", "Nq", "d"))
        lens, shared, heads, groups = _members(case)
        B = len(lens)
        used = sum((n + P - 1) // P - c for n, c in zip(lens, shared))
        table, _ = _table(lens, shared, heads, P, (max(lens) + P - 1) // P, used + 3, rng)
        s["page_table"] = torch.from_numpy(table).cuda()
        s["kv_lens"] = torch.tensor(lens, **i32)
        s["groups"] = torch.tensor(groups, **i32)
        s["q"] = _randn((B, H, Nq, d), g)
        s["k_pages"], s["v_pages"] = (_pages(case, g, used + 3, k) for k in (True, False))
        s["scale"] = 1.0 / math.sqrt(d)
        s["lens"] = lens
        return s
    plan = _plan(case)
    S, M, N = case["S"], plan["max_pages"], plan["num_pages"]
    heads = [b - b % case["fan"] for b in range(S)]
    table, refs = _table(plan["lens"], plan["shared"], heads, P, M, N, rng)
    # The table, the rows' tokens and the pages' uses in one buffer: a pass starts from the same
    # ones each time, which one copy puts back.
    parts = [table.ravel(), np.array(plan["lens"], dtype=np.int32), refs]
    places, at = [], 0
    for x in parts:
        places.append(at)
        at += (len(x) + 63) // 64 * 64
    start = np.zeros(at, dtype=np.int32)
    for x, p in zip(parts, places):
        start[p:p + len(x)] = x
    s["start"] = torch.from_numpy(start).cuda()
    s["live"] = s["start"].clone()
    views = [s["live"][p:p + len(x)] for x, p in zip(parts, places)]
    s["page_table"], s["lens"], s["refs"] = views[0].view(S, M), views[1], views[2]
    for name in ("new", "src", "dst", "rows", "keep"):
        if name in plan:
            s[name] = torch.tensor(plan[name], **i32)
    if "cache" in case:
        s["k_pages"], s["v_pages"] = (_pages(case, g, N, k) for k in (True, False))
    return s


def _members(case):
    """Tokens of the sequences, the pages that each shares, with which row, and the groups."""
    r = random.Random("%s %d %d" % (case["sizes"], case["prefix"], case["own"]))
    lens, shared, heads, groups = [], [], [], []
    for j, n in enumerate(map(int, case["sizes"].split())):
        prefix = case["prefix"] if j == 0 else int(case["prefix"] * r.uniform(0.2, 1.0))
        head = len(lens)
        for i in range(n):
            lens.append(prefix + max(case["Nq"], int(case["own"] * r.uniform(0.05, 1.0))))
            shared.append(prefix // case["page"] if i else 0)
            heads.append(head)
            groups.append(j)
    return lens, shared, heads, groups


# ------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------
def _free_pages(refs):
    """The free pages in order, -1 behind the last one, and each page's rank among them."""
    free = refs <= 0
    rank = free.cumsum(0) - 1
    n = refs.numel()
    ids = torch.full((n + 1,), -1, dtype=torch.int32, device="cuda")
    ids.scatter_(0, torch.where(free, rank, n), torch.arange(n, dtype=torch.int32, device="cuda"))
    ids[n] = -1
    return ids, torch.where(free, rank, n)


def _plain_grow(s):
    case, table, lens, refs = s["case"], s["page_table"], s["lens"], s["refs"]
    P, d = case["page"], case["d"]
    old = lens.clone()
    new = (old + s["new"]).clamp(max=table.shape[1] * P)
    last = (old // P).clamp(max=table.shape[1] - 1)
    holds = table.gather(1, last[:, None].long()).squeeze(1)
    # a last page that is not full and that others use too is replaced by a copy
    copies = (new > old) & (old % P > 0) & (refs[holds.clamp(min=0)] > 1)
    first = torch.where(copies, last, (old + P - 1) // P)
    need = (new + P - 1) // P - first
    before = need.cumsum(0) - need
    ids, rank = _free_pages(refs)
    j = torch.arange(table.shape[1], device="cuda")
    mine = (j >= first[:, None]) & (j < ((new + P - 1) // P)[:, None])
    at = (before[:, None] + j - first[:, None]).clamp(0, len(ids) - 1)
    table.copy_(torch.where(mine, ids[at], table))
    refs.copy_(torch.where(rank < need.sum(), 1, refs))
    a = holds[copies].long()
    b = table.gather(1, last[:, None].long()).squeeze(1)[copies].long()
    refs.index_add_(0, a, torch.full_like(a, -1, dtype=torch.int32))
    keep = torch.arange(P, device="cuda") < (old % P)[copies][:, None]  # [copies, P]
    for pages in (s["k_pages"], s["v_pages"]):
        if case["cache"] == "bf16":
            pages[b] = torch.where(keep[:, None, :, None], pages[a], pages[b])
        else:
            codes = keep.repeat_interleave(d // 2, 1)
            words = keep.repeat_interleave(d // 32, 1)
            pages[b] = torch.where(torch.cat((codes, words), 1)[:, None], pages[a], pages[b])
    lens.copy_(new)
    return table, lens, refs, old, s["k_pages"], s["v_pages"]


def _plain_fork(s):
    P, table, lens, refs = s["case"]["page"], s["page_table"], s["lens"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    L = lens[src]
    here = torch.arange(table.shape[1], device="cuda") < ((L + P - 1) // P)[:, None]
    rows = torch.where(here, table[src], table[dst])
    refs.scatter_add_(0, rows.clamp(min=0).long().flatten(), here.to(torch.int32).flatten())
    table[dst] = rows
    lens[dst] = L
    return table, lens, refs


def _plain_free(s):
    P, table, lens, refs = s["case"]["page"], s["page_table"], s["lens"], s["refs"]
    rows = s["rows"].long()
    keep = torch.minimum(s["keep"], lens[rows])
    j = torch.arange(table.shape[1], device="cuda")
    gone = (j >= ((keep + P - 1) // P)[:, None]) & (j < ((lens[rows] + P - 1) // P)[:, None])
    pages = table[rows].clamp(min=0).long()
    refs.scatter_add_(0, pages.flatten(), -gone.to(torch.int32).flatten())
    refs.clamp_(min=0)
    lens[rows] = keep
    return lens, refs


def _plain_compact(s):
    case, table, lens, refs = s["case"], s["page_table"], s["lens"], s["refs"]
    P, n = case["page"], refs.numel()
    page = torch.arange(n, device="cuda")
    taken = refs > 0
    used = taken.sum()
    source = (taken & (page >= used)).nonzero().squeeze(-1)
    to = (~taken & (page < used)).nonzero().squeeze(-1)
    where = torch.where(taken, page, -1)
    where[source] = to
    where = where.to(torch.int32)
    refs[to] = refs[source]
    refs[source] = 0
    for pages in (s["k_pages"], s["v_pages"]):
        pages[to] = pages[source]
    here = torch.arange(table.shape[1], device="cuda") < ((lens + P - 1) // P)[:, None]
    table.copy_(torch.where(here, where[table.clamp(min=0).long()], table))
    return table, refs, where, used.to(torch.int32).view(1), s["k_pages"], s["v_pages"]


def _values(pages, case):
    """Values [pages, heads, page, d] in 32 bits."""
    if case["cache"] == "bf16":
        return pages.float()
    P, d = case["page"], case["d"]
    b = pages[..., : P * d // 2].unflatten(-1, (P, d // 2))
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (d // GROUP, GROUP))
    w = pages[..., P * d // 2:].contiguous().view(torch.int16).unflatten(-1, (P, d // GROUP, 1))
    w = w.to(torch.int32)
    return (((w & 0xffc0) << 15).view(torch.float32) * (((w & 63) ^ 32) - 32 + c)).flatten(-2)


def _plain_shared(s):
    case = s["case"]
    H, Hkv, Nq, d, P = (case[k] for k in ("H", "Hkv", "Nq", "d", "page"))
    outs, lses = [], []
    for b, n in enumerate(s["lens"]):
        ids = s["page_table"][b, : (n + P - 1) // P].long()
        k, v = (_values(s[t][ids], case).transpose(0, 1).flatten(1, 2)[:, :n]
                for t in ("k_pages", "v_pages"))
        q = s["q"][b].float().view(Hkv, (H // Hkv) * Nq, d)
        x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(H, Nq, n)
        if case["causal"]:
            i, j = torch.arange(Nq, device="cuda"), torch.arange(n, device="cuda")
            x.masked_fill_(j > n - Nq + i[:, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = x.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        o = (p.view(Hkv, -1, n) @ v).view(H, Nq, d) / total
        outs.append(o.to(torch.bfloat16))
        lses.append((m + total.log()).squeeze(-1))
    return torch.stack(outs), torch.stack(lses)


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def _own(s):
    from online_softmax_tiled_attn_gb300 import binding as osm

    case = s["case"]
    op, page = case["op"], case["page"]
    if op == "shared":
        return osm.fa_fwd_paged_shared(s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                                       s["kv_lens"], groups=s["groups"], scale=s["scale"],
                                       causal=case["causal"])
    table, lens, refs = s["page_table"], s["lens"], s["refs"]
    if op == "grow":
        old = osm.osm_kv_grow(s["k_pages"], s["v_pages"], table, lens, s["new"], refs, case["d"])
        return table, lens, refs, old, s["k_pages"], s["v_pages"]
    if op == "free":
        osm.osm_kv_free(table, lens, refs, page, rows=s["rows"], keep_lens=s["keep"])
        return lens, refs
    if op == "fork":
        osm.osm_kv_fork(table, lens, refs, page, s["src"], s["dst"])
        return table, lens, refs
    where, used = osm.osm_kv_compact(s["k_pages"], s["v_pages"], table, lens, refs, case["d"])
    return table, refs, where, used, s["k_pages"], s["v_pages"]


def run(state):
    op = state["case"]["op"]
    if op != "shared":
        state["live"].copy_(state["start"])
    if own:
        return _own(state)
    return {"grow": _plain_grow, "fork": _plain_fork, "free": _plain_free,
            "compact": _plain_compact, "shared": _plain_shared}[op](state)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    P = case["page"]
    if "cache" in case:
        d = case["d"]
        row = 2 * d if case["cache"] == "bf16" else d // 2 + d // 32  # a token's head
    if case["op"] == "shared":
        H, Hkv, Nq = case["H"], case["Hkv"], case["Nq"]
        lens, shared, _, _ = _members(case)
        tokens = sum(n - c * P for n, c in zip(lens, shared))
        pairs = sum(sum(n - Nq + i + 1 for i in range(Nq)) if case["causal"] else n * Nq
                    for n in lens)
        return {"bytes": 2 * tokens * Hkv * row + len(lens) * H * Nq * (4 * d + 4),
                "flops": 4 * pairs * H * d}
    plan = _plan(case)
    lens, N = plan["lens"], plan["num_pages"]

    def pages(n):
        return (n + P - 1) // P

    if case["op"] == "grow":
        room = plan["max_pages"] * P
        given = sum(pages(min(n + m, room)) - pages(n) for n, m in zip(lens, plan["new"]))
        tokens = sum(lens[b] % P for b in plan["copies"])
        return {"bytes": 4 * N + 8 * (given + len(plan["copies"])) + 16 * len(lens) +
                4 * tokens * case["Hkv"] * row, "flops": 0}
    if case["op"] == "free":
        gone = sum(pages(lens[b]) - pages(min(k, lens[b]))
                   for b, k in zip(plan["rows"], plan["keep"]))
        return {"bytes": 12 * gone + 16 * len(plan["rows"]), "flops": 0}
    if case["op"] == "fork":  # entries read and written, their pages' uses read and written
        return {"bytes": sum(16 * pages(lens[b]) + 12 for b in plan["src"]), "flops": 0}
    used = sum(pages(n) - c for n, c in zip(lens, plan["shared"]))
    moved = used * (N - used) // N  # pages scattered evenly over the pool
    return {"bytes": 4 * moved * P * case["Hkv"] * row + 12 * N + 4 * sum(map(pages, lens)),
            "flops": 0}


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------
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
    """Of the attention; what the other operators return is whole numbers and copies."""
    if case["op"] != "shared":
        return None
    s = prepare(case, seed)
    H, Hkv, Nq, d, P = (case[k] for k in ("H", "Hkv", "Nq", "d", "page"))
    B = len(s["lens"])
    o = torch.zeros((B, H, Nq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H, Nq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"]):
        ids = s["page_table"][b, : (n + P - 1) // P]
        K, V = (_read(s[t], ids, case)[:, :n] for t in ("k_pages", "v_pages"))
        for h in range(H):
            x = s["q"][b, h].double() @ K[h // (H // Hkv)].T * s["scale"]
            if case["causal"]:
                x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(n - Nq + 1), -math.inf)
            lse[b, h] = torch.logsumexp(x, -1)
            o[b, h] = torch.softmax(x, -1) @ V[h // (H // Hkv)]
    return o, lse
