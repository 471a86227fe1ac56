"""fa_fwd_paged_shared on the GPU against plain fp64 restatements: groups of sequences whose first
pages are the same ones.  The tolerances are those of the paged attention (cache_ref.attend): the
common part's shares are rounded to bf16 as counted there, its products are of exact bf16 values, and
joining two states adds a handful of fp32 roundings to the n / 16 + 16 that are counted.

Sequences that could not have much in common are fa_fwd_paged's, by the shape of the call: so the
tables here are wide, with nonsense in the entries that no token needs."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding
from test_kv_cache_gpu import check, filled, i32, rand

pytestmark = pytest.mark.gpu


def tables(sizes, prefix, lens, P, seed, width=None):
    """(table, pages in the pool, groups): group j's sequences share the pages that are full within
    prefix[j] tokens; the other pages are their own, scattered; unused entries hold nonsense."""
    n = [(x + P - 1) // P for x in lens]
    M = width or max(n)
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(sum(n) + 3, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(M, 1)), -7, dtype=torch.int32)
    at, b, groups = 0, 0, []
    for j, size in enumerate(sizes):
        head = b
        for i in range(size):
            c = min(prefix[j] // P, n[b], n[head]) if i else 0
            table[b, :c] = table[head, :c]
            table[b, c:n[b]] = ids[at:at + n[b] - c]
            at += n[b] - c
            groups.append(7 - 3 * j)
            b += 1
    return table, sum(n) + 3, groups


def wide(B, Hkv, P):
    """Entries of a row for which the call shares what it can: 2^22 tokens over the heads and the
    sequences but one."""
    return -(-(1 << 22) // ((B - 1) * Hkv * P))


def widened(table, entries):
    M = max(entries, table.shape[1])
    return torch.cat((table, torch.full((len(table), M - table.shape[1]), -3, dtype=torch.int32)), 1)


def run(q, kp, vp, table, lens, groups, q_lens, causal, P, **kw):
    B, H, Nq, d = q.shape
    table = widened(table, wide(B, kp.shape[1], P))
    fmt = "bf16" if kp.dtype == torch.bfloat16 else "int4"
    shape = (B, H, kp.shape[1], Nq, d, fmt, P, table.shape[1])
    assert binding.paged_shared_plan(*shape) > binding.paged_plan(*shape)  # it shares
    O, L = binding.fa_fwd_paged_shared(q, kp, vp, table.cuda(), i32(lens),
                                       groups=None if groups is None else i32(groups),
                                       q_lens=None if q_lens is None else i32(q_lens),
                                       causal=causal, **kw)
    torch.cuda.synchronize()
    return O, L


# sizes, prefix, own tokens (cycled), H, Hkv, Nq, d, page, q_lens (cycled) or None, causal
CASES = [
    ([2], [256], [1], 1, 1, 1, 64, 16, None, True),
    ([8], [1000], [40, 3, 77], 16, 4, 1, 64, 16, None, True),
    ([5], [300], [20, 1], 8, 2, 3, 128, 48, [3, 1, 0, 2], True),
    ([3, 4, 1, 2], [700, 140, 999, 2500], [9, 200, 31], 8, 1, 2, 128, 32, None, True),
    ([33], [513], [5, 130], 12, 4, 1, 128, 64, None, True),       # 99 rows: one block, alternate tiles
    ([50], [400], [12, 300], 8, 2, 1, 64, 128, None, False),      # 200 rows: two halves
    ([80], [1300], [2, 65, 128], 16, 4, 1, 128, 16, None, True),  # 320 rows: a block and a half
    ([3], [128], [1], 4, 4, 1, 128, 16, None, True),              # just too little to share
    ([3], [144], [130, 1], 4, 4, 1, 128, 16, None, True),
    ([2, 2], [5000, 5000], [17], 4, 2, 1, 64, 1024, None, True),
    ([4], [9000], [100, 1, 33], 8, 8, 1, 128, 16, None, True),    # items over many shares
    ([20] * 4, [260, 400, 1024, 90], [8, 16, 33], 4, 2, 2, 64, 16, [2, 2, 1], False),
    ([7], [20000], [50], 64, 1, 1, 128, 64, None, True),
    ([130], [384], [1, 2, 3], 3, 3, 1, 64, 16, None, True),
    ([3], [1000], [60, 77], 5, 1, 51, 64, 16, [51, 50, 3], True),  # 255 rows a sequence
    ([3], [530], [90], 17, 1, 15, 128, 48, None, False),
    ([2, 3, 2, 2, 9, 2], [600, 129, 5000, 256, 384, 3000], [3, 40], 8, 4, 1, 128, 16, None, True),
    ([4] * 24, [300], [1, 9], 16, 8, 1, 64, 16, None, True),      # more items than CTAs
    ([3] * 21, [5200], [1, 9], 16, 8, 1, 64, 32, None, True),     # and shares that cut them
    ([2] * 32, [260], [5, 70], 8, 2, 1, 64, 16, None, True),      # as many groups as lanes
    ([2] * 33, [260], [5, 70], 8, 2, 1, 64, 16, None, True),      # and one more
    ([3] * 70, [300], [1, 20], 16, 4, 1, 128, 32, None, True),
    ([6], [256], [9000, 4000, 100], 8, 2, 1, 128, 64, None, True),   # most work in the own tokens
    ([2, 3], [16, 300], [3000], 8, 2, 2, 64, 16, [2, 1], True),
    ([5], [12000], [6000, 1], 8, 2, 1, 128, 32, None, True),         # about as much in both
]


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("sizes,prefix,own,H,Hkv,Nq,d,P,q_lens,causal", CASES,
                         ids=lambda v: str(v)[:20])
def test_groups(sizes, prefix, own, H, Hkv, Nq, d, P, q_lens, causal, fmt):
    lens, ql = [], None
    prefix = prefix * (len(sizes) if len(prefix) == 1 else 1)
    for j, n in enumerate(sizes):
        lens += [prefix[j] + max(Nq, own[(len(lens) + i) % len(own)]) for i in range(n)]
    B = len(lens)
    if q_lens is not None:
        ql = [q_lens[b % len(q_lens)] for b in range(B)]
    table, num, groups = tables(sizes, prefix, lens, P, 5)
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((B, H, Nq, d), 30).cuda()
    O, L = run(q, kp, vp, table, lens, groups, ql, causal, P)
    assert binding.device_status() == 0
    check(q, kp, vp, table, lens, ql, causal, P, O=O, L=L)
    # the shape of the groups changes the order of sums only: one group, and none at all
    for g in (None, list(range(B))):
        O2, L2 = run(q, kp, vp, table, lens, g, ql, causal, P)
        check(q, kp, vp, table, lens, ql, causal, P, O=O2, L=L2)
    O3, L3 = run(q, kp, vp, table, lens, groups, ql, causal, P)
    assert torch.equal(O3, O) and torch.equal(L3, L)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_members_that_do_not_join(fmt):
    """In one group: empty and padded sequences, one shorter than the prefix, one with other pages, one
    with no query, equal rows (forks that have not grown) and a first one that is idle."""
    P, d, H, Hkv, Nq = 16, 128, 8, 2, 2
    lens = [0, 700, 690, 100, 680, 0, 680, 660, 700, 1, 680]
    ql = [2, 2, 1, 2, 2, 0, 0, 2, 2, 2, 2]
    table, num, _ = tables([1] + [10], [0, 656], lens, P, 5)
    table[7, :42] = table[7, :42].flip(0)     # the same pages, another order
    table[8] = table[1]
    lens[8] = lens[1]
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((len(lens), H, Nq, d), 30).cuda()
    O, L = run(q, kp, vp, table, lens, None, ql, True, P)
    assert binding.device_status() == 0
    check(q, kp, vp, table, lens, ql, True, P, O=O, L=L)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_bad_page_in_the_prefix(fmt):
    """An entry that is no page ends what is shared; its tokens take no part, for every sequence."""
    P, d, H, Hkv = 16, 64, 4, 2
    lens = [500, 520, 510]
    table, num, _ = tables([3], [480], lens, P, 5)
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((3, H, 1, d), 30).cuda()
    bad = table.clone()
    bad[:, 20] = num
    O, L = run(q, kp, vp, bad, lens, None, None, True, P)
    assert binding.device_status() == binding.FA_ERR_PAGE
    short = torch.cat((table[:, :20], table[:, 21:]), 1).contiguous()
    check(q, kp, vp, short, [n - P for n in lens], None, True, P, O=O, L=L)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(d, fmt):
    """Scores of sd 30 and more, keys that climb: the running max moves in the shared part too."""
    P, Hkv = 32, 2
    lens = [900 + i for i in range(40)]
    table, num, _ = tables([40], [896], lens, P, 5)
    x = [(rand((num, Hkv, P, d), 40 + i, 3.0) + 2.0 * (1 - i)) for i in range(2)]
    order = torch.empty(num)
    order[table[0, :28].long()] = torch.arange(28).float()
    x[0][table[0, :28].long()] *= (1 + order[table[0, :28].long()] / 8)[:, None, None, None].to(
        torch.bfloat16)
    if fmt == "int4":
        x = [torch.from_numpy(ref.head_bytes(t.double().numpy())) for t in x]
    q = rand((40, 8, 1, d), 41, 10.0).cuda()
    kp, vp = (t.cuda() for t in x)
    O, L = run(q, kp, vp, table, lens, None, None, True, P)
    check(q, kp, vp, table, lens, None, True, P, O=O, L=L)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_what_a_sequence_does_not_see(fmt):
    """NaN and infinities behind the sequences, in pages that are nobody's, in padding queries and in
    other sequences' own pages and queries do not reach a row."""
    P, d, H, Hkv, Nq = 16, 128, 8, 2, 2
    lens, ql = [400, 390, 401, 395], [2, 1, 2, 2]
    table, num, _ = tables([4], [384], [n + P for n in lens], P, 6)
    kp, vp = (filled(num, Hkv, P, d, "bf16", 50 + i) for i in range(2))
    q = rand((4, H, Nq, d), 51).cuda()
    used = torch.zeros((num, P), dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // P], j % P] = True
    good = [t.clone() for t in (kp, vp)]
    poison = torch.where(torch.arange(d) % 2 == 0, float("nan"), float("inf")).to(torch.bfloat16)
    own = torch.zeros((num, P), dtype=torch.bool)
    for j in range(384, lens[3]):
        own[table[3, j // P], j % P] = True
    for x in (kp, vp):
        x.permute(0, 2, 1, 3)[(~used | own).cuda()] = poison.cuda()
    q[1, :, 1] = float("nan")
    q[3, 2, 0] = float("inf")
    if fmt == "int4":
        with np.errstate(invalid="ignore"):
            kp, vp, *good = (torch.from_numpy(ref.head_bytes(t.cpu().double().nan_to_num(
                0, 0, 0).numpy())) for t in (kp, vp, *good))
        # a group with a NaN takes a step of NaN
        w = P * d // 2
        for x in (kp, vp):
            words = x[..., w:].view(torch.int16).view(num, Hkv, P, d // 64)
            words.permute(0, 2, 1, 3)[~used | own] = (0x3fe << 6) - (1 << 16)
        kp, vp, *good = (t.cuda() for t in (kp, vp, *good))
    O, L = run(q, kp, vp, table, lens, None, ql, True, P)
    assert binding.device_status() == 0
    check(q[:3], good[0], good[1], table[:3], lens[:3], ql[:3], True, P, O=O[:3], L=L[:3])
    assert torch.isnan(O[3].float()).any()


def test_a_token_of_the_prefix_that_is_not_finite():
    """Every sequence of the group sees it, as each would alone."""
    P, d, H, Hkv = 16, 64, 4, 1
    lens = [300, 310]
    table, num, _ = tables([2], [288], lens, P, 6)
    kp, vp = (filled(num, Hkv, P, d, "bf16", 50 + i) for i in range(2))
    vp[table[0, 3], 0, 5, 7] = float("inf")
    q = rand((2, H, 1, d), 51).cuda()
    O, _ = run(q, kp, vp, table, lens, None, None, True, P)
    O1, _ = binding.fa_fwd_paged(q, kp, vp, table.cuda(), i32(lens))
    assert torch.equal(torch.isinf(O), torch.isinf(O1)) and torch.isinf(O[..., 7]).all()
    assert not torch.isnan(O).any()


def test_many_sequences():
    """More than the plan keeps in shared memory, in groups of several sizes."""
    P, d, H, Hkv, B = 16, 64, 2, 1, 1500
    r = np.random.RandomState(1)
    sizes = []
    while sum(sizes) < B:
        sizes.append(int(min(r.choice([1, 2, 30, 200]), B - sum(sizes))))
    prefix = [int(x) for x in r.choice([100, 140, 300, 420], len(sizes))]
    lens = []
    for n, x in zip(sizes, prefix):
        lens += [int(x + y) for y in r.randint(0, 40, n)]
    lens[7] = 0
    table, num, groups = tables(sizes, prefix, lens, P, 3)
    kp, vp = (filled(num, Hkv, P, d, "int4", 20 + i) for i in range(2))
    q = rand((B, H, 1, d), 30).cuda()
    O, L = run(q, kp, vp, table, lens, groups, None, True, P)
    assert binding.device_status() == 0
    check(q, kp, vp, table, lens, None, True, P, O=O, L=L)


def test_pages_past_four_gigabytes():
    P, d, H, Hkv = 64, 128, 4, 2
    num = 5 * (1 << 30) // (P * d * 2 * Hkv)
    lens = [700, 712, 705]
    table, used, _ = tables([3], [680], lens, P, 5)
    kp, vp = (torch.zeros((num, Hkv, P, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = [filled(used, Hkv, P, d, "bf16", 20 + i) for i in range(2)]
    far = num - used
    kp[far:], vp[far:] = small
    q = rand((3, H, 1, d), 30).cuda()
    O, L = run(q, kp, vp, torch.where(table >= 0, table + far, table), lens, None, None, True, P)
    assert binding.device_status() == 0
    check(q, *small, table, lens, None, True, P, O=O, L=L)


def test_little_to_share_is_paged():
    """Shapes that cannot save much run as fa_fwd_paged, with its workspace."""
    P, d, H, Hkv = 16, 64, 8, 2
    lens = [400, 420, 0]
    table, num, _ = tables([3], [320], lens, P, 6)
    kp, vp = (filled(num, Hkv, P, d, "int4", 50 + i) for i in range(2))
    q = rand((3, H, 1, d), 51).cuda()
    shape = (3, H, Hkv, 1, d, "int4", P, table.shape[1])
    assert binding.paged_shared_plan(*shape) == binding.paged_plan(*shape)
    O, L = binding.fa_fwd_paged_shared(q, kp, vp, table.cuda(), i32(lens))
    O1, L1 = binding.fa_fwd_paged(q, kp, vp, table.cuda(), i32(lens))
    assert torch.equal(O, O1) and torch.equal(L, L1)


def test_many_rows_a_sequence():
    """From 256 rows a head on nothing is shared."""
    P, d, H, Hkv, Nq = 16, 64, 8, 1, 40
    lens = [400, 420]
    table, num, _ = tables([2], [320], lens, P, 6)
    table = widened(table, wide(2, Hkv, P))
    kp, vp = (filled(num, Hkv, P, d, "bf16", 50 + i) for i in range(2))
    q = rand((2, H, Nq, d), 51).cuda()
    O, L = binding.fa_fwd_paged_shared(q, kp, vp, table.cuda(), i32(lens))
    O1, L1 = binding.fa_fwd_paged(q, kp, vp, table.cuda(), i32(lens))
    assert torch.equal(O, O1) and torch.equal(L, L1)


def test_replays_and_streams():
    """Captured once, replayed over other lengths, groups, tables and queries (all device data); two
    graphs with a workspace each run side by side; a stream of the caller's."""
    P, d, H, Hkv, B = 16, 128, 8, 2, 6
    M = wide(B, Hkv, P)
    sets = []
    for k, (sizes, prefix) in enumerate([([6], [700]), ([2, 4], [900, 300]), ([3, 3], [0, 140])]):
        lens = [prefix[0 if b < sizes[0] else 1] + 5 + 3 * b for b in range(B)]
        table, num, groups = tables(sizes, prefix, lens, P, k, width=M)
        sets.append((table, lens, groups, rand((B, H, 1, d), 70 + k)))
    num = 400
    kp, vp = (filled(num, Hkv, P, d, "int4", 50 + i) for i in range(2))
    need = binding.paged_shared_plan(B, H, Hkv, 1, d, "int4", P, M)
    side = torch.cuda.Stream()
    graphs = []
    for k in range(2):
        s = dict(q=sets[0][3].cuda(), table=sets[0][0].cuda(), lens=i32(sets[0][1]),
                 groups=i32(sets[0][2]), ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, H, 1), device="cuda")

        def call(s=s, stream=None):
            binding.fa_fwd_paged_shared(s["q"], kp, vp, s["table"], s["lens"], groups=s["groups"],
                                        out=s["out"], lse=s["lse"], workspace=s["ws"], stream=stream)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, s, call))
    for k in range(4):
        for j, (graph, s, _) in enumerate(graphs):
            table, lens, groups, q = sets[(k + j) % 3]
            s["q"].copy_(q), s["table"].copy_(table), s["lens"].copy_(i32(lens))
            s["groups"].copy_(i32(groups)), s["out"].fill_(7.0)
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        for j, (_, s, _) in enumerate(graphs):
            table, lens, groups, q = sets[(k + j) % 3]
            check(s["q"], kp, vp, table, lens, None, True, P, O=s["out"], L=s["lse"])
    _, s, call = graphs[0]
    want = s["out"].clone()
    s["out"].fill_(3.0)
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    assert torch.equal(s["out"], want)


def test_forks_then_decoding():
    """Rows grown, filled, forked, grown on and attended to, through the pool's own calls."""
    P, d, H, Hkv, rows, num = 16, 64, 8, 2, 9, 256
    kp, vp = binding.kv_pages(num, Hkv, P, d, "bf16")
    table = torch.full((rows, wide(rows, Hkv, P)), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (rows, num))

    def append(new, seed):
        old = binding.osm_kv_grow(kp, vp, table, lens, i32(new), refs, d)
        k, v = (rand((rows, Hkv, max(new), d), seed + i).cuda() for i in range(2))
        binding.osm_kv_append(k, v, kp, vp, table, old, new_lens=i32(new))

    append([333] + [0] * 8, 1)
    binding.osm_kv_fork(table, lens, refs, P, i32([0] * 7), i32(range(1, 8)))
    for step in range(3):
        append([1] * 8 + [5], 10 + step)
        q = rand((rows, H, 1, d), 30 + step).cuda()
        O, L = binding.fa_fwd_paged_shared(q, kp, vp, table, lens, groups=i32([0] * 8 + [1]))
        torch.cuda.synchronize()
        n = lens.tolist()
        assert n == [334 + step] * 8 + [5 * (step + 1)] and binding.device_status() == 0
        check(q, kp, vp, table.cpu(), n, None, True, P, O=O, L=L)
    assert int(refs[:20].max()) == 8 and int((refs > 0).sum()) == 20 + 8 + 1
