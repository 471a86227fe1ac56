"""osm_kv_grow, osm_kv_fork, osm_kv_free and osm_kv_compact on the GPU against a plain restatement:
whole numbers and copies, so every comparison is for equality."""
import numpy as np
import pytest
import torch

import pool_ref as ref
from online_softmax_tiled_attn_gb300 import binding

pytestmark = pytest.mark.gpu


def status():
    torch.cuda.synchronize()
    return binding.device_status()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def same(t, x):
    assert (t.cpu().numpy() == x).all()


def pool(rows, max_pages, num_pages, P, seed, fill=0.6, share=0.0, most=None):
    """A pool in use: rows of different lengths (some 0), scattered pages, some of them shared;
    entries behind a row's last hold nonsense, free pages' refs may be below 0."""
    r = np.random.RandomState(seed)
    ids = list(r.permutation(num_pages))
    table = r.randint(-9, num_pages + 9, (rows, max_pages)).astype(np.int32)
    lens, refs = np.zeros(rows, np.int32), np.zeros(num_pages, np.int32)
    for b in range(rows):
        if r.rand() < 0.15:
            continue
        n = int(r.randint(1, (most or max_pages * P) + 1))
        n = min(n, int(len(ids) * fill) * P)
        for j in range(ref.count(n, P)):
            if share and b and r.rand() < share and j < ref.count(lens[b - 1], P):
                table[b, j] = table[b - 1, j]
            else:
                table[b, j] = ids.pop()
            refs[table[b, j]] += 1
        lens[b] = n
    refs[(refs == 0) & (r.rand(num_pages) < 0.1)] = -3
    return table, lens, refs, r


def page_arrays(num_pages, Hkv, P, d, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = binding.kv_page_bytes(fmt, P, d)
    raw = [torch.randint(0, 256, (num_pages, Hkv, n), generator=g, device="cuda", dtype=torch.uint8)
           for _ in range(2)]
    if fmt == "bf16":  # any bits, NaN and infinities among them
        return [x.view(torch.bfloat16).view(num_pages, Hkv, P, d) for x in raw]
    return raw


def raw(pages):
    return pages.view(torch.uint8).flatten(2).cpu().numpy()


def copy_tokens(pages, a, b, n, P, d, fmt):
    """The first n tokens of every head of page a, in page b."""
    if fmt == "bf16":
        pages[b, :, : n * 2 * d] = pages[a, :, : n * 2 * d]
        return
    w, s = P * d // 2, d // 32
    pages[b, :, : n * d // 2] = pages[a, :, : n * d // 2]
    pages[b, :, w:w + n * s] = pages[a, :, w:w + n * s]


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("rows, max_pages, num_pages, P, top, Hkv, d", [
    (1, 1, 1, 16, 16, 1, 64), (3, 5, 40, 16, 40, 2, 64), (64, 40, 5000, 16, 1, 1, 128),
    (7, 300, 4096, 48, 9000, 1, 64), (1500, 9, 20000, 32, 100, 1, 64),
    (33, 2000, 70001, 16, 20000, 1, 64), (2, 3, 0, 16, 5, 1, 64), (20, 6, 300, 64, 9, 3, 128),
    (5000, 4, 30000, 16, 30, 1, 64), (1100, 5, 9000, 32, 20, 2, 64),
    (1500, 9, 20000, 16, 100, 1, 64), (40, 3, 300, 1024, 500, 8, 64),
])
def test_grow(rows, max_pages, num_pages, P, top, Hkv, d, fmt):
    if num_pages:
        table, lens, refs, r = pool(rows, max_pages, num_pages, P, rows + P, fill=0.1, share=0.4)
    else:
        table, lens, refs = (np.full(s, -1, np.int32) for s in ((rows, max_pages), rows, 0))
        r = np.random.RandomState(0)
    for b in range(1, rows):  # rows that share all: a last page that is not full with two or more uses
        if lens[b] == 0 and r.rand() < 0.7:
            ref.fork(table, lens, refs, P, [b - 1], [b])
    new = r.randint(-2, top + 1, rows).astype(np.int32)
    lens[-1] = -4 if rows > 1 and lens[-1] == 0 else lens[-1]
    kp, vp = page_arrays(num_pages, Hkv, P, d, fmt, 5)
    k, v = raw(kp), raw(vp)
    t, l, f = dev(table), dev(lens), dev(refs)
    old = binding.osm_kv_grow(kp, vp, t, l, dev(new), f, d)
    want, copies, short = ref.grow(table, lens, new, refs, P)
    for a, b, n in copies:
        copy_tokens(k, a, b, n, P, d, fmt)
        copy_tokens(v, a, b, n, P, d, fmt)
    assert status() == (binding.FA_ERR_PAGE if short else 0)
    same(t, table), same(l, lens), same(f, refs), same(old, want)
    assert (raw(kp) == k).all() and (raw(vp) == v).all()


def test_grow_past_the_room_and_the_pool():
    """Rows stop at the table's width; the pool's last page goes out and the rest get -1, a copy that
    cannot be made among them."""
    table = np.array([[0, 1, 3, 4], [7, 7, 7, 7], [5, 6, 7, 5], [5, 6, 7, 5]], np.int32)
    lens = np.array([60, 0, 2 ** 31 - 1, 17], np.int32)
    refs = np.array([1, 1, 0, 1, 1, 2, 2, 2, 0], np.int32)
    new = np.array([2 ** 31 - 1, 33, 5, 1], np.int32)
    kp, vp = page_arrays(9, 1, 16, 64, "bf16", 1)
    k = raw(kp)
    t, l, f = dev(table), dev(lens), dev(refs)
    old = binding.osm_kv_grow(kp, vp, t, l, dev(new), f, 64)
    want, copies, short = ref.grow(table, lens, new, refs, 16)
    assert short and not copies and status() == binding.FA_ERR_PAGE
    assert list(lens) == [64, 33, 64, 18] and list(table[1]) == [2, 8, -1, 7]
    assert list(table[3]) == [5, -1, 7, 5] and refs[6] == 1
    same(t, table), same(l, lens), same(f, refs), same(old, want)
    assert (raw(kp) == k).all()


@pytest.mark.parametrize("rows, max_pages, num_pages, P, pairs", [
    (2, 1, 3, 16, 1), (9, 7, 90, 16, 6), (40, 30, 900, 48, 30), (2000, 3, 9000, 16, 1500),
    (12, 3000, 9000, 16, 11), (3000, 4, 20000, 16, 2500), (40, 40000, 90000, 16, 30),
])
def test_fork(rows, max_pages, num_pages, P, pairs):
    table, lens, refs, r = pool(rows, max_pages, num_pages, P, pairs + P, fill=0.2, share=0.3)
    lens[rows // 2:] = 0  # (their pages stay counted: the caller may hold uses of its own)
    free = list(r.permutation(np.arange(rows // 2, rows)))
    src, dst = r.randint(0, rows, pairs), np.array([free[i % len(free)] for i in range(pairs)])
    t, l, f = dev(table), dev(lens), dev(refs)
    binding.osm_kv_fork(t, l, f, P, dev(src), dev(dst))
    bad = ref.fork(table, lens, refs, P, src, dst)
    assert status() == (binding.FA_ERR_PAGE if bad else 0)
    same(t, table), same(l, lens), same(f, refs)


def test_fork_pairs_that_do_nothing():
    """Padding, rows past the table, full destinations, one destination twice, a row onto itself, bad
    entries: the rest is done all the same."""
    table = np.full((8, 3), -5, np.int32)
    table[0] = [4, 99, 2]  # an entry that is no page
    table[1] = [1, 0, -1]
    table[6] = [3, -2, 9]  # its last page is none
    lens = np.array([40, 30, 0, 0, 0, 0, 20, 0], np.int32)
    refs = np.array([1, 1, 1, 1, 1, 0, 0], np.int32)
    src = [0, -1, 8, 1, 1, 1, 6, 2, 1, 0]
    dst = [2, 3, 3, 0, 3, 3, 4, 2, 5, 7]
    t, l, f = dev(table), dev(lens), dev(refs)
    binding.osm_kv_fork(t, l, f, 16, dev(src), dev(dst))
    bad = ref.fork(table, lens, refs, 16, src, dst)
    assert bad and list(table[4]) == [3, -2, -5] and lens[7] == 40 and refs[1] == 3
    assert status() == binding.FA_ERR_PAGE
    same(t, table), same(l, lens), same(f, refs)


@pytest.mark.parametrize("rows, max_pages, num_pages, P, n", [
    (1, 1, 2, 16, 1), (50, 20, 2000, 16, 37), (9, 3000, 40000, 32, 9), (700, 5, 9000, 48, 900),
])
@pytest.mark.parametrize("how", ["all", "keep", "every row"])
def test_free(rows, max_pages, num_pages, P, n, how):
    table, lens, refs, r = pool(rows, max_pages, num_pages, P, n + P, fill=0.5, share=0.5)
    lst = r.randint(-1, rows + (rows > 1), n)  # rows more than once, padding, one past the last
    keep = r.randint(-3, max_pages * P + 9, n) if how == "keep" else np.zeros(n, int)
    t, l, f = dev(table), dev(lens), dev(refs)
    if how == "every row":
        binding.osm_kv_free(t, l, f, P)
        bad = ref.release(table, lens, refs, P, range(rows), [0] * rows)
    else:
        binding.osm_kv_free(t, l, f, P, rows=dev(lst),
                            keep_lens=dev(keep) if how == "keep" else None)
        bad = ref.release(table, lens, refs, P, lst, keep)
    assert status() == (binding.FA_ERR_PAGE if bad else 0)
    same(t, table), same(l, lens), same(f, refs)


def test_free_counts_stop_at_zero():
    """More entries than uses: the count ends at 0 whatever the order."""
    table = np.full((64, 40), 3, np.int32)
    table[:, 1::2] = 4
    lens, refs = np.full(64, 640, np.int32), np.array([1, 1, 1, 5, 2000, 1], np.int32)
    t, l, f = dev(table), dev(lens), dev(refs)
    binding.osm_kv_free(t, l, f, 16)
    assert status() == 0
    same(f, [1, 1, 1, 0, 2000 - 64 * 20, 1]), same(l, np.zeros(64))


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("rows, max_pages, num_pages, P, Hkv, d, fill", [
    (1, 1, 1, 16, 1, 64, 1.0), (5, 7, 200, 16, 1, 64, 0.2), (30, 9, 700, 48, 3, 64, 0.5),
    (12, 40, 700, 32, 2, 128, 0.9), (200, 20, 40000, 16, 1, 64, 0.02), (3, 2, 50, 1024, 1, 64, 0.3),
])
def test_compact(rows, max_pages, num_pages, P, Hkv, d, fill, fmt):
    table, lens, refs, _ = pool(rows, max_pages, num_pages, P, rows + P, fill=fill, share=0.2)
    refs[-1] = max(refs[-1], 2)  # a use that no row shows
    kp, vp = page_arrays(num_pages, Hkv, P, d, fmt, 7)
    k, v = raw(kp), raw(vp)
    t, l, f = dev(table), dev(lens), dev(refs)
    where, used = binding.osm_kv_compact(kp, vp, t, l, f, d)
    want, n, moves = ref.compact(table, lens, refs, P)
    for a, b in moves:
        k[b], v[b] = k[a], v[a]
    assert status() == 0
    same(t, table), same(l, lens), same(f, refs), same(where, want), same(used, [n])
    assert (raw(kp) == k).all() and (raw(vp) == v).all()


def test_compact_nothing_to_move():
    """A full pool, an empty one, and one without gaps."""
    kp, vp = page_arrays(6, 1, 16, 64, "bf16", 2)
    before = raw(kp)
    for refs in ([2, 1, 1, 1, 1, 9], [0] * 6, [1, 1, 4, 0, 0, -1]):
        table, lens = np.array([[0, 1, 2]], np.int32), np.array([48 if refs[0] else 0], np.int32)
        f, t = dev(refs), dev(table)
        where, used = binding.osm_kv_compact(kp, vp, t, dev(lens), f, 64)
        n = sum(x > 0 for x in refs)
        same(where, [i if x > 0 else -1 for i, x in enumerate(refs)]), same(used, [n])
        same(f, refs), same(t, table)
    assert status() == 0 and (raw(kp) == before).all()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_a_pool_in_use(fmt):
    """The calls together as a server makes them, with the append and the read-out between: what the
    rows hold is what was appended, through forks, refused tokens, finished rows and compaction."""
    P, d, Hkv, rows, num = 16, 64, 2, 6, 64
    kp, vp = binding.kv_pages(num, Hkv, P, d, fmt)
    table = torch.full((rows, 8), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (rows, num))
    held = [np.zeros((Hkv, 0, d)) for _ in range(rows)]
    g = torch.Generator(device="cuda").manual_seed(11)
    r = np.random.RandomState(4)

    def append(new):
        new = np.array(new, np.int32)
        old = binding.osm_kv_grow(kp, vp, table, lens, dev(new), refs, d)
        N = int(new.max())
        # small whole numbers: 4 bits hold them as bf16 does
        k, v = (torch.randint(0, 16, (rows, Hkv, N, d), generator=g, device="cuda")
                .to(torch.bfloat16) for _ in range(2))
        k[..., ::64], v[..., ::64], k[..., 1::64], v[..., 1::64] = 0, 0, 15, 15
        binding.osm_kv_append(k, v, kp, vp, table, old, new_lens=dev(new))
        for b in range(rows):
            held[b] = np.concatenate((held[b], k[b, :, : new[b]].float().cpu().numpy()), 1)

    def check():
        n = [h.shape[1] for h in held]
        same(lens, n)
        K, _ = binding.osm_kv_gather(kp, vp, table, lens, max(max(n), 1), d)
        for b in range(rows):
            assert (K[b, :, : n[b]].float().cpu().numpy() == held[b]).all()
        t, f = table.cpu().numpy(), np.zeros(num, np.int32)
        for b in range(rows):
            for e in t[b, : ref.count(n[b], P)]:
                f[e] += 1
        same(refs, f)

    append([40, 17, 16, 0, 0, 0])
    check()
    for step in range(5):
        empty = [b for b in range(rows) if held[b].shape[1] == 0]
        src = [b for b in range(rows) if held[b].shape[1]][: len(empty)]
        binding.osm_kv_fork(table, lens, refs, P, dev(src), dev(empty[: len(src)]))
        for s, t in zip(src, empty):
            held[t] = held[s].copy()
        check()
        append([int(x) if held[b].shape[1] < 90 and held[b].shape[1] else 0
                for b, x in enumerate(r.randint(1, 20, rows))])
        check()
        keep = [max(0, h.shape[1] - 3) for h in held]
        keep[step % rows] = 0
        binding.osm_kv_free(table, lens, refs, P, keep_lens=dev(keep))
        held = [h[:, :k] for h, k in zip(held, keep)]
        check()
        where, used = binding.osm_kv_compact(kp, vp, table, lens, refs, d)
        assert (refs[: int(used)] > 0).all() and (refs[int(used):] == 0).all()
        check()
    assert status() == 0


def test_pages_past_four_gigabytes():
    """A copy on growing, and a page moved, between the ends of a pool of 5 GB."""
    P, d, Hkv = 64, 128, 2
    num = 5 * (1 << 30) // (P * d * 2 * Hkv)
    kp, vp = (torch.zeros((num, Hkv, P, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    last = num - 1
    for x, seed in ((kp, 1), (vp, 2)):
        x[last] = torch.randn((Hkv, P, d), generator=torch.Generator().manual_seed(seed)).to(x.dtype)
    table, lens = dev([[last, -1], [last, -1]]), dev([40, 40])
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    refs[last] = 2
    binding.osm_kv_grow(kp, vp, table, lens, dev([30, 0]), refs, d)
    same(table, [[0, 1], [last, -1]])
    for x in (kp, vp):
        assert torch.equal(x[0, :, :40], x[last, :, :40]) and not x[0, :, 40:].any()
    where, used = binding.osm_kv_compact(kp, vp, table, lens, refs, d)
    same(table, [[0, 1], [2, -1]]), same(used, [3])
    assert status() == 0 and int(where[last]) == 2
    assert torch.equal(kp[2], kp[last]) and torch.equal(vp[2], vp[last])


def test_two_pools_at_once():
    """Calls on two pools, on two streams, replayed side by side."""
    P, d = 16, 64
    pools, graphs = [], []
    for k in range(2):
        table, lens, refs, _ = pool(40, 50, 9000, P, 20 + k, fill=0.05, share=0.3)
        kp, vp = page_arrays(9000, 1, P, d, "int4", k)
        x = [kp, vp, dev(table), dev(lens), dev(refs), dev([3] * 40)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())

        def call(x=x):
            old = binding.osm_kv_grow(x[0], x[1], x[2], x[3], x[5], x[4], d)
            where, used = binding.osm_kv_compact(x[0], x[1], x[2], x[3], x[4], d)
            return old, where, used

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        pools.append((x, [table, lens, refs, raw(kp)], out))
        graphs.append((graph, s))
    for _ in range(5):
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    assert status() == 0
    for (kp, vp, t, l, f, _), (table, lens, refs, k), (old, where, used) in pools:
        for _ in range(5):
            want, copies, _ = ref.grow(table, lens, [3] * 40, refs, P)
            for a, b, n in copies:
                copy_tokens(k, a, b, n, P, d, "int4")
            w, n, moves = ref.compact(table, lens, refs, P)
            for a, b in moves:
                k[b] = k[a]
        same(t, table), same(l, lens), same(f, refs), same(old, want), same(where, w), same(used, [n])
        assert (raw(kp) == k).all()


def test_pool_calls_in_a_graph():
    """Captured and replayed: each replay starts from the state it finds; nothing is kept between."""
    P, d = 16, 64
    table, lens, refs, _ = pool(12, 30, 1500, P, 3, fill=0.05)
    lens[8:] = 0
    kp, vp = page_arrays(1500, 1, P, d, "bf16", 3)
    k = raw(kp)
    t, l, f = dev(table), dev(lens), dev(refs)
    new, src, dst = dev([1] * 8 + [0] * 4), dev([0, 1]), dev([8, 9])
    keep = dev([0, 0])
    out = dev(np.zeros(1500)), dev([0])

    def calls(s=None):
        binding.osm_kv_grow(kp, vp, t, l, new, f, d, stream=s)
        binding.osm_kv_fork(t, l, f, P, src, dst, stream=s)
        binding.osm_kv_compact(kp, vp, t, l, f, d, page_map=out[0], used=out[1], stream=s)
        binding.osm_kv_free(t, l, f, P, rows=dst, keep_lens=keep, stream=s)

    def reference():
        nonlocal k
        _, copies, _ = ref.grow(table, lens, [1] * 8 + [0] * 4, refs, P)
        for a, b, n in copies:
            copy_tokens(k, a, b, n, P, d, "bf16")
        ref.fork(table, lens, refs, P, [0, 1], [8, 9])
        _, _, moves = ref.compact(table, lens, refs, P)
        for a, b in moves:
            k[b] = k[a]
        ref.release(table, lens, refs, P, [8, 9], [0, 0])

    calls()
    reference()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        graph.replay()
        reference()
        assert status() == 0
        same(t, table), same(l, lens), same(f, refs)
        assert (raw(kp) == k).all()
    # and on a stream of the caller's
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    s.synchronize()
    reference()
    same(t, table), same(l, lens), same(f, refs)
    assert status() == 0


def test_refusals_of_the_binding():
    t, v = dev(np.zeros((4, 5))), dev(np.zeros(4))
    f = dev(np.zeros(8))
    kp, vp = page_arrays(8, 1, 16, 64, "bf16", 0)
    with pytest.raises(ValueError):
        binding.osm_kv_grow(kp, vp, t, dev(np.zeros(3)), v, f, 64)
    with pytest.raises(TypeError):
        binding.osm_kv_grow(kp, vp, t, v, v.long(), f, 64)
    with pytest.raises(binding.FaError):
        binding.osm_kv_fork(t, v, f, 24, v[:1], v[1:2])
    with pytest.raises(binding.FaError):
        binding.osm_kv_grow(kp, vp, t, v, v, f, 64)  # new_lens is lens
    with pytest.raises(ValueError):
        binding.osm_kv_grow(kp, vp, t, v, dev(np.zeros(4)), dev(np.zeros(9)), 64)
    with pytest.raises(ValueError):
        binding.osm_kv_fork(t, v, f, 16, dev([0]), dev([1, 2]))
    with pytest.raises(ValueError):
        binding.osm_kv_free(t, v, f, 16, rows=dev([0]), keep_lens=dev([1, 2]))
    with pytest.raises(ValueError):
        binding.osm_kv_compact(kp, vp, t, v, f, 64, page_map=dev(np.zeros(9)))
    with pytest.raises(ValueError):
        binding.osm_kv_compact(kp, vp, t, v, f, 64,
                               workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))
    assert status() == 0
