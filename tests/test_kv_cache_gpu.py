"""osm_kv_append, osm_kv_gather and fa_fwd_paged on the GPU against plain fp64 restatements."""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(torch.bfloat16)


def page_table(counts, seed, spare=3, width=None):
    """Scattered pages, `counts[b]` of them for sequence b; unused entries hold nonsense."""
    total = sum(counts)
    ids = torch.randperm(total + spare, generator=gen(seed))[:total].to(torch.int32)
    table = torch.full((len(counts), width or max(1, max(counts))), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, total + spare


def pages_of(lens, P):
    return [(n + P - 1) // P for n in lens]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def values(pages, P, d):
    """fp64 values [num, heads, P, d] of a page array, and the step of each (0 for bf16)."""
    raw = pages.cpu()
    if raw.dtype == torch.bfloat16:
        x = raw.double().numpy()
        return x, np.zeros_like(x)
    with np.errstate(invalid="ignore"):
        return ref.head_values(raw.numpy(), P, d), ref.head_steps(raw.numpy(), P, d)


def filled(num, Hkv, P, d, fmt, seed):
    """A page array full of tokens, outlying channels among them."""
    x = rand((num, Hkv, P, d), seed)
    x[..., ::37] *= 5
    if fmt == "bf16":
        return x.cuda()
    return torch.from_numpy(ref.head_bytes(x.double().numpy())).cuda()


# ------------------------------------------------------------------------------------------
# append and gather
# ------------------------------------------------------------------------------------------
# B, H, Hkv, N, d, page, past, new, rot
APPEND = [
    (1, 1, 1, 1, 64, 16, [0], [1], 64),
    (3, 8, 2, 5, 128, 16, [0, 14, 31], [5, 3, 0], 128),
    (2, 4, 4, 70, 64, 48, [100, 0], [70, 33], 32),
    (2, 6, 2, 40, 128, 32, [7, 90], [40, 1], 64),
    (2, 7, 1, 19, 128, 128, [3, 250], [19, 18], 24),
    (2, 2, 2, 33, 64, 64, [0, 1], [33, 32], 0),
    (65, 32, 8, 1, 128, 16, list(range(65)), [1] * 65, 128),
]


def run_append(B, H, Hkv, N, d, P, past, new, rot, layout, fmt, seed, packed=True):
    total = [a + b for a, b in zip(past, new)]
    table, num = page_table(pages_of(total, P), seed)
    if packed:  # the projection's output, [B, N, heads, d], read in place
        qkv = rand((B, N, H + 2 * Hkv, d), seed + 1)
        qkv[:, :, :, 5] *= 6
        q, k, v = (t.transpose(1, 2) for t in qkv.cuda().split([H, Hkv, Hkv], 2))
    else:
        q, k, v = (rand((B, n, N, d), seed + 1 + i).cuda() for i, n in enumerate((H, Hkv, Hkv)))
    kp, vp = (filled(num, Hkv, P, d, fmt, seed + 5 + i) for i in range(2))
    before = kp.clone(), vp.clone()
    w = ref.rates(rot) if rot else []
    q_out = torch.full((B, H, N, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got = binding.osm_kv_append(k, v, kp, vp, table.cuda(), i32(past), new_lens=i32(new),
                                table=binding.rope_table(w) if rot else None, layout=layout, q=q,
                                q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out and binding.device_status() == 0
    return q, k, v, kp, vp, before, table, w, q_out, total


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hkv,N,d,P,past,new,rot", APPEND, ids=lambda v: str(v)[:24])
def test_append_writes_the_slots_and_nothing_else(B, H, Hkv, N, d, P, past, new, rot, layout, fmt):
    q, k, v, kp, vp, before, table, w, q_out, total = run_append(
        B, H, Hkv, N, d, P, past, new, rot, layout, fmt, 100 + N + d + P)
    pos = np.array(past)[:, None] + np.arange(N)
    kr = ref.rotate(k.double().cpu().numpy(), pos, w, layout) if rot else k.double().cpu().numpy()
    want_v = v.double().cpu().numpy()
    bound = np.zeros((B, Hkv, N, d))
    if rot:
        k64 = np.abs(k.double().cpu().numpy())
        bound[..., :rot] = 6e-7 * 2 * k64[..., :rot].max(-1, keepdims=True)
    for pages, old, x, slack in ((kp, before[0], kr, bound), (vp, before[1], want_v, 0 * bound)):
        if fmt == "bf16":
            want, _ = values(old, P, d)
            tol = np.zeros_like(want)
            for b in range(B):
                for n in range(new[b]):
                    p = past[b] + n
                    want[table[b, p // P], :, p % P] = x[b, :, n]
                    tol[table[b, p // P], :, p % P] = \
                        2.0 ** -8 * np.abs(x[b, :, n]) + slack[b, :, n] if pages is kp else 0
            assert np.all(np.abs(pages.double().cpu().numpy() - want) <= tol)
        else:  # the stored bits themselves
            want = old.cpu().numpy()
            heads = np.zeros((kp.shape[0], Hkv, P, d // 2 + d // 32), np.uint8)
            row = np.zeros(kp.shape[:1] + (P,), bool)
            for b in range(B):
                for n in range(new[b]):
                    p = past[b] + n
                    one = ref.head_bytes(x[b, :, n][:, None])  # a page head of one token
                    heads[table[b, p // P], :, p % P] = one
                    row[table[b, p // P], p % P] = True
            body = want[..., : P * d // 2].reshape(-1, Hkv, P, d // 2).copy()
            tail = want[..., P * d // 2:].reshape(-1, Hkv, P, d // 32).copy()
            for h in range(Hkv):
                body[:, h][row] = heads[:, h][row][:, : d // 2]
                tail[:, h][row] = heads[:, h][row][:, d // 2:]
            want = np.concatenate((body.reshape(-1, Hkv, P * d // 2),
                                   tail.reshape(-1, Hkv, P * d // 32)), -1)
            assert np.array_equal(pages.cpu().numpy(), want)
    qr = ref.rotate(q.double().cpu().numpy(), pos, w, layout) if rot else q.double().cpu().numpy()
    qo = q_out.double().cpu().numpy()
    for b in range(B):
        err = np.abs(qo[b, :, :new[b]] - qr[b, :, :new[b]])
        mag = np.abs(q[b, :, :new[b]].double().cpu().numpy()).max(-1, keepdims=True) \
            if new[b] else 0
        assert np.all(err <= 2.0 ** -8 * np.abs(qr[b, :, :new[b]]) + 6e-7 * 2 * mag)
        assert (qo[b, :, new[b]:] == 3.0).all()


def test_layouts_of_the_input_do_not_matter():
    """[B, N, heads, d] views, contiguous tensors and rows off any boundary store the same bits."""
    B, H, Hkv, N, d, P = 2, 4, 2, 21, 128, 16
    table, num = page_table([4, 4], 1)
    for fmt in ("bf16", "int4"):
        outs = []
        for form in range(3):
            wide = rand((B, N, H + 2 * Hkv, d + 1), 77).cuda()
            src = wide[..., 1:]
            if form == 1:
                src = src.contiguous()
            q, k, v = (t.transpose(1, 2) for t in src.split([H, Hkv, Hkv], 2))
            if form == 2:
                q, k, v = (t.contiguous() for t in (q, k, v))
            kp, vp = binding.kv_pages(num, Hkv, P, d, fmt)
            q_out = q if form == 2 else None  # in place where q is contiguous
            q_out = binding.osm_kv_append(k, v, kp, vp, table.cuda(), i32([40, 3]),
                                          table=binding.rope_table(binding.rope_rates(d)), q=q,
                                          q_out=q_out)
            outs.append((kp, vp, q_out))
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("d", [64, 128])
def test_four_bit_rows_of_hard_values(d):
    """Ties, steps on the border, one-sided groups, equal values, zeros, tiny and huge values."""
    rows = [np.arange(d) % 16 * 0.25, np.arange(d) % 16 * 0.25 - 1.875, np.full(d, 5.0),
            np.zeros(d), np.where(np.arange(d) == 3, -40.0, 0.0), 10 + np.arange(d) % 7 * 0.0625,
            -10 - np.arange(d) % 7 * 0.0625, (np.arange(d) - d / 2) * 1e-30,
            (np.arange(d) - d / 2) * 1e-39, (np.arange(d) - d / 2) * 1e34,
            np.where(np.arange(d) % 2 == 0, 3e38, -3e38), np.arange(d) % 31 * 0.5 - 7.5,
            (np.arange(d) % 32) / 2 * 1.25, (np.arange(d) % 32 - 16) / 2 * 1.75]
    x = torch.tensor(np.array(rows)).to(torch.bfloat16)[None, None]  # [1, 1, N, d]
    N = x.shape[2]
    kp, vp = binding.kv_pages(1, 1, 16, d, "int4")
    binding.osm_kv_append(x.cuda(), x.cuda(), kp, vp, i32([[0]]), i32([0]))
    x64 = x.double().numpy()[0]
    want = ref.head_bytes(np.concatenate((x64, np.zeros((1, 16 - N, d))), 1))
    assert np.array_equal(kp.cpu().numpy()[0], want) and torch.equal(kp, vp)
    K, _ = binding.osm_kv_gather(kp, vp, i32([[0]]), i32([N]), N, d)
    back = K.double().cpu().numpy()[0, 0]
    codes, s, b = ref.quantise(x64[0])
    fine = np.abs(back) < 1e38
    # a step of 0 stands for one below 2^-126: |min| < 31 and max - min < 15 such steps
    half = np.repeat(np.where(s > 0, s / 2, 46 * 2.0 ** -126), 64, -1)
    assert np.all(np.abs(back - x64[0])[fine] <= half[fine])


def test_non_finite_groups_read_back_as_nan():
    d = 128
    x = torch.ones((1, 1, 4, d), dtype=torch.bfloat16)
    x[0, 0, 0, 3] = float("nan")
    x[0, 0, 1, 70] = float("inf")
    x[0, 0, 2, 127] = float("-inf")
    kp, vp = binding.kv_pages(1, 1, 16, d, "int4")
    binding.osm_kv_append(x.cuda(), x.cuda(), kp, vp, i32([[0]]), i32([0]))
    K, V = binding.osm_kv_gather(kp, vp, i32([[0]]), i32([4]), 4, d)
    bad = torch.isnan(K.cpu())[0, 0].view(4, 2, 64)
    assert bad.all(-1).tolist() == [[True, False], [False, True], [False, True], [False, False]]
    assert torch.equal(bad.all(-1), bad.any(-1))


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("d,P,lens,N", [(64, 16, [0, 1, 16, 50], 50), (128, 48, [96, 13], 111),
                                        (128, 128, [200], 129), (64, 32, [5], 1)])
def test_gather(fmt, d, P, lens, N):
    Hkv = 3
    table, num = page_table(pages_of(lens, P), d + P)
    kp, vp = (filled(num, Hkv, P, d, fmt, i) for i in range(2))
    K, V = binding.osm_kv_gather(kp, vp, table.cuda(), i32(lens), N, d)
    assert binding.device_status() == 0
    for out, pages in ((K, kp), (V, vp)):
        x = values(pages, P, d)[0]
        want = np.zeros((len(lens), Hkv, N, d))
        for b, n in enumerate(lens):
            n = min(n, N)
            want[b, :, :n] = ref.dense(x, table[b].numpy(), n)
        assert np.array_equal(out.double().cpu().numpy(), want)


def test_bad_pages_are_reported_and_skipped():
    """An entry that is no page: nothing is written, zeros come back, the keys take no part."""
    d, P, Hkv = 64, 16, 2
    for bad in (-1, 3, 2 ** 31 - 1):
        kp, vp = (filled(3, Hkv, P, d, "bf16", i) for i in range(2))
        old = kp.clone(), vp.clone()
        table = i32([[0, bad, 2]])
        k = rand((1, Hkv, 20, d), 1).cuda()
        binding.osm_kv_append(k, k, kp, vp, table, i32([14]))  # positions 14 .. 33
        assert binding.device_status() == binding.FA_ERR_PAGE
        assert torch.equal(kp[0, :, :14], old[0][0, :, :14])
        assert torch.equal(kp[0, :, 14:], k[0, :, :2]) and torch.equal(kp[1], old[0][1])
        assert torch.equal(kp[2, :, :2], k[0, :, 18:]) and torch.equal(kp[2, :, 2:], old[0][2, :, 2:])
        K, _ = binding.osm_kv_gather(kp, vp, table, i32([34]), 34, d)
        assert binding.device_status() == binding.FA_ERR_PAGE
        assert (K[0, :, 16:32] == 0).all() and torch.equal(K[0, :, 32:], kp[2, :, :2])
        q = rand((1, Hkv, 1, d), 2).cuda()
        O, L = binding.fa_fwd_paged(q, kp, vp, table, i32([34]))
        assert binding.device_status() == binding.FA_ERR_PAGE
        # the same as a sequence of the two good pages
        O2, L2 = binding.fa_fwd_paged(q, kp, vp, i32([[0, 2]]), i32([18]))
        assert binding.device_status() == 0
        assert (O.float() - O2.float()).abs().max() <= 2 ** -7 * O2.float().abs().max()
        assert (L - L2).abs().max() <= 1e-5


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_queries_in_place_at_an_odd_rotated_width(layout):
    """A rotated width off the fast path: partners of a pair belong to different threads."""
    B, H, N, d = 2, 5, 33, 64
    rt = binding.rope_table(binding.rope_rates(38))
    k, q = rand((B, 1, N, d), 91).cuda(), rand((B, H, N, d), 92).cuda()
    kp, vp = binding.kv_pages(8, 1, 16, d, "bf16")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(B, 4)
    lens = i32([5, 0])
    want = binding.osm_kv_append(k, k, kp, vp, table, lens, table=rt, layout=layout, q=q)
    assert binding.osm_kv_append(k, k, kp, vp, table, lens, table=rt, layout=layout, q=q,
                                 q_out=q) is q
    assert torch.equal(q, want)


@pytest.mark.parametrize("Nq", [1, 300])
def test_a_cache_without_pages(Nq):
    kp, vp = binding.kv_pages(0, 2, 16, 64, "int4")
    table = torch.full((1, 30), -1, dtype=torch.int32, device="cuda")
    O, L = binding.fa_fwd_paged(rand((1, 2, Nq, 64), 1).cuda(), kp, vp, table, i32([400]))
    assert binding.device_status() == binding.FA_ERR_PAGE
    assert (O == 0).all() and torch.isneginf(L).all()
    K, _ = binding.osm_kv_gather(kp, vp, table, i32([400]), 40, 64)
    assert binding.device_status() == binding.FA_ERR_PAGE and (K == 0).all()


@pytest.mark.parametrize("Nq", [1, 300])
def test_a_table_without_entries(Nq):
    """kv_lens is clamped to what the table holds: nothing; tokens to append have no page."""
    kp, vp = (filled(3, 2, 16, 64, "int4", 8 + i) for i in range(2))
    before = kp.clone()
    table = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    O, L = binding.fa_fwd_paged(rand((2, 4, Nq, 64), 1).cuda(), kp, vp, table, i32([40, 0]))
    assert binding.device_status() == 0
    assert (O == 0).all() and torch.isneginf(L).all()
    k = rand((2, 2, 3, 64), 2).cuda()
    binding.osm_kv_append(k, k, kp, vp, table, i32([0, 5]))
    assert binding.device_status() == binding.FA_ERR_PAGE and torch.equal(kp, before)


def test_tokens_past_the_table_are_reported():
    d, P = 64, 16
    kp, vp = binding.kv_pages(2, 1, P, d, "int4")
    old = kp.clone()
    k = rand((1, 1, 8, d), 1).cuda()
    binding.osm_kv_append(k, k, kp, vp, i32([[0]]), i32([12]))
    assert binding.device_status() == binding.FA_ERR_PAGE
    assert not torch.equal(kp[0], old[0]) and torch.equal(kp[1], old[1])


# ------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------
def check(q, kp, vp, table, lens, q_lens, causal, P, scale=None, O=None, L=None):
    """fa_fwd_paged (or the given outputs) within the derived tolerances of the fp64 result."""
    B, H, Nq, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    if O is None:
        O, L = binding.fa_fwd_paged(q, kp, vp, table.cuda(), i32(lens),
                                    q_lens=None if q_lens is None else i32(q_lens), scale=scale,
                                    causal=causal)
        torch.cuda.synchronize()
        assert binding.device_status() == 0
    kx, kstep = values(kp, P, d)
    vx, vstep = values(vp, P, d)
    kmag = 136 * kstep if kp.dtype == torch.uint8 else np.abs(kx)
    qn = q.double().cpu().numpy()
    for b, n in enumerate(lens):
        t = table[b].cpu().numpy()
        k, v, km, vs = (ref.dense(x, t, n) for x in (kx, vx, kmag, vstep))
        ql = Nq if q_lens is None else min(max(q_lens[b], 0), Nq)
        Or, Lr, tO, tL = ref.attend(qn[b], k, v, km, vs, scale, causal, ql)
        Ob, Lb = O[b].double().cpu().numpy(), L[b].double().cpu().numpy()
        empty = np.isneginf(Lr)
        assert np.array_equal(np.isneginf(Lb), empty), (b, n)
        assert np.all(Ob[empty] == 0)
        e = np.abs(Ob - Or) - tO
        assert np.all(e <= 0), (b, n, e.max(), np.unravel_index(e.argmax(), e.shape))
        e = np.abs(Lb[~empty] - Lr[~empty]) - tL[~empty]
        assert np.all(e <= 0), (b, n, e.max())
    return O, L


# B, H, Hkv, Nq, d, page, lens, q_lens, causal
ATTEND = [
    (1, 1, 1, 1, 64, 16, [1], None, True),
    (1, 8, 1, 1, 128, 16, [15], None, True),
    (4, 8, 2, 1, 128, 16, [0, 1, 33, 300], None, True),
    (3, 4, 4, 1, 64, 48, [47, 49, 1000], None, False),
    (2, 16, 2, 1, 128, 32, [2049, 31], None, True),
    (2, 12, 4, 3, 128, 64, [100, 2], None, True),       # more queries than keys
    (3, 8, 4, 7, 64, 128, [130, 7, 0], [7, 3, 2], True),
    (2, 8, 8, 5, 128, 16, [77, 16], [5, 0], False),
    (1, 32, 2, 1, 64, 16, [5000], None, True),
    (1, 3, 1, 9, 128, 32, [64], [9], True),
    (2, 10, 2, 33, 64, 16, [200, 33], [33, 20], True),
    (1, 64, 1, 1, 128, 1024, [1500], None, True),
    (1, 4, 2, 150, 128, 64, [333], None, True),
    (20, 4, 2, 1, 128, 16, [17 * i for i in range(20)], None, True),
    (70, 8, 2, 3, 64, 16, [(5 * i) % 40 for i in range(70)], [i % 4 for i in range(70)], True),
    (37, 12, 1, 2, 128, 32, [0] * 33 + [90, 0, 1, 64], None, False),
]


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("B,H,Hkv,Nq,d,P,lens,q_lens,causal", ATTEND, ids=lambda v: str(v)[:24])
def test_attention(B, H, Hkv, Nq, d, P, lens, q_lens, causal, fmt):
    table, num = page_table(pages_of(lens, P), 5)
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((B, H, Nq, d), 30).cuda()
    check(q, kp, vp, table, lens, q_lens, causal, P)


# Query rows enough for the dense chunk path (256 rows a key/value head on), and just too few.
CHUNKS = [
    (2, 8, 2, 70, 128, 16, [70, 333], [70, 41], True),
    (2, 4, 4, 300, 64, 48, [300, 1000], None, True),
    (3, 8, 1, 40, 128, 64, [2000, 0, 129], [40, 3, 0], False),
    (1, 16, 4, 64, 64, 128, [20], None, True),          # more queries than keys
    (2, 16, 2, 31, 128, 32, [900, 31], None, True),
    (1, 2, 2, 257, 128, 16, [4000], None, True),        # split keys
]


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("B,H,Hkv,Nq,d,P,lens,q_lens,causal", CHUNKS, ids=lambda v: str(v)[:24])
def test_chunks(B, H, Hkv, Nq, d, P, lens, q_lens, causal, fmt):
    table, num = page_table(pages_of(lens, P), 5)
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((B, H, Nq, d), 30).cuda()
    check(q, kp, vp, table, lens, q_lens, causal, P)


def test_chunks_a_group_of_sequences_at_a_time():
    """A table so wide that the dense copy holds two of the three sequences."""
    B, H, Hkv, Nq, d, P = 3, 8, 8, 256, 128, 16
    lens = [300, 500, 256]
    table, num = page_table(pages_of(lens, P), 5, width=8192)
    need = binding.paged_plan(B, H, Hkv, Nq, d, "int4", P, 8192)
    assert 2 * 2 * Hkv * 131072 * d * 2 <= need < 2 * 3 * Hkv * 131072 * d * 2
    kp, vp = (filled(num, Hkv, P, d, "int4", 20 + i) for i in range(2))
    check(rand((B, H, Nq, d), 30).cuda(), kp, vp, table, lens, None, True, P)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_chunk_with_a_page_that_is_none(fmt):
    """Sequence 0 has a bad page (its tokens take no part); sequence 1 is as ever."""
    B, H, Hkv, Nq, d, P = 2, 4, 1, 80, 128, 16
    lens = [200, 130]
    table, num = page_table(pages_of(lens, P), 5)
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((B, H, Nq, d), 30).cuda()
    O, L = binding.fa_fwd_paged(q, kp, vp, table.cuda(), i32(lens))
    assert binding.device_status() == 0
    bad = table.clone()
    bad[0, 3] = num
    O2, L2 = binding.fa_fwd_paged(q, kp, vp, bad.cuda(), i32(lens))
    assert binding.device_status() == binding.FA_ERR_PAGE
    assert torch.equal(O2[1], O[1]) and torch.equal(L2[1], L[1])
    # without that page: the sequence of the other pages, 16 tokens shorter
    short = torch.cat((table[:1, :3], table[:1, 4:]), 1).contiguous()
    check(q[:1], kp, vp, short, [lens[0] - P], None, True, P, O=O2[:1], L=L2[:1])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(d, fmt):
    """Scores of sd 30 and keys far from zero: the running max moves, shares underflow."""
    P, lens, Hkv = 16, [700], 2
    table, num = page_table(pages_of(lens, P), 5)
    kp, vp = (rand((num, Hkv, P, d), 40 + i, 3.0) + 2.0 * (1 - i) for i in range(2))
    if fmt == "int4":
        kp, vp = (torch.from_numpy(ref.head_bytes(x.double().numpy())) for x in (kp, vp))
    q = rand((1, 8, 2, d), 41, 10.0).cuda()
    check(q, kp.cuda(), vp.cuda(), table, lens, None, True, P)


@pytest.mark.parametrize("Nq", [1, 9])
def test_small_steps_beside_a_large_one(Nq):
    """Tokens whose step is 2^-15 of another's: what the products' alignment may drop of them."""
    d, P = 64, 16
    v = np.full((1, 1, P, d), 1.75 * 2.0 ** -16)
    v[..., 0] = 0
    v[..., 63] *= 15
    v[0, 0, 5] = 0
    v[0, 0, 5, 63] = 15.0
    vp = torch.from_numpy(ref.head_bytes(v))
    x, s = values(vp, P, d)
    assert np.array_equal(x, v) and s[0, 0, 5, 0] == 1 and s[0, 0, 4, 0] == 1.75 * 2.0 ** -16
    kp = filled(1, 1, P, d, "int4", 3)
    table = torch.zeros((1, 1), dtype=torch.int32)
    for q in (torch.zeros((1, 4, Nq, d), dtype=torch.bfloat16), rand((1, 4, Nq, d), 4)):
        check(q.cuda(), kp, vp.cuda(), table, [P], None, False, P)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("Nq", [1, 4, 40, 150])
def test_what_lies_outside_takes_no_part(fmt, Nq):
    """NaN and infinities in the places behind a sequence, in other pages, in padding queries and,
    where the causal mask hides them, in keys and values."""
    d, P, Hkv, H = 128, 16, 2, 8
    lens = [Nq + 37, Nq + 16]
    q_lens = [Nq, max(1, Nq - 1)]
    table, num = page_table([c + 1 for c in pages_of(lens, P)], 6)  # a page behind each sequence
    kp, vp = (filled(num, Hkv, P, d, "bf16", 50 + i) for i in range(2))
    good = kp.clone(), vp.clone()
    used = torch.zeros((num, P), dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // P], j % P] = True
    poison = torch.where(torch.arange(d) % 2 == 0, float("nan"), float("inf")).to(torch.bfloat16)
    for x in (kp, vp):
        x.permute(0, 2, 1, 3)[~used.cuda()] = poison.cuda()
    q = rand((2, H, Nq, d), 51).cuda()
    if q_lens[1] < Nq:
        q[1, :, q_lens[1]:] = float("nan")

    def cache(k, v):
        if fmt == "bf16":
            return k, v
        out = []
        for x in (k, v):
            p4, _ = binding.kv_pages(num, Hkv, P, d, "int4")
            ident = torch.arange(num, dtype=torch.int32, device="cuda")[:, None]
            binding.osm_kv_append(x, x, p4, torch.empty_like(p4), ident, i32([0] * num))
            out.append(p4)
        return out

    kc, vc = cache(kp, vp)
    kg, vg = cache(*good)
    args = (table.cuda(), i32(lens))
    O, L = binding.fa_fwd_paged(q, kc, vc, *args, q_lens=i32(q_lens))
    assert binding.device_status() == 0
    Og, Lg = binding.fa_fwd_paged(torch.nan_to_num(q), kg, vg, *args, q_lens=i32(q_lens))
    assert torch.equal(O, Og) and torch.equal(L, Lg)
    if Nq == 1:
        return
    # the last token's value is hidden from every query but the last
    p = lens[0] - 1
    vp[table[0, p // P], :, p % P] = poison.cuda()
    kp[table[0, p // P], :, p % P] = poison.cuda()
    kc, vc = cache(kp, vp)
    O2, L2 = binding.fa_fwd_paged(q, kc, vc, *args, q_lens=i32(q_lens))
    a, b = (O2[0, :, :-1], L2[0, :, :-1]), (O[0, :, :-1], L[0, :, :-1])
    if Nq * H // Hkv < 256:
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    else:
        # Another kernel computes such a sequence of a long chunk.  Each result is off by a rounding
        # of O and one of the shares to bf16, 2^-8 |O| + 2^-8 sum p |V|, both at most
        # 2^-8 max |V|; LSE by the scores' and sums' fp32 roundings (2^-20 of scores below 64).
        assert (a[0].float() - b[0].float()).abs().max() <= 4.04 * 2.0 ** -8 * good[1].abs().max()
        assert (a[1] - b[1]).abs().max() <= 2 * 64 * 2.0 ** -20
    assert torch.isnan(O2[0, :, -1]).any(-1).all()


def test_repeats_bit_for_bit_and_replays():
    """Twice the same call, a captured and replayed one, and one on a side stream agree."""
    B, H, Hkv, Nq, d, P = 3, 8, 2, 2, 128, 32
    lens = [3000, 5, 800]
    table, num = page_table(pages_of([3000, 700, 800], P), 8)  # both lengths' pages
    kp, vp = (filled(num, Hkv, P, d, "int4", 60 + i) for i in range(2))
    q = rand((B, H, Nq, d), 61).cuda()
    t, n = table.cuda(), i32(lens)
    O, L = binding.fa_fwd_paged(q, kp, vp, t, n)
    O2, L2 = binding.fa_fwd_paged(q, kp, vp, t, n)
    assert torch.equal(O, O2) and torch.equal(L, L2)
    need = binding.paged_plan(B, H, Hkv, Nq, d, "int4", P, t.shape[1])
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    out, lse = torch.empty_like(q), torch.empty_like(L)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.fa_fwd_paged(q, kp, vp, t, n, out=out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(O, out) and torch.equal(L, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.fa_fwd_paged(q, kp, vp, t, n, out=out, lse=lse, workspace=ws)
    n.copy_(i32([2000, 700, 0]))  # the lengths are read when the graph runs
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(q, kp, vp, table, [2000, 700, 0], None, True, P, O=out, L=lse)


def test_a_side_stream_allocates_its_own():
    """Results and workspaces made for a call on another stream come from that stream's memory, so
    that work still queued on the current stream cannot meet them."""
    d, P, Hkv = 128, 16, 2
    kp, vp = (filled(8, Hkv, P, d, "int4", 75 + i) for i in range(2))
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    q = rand((1, 8, 40, d), 76).cuda()
    rt = binding.rope_table(binding.rope_rates(d))
    want, _ = binding.fa_fwd_paged(q, kp, vp, table, i32([120]))
    turned = binding.osm_rope(q, rt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.empty(1 << 26, device="cuda")
    lens = i32([120])
    torch.cuda.synchronize()
    for _ in range(20):  # memory freed on the current stream while that is still writing it
        t = torch.empty_like(want)
        busy.fill_(1.0)
        t.fill_(7.0)
        del t
        O, _ = binding.fa_fwd_paged(q, kp, vp, table, lens, stream=side)
        y = binding.osm_rope(q, rt, stream=side)
        side.synchronize()
        torch.cuda.current_stream().synchronize()
        assert torch.equal(O, want) and torch.equal(y, turned)


def test_shared_prefix_pages():
    """Two sequences whose first pages are the same pages."""
    d, P, Hkv = 128, 16, 2
    table = torch.tensor([[0, 1, 2], [0, 1, 3]], dtype=torch.int32)
    kp, vp = (filled(4, Hkv, P, d, "int4", 70 + i) for i in range(2))
    check(rand((2, 4, 1, d), 71).cuda(), kp, vp, table, [40, 44], None, True, P)


def test_pages_past_four_gigabytes():
    """Page offsets pass 32 bits."""
    d, P, Hkv = 128, 1024, 8
    num = 2200  # 2200 * 8 * 1024 * 256 bytes = 4.6 GB an array
    kp = torch.empty((num, Hkv, P, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    last = num - 1
    table = torch.tensor([[last, 0]], dtype=torch.int32)
    for i, x in enumerate((kp, vp)):
        x[0], x[last] = (filled(1, Hkv, P, d, "bf16", 80 + 2 * i + j)[0] for j in range(2))
    k = rand((1, Hkv, 2, d), 85).cuda()
    binding.osm_kv_append(k, k, kp, vp, table.cuda(), i32([1022]))
    q = rand((1, 8, 1, d), 86).cuda()
    O, L = binding.fa_fwd_paged(q, kp, vp, table.cuda(), i32([1030]))
    K, V = binding.osm_kv_gather(kp, vp, table.cuda(), i32([1030]), 1030, d)
    assert binding.device_status() == 0
    assert torch.equal(K[0, :, 1022:1024], k[0]) and torch.equal(V[0, :, :1022], vp[last, :, :1022])
    assert torch.equal(K[0, :, 1024:], kp[0, :, :6])
    small = torch.stack((kp[last], kp[0])), torch.stack((vp[last], vp[0]))
    check(q, *small, torch.tensor([[0, 1]], dtype=torch.int32), [1030], None, True, P, O=O, L=L)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_prompt_then_decoding(fmt):
    """A prompt in two chunks, then tokens one by one: every query's output is that of the whole
    sequence's causal attention over what the cache gives back."""
    B, H, Hkv, d, P, rot = 2, 8, 2, 128, 16, 64
    plan = [(40, [40, 25]), (9, [9, 9])] + [(1, [1, 1])] * 6
    table, num = page_table([6, 6], 9)
    t = table.cuda()
    kp, vp = binding.kv_pages(num, Hkv, P, d, fmt)
    rt = binding.rope_table(binding.rope_rates(rot, scaling="bands", factor=4.0, orig_len=64.0,
                                               low=1.0, high=4.0))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    qs, outs = [[] for _ in range(B)], [[] for _ in range(B)]
    for step, (N, new) in enumerate(plan):
        qkv = rand((B, N, H + 2 * Hkv, d), 90 + step).cuda()
        q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
        nl = i32(new)
        qr = binding.osm_kv_append(k, v, kp, vp, t, lens, new_lens=nl, table=rt, q=q)
        # the same rotation as the operator of its own
        pos = lens[:, None] + torch.arange(N, dtype=torch.int32, device="cuda")
        alone = binding.osm_rope(q, rt, positions=pos)
        lens += nl
        O, L = binding.fa_fwd_paged(qr, kp, vp, t, lens, q_lens=nl)
        for b in range(B):
            assert torch.equal(alone[b, :, :new[b]], qr[b, :, :new[b]])
            qs[b].append(qr[b, :, :new[b]])
            outs[b].append((O[b, :, :new[b]], L[b, :, :new[b]]))
    assert binding.device_status() == 0
    for b in range(B):
        n = lens[b].item()
        q = torch.cat(qs[b], 1)[None].contiguous()
        O = torch.cat([o for o, _ in outs[b]], 1)[None]
        L = torch.cat([l for _, l in outs[b]], 1)[None]
        check(q, kp, vp, table[b:b + 1], [n], None, True, P, O=O, L=L)
        # and the framework's dense attention over the cache read out
        K, V = binding.osm_kv_gather(kp, vp, t[b:b + 1], lens[b:b + 1], n, d)
        Od, Ld = binding.fa_fwd_gqa(q, K, V, causal=True)
        # each is off by a rounding of O and of the shares to bf16: 2^-8 |O| + 2^-8 sum p |V|, and
        # |O| <= sum p |V| <= max |V|: 4 * 2^-8 max |V| between the two (an absolute bound would
        # not do: one bf16 step of an output above 2 is 2^-6)
        assert (Od.float() - O.float()).abs().max() <= 4.04 * 2.0 ** -8 * V.float().abs().max()
        assert (Ld - L).abs().max() <= 1e-3
