"""The calls on the pool of cache pages refuse bad arguments on the host, before any CUDA call; the
restatement that the GPU tests use keeps a pool's books."""
import ctypes

import numpy as np
import pytest

import pool_ref as ref
from online_softmax_tiled_attn_gb300 import binding

P = 1 << 20
T = 1 << 20  # bytes between the fake addresses
BAD, UNSUP, OK = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_OK

SHARED = [
    (dict(rows=-1), BAD), (dict(maxp=-1), BAD), (dict(nump=-1), BAD), (dict(nump=1 << 31), BAD),
    (dict(page=0), BAD), (dict(page=24), UNSUP), (dict(page=2048), UNSUP),
    (dict(maxp=(1 << 26) + 1), BAD), (dict(rows=1 << 20, maxp=1 << 12), UNSUP),
    (dict(pt=0), BAD), (dict(pt=P + 2), BAD), (dict(lens=0), BAD), (dict(lens=P + T + 1), BAD),
    (dict(refs=0), BAD), (dict(refs=P + 2 * T + 3), BAD),
    (dict(lens=P + 4), BAD), (dict(refs=P + T), BAD),       # arrays on one another
]
WS = [(dict(ws=0), BAD), (dict(ws=P + 20 * T + 8), BAD), (dict(wsb=0), BAD), (dict(ws=P), BAD)]
MANY = dict(rows=3000)  # more rows than the calls without a workspace take
WS_MANY = [({**MANY, **over}, want) for over, want in WS] + [(dict(wsb=-1), BAD)]
PAGES = [(dict(d=96), UNSUP), (dict(fmt=2), BAD), (dict(kp=0), BAD), (dict(vp=P + 9 * T + 8), BAD),
         (dict(kp=P + 9 * T), BAD), (dict(Hkv=-1), BAD), (dict(Hkv=1 << 20), UNSUP),
         (dict(kp=P + 2 * T), BAD)]


def base(over, **more):
    """5 rows of 8 entries, 16 pages of 16 tokens, at distinct fake addresses."""
    a = dict(pt=P, maxp=8, page=16, lens=P + T, refs=P + 2 * T, nump=16, rows=5, ws=P + 20 * T,
             wsb=1 << 40, kp=P + 8 * T, vp=P + 9 * T, fmt=0, Hkv=2, d=128)
    a.update(more)
    a.update(over)
    return a


@pytest.mark.parametrize("over, want", SHARED + WS_MANY + PAGES + [
    (dict(rows=0), OK), (dict(rows=0, pt=0, lens=0, new=0, ws=0), OK), (dict(new=0), BAD),
    (dict(new=P + 3 * T + 2), BAD), (dict(old=P + 4 * T + 1), BAD), (dict(old=P + 3 * T), BAD),
    (dict(new=P + T), BAD), (dict(old=P + T), BAD), (dict(new=P + 9 * T + 64), BAD),
])
def test_grow_refusals(over, want):
    a = base(over, **{k: v for k, v in dict(new=P + 3 * T, old=P + 4 * T).items() if k not in over})
    assert binding.lib().osm_kv_grow(a["kp"] or None, a["vp"] or None, a["fmt"], a["nump"],
                                     a["page"], a["pt"] or None, a["maxp"], a["lens"] or None,
                                     a["new"] or None, a["old"] or None, a["refs"] or None,
                                     a["rows"], a["Hkv"], a["d"], a["ws"] or None, a["wsb"],
                                     None) == want


@pytest.mark.parametrize("over, want", SHARED + WS_MANY + [
    (dict(n=0), OK), (dict(n=0, src=0, dst=0, ws=0), OK), (dict(n=-1), BAD), (dict(src=0), BAD),
    (dict(dst=0), BAD), (dict(src=P + 3 * T + 2), BAD), (dict(dst=P + T), BAD),
    (dict(n=1 << 30), UNSUP),
])
def test_fork_refusals(over, want):
    a = base(over, **{k: v for k, v in dict(src=P + 3 * T, dst=P + 4 * T, n=3).items()
                      if k not in over})
    assert binding.lib().osm_kv_fork(a["pt"] or None, a["maxp"], a["page"], a["lens"] or None,
                                     a["refs"] or None, a["nump"], a["src"] or None,
                                     a["dst"] or None, a["n"], a["rows"], a["ws"] or None, a["wsb"],
                                     None) == want


@pytest.mark.parametrize("over, want", SHARED + [
    (dict(n=0), OK), (dict(n=-1), BAD), (dict(list=P + 3 * T + 2), BAD), (dict(list=0, n=6), BAD),
    (dict(keep=P + 4 * T + 1), BAD), (dict(list=P + T), BAD), (dict(keep=P + 2 * T), BAD),
    (dict(n=1 << 30), UNSUP),
])
def test_free_refusals(over, want):
    a = base(over, **{k: v for k, v in dict(list=P + 3 * T, keep=P + 4 * T, n=3).items()
                      if k not in over})
    assert binding.lib().osm_kv_free(a["pt"] or None, a["maxp"], a["page"], a["lens"] or None,
                                     a["refs"] or None, a["nump"], a["list"] or None,
                                     a["keep"] or None, a["n"], a["rows"], None) == want


@pytest.mark.parametrize("over, want", SHARED + WS + PAGES + [
    (dict(map=0), BAD), (dict(map=P + 3 * T + 2), BAD), (dict(used=0), BAD),
    (dict(used=P + 4 * T + 2), BAD), (dict(map=P + 2 * T), BAD), (dict(used=P + 3 * T), BAD),
])
def test_compact_refusals(over, want):
    a = base(over, **{k: v for k, v in dict(map=P + 3 * T, used=P + 4 * T).items() if k not in over})
    assert binding.lib().osm_kv_compact(a["kp"] or None, a["vp"] or None, a["fmt"], a["nump"],
                                        a["page"], a["pt"] or None, a["maxp"], a["lens"] or None,
                                        a["refs"] or None, a["map"] or None, a["used"] or None,
                                        a["rows"], a["Hkv"], a["d"], a["ws"] or None, a["wsb"],
                                        None) == want


@pytest.mark.parametrize("over, want", [
    (dict(Nq=0), OK), (dict(B=0), OK), (dict(Nq=-1), BAD), (dict(Hkv=3), BAD), (dict(d=96), UNSUP),
    (dict(page=40), UNSUP), (dict(scale=0.0), BAD), (dict(q=0), BAD), (dict(o=P + 4 * T + 8), BAD),
    (dict(groups=P + 7 * T + 2), BAD), (dict(groups=P + 4 * T), BAD), (dict(kl=0), BAD),
    (dict(ql=P + 5 * T), BAD), (dict(ws=0), BAD), (dict(ws=P + 20 * T + 8), BAD), (dict(wsb=0), BAD),
    (dict(ws=P), BAD), (dict(kp=0), BAD),
])
def test_shared_attention_refusals(over, want):
    """B2 H8 H_kv 2 Nq3 d128 at distinct fake addresses, 64 pages of 16."""
    a = dict(q=P, kp=P + T, vp=P + 2 * T, fmt=1, nump=8, page=16, pt=P + 3 * T, maxp=64,
             kl=P + 6 * T, ql=0, groups=P + 7 * T, o=P + 4 * T, lse=P + 5 * T, B=2, H=8, Hkv=2,
             Nq=3, d=128, scale=0.1, ws=P + 20 * T, wsb=1 << 40)
    a.update(over)
    assert binding.lib().fa_fwd_paged_shared(
        a["q"] or None, a["kp"] or None, a["vp"], a["fmt"], a["nump"], a["page"], a["pt"], a["maxp"],
        a["kl"] or None, a["ql"] or None, a["groups"], a["o"], a["lse"], a["B"], a["H"], a["Hkv"],
        a["Nq"], a["d"], a["scale"], 1, a["ws"] or None, a["wsb"], None) == want


def test_plans():
    assert binding.kv_grow_plan(64, "int4", 16, 8, 128) == 0  # one launch, lists in shared memory
    assert binding.kv_grow_plan(5000, "int4", 16, 1, 64) >= 4 * 20001
    assert binding.kv_grow_plan(64, "bf16", 1024, 8, 128) >= 4 * 257
    assert binding.kv_fork_plan(64, 512, 60) == 0 and binding.kv_fork_plan(0, 0, 0) == 0
    assert binding.kv_fork_plan(5000, 1, 1) >= 4 * 5001
    assert binding.kv_fork_plan(64, 1 << 20, 60) >= 4 * 124
    assert binding.kv_compact_plan(1000) >= 4 * 1001
    n = ctypes.c_int64(0)
    r = ctypes.byref(n)
    L = binding.lib()
    assert L.osm_kv_grow_plan(-1, 0, 16, 1, 64, r) == BAD and L.osm_kv_grow_plan(1, 2, 16, 1, 64, r) == BAD
    assert L.osm_kv_grow_plan(1, 0, 24, 1, 64, r) == UNSUP and L.osm_kv_grow_plan(1, 0, 16, 1, 64, None) == BAD
    assert L.osm_kv_grow_plan(1, 0, 16, 1 << 40, 64, r) == UNSUP
    assert L.osm_kv_grow_plan(1 << 30, 0, 16, 1, 64, r) == UNSUP
    assert L.osm_kv_fork_plan(1, 1, -1, r) == BAD and L.osm_kv_fork_plan(1 << 30, 1, 1, r) == UNSUP
    assert L.osm_kv_fork_plan(1, 1, 1, None) == BAD
    assert L.osm_kv_compact_plan(1 << 31, r) == BAD and L.osm_kv_compact_plan(5, None) == BAD


def test_binding_refuses_host_tensors():
    import torch

    t = torch.zeros((2, 4), dtype=torch.int32)
    v = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        binding.osm_kv_fork(t, v, v, 16, v, v)
    with pytest.raises(TypeError):
        binding.osm_kv_free(t, v, v, 16)
    pages = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.osm_kv_grow(pages, pages, t, v, v, v, 64)
    with pytest.raises(TypeError):
        binding.osm_kv_compact(pages, pages, t, v, v, 64)


def books(table, lens, refs, P):
    """refs are the rows' entries in use, counted."""
    want = np.zeros_like(refs)
    for b, n in enumerate(lens):
        for e in table[b, : ref.count(n, P)]:
            want[e] += 1
    assert (want == refs).all()


def test_reference_pool():
    P, r = 16, np.random.RandomState(3)
    table, lens = np.full((8, 10), -1, np.int32), np.zeros(8, np.int32)
    refs = np.zeros(60, np.int32)
    for step in range(40):
        new = r.randint(0, 30, 8) * (r.rand(8) < 0.5) * (lens > 0) + (lens == 0) * r.randint(0, 40, 8)
        if (refs == 0).sum() > 30:
            old, copies, bad = ref.grow(table, lens, new, refs, P)
            assert not bad and (lens >= old).all() and all(0 < n < P for _, _, n in copies)
        books(table, lens, refs, P)
        rows = r.randint(-1, 8, 3)
        assert not ref.release(table, lens, refs, P, rows, r.randint(0, 60, 3))
        books(table, lens, refs, P)
        empty = [b for b in range(8) if lens[b] == 0]
        if empty and (refs == 0).sum() > 8:
            assert not ref.fork(table, lens, refs, P, [r.randint(8)], empty[:1])
        books(table, lens, refs, P)
        where, used, moves = ref.compact(table, lens, refs, P)
        assert (refs[:used] > 0).all() and (refs[used:] == 0).all()
        books(table, lens, refs, P)
