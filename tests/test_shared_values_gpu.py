"""Which tokens fa_fwd_paged_shared reads once for a group, and how it takes their 4-bit values.  Keys
whose groups lie far to one side of zero have values that bf16 cannot hold: the common part takes
them rounded, as osm_kv_gather gives them, a sequence's own tokens are exact.  The LSE tells the two
apart by much more than its tolerance, so it shows which tokens were common."""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding
from test_kv_cache_gpu import filled, i32, rand, values
from test_shared_gpu import tables, wide, widened

pytestmark = pytest.mark.gpu

TILE = 128


def one_sided(num, Hkv, P, d, seed):
    """4-bit pages of keys 7/4 2^-6 times 37, 41 or 45: the base 31 and codes 6, 10 or 14."""
    r = np.random.RandomState(seed)
    codes = r.choice([6, 10, 14], (num, Hkv, P, d)).astype(np.uint8)
    body = (codes[..., 0::2] | codes[..., 1::2] << 4).reshape(num, Hkv, -1)
    step = int(np.float32(1.75 / 64).view(np.uint32)) >> 21
    words = np.full((num, Hkv, P * d // 64), step << 6 | 31, dtype="<u2").view(np.uint8)
    return torch.from_numpy(np.concatenate((body, words), -1)).cuda()


def held(lens, Nq, q_lens, causal):
    """Tokens of each sequence that it may share."""
    ql = [Nq] * len(lens) if q_lens is None else q_lens
    return [0 if k == 0 else (n - k if causal else n - 1) for n, k in zip(lens, ql)]


def lse_and_o(q, kx, kr, vx, vstep, kstep, table, n, ql, causal, common):
    """The fp64 result with the first `common` keys as kr, the others as kx, and its tolerances."""
    k, r, v, vs, ks = (ref.dense(x, table, n) for x in (kx, kr, vx, vstep, kstep))
    k[:, :common] = r[:, :common]
    return ref.attend(q, k, v, 136 * ks, vs, 1 / math.sqrt(q.shape[-1]), causal, ql)


def run(H, Hkv, Nq, d, P, table, num, lens, q_lens, groups, causal, common):
    """The call on one-sided keys: its result is that of `common[b]` rounded keys of each sequence, and
    for a sequence that shares, not that of none or of a tile more or less."""
    B = len(lens)
    kp, vp = one_sided(num, Hkv, P, d, 3), filled(num, Hkv, P, d, "int4", 4)
    q = rand((B, H, Nq, d), 5).abs().cuda()
    full = widened(table, wide(B, Hkv, P)).cuda()
    shape = (B, H, Hkv, Nq, d, "int4", P, full.shape[1])
    assert binding.paged_shared_plan(*shape) > binding.paged_plan(*shape)
    O, L = binding.fa_fwd_paged_shared(q, kp, vp, full, i32(lens), causal=causal,
                                       groups=None if groups is None else i32(groups),
                                       q_lens=None if q_lens is None else i32(q_lens))
    assert binding.device_status() == 0
    kx, kstep = values(kp, P, d)
    vx, vstep = values(vp, P, d)
    kr = torch.from_numpy(kx).to(torch.bfloat16).double().numpy()
    assert (kr != kx).all()
    # the read-out gives these
    K, _ = binding.osm_kv_gather(kp, vp, full, i32(lens), max(lens), d)
    t = table.numpy()
    for b, n in enumerate(lens):
        assert np.array_equal(K[b, :, :n].double().cpu().numpy(), ref.dense(kr, t[b], n))
        ql = Nq if q_lens is None else q_lens[b]
        qb = q[b].double().cpu().numpy()
        args = (qb, kx, kr, vx, vstep, kstep, t[b], n, ql, causal)
        Or, Lr, tO, tL = lse_and_o(*args, common[b])
        Ob, Lb = O[b].double().cpu().numpy(), L[b].double().cpu().numpy()
        some = np.isfinite(Lr)
        assert np.array_equal(np.isfinite(Lb), some)
        assert (np.abs(Lb[some] - Lr[some]) <= tL[some]).all(), b
        assert (np.abs(Ob - Or) <= tO).all(), b
        for other in {0, common[b] - TILE, common[b] + TILE} - {common[b]}:
            if 0 <= other <= n and ql:
                _, Lo, _, _ = lse_and_o(*args, other)
                assert (np.abs(Lo[some] - Lr[some]) > 10 * tL[some]).all(), (b, other)


@pytest.mark.parametrize("Nq, causal, lens", [
    (1, True, 128), (1, True, 129), (1, False, 128), (1, False, 129), (3, True, 130), (3, True, 131),
    (3, False, 128), (3, False, 129), (2, True, 257), (2, True, 258), (1, False, 257),
])
@pytest.mark.parametrize("d", [64, 128])
def test_the_least_that_is_shared(Nq, causal, lens, d):
    """128 tokens that all queries see, on either side; whole tiles.  (Equal rows: all pages are common,
    and one token stays a sequence's own.)"""
    P = 16
    table, num, _ = tables([2], [lens + P], [lens] * 2, P, 5)
    table[1] = table[0]
    n = held([lens], Nq, None, causal)[0] // TILE * TILE
    assert n == {128: 0, 130: 0, 129: 128, 131: 128, 257: 256 if Nq == 1 else 128, 258: 256}[lens]
    run(2, 1, Nq, d, P, table, num, [lens] * 2, None, None, causal, [n] * 2)


@pytest.mark.parametrize("sizes, prefix, own, q_lens, groups, common", [
    # the least of three, one that falls short, one that is idle
    ([5], [600], [40, 400, 1, 200, 30], [2, 2, 2, 0, 1], None, [512, 512, 512, 0, 512]),
    # two groups; the second's sequences have a tile in common
    ([2, 3], [300, 150], [9, 30], None, "given", [256, 256, 128, 128, 128]),
    # both as one group: the first one's pages count, and the others have none of them
    ([2, 3], [300, 150], [9, 30], None, None, [256, 256, 0, 0, 0]),
    # one sequence with other pages in front: nothing in common
    ([1, 4], [300, 300], [9, 30], None, None, [0, 0, 0, 0, 0]),
    # the same one, too short to share: it is passed over
    ([1, 4], [100, 300], [9, 30], None, None, [0, 256, 256, 256, 256]),
    # one with other pages between them
    ([2, 1], [400, 300], [9, 30], None, None, [384, 384, 0]),
])
def test_what_is_found_in_common(sizes, prefix, own, q_lens, groups, common):
    P, Nq = 16, 2
    lens = []
    for j, n in enumerate(sizes):
        lens += [prefix[j] + max(Nq, own[(len(lens) + i) % len(own)]) for i in range(n)]
    table, num, given = tables(sizes, prefix, lens, P, 5)
    run(4, 2, Nq, 64, P, table, num, lens, q_lens, given if groups else None, True, common)
