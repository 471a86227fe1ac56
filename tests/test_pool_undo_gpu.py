"""A pool that runs out: osm_kv_grow is undone by the table, lens and refs from before it, whatever was
appended since, and done again once pages were given back."""
import numpy as np
import pytest
import torch

import pool_ref as ref
from online_softmax_tiled_attn_gb300 import binding
from test_pool_gpu import dev, same, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("P, d, Hkv", [(16, 64, 2), (48, 128, 1), (1024, 128, 8)])
def test_running_out_and_trying_again(P, d, Hkv, fmt):
    """One row and two forks of it, all with a page that is not full, and a row of its own; the pool has
    a page left, then none.  (The last size takes the two launches of larger copies.)"""
    rows, num = 5, 8
    assert (binding.kv_grow_plan(rows, fmt, P, Hkv, d) > 0) == (P == 1024)
    kp, vp = binding.kv_pages(num, Hkv, P, d, fmt)
    table = torch.full((rows, 4), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (rows, num))
    held = [np.zeros((2, Hkv, 0, d)) for _ in range(rows)]
    g = torch.Generator(device="cuda").manual_seed(11)

    def append(old, new, keep=True):
        N = int(max(new))
        # small whole numbers: 4 bits hold them as bf16 does
        k, v = (torch.randint(0, 16, (rows, Hkv, N, d), generator=g, device="cuda")
                .to(torch.bfloat16) for _ in range(2))
        k[..., ::64], v[..., ::64], k[..., 1::64], v[..., 1::64] = 0, 0, 15, 15
        binding.osm_kv_append(k, v, kp, vp, table, old, new_lens=dev(new))
        for b in range(rows if keep else 0):
            x = torch.stack((k[b, :, : new[b]], v[b, :, : new[b]])).float().cpu().numpy()
            held[b] = np.concatenate((held[b], x), 2)

    def grow(new):
        return binding.osm_kv_grow(kp, vp, table, lens, dev(new), refs, d)

    def check():
        n = [h.shape[2] for h in held]
        same(lens, n)
        K, V = binding.osm_kv_gather(kp, vp, table, lens, max(n), d)
        for b in range(rows):
            for x, y in zip((K, V), held[b]):
                assert (x[b, :, : n[b]].float().cpu().numpy() == y).all()
        t, f = table.cpu().numpy(), np.zeros(num, np.int32)
        for b in range(rows):
            for e in t[b, : ref.count(n[b], P)]:
                f[e] += 1
        same(refs, f)

    new = [2 * P + 9, P + 3, 0, 0, 2 * P]
    append(grow(new), new)
    binding.osm_kv_fork(table, lens, refs, P, dev([0, 0]), dev([2, 3]))
    for b in (2, 3):
        held[b] = held[0].copy()
    check()
    assert status() == 0 and int((refs <= 0).sum()) == 1
    # three copies are wanted, a page of a row's own, and there is one page
    new = [5, P - 2, 3, 4, 0]
    before = [t.clone() for t in (table, lens, refs)]
    append(grow(new), new, keep=False)
    assert status() == binding.FA_ERR_PAGE and int((table[:, 2] < 0).sum()) >= 2
    for t, old in zip((table, lens, refs), before):
        t.copy_(old)
    check()
    binding.osm_kv_free(table, lens, refs, P, rows=dev([4, 1]))
    held[4], held[1] = held[4][:, :, :0], held[1][:, :, :0]
    new = [5, 0, 3, 4, 0]
    append(grow(new), new)
    check()
    assert status() == 0
