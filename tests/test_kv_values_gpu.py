"""4-bit values that bf16 does not hold (nine bits: a step of 1.75 times 37, 39, .. 45): the paths over
the cache round them as include/osm_attn.h says."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding
from test_kv_cache_gpu import check, i32, page_table, pages_of, rand, values

pytestmark = pytest.mark.gpu


def wide(shape, seed):
    """Values [.., d] whose groups have a step of 1.75 times a power of two and a base above 21."""
    rng = np.random.default_rng(seed)
    x = rng.uniform(52.5, 78.5, shape)
    x[..., ::64] = 52.5
    return x * 2.0 ** rng.integers(-3, 3, shape[:-1] + (1,))


def pages(num, Hkv, P, d, seed):
    x = wide((num, Hkv, P, d), seed)
    raw = torch.from_numpy(ref.head_bytes(x)).cuda()
    v, s = values(raw, P, d)
    assert np.all(np.frexp(s)[0] == 0.875) and np.all(np.abs(v - x) <= s / 2)
    return raw, v


def test_the_read_out_rounds_once():
    Hkv, d, P, lens = 3, 128, 32, [70, 33]
    table, num = page_table(pages_of(lens, P), 1)
    (kp, k), (vp, v) = (pages(num, Hkv, P, d, i) for i in range(2))
    K, V = binding.osm_kv_gather(kp, vp, table.cuda(), i32(lens), 70, d)
    for out, x in ((K, k), (V, v)):
        assert not np.array_equal(torch.from_numpy(x).to(torch.bfloat16).double().numpy(), x)
        for b, n in enumerate(lens):
            want = torch.from_numpy(ref.dense(x, table[b].numpy(), n)).to(torch.bfloat16)
            assert torch.equal(out[b, :, :n].cpu(), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 3, 40, 64])
def test_attention_of_values_of_nine_bits(d, Nq):
    """A few queries see the values as stored, a chunk (256 rows a key/value head) what the read-out
    gives."""
    H, Hkv, P, lens = 8, 2, 16, [150, 97]
    table, num = page_table(pages_of(lens, P), 2)
    (kp, k), (vp, v) = (pages(num, Hkv, P, d, 3 + i) for i in range(2))
    q = rand((2, H, Nq, d), 7, 0.02).cuda()
    O, L = binding.fa_fwd_paged(q, kp, vp, table.cuda(), i32(lens))
    assert binding.device_status() == 0
    if Nq * H // Hkv >= 256:
        kp, vp = (torch.from_numpy(x).to(torch.bfloat16).cuda() for x in (k, v))
    check(q, kp, vp, table, lens, None, True, P, O=O, L=L)
