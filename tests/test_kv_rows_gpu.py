"""What osm_kv_append stores in 4 bits where the quantiser's decisions are close, bit for bit against
the fp64 restatement."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding
from test_kv_cache_gpu import i32

pytestmark = pytest.mark.gpu


def stored(k, v, past, rates=None, layout="half"):
    """The page bytes (keys, values) uint8 [B, H_kv, bytes] of one token for each of B sequences: k, v
    bf16 [B, H_kv, 1, d], sequence b's at position past[b], which is the first place of a page."""
    B, Hkv, _, d = k.shape
    pages = [p // 16 for p in past]
    assert all(p % 16 == 0 for p in past)
    table = torch.full((B, max(pages) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        table[b, n] = b
    kp, vp = binding.kv_pages(B, Hkv, 16, d, "int4")
    binding.osm_kv_append(k.cuda(), v.cuda(), kp, vp, table.cuda(), i32(past),
                          table=None if rates is None else binding.rope_table(rates),
                          layout=layout)
    assert binding.device_status() == 0
    return kp.cpu().numpy(), vp.cpu().numpy()


def wanted(x):
    """Page bytes of x [B, H_kv, 1, d] float64 in the first place of a page of 16."""
    return ref.head_bytes(np.concatenate((x, np.zeros(x.shape[:2] + (15, x.shape[3]))), 2))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot", [0, 32])
def test_a_span_just_above_a_step(d, rot):
    """15 s >= max - min where the span passes 15 steps by less than a float of it shows: 15 and -1e-9
    want a step of 1.25, not of 1."""
    rows = []
    for top in (15.0, 60.0, 75.0, 90.0, 105.0, 15.0 * 2 ** 20, 105.0 * 2.0 ** -60):
        for low in (-1e-9, -1e-12):
            x = np.zeros(d)
            x[d - 20], x[d - 7] = top, low * top
            rows += [x, -x[::-1] if rot == 0 else x]
    x = torch.tensor(np.array(rows)).to(torch.bfloat16)[:, None, None]  # [B, 1, 1, d]
    B = x.shape[0]
    # at position 0 a rotation changes nothing
    kp, vp = stored(x, x, [0] * B, ref.rates(rot) if rot else None)
    want = wanted(x.double().numpy())
    assert np.array_equal(vp, want) and np.array_equal(kp, want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_partners_much_larger_than_the_group(layout):
    """In the half layout at d = 128 value i's partner is in the other group.  Keys whose second half
    is hundreds of steps of the first, at angles so near whole half turns that little of it comes
    over: what does carries an error of its partner's size, which decides codes and steps."""
    B, Hkv, d = 64, 32, 128
    g = torch.Generator().manual_seed(11)
    k = torch.randn((B, Hkv, 1, d), generator=g)
    k[..., d // 2:] = (200 + 800 * torch.rand((B, Hkv, 1, d // 2), generator=g)) * \
        torch.sign(k[..., d // 2:])
    k = k.to(torch.bfloat16)
    w = [float(np.pi / 16 * (1 + 1e-4 * (2 * r - 1))) for r in torch.rand(d // 2, generator=g)]
    past = [16 * (b % 7 + 1) for b in range(B)]
    kp, vp = stored(k, k, past, w, layout)
    x = k.double().numpy()
    assert np.array_equal(vp, wanted(x))
    assert np.array_equal(kp, wanted(ref.rotate(x, np.array(past)[:, None], w, layout)))
