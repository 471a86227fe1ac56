"""fa_fwd_paged_shared where the sequences' own tokens are of very different numbers: fresh forks beside
long ones.  Results, and that sharing pays there too."""
import pytest
import torch

from online_softmax_tiled_attn_gb300 import binding
from test_kv_cache_gpu import check, filled, i32, rand
from test_shared_gpu import run, tables

pytestmark = pytest.mark.gpu

OWN = {
    "half": lambda B: [1000] * (B // 2) + [3] * (B - B // 2),
    "first": lambda B: [9000] + [4] * (B - 1),
    "last": lambda B: [4] * (B - 1) + [3000],
    "alternating": lambda B: [700 if b % 2 else 5 for b in range(B)],
    "ones": lambda B: [3] * B,
}


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("B, H, Hkv, Nq, d, P", [
    (24, 8, 2, 1, 128, 16), (24, 8, 2, 3, 64, 64), (7, 12, 4, 3, 128, 48), (40, 8, 8, 1, 64, 32),
])
@pytest.mark.parametrize("own", OWN)
def test_uneven(own, B, H, Hkv, Nq, d, P, fmt):
    """Equal shares of the work begin and end anywhere: between items, within them, and within what an
    item costs before its first tile."""
    lens = [512 + n for n in OWN[own](B)]
    table, num, _ = tables([B], [512], lens, P, 5)
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((B, H, Nq, d), 30).cuda()
    for ql in (None, [Nq if b % 5 else max(0, Nq - b % 3) for b in range(B)]):
        O, L = run(q, kp, vp, table, lens, None, ql, True, P)
        assert binding.device_status() == 0
        check(q, kp, vp, table, lens, ql, True, P, O=O, L=L)


@pytest.mark.parametrize("fmt, Nq", [("bf16", 1), ("int4", 3)])
def test_forks_of_a_long_prompt_beside_long_answers(fmt, Nq):
    """32 sequences with 1000 tokens of their own and 32 with a few, behind 16384 common ones: sharing
    takes a third of the time (0.26 and 0.33 of it; 1.1 and 1.7 times it where equal numbers of tiles
    were an equal share)."""
    P, d, H, Hkv, B = 64, 128, 32, 8, 64
    lens = [16384 + (1000 if b < 32 else 10) for b in range(B)]
    table, num, _ = tables([B], [16384], lens, P, 5)
    kp, vp = binding.kv_pages(num, Hkv, P, d, fmt)
    q, table, lens = rand((B, H, Nq, d), 30).cuda(), table.cuda(), i32(lens)

    def time(call):
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                call(q, kp, vp, table, lens)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    alone = time(binding.fa_fwd_paged)
    assert time(binding.fa_fwd_paged_shared) < 0.7 * alone
    assert binding.device_status() == 0
