"""fa_fwd_paged_shared for thousands of sequences: the plan's passes over them, and what they cost."""
import numpy as np
import pytest
import torch

from online_softmax_tiled_attn_gb300 import binding
from test_kv_cache_gpu import check, filled, i32, rand
from test_shared_gpu import run, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("what", ["late", "pairs", "steps", "one"])
def test_thousands_of_sequences(what, fmt):
    """More than a step of the plan's passes takes: one run whose first sequences cannot share, pairs,
    runs that begin and end around the steps of 1024, one run of all."""
    P, d, H, Hkv = 16, 64, 2, 1
    r = np.random.RandomState(3)
    if what == "late":      # 2100 idle, empty or short ones, then a common prefix
        sizes, prefix = [1] * 2100 + [900], [0] * 2100 + [300]
        lens = [int(x) for x in r.randint(0, 120, 2100)] + [301 + i % 40 for i in range(900)]
    elif what == "pairs":
        sizes = [2] * 1300
        prefix = [int(x) for x in r.choice([100, 130, 260], 1300)]
        lens = [prefix[b // 2] + 1 + b % 5 for b in range(2600)]
    elif what == "steps":
        sizes = [1023, 2, 1022, 1, 1, 1024, 30, 2]
        prefix = [140, 300, 129, 0, 500, 260, 128, 400]
        lens = [prefix[j] + 1 + i % 7 for j, n in enumerate(sizes) for i in range(n)]
    else:
        sizes, prefix = [2200], [270]
        lens = [271 + i % 33 for i in range(2200)]
    table, num, groups = tables(sizes, prefix, lens, P, 3)
    if what in ("late", "one"):
        groups = None
    elif what == "pairs":
        groups = [b // 2 % 7 for b in range(2600)]
    kp, vp = (filled(num, Hkv, P, d, fmt, 20 + i) for i in range(2))
    q = rand((len(lens), H, 1, d), 30).cuda()
    O, L = run(q, kp, vp, table, lens, groups, None, True, P)
    assert binding.device_status() == 0
    check(q, kp, vp, table, lens, None, True, P, O=O, L=L)


def test_looking_for_common_pages_stays_cheap():
    """8192 sequences as one group in a table four times as wide as they need: less than twice as long
    as each by itself (1.5 times; 2.7 where one warp walked over all of them for each step)."""
    P, d, H, Hkv, B = 16, 64, 4, 1, 8192
    lens = [256 + 1 + i % 20 for i in range(B)]
    table, num, _ = tables([B], [256], lens, P, 3, width=64)
    kp, vp = binding.kv_pages(num, Hkv, P, d, "bf16")
    q, table, lens = rand((B, H, 1, d), 30).cuda(), table.cuda(), i32(lens)
    shape = (B, H, Hkv, 1, d, "bf16", P, 64)
    assert binding.paged_shared_plan(*shape) > binding.paged_plan(*shape)

    def time(call):
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(5):
                call(q, kp, vp, table, lens)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    alone = time(binding.fa_fwd_paged)
    assert time(binding.fa_fwd_paged_shared) < 2 * alone
    assert binding.device_status() == 0
