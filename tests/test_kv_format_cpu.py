"""What the 4-bit format can hold, over all steps' fractions and all integers that the quantiser can
give them; and pages too large for the attention's addresses."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding


def reachable():
    """(fraction in quarters, b + code): the base is rint(min / s) with |min| <= 31 s, a code at most
    15 above it."""
    return [(f, n) for f in (4, 5, 6, 7) for n in range(-31, 31 + 15 + 1)]


def test_values_that_bf16_rounds():
    """A value is a bf16 number but for five integers at a step of 7/4: those lie half way between two,
    a seventh of the step from each."""
    wide = []
    for f, n in reachable():
        for e in (-126, -2, 0, 100):
            x = np.ldexp(f * n / 4, e)  # 9 bits at most: exact
            y = torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).item()
            if x != y:
                wide.append((f, n))
                assert abs(x - y) == np.ldexp(0.25, e) and abs(x - y) * 7 == np.ldexp(f / 4, e)
    assert sorted(set(wide)) == [(7, n) for n in (37, 39, 41, 43, 45)] and len(wide) == 20


def test_groups_reach_them():
    """Far from zero: the least value 22 steps or more up."""
    x = np.linspace(52.5, 78.5, 64)
    codes, s, b = ref.quantise(x)
    assert s[0] == 1.75 and b[0] == 30
    stored = ref.stored(x)
    back = torch.from_numpy(stored).to(torch.bfloat16).double().numpy()
    assert np.abs(stored - x).max() <= s[0] / 2
    assert np.array_equal(back != stored, np.isin(codes + b[0], (37, 39, 41, 43, 45)))
    assert (back != stored).any()
    assert s[0] / 2 < np.abs(back - x).max() <= s[0] / 2 + s[0] / 7


def test_groups_that_hold_zero_never_do():
    """A group with a value of no more than 21 steps has none of them: the quantiser's rows of any
    cache whose groups straddle zero are bf16 numbers."""
    for f, n in reachable():
        for base in range(-31, 22):
            if base <= n <= base + 15:
                x = f * n / 4
                assert torch.tensor(x).to(torch.bfloat16).item() == x


@pytest.mark.parametrize("fmt,H_kv,want", [
    (0, 8191, binding.FA_OK), (0, 8192, binding.FA_ERR_UNSUPPORTED),
    (1, 30840, binding.FA_OK), (1, 30841, binding.FA_ERR_UNSUPPORTED),
])
def test_pages_of_two_gigabytes_are_refused_before_anything_runs(fmt, H_kv, want):
    """2^18 or 69632 bytes a head of a page of 1024 tokens of 128 values.  300 queries: a chunk, whose
    read-out and dense attention come before the kernel that cannot address such pages."""
    n = ctypes.c_int64(0)
    assert binding.lib().fa_fwd_paged_plan(1, H_kv, H_kv, 300, 128, fmt, 1024, 1,
                                           ctypes.byref(n)) == want
