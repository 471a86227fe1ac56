"""fa_fwd_paged_shared on the host: which calls share, as the header states it."""
import pytest

from online_softmax_tiled_attn_gb300 import binding


def shares(*shape):
    """A call shares where its plan returns more than fa_fwd_paged_plan."""
    more = binding.paged_shared_plan(*shape) - binding.paged_plan(*shape)
    assert more >= 0
    return more > 0


@pytest.mark.parametrize("fmt, least", [("bf16", 7 << 24), ("int4", 10 << 24)])
@pytest.mark.parametrize("B, H, Hkv, Nq, d, P", [
    (2, 1, 1, 1, 64, 16), (8, 32, 8, 1, 128, 64), (65, 16, 4, 2, 64, 48), (3, 24, 1, 1, 128, 16),
    (5, 4, 4, 16, 64, 32), (5, 4, 4, 17, 64, 32), (9, 8, 1, 31, 128, 1024), (1025, 2, 1, 1, 64, 16),
])
def test_which_calls_share(B, H, Hkv, Nq, d, P, fmt, least):
    """By the sequences but one, the blocks of 16 rows and the table's width, not by lengths."""
    rows = Nq * H // Hkv
    page = (B - 1) * -(-rows // 16) * P * Hkv * d  # values that a page of the table's width counts
    pages = -(-least // page)
    assert shares(B, H, Hkv, Nq, d, fmt, P, pages)
    assert not shares(B, H, Hkv, Nq, d, fmt, P, pages - 1)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_what_never_shares(fmt):
    assert not shares(1, 32, 8, 1, 128, fmt, 64, 1 << 20)        # one sequence
    assert shares(2, 8, 1, 31, 64, fmt, 16, 1 << 20)
    assert not shares(2, 8, 1, 32, 64, fmt, 16, 1 << 20)         # 256 rows of a sequence and head
    assert not shares(1 << 20, 8, 8, 1, 64, fmt, 16, 1 << 14)    # 2^39 tiles of 16 tokens
