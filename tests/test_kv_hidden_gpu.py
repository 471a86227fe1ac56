"""fa_fwd_paged over 4-bit pages: large finite values that some queries do not see."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from test_kv_cache_gpu import check, filled, page_table, pages_of, rand

pytestmark = pytest.mark.gpu

# H, Hkv, Nq, d, page, lens, q_lens
CASES = [
    (2, 2, 2, 64, 16, [40, 3], None),
    (8, 2, 5, 128, 16, [5, 77], None),          # every tile is hidden from some query
    (8, 8, 8, 128, 64, [300, 64], [8, 3]),
    (4, 1, 4, 64, 32, [1000, 4], None),
    (6, 2, 33, 128, 48, [200, 50], [33, 20]),   # blocks of rows that see none of the last tiles
    (2, 1, 16, 128, 16, [530, 12], [16, 16]),   # more queries than keys
    (32, 2, 4, 128, 16, [2500, 9], None),       # items that span shares
]


@pytest.mark.parametrize("big", [2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("H,Hkv,Nq,d,P,lens,q_lens", CASES, ids=lambda v: str(v)[:24])
def test_large_values_that_a_query_does_not_see(H, Hkv, Nq, d, P, lens, q_lens, big):
    """The last tokens' values are `big` times the others', so that their steps pass those of the
    tokens before by what no fp16 share can span.  A query is held to the steps that it sees."""
    table, num = page_table(pages_of(lens, P), 5)
    v = rand((num, Hkv, P, d), 21).double().numpy()
    for b, n in enumerate(lens):
        ql = Nq if q_lens is None else q_lens[b]
        for j in range(max(0, n - ql), n):
            if j % 3 != 1:  # ordinary ones between them, and one group of two of some
                v[table[b, j // P], :, j % P, :64 if j % 3 == 2 else d] *= big
    vp = torch.from_numpy(ref.head_bytes(v)).cuda()
    kp = filled(num, Hkv, P, d, "int4", 20)
    q = rand((len(lens), H, Nq, d), 30).cuda()
    check(q, kp, vp, table, lens, q_lens, True, P)
