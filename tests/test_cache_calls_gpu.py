"""The key/value cache's calls: their status, arguments and streams."""
from __future__ import annotations

import pytest
import torch

from cache_helpers import DEV, Cache
from io_aware_exact_23_b200 import binding as fa

pytestmark = pytest.mark.gpu


def setup(e4m3=False, seed=0):
    c = Cache([200, 0, 90], 2, 64, 16, e4m3, seed=seed)
    q = torch.randn(3, 4, 64, device=DEV).to(torch.bfloat16)
    o, L = torch.empty_like(q), torch.empty(3, 4, device=DEV)
    ws = torch.empty(fa.fa_decode_workspace_bytes(3, 4, 2, 64), dtype=torch.uint8, device=DEV)
    return c, q, o, L, ws


# ------------------------------------------------------------------ status
def test_a_bad_page_does_not_hide_a_timeout():
    """A wait that gave up is what the status says, whatever a table brought before it."""
    c, q, o, L, ws = setup()
    c.table[0, 3] = c.num
    fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=0.1, workspace=ws, **c.args)
    fa.fa_selftest_timeout()
    st, info = fa.fa_device_status(info=True)
    assert st == 7 and info[:3] == [5, 1, 0] and info[3] > 0, (st, info)
    assert fa.fa_device_status() == 0
    # The other way round, the timeout stays too.
    fa.fa_selftest_timeout()
    fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=0.1, workspace=ws, **c.args)
    st, info = fa.fa_device_status(info=True)
    assert st == 7 and info[:2] == [5, 1], (st, info)
    fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=0.1, workspace=ws, **c.args)
    st, info = fa.fa_device_status(info=True)
    assert st == 9 and info[:2] == [8, 0] and info[3] > 0, (st, info)
    assert fa.fa_device_status() == 0
