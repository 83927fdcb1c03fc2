"""The key/value cache's calls: their status, arguments and streams."""
from __future__ import annotations

import pytest
import torch

from cache_helpers import DEV, Cache, check_decode, decode_exact
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


# ----------------------------------------------------------------- streams
@pytest.mark.parametrize("e4m3", [False, True])
def test_wrapper_on_a_stream(e4m3):
    """KVCache's calls on a stream that is not the current one: results, and memory that is
    not handed out again while they run."""
    ref = Cache([90, 0, 33], 2, 64, 16, e4m3, seed=3, fill=False)
    c = fa.KVCache(ref.num, 2, 16, 64, e4m3)
    new = torch.randn(2, 123, 2, 64, device=DEV).to(torch.bfloat16)
    cu = torch.tensor([0, 90, 90, 123], dtype=torch.int32, device=DEV)
    q = torch.randn(3, 4, 64, device=DEV).to(torch.bfloat16)
    ref.k, ref.v, ref.ks, ref.vs = c.k, c.v, c.k_scale, c.v_scale
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # what follows is still to run when the calls return
    c.append(new[0], new[1], ref.table, ref.lens, cu, stream=s)
    o, L = c.decode(q, ref.table, ref.lens, 0.2, stream=s)
    k, v = c.gather(ref.table, ref.lens, 90, rep=2, stream=s)
    for _ in range(20):  # the current stream's own allocations of the same sizes
        for t in (o, L, k):
            torch.empty_like(t).fill_(7)
        torch.empty(fa.fa_decode_workspace_bytes(3, 4, 2, 64), dtype=torch.uint8, device=DEV).fill_(0xFF)
    s.synchronize()
    assert fa.fa_device_status() == 0
    check_decode(o, L, decode_exact(ref, q, 0.2))
    for b, n in ((0, 90), (2, 33)):
        for t, nm in ((k, "k"), (v, "v")):
            want = ref.rows(nm, b, n).repeat_interleave(2, 0)
            assert ((t[b, :, :n].double() - want).abs() <= (2.0**-8 + 2.0**-23) * want.abs()).all()
    assert (k[1] == 0).all() and (v[2, :, 33:] == 0).all()
