"""The key/value cache's calls: their status, arguments and streams."""
from __future__ import annotations

import pytest
import torch

from cache_bounds import check_tight, decode_tight
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


# ------------------------------------------------ calls that begin while the last one ends
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_decode_s_output_is_the_next_one_s_query(e4m3):
    """No kernel in between: each call may start while the one that writes its q still runs."""
    c = [Cache([700, 0, 90, 33], 2, 128, 16, e4m3, layout, seed=i) for i, layout in enumerate(("hnd", "nhd"))]
    start = torch.randn(4, 8, 128, device=DEV).to(torch.bfloat16)
    ws = torch.empty(fa.fa_decode_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device=DEV)

    def chain(wait):
        x, out = start.clone(), []
        for t in range(24):
            y = torch.empty_like(x)
            if wait:
                torch.cuda.synchronize()
            cc = c[t % 2]
            fa.fa_decode(x, cc.k, cc.v, o=y, lse=None, scale=0.3, workspace=ws, **cc.args)
            out.append(y)
            x = y
        return out

    slow = chain(True)
    torch.cuda.synchronize()
    for _ in range(5):
        got = chain(False)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
        for t, (a, b) in enumerate(zip(got, slow)):
            assert torch.equal(a, b), f"step {t}"


@pytest.mark.parametrize("layout", ["hnd", "nhd", "padded"])
@pytest.mark.parametrize("H", [1, 3])
def test_decodes_see_each_append_s_factors(H, layout):
    """Steps of append and decode in a row over the same lines of factors, tokens adjacent or not:
    what a decode has read of them before is not what the next one uses."""
    steps, B, d = 50, 3, 64
    c = Cache([steps + 40] * B, H, d, 16, True, layout, seed=7)
    c.lens.copy_(torch.tensor([30, 1, 17], dtype=torch.int32))
    q = torch.randn(B, 4 * H, d, device=DEV).to(torch.bfloat16)
    ws = torch.empty(fa.fa_decode_workspace_bytes(B, 4 * H, H, d), dtype=torch.uint8, device=DEV)
    # Sizes that change from step to step: a factor of the step before would show.
    size = torch.exp2(torch.arange(steps, device=DEV) * 5 % 17 - 8.0)[:, None, None, None, None]
    new = (torch.randn(steps, 2, B, H, d, device=DEV) * size).to(torch.bfloat16)
    lens = [c.lens + t + 1 for t in range(steps)]
    out = []
    torch.cuda.synchronize()
    for t in range(steps):
        args = dict(c.args, seq_lens=lens[t])
        fa.fa_cache_append(new[t, 0], new[t, 1], c.k, c.v, **args)
        o, L = torch.empty_like(q), torch.empty(B, 4 * H, device=DEV)
        fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=0.02, workspace=ws, **args)
        out.append((o, L))
    assert fa.fa_device_status() == 0
    for t in range(steps):
        check_decode(*out[t], decode_exact(c, q, 0.02, lens=lens[t].tolist()), f"step {t}")
        for b in range(B):
            ref = decode_tight(c, q[b], 0.02, b=b, n=int(lens[t][b]))
            check_tight(out[t][0][b], out[t][1][b], ref, f"step {t}, sequence {b}")
