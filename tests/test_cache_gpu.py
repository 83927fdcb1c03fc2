"""GPU tests of the paged key/value cache: append, gather and decode against their
definitions in 64 bits, at the lengths, layouts and sharings where they can go
wrong, and as they are used together."""
from __future__ import annotations

import math

import pytest
import torch

from cache_helpers import BF16_HALF, DEV, Cache, check_decode, decode_exact
from io_aware_exact_23_b200 import binding as fa

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 300, 1000]


def ok():
    st, info = fa.fa_device_status(info=True)
    assert st == 0, f"device status {st} {info}"


def make_q(B, Hq, d, seed=0, mult=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed + 77)
    return (torch.randn(B, Hq, d, generator=g) * mult).to(torch.bfloat16).to(DEV)


def decode(c, q, scale=None, window=0, lse=True, ws=None, stream=None, out=None):
    B, Hq, d = q.shape
    o = torch.full_like(q, float("nan")) if out is None else out
    L = torch.full((B, Hq), float("nan"), device=DEV) if lse else None
    if ws is None:
        ws = torch.full((fa.fa_decode_workspace_bytes(B, Hq, c.H, d),), 0xFF, dtype=torch.uint8, device=DEV)
    fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=scale or 1 / math.sqrt(d), workspace=ws, window=window, stream=stream,
                 **c.args)
    return o, L


def run_decode(c, q, label="", **kw):
    o, L = decode(c, q, **kw)
    ok()
    w = kw.get("window", 0)
    check_decode(o, L, decode_exact(c, q, kw.get("scale") or 1 / math.sqrt(q.shape[2]), w), label)
    return o, L


# ------------------------------------------------------------------- decode
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128, 256])
def test_decode_lengths(d, page, e4m3):
    c = Cache(EDGES, 2, d, page, e4m3, "nhd" if page == 16 else "hnd", seed=page)
    run_decode(c, make_q(c.B, 8, d))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 24, 31, 32, 33, 40, 64, 71])
def test_decode_shared_heads(G, e4m3):
    d = 128 if G % 2 else 64
    c = Cache([5, 0, 200, 513], 2, d, 32, e4m3, seed=G)
    run_decode(c, make_q(c.B, 2 * G, d, seed=G))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "joint", "padded"])
@pytest.mark.parametrize("page", [16, 32, 384])
def test_decode_layouts(layout, page, e4m3):
    for d in (64, 128):
        c = Cache([130, 7, 900], 3, d, page, e4m3, layout, seed=3)
        run_decode(c, make_q(c.B, 6, d), f"{layout} {page} {d}")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [1, 2, 100, 127, 128, 129, 500, 5000])
def test_decode_window(window, e4m3):
    c = Cache([0, 1, 128, 129, 300, 1025], 2, 128 if window % 2 else 64, 16, e4m3, seed=window)
    run_decode(c, make_q(c.B, 8, c.d), window=window)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_large_logits(d, e4m3):
    """Nearly one-hot rows whose maximum keeps moving: the running maximum has to rescale."""
    c = Cache([700, 1, 2049], 2, d, 64, e4m3, seed=5, mult=8.0)
    run_decode(c, make_q(c.B, 8, d, mult=8.0))
    # Scores that climb by 20 from each token to the next, and that fall.
    for sign in (1.0, -1.0):
        c = Cache([400], 1, d, 16, e4m3, seed=6)
        q = torch.zeros(1, 4, d, device=DEV, dtype=torch.bfloat16)
        q[:, :, 0] = 1
        r = torch.zeros(400, 1, d, device=DEV, dtype=torch.bfloat16)
        r[:, 0, 0] = torch.arange(400, device=DEV) * 20 * sign
        c.put(c.k, c.ks, 0, torch.arange(400, device=DEV), r)
        run_decode(c, q, scale=1.0)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_e4m3_factors_of_every_size(d):
    """Factors that differ by 2^40 from row to row, and rows of zeros."""
    c = Cache([600, 37], 2, d, 16, True, seed=8)
    g = torch.Generator(device="cpu").manual_seed(1)
    for b, n in enumerate((600, 37)):
        pos = torch.arange(n, device=DEV)
        f = torch.exp2(torch.randint(-20, 20, (n, 1, 1), generator=g).float()).to(DEV)
        r = torch.randn(n, 2, d, generator=g).to(DEV) * f
        r[::7] = 0
        c.put(c.v, c.vs, b, pos, r.to(torch.bfloat16))
    run_decode(c, make_q(2, 8, d))


def test_decode_sink_and_many_small():
    """One key far above many others whose weights only count together."""
    for e4m3 in (False, True):
        n = 20000
        c = Cache([n], 1, 64, 64, e4m3, seed=9, mult=0.05)
        r = torch.zeros(1, 1, 64, device=DEV, dtype=torch.bfloat16)
        r[0, 0, :] = 1
        c.put(c.k, c.ks, 0, torch.zeros(1, dtype=torch.long, device=DEV), r)
        q = torch.ones(1, 8, 64, device=DEV, dtype=torch.bfloat16)
        run_decode(c, q, scale=9.0 / 64)  # the sink's score is 9: about as much weight as the rest


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_many_sequences_and_few_tiles(e4m3):
    """More sequences than threads of a block, and grids with fewer tiles than SMs."""
    r = torch.Generator(device="cpu").manual_seed(4)
    lens = torch.randint(0, 40, (700,), generator=r).tolist()
    lens[100:400] = [0] * 300
    c = Cache(lens, 1, 64, 16, e4m3, seed=10)
    run_decode(c, make_q(700, 2, 64))
    for n in (1, 129, 3000, 18944, 19000):
        c = Cache([n], 1, 128, 128, e4m3, seed=n)
        run_decode(c, make_q(1, 5, 128), f"n = {n}")


def test_decode_all_idle():
    c = Cache([0, 0, 0], 2, 64, 16, False)
    o, L = run_decode(c, make_q(3, 4, 64))
    assert (o == 0).all() and (L == -math.inf).all()


def test_decode_without_lse_and_odd_scale():
    c = Cache([77, 300], 2, 128, 32, False, seed=12)
    run_decode(c, make_q(2, 8, 128), lse=False, scale=0.37)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_repeats_bit_for_bit_wherever_the_pages_lie(e4m3):
    lens = [3000, 17, 0, 900, 128]
    a, b = (Cache(lens, 4, 128, 16, e4m3, seed=20) for _ in range(2))
    b.table.copy_(torch.where(b.table >= 0, b.num - 1 - b.table, b.table))
    b.k, b.v = a.k.flip(0), a.v.flip(0)
    if e4m3:
        b.ks, b.vs = a.ks.flip(0), a.vs.flip(0)
    q = make_q(5, 16, 128)
    o, L = run_decode(a, q)
    for c in (a, a, b):
        o2, L2 = decode(c, q)
        assert torch.equal(o, o2) and torch.equal(L, L2)
    ok()


def test_decode_shared_prefix():
    """Two sequences whose tables name the same pages."""
    c = Cache([256, 256], 2, 64, 64, False, seed=21)
    c.table[1] = c.table[0]
    q = make_q(1, 4, 64).expand(2, -1, -1).contiguous()
    o, L = run_decode(c, q)
    assert torch.equal(o[0], o[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_offsets_beyond_32_bits(e4m3):
    """Pages that start more than 2^32 elements into the cache."""
    dt = torch.uint8 if e4m3 else torch.bfloat16
    page, d = 128, 128
    P = (1 << 32) // (page * d) + 40
    big = torch.empty((P, 1, page, d), dtype=dt, device=DEV)
    c = Cache([200, 300], 1, d, page, e4m3, seed=22)
    at = P - c.num
    big[at:] = c.k
    c.k = big
    vbig = torch.empty((P, 1, page, d), dtype=dt, device=DEV)
    vbig[at:] = c.v
    c.v = vbig
    if e4m3:
        pad = torch.full((at, 1, page), float("nan"), device=DEV)
        c.ks, c.vs = torch.cat([pad, c.ks]), torch.cat([pad, c.vs])
    c.table.copy_(torch.where(c.table >= 0, c.table + at, c.table))
    run_decode(c, make_q(2, 4, d))
    new = torch.randn(2, 1, d, device=DEV).to(torch.bfloat16)
    fa.fa_cache_append(new, new, c.k, c.v, **c.args)
    out = torch.empty(2, 1, 300, d, dtype=torch.bfloat16, device=DEV)
    fa.fa_cache_gather(c.k, c.v, k_out=out, v_out=None, **c.args)
    ok()
    if not e4m3:
        assert torch.equal(out[0, 0, 199], new[0, 0]) and torch.equal(out[1, 0, 299], new[1, 0])
    ref = c.rows("k", 1, 300)[0]
    assert ((out[1, 0].double() - ref).abs() <= BF16_HALF * ref.abs()).all()


def test_decode_on_another_stream_and_two_at_once():
    c = Cache([5000, 300], 2, 128, 64, False, seed=23)
    c2 = Cache([4000, 900, 2], 2, 64, 64, True, seed=24)
    q, q2 = make_q(2, 8, 128), make_q(3, 8, 64)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((decode(c, q, stream=s1), decode(c2, q2, stream=s2)))
        torch.cuda.synchronize()
    ok()
    for a, b in got:
        check_decode(*a, decode_exact(c, q, 1 / math.sqrt(128)))
        check_decode(*b, decode_exact(c2, q2, 1 / math.sqrt(64)))


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_in_a_graph_follows_its_inputs(e4m3):
    """A captured step replayed with other lengths, tables, keys and queries."""
    c = Cache([700] * 4, 2, 128, 16, e4m3, seed=25)  # every row that a step may read is written
    q = make_q(4, 8, 128)
    new = torch.randn(2, 4, 2, 128, device=DEV).to(torch.bfloat16)
    ws = torch.empty(fa.fa_decode_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device=DEV)
    o, L = decode(c, q, ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs that share the workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_cache_append(new[0], new[1], c.k, c.v, **c.args)
            fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=0.1, workspace=ws, **c.args)
        graphs.append(g)
    for step, lens in enumerate(([700, 400, 128, 33], [1, 0, 300, 600], [0, 0, 0, 0], [650, 1, 17, 700])):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(make_q(4, 8, 128, seed=step))
        new.normal_()
        o.fill_(float("nan"))
        graphs[step % 2].replay()
        ok()
        check_decode(o, L, decode_exact(c, q, 0.1), f"step {step}")


def test_decode_nan_stays_in_its_sequence():
    """A NaN in a visible row reaches that sequence's heads and no other's."""
    c = Cache([300, 300, 40], 2, 64, 16, False, seed=26)
    page, off = c.where(1, torch.tensor([150], device=DEV))
    c.v[page[0], 0, off[0]] = float("nan")
    q = make_q(3, 4, 64)
    o, _ = decode(c, q)
    ok()
    assert torch.isnan(o[1, :2]).all() and torch.isfinite(o[1, 2:]).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length"])
def test_bad_tables_are_reported(what, e4m3):
    """A page id or length out of range is recorded, never followed, and leaves the others' rows right."""
    c = Cache([200, 200, 90], 2, 64, 16, e4m3, seed=27)
    q = make_q(3, 4, 64)
    ref = decode_exact(c, q, 1 / 8)
    if what.endswith("page"):
        c.table[1, 3] = c.num if what == "page" else -1
    else:
        c.lens[1] = 16 * c.per + 1 if what == "length" else -3
    if what == "length":
        c.table[1] = c.table[0, 0]  # every page the clamped length reaches is a valid one
    o, L = decode(c, q)
    st, info = fa.fa_device_status(info=True)
    assert st == 9 and info[:2] == [8, 1], (st, info)
    assert fa.fa_device_status() == 0
    keep = torch.tensor([0, 2], device=DEV)
    check_decode(o[keep], L[keep], tuple(x[keep] for x in ref))
    new = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    if what.endswith("length"):
        fa.fa_cache_append(new, new, c.k, c.v, **c.args)
        assert fa.fa_device_status(info=True)[1][:2] == [6, 1]
    out = torch.empty(3, 2, 200, 64, dtype=torch.bfloat16, device=DEV)
    fa.fa_cache_gather(c.k, c.v, k_out=out, v_out=None, **c.args)
    st, info = fa.fa_device_status(info=True)
    assert st == 9 and info[:2] == [7, 1]


# ------------------------------------------------------------------- append
def append_reference(c, k_new, v_new, counts):
    """The cache's tensors after the append, from the definition (a copy)."""
    want = [x if x is None else x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    at = 0
    for b, m in enumerate(counts):
        n = int(c.lens[b])
        pos = torch.arange(n - m, n, device=DEV)
        keep = pos >= 0
        for x, f, new in ((want[0], want[2], k_new), (want[1], want[3], v_new)):
            if keep.any():
                c.put(x, f, b, pos[keep], new[at:at + m][keep])
        at += m
    return want


def same(a, b):
    if a is None:
        return b is None
    if a.dtype == torch.uint8:  # codes stand for values: both NaN codes are one
        a, b = a.view(torch.float8_e4m3fn).float(), b.view(torch.float8_e4m3fn).float()
    return torch.equal(torch.nan_to_num(a.float(), nan=12345.0), torch.nan_to_num(b.float(), nan=12345.0))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "joint", "padded"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_one_token(d, layout, e4m3):
    c = Cache([1, 0, 16, 17, 128, 129, 40], 3, d, 16, e4m3, layout, seed=30)
    qkv = torch.randn(7, 5, 3, d, device=DEV).to(torch.bfloat16)  # K and V sliced out of wider rows
    k, v = qkv[:, 1], qkv[:, 3]
    want = append_reference(c, k, v, [1] * 7)
    fa.fa_cache_append(k, v, c.k, c.v, **c.args)
    ok()
    for got, w in zip((c.k, c.v, c.ks, c.vs), want):
        assert same(got, w)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 128])
def test_append_prompts(page, e4m3):
    """Whole prompts, parts, none, more tokens than the sequence holds, and padding behind the last."""
    lens, counts = [300, 5, 0, 128, 40, 1], [300, 2, 0, 128, 45, 0]
    c = Cache(lens, 2, 128, page, e4m3, "nhd", seed=31)
    T = sum(counts)
    new = torch.randn(2, T + 9, 2, 128, device=DEV).to(torch.bfloat16)
    want = append_reference(c, new[0], new[1], counts)
    cu = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    fa.fa_cache_append(new[0], new[1], c.k, c.v, cu_new=cu, **c.args)
    ok()
    for got, w in zip((c.k, c.v, c.ks, c.vs), want):
        assert same(got, w)


def test_append_many_sequences():
    counts = [(i * 7) % 5 for i in range(600)]
    c = Cache([n + 3 for n in counts], 1, 64, 16, True, seed=32)
    new = torch.randn(2, sum(counts), 1, 64, device=DEV).to(torch.bfloat16)
    want = append_reference(c, new[0], new[1], counts)
    cu = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    fa.fa_cache_append(new[0], new[1], c.k, c.v, cu_new=cu, **c.args)
    ok()
    for got, w in zip((c.k, c.v, c.ks, c.vs), want):
        assert same(got, w)


def test_append_of_hard_values():
    """Zeros, subnormals, the largest numbers, ties, infinities and NaN."""
    d = 64
    c = Cache([1] * 7, 1, d, 16, True, seed=33)
    x = torch.randn(7, 1, d, device=DEV).to(torch.bfloat16)
    x[0] = 0
    x[1] *= 1e-38
    x[2] *= 1e38
    x[3] = torch.arange(d, device=DEV).to(torch.bfloat16) * 7  # 441 = 448 - 7: codes between which ties fall
    x[3, 0, 0] = 448
    x[4, 0, 5] = float("inf")
    x[5, 0, 9] = float("nan")
    x[6] *= 1e-30
    want = append_reference(c, x, x, [1] * 7)
    fa.fa_cache_append(x, x, c.k, c.v, **c.args)
    ok()
    for got, w in zip((c.k, c.v, c.ks, c.vs), want):
        assert same(got, w)


def test_append_of_nothing():
    c = Cache([3, 4], 1, 64, 16, False)
    z = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    before = c.k.clone()
    fa.fa_cache_append(z, z, c.k, c.v, cu_new=cu, **c.args)
    ok()
    assert same(before, c.k)


# ------------------------------------------------------------------- gather
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "joint", "padded"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rep,N", [(1, 1), (3, 130), (4, 700)])
def test_gather(d, layout, e4m3, rep, N):
    lens = [1, 0, 64, 129, 513]
    c = Cache(lens, 2, d, 64 if d == 64 else 16, e4m3, layout, seed=40)
    out = [torch.full((5, 2 * rep, N, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    fa.fa_cache_gather(c.k, c.v, k_out=out[0], v_out=out[1], **c.args)
    ok()
    for nm, got in zip("kv", out):
        want = torch.zeros(5, 2, N, d, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            m = min(n, N)
            if m:
                want[b, :, :m] = c.rows(nm, b, m)
        want = want.repeat_interleave(rep, 1)
        if e4m3:  # code * factor in fp32, then bf16: two roundings
            assert ((got.double() - want).abs() <= (BF16_HALF + 2.0 ** -23) * want.abs()).all()
        else:
            assert torch.equal(got.double(), want)


def test_gather_one_of_two():
    c = Cache([70], 2, 64, 16, False, seed=41)
    a, b = (torch.full((1, 2, 70, 64), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fa.fa_cache_gather(c.k, c.v, k_out=a, v_out=None, **c.args)
    fa.fa_cache_gather(c.k, c.v, k_out=None, v_out=b, **c.args)
    ok()
    assert torch.equal(a.double()[0], c.rows("k", 0, 70)) and torch.equal(b.double()[0], c.rows("v", 0, 70))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_then_tokens(d, e4m3):
    """As a server runs them: fa_fwd over the prompts, one append of their keys and
    values, then tokens one at a time; and the cache read back into fa_fwd."""
    prompts, steps, H, G, page = [150, 31, 128], 20, 2, 4, 16
    ends = [n + steps for n in prompts]
    c = Cache(ends, H, d, page, e4m3, seed=50, fill=False)
    N = max(ends)
    g = torch.Generator(device="cpu").manual_seed(51)
    q, k, v = (torch.randn(3, h, N, d, generator=g).to(torch.bfloat16).to(DEV) for h in (H * G, H, H))
    c.lens.copy_(torch.tensor(prompts, dtype=torch.int32))
    pk = torch.cat([k[b, :, :n].transpose(0, 1) for b, n in enumerate(prompts)])
    pv = torch.cat([v[b, :, :n].transpose(0, 1) for b, n in enumerate(prompts)])
    cu = torch.tensor([0, 150, 181, 309], dtype=torch.int32, device=DEV)
    fa.fa_cache_append(pk, pv, c.k, c.v, cu_new=cu, **c.args)
    scale = 1 / math.sqrt(d)
    got = []
    for t in range(steps):
        c.lens += 1
        at = c.lens.long() - 1
        b = torch.arange(3, device=DEV)
        fa.fa_cache_append(k[b, :, at], v[b, :, at], c.k, c.v, **c.args)
        o, L = decode(c, q[b, :, at].contiguous(), scale)
        ref = decode_exact(c, q[b, :, at], scale)
        check_decode(o, L, ref, f"step {t}")
        got.append((at.tolist(), o, L))
    ok()
    # The whole sequences at once, from the cache: fa_fwd's causal rows are the steps' rows.
    K, V = (torch.empty(3, H * G, N, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fa.fa_cache_gather(c.k, c.v, k_out=K, v_out=V, **c.args)
    o, lse = torch.empty_like(q), torch.empty(3, H * G, N, device=DEV)
    fa.fa_fwd(q, K, V, o, lse, scale, True)
    ok()
    for at, od, Ld in got:
        for b, n in enumerate(at):
            # Both are within 1e-2 of exact attention (fa_fwd's gate; the read-back of e4m3
            # rows rounds them to bf16 once more, 2^-9 of values below 5).
            assert (o[b, :, n] - od[b]).abs().max() <= (4e-2 if e4m3 else 2e-2)
            assert (lse[b, :, n] - Ld[b]).abs().max() <= (2e-2 if e4m3 else 2e-3)


# ---------------------------------------------------------------- refusals
def test_binding_refusals():
    c = Cache([20, 30], 2, 64, 16, False)
    e = Cache([20, 30], 2, 64, 16, True)
    q = make_q(2, 4, 64)
    o, L = torch.empty_like(q), torch.empty(2, 4, device=DEV)
    ws = torch.empty(fa.fa_decode_workspace_bytes(2, 4, 2, 64), dtype=torch.uint8, device=DEV)

    def call(cc=c, **kw):
        a = dict(q=q, k_cache=cc.k, v_cache=cc.v, o=o, lse=L, scale=0.1, workspace=ws, **cc.args)
        a.update(kw)
        fa.fa_decode(**a)

    call()
    call(e)
    for bad in (dict(seq_lens=c.lens.long()), dict(q=q.float()), dict(v_cache=e.v), dict(lse=L.double()),
                dict(workspace=None), dict(workspace=ws.float())):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    for bad in (dict(seq_lens=c.lens[:1]), dict(q=q[:1]), dict(o=o[:, :2]), dict(q=q.transpose(0, 1)), dict(lse=L[:1]),
                dict(block_table=c.table[:1]), dict(block_table=c.table.t()), dict(v_cache=c.v[:1]),
                dict(k_cache=c.k.transpose(2, 3), v_cache=c.v.transpose(2, 3)), dict(k_scale=e.ks),
                dict(block_table=c.table.cpu()), dict(seq_lens=c.lens.cpu())):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    with pytest.raises((TypeError, ValueError)):
        call(e, k_scale=None)
    with pytest.raises((TypeError, ValueError)):
        call(e, v_scale=e.vs[:1])
    for bad, code in ((dict(workspace=ws[:16]), 4), (dict(scale=0.0), 1), (dict(window=-1), 1),
                      (dict(q=make_q(2, 3, 64), o=torch.empty(2, 3, 64, dtype=torch.bfloat16, device=DEV), lse=None), 1)):
        with pytest.raises(fa.FaError) as err:
            call(**bad)
        assert err.value.code == code
    odd = torch.empty(c.num, 2, 16, 65, dtype=torch.bfloat16, device=DEV)[..., :64]  # rows off the 16-byte grid
    with pytest.raises(fa.FaError) as err:
        call(k_cache=odd, v_cache=odd)
    assert err.value.code == 3
    new = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(k_new=new[:1], v_new=new[:1]), dict(k_new=new.float()), dict(v_new=new[:, :1]),
                dict(cu_new=torch.zeros(2, dtype=torch.int32, device=DEV)),
                dict(cu_new=torch.zeros(3, dtype=torch.int64, device=DEV))):
        a = dict(k_new=new, v_new=new, k_cache=c.k, v_cache=c.v, **c.args)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            fa.fa_cache_append(**a)
    out = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(k_out=None, v_out=None), dict(k_out=out[:, :3]), dict(k_out=out[:1]), dict(k_out=out.float()),
                dict(k_out=out, v_out=out[:, :2]), dict(k_out=out.transpose(0, 1).contiguous().transpose(0, 1))):
        a = dict(k_cache=c.k, v_cache=c.v, k_out=out, v_out=out, **c.args)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            fa.fa_cache_gather(**a)
    ok()


# ------------------------------------------------------- calls in other settings
CAPTURE_FIRST = """
import math, sys
sys.path[:0] = [{tests!r}, {root!r}]
import torch
from cache_helpers import Cache, check_decode, decode_exact, DEV
from io_aware_exact_23_b200 import binding as fa
fa.fa_device_status()  # the device's first call
for e4m3, Hq, d in ((False, 2, 64), (True, 40, 128)):
    c = Cache([300, 0, 129], 1, d, 16, e4m3, seed=60)
    q = torch.randn(3, Hq, d, device=DEV).to(torch.bfloat16)
    new = torch.randn(3, 1, d, device=DEV).to(torch.bfloat16)
    o, L = torch.empty_like(q), torch.empty(3, Hq, device=DEV)
    out = torch.empty(3, Hq, 300, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(fa.fa_decode_workspace_bytes(3, Hq, 1, d), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_cache_append(new, new, c.k, c.v, **c.args)
        fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=0.1, workspace=ws, **c.args)
        fa.fa_cache_gather(c.k, c.v, k_out=out, v_out=None, **c.args)
    for _ in range(3):
        o.fill_(float("nan"))
        g.replay()
    assert fa.fa_device_status() == 0
    check_decode(o, L, decode_exact(c, q, 0.1))
    ref = c.rows("k", 0, 300)
    assert ((out[0, 0].double() - ref[0]).abs() <= 2.0 ** -8 * ref[0].abs()).all()
print("captured")
"""


def test_captured_before_any_other_call_of_its_kind():
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = CAPTURE_FIRST.format(tests=tests, root=os.path.dirname(tests))
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "captured" in got.stdout, got.stderr[-2000:]


def test_two_graphs_at_once_with_a_workspace_each():
    q = [make_q(2, 8, 128, seed=s) for s in (1, 2)]
    c = [Cache([2500, 700], 2, 128, 16, e, seed=61 + e) for e in (False, True)]
    res, graphs = [], []
    for i in range(2):
        res.append(decode(c[i], q[i]))
        ws = torch.empty(fa.fa_decode_workspace_bytes(2, 8, 2, 128), dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(8):
                decode(c[i], q[i], ws=ws, out=res[i][0])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    ok()
    for i in range(2):
        check_decode(*res[i], decode_exact(c[i], q[i], 1 / math.sqrt(128)))


def test_decode_from_two_threads():
    import threading
    c = [Cache([900, 31, 400], 2, 64, 32, e, seed=63 + e) for e in (False, True)]
    q = [make_q(3, 4, 64, seed=s) for s in (3, 4)]
    res, errors = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    res[i] = decode(c[i], q[i])
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    ok()
    for i in range(2):
        check_decode(*res[i], decode_exact(c[i], q[i], 1 / 8))


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_thousands_of_idle_slots(e4m3):
    """A padded batch of which only a few slots are taken."""
    lens = [0] * 5000
    for b in (0, 31, 32, 383, 384, 385, 2999, 4999):
        lens[b] = 7 + b % 300
    c = Cache(lens, 1, 64, 16, e4m3, seed=65)
    run_decode(c, make_q(5000, 1, 64))


def test_decode_window_larger_than_any_length():
    c = Cache([300, 1, 0], 2, 64, 16, False, seed=66)
    q = make_q(3, 4, 64)
    a, b = run_decode(c, q, window=2 ** 31 - 1), run_decode(c, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_the_same_page_twice():
    """One sequence whose table names a page twice."""
    c = Cache([64, 64], 2, 64, 16, False, seed=67)
    c.table[0, 2] = c.table[0, 0]
    run_decode(c, make_q(2, 4, 64))


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_follows_an_append_without_a_wait(e4m3):
    """Each kernel may start while the one before it ends: many short steps in a row."""
    steps, B, H, d = 60, 5, 2, 128
    c = Cache([steps + 130] * B, H, d, 16, e4m3, seed=68)  # room for the longest one's steps
    c.lens.copy_(torch.tensor([70, 1, 0, 127, 128 - steps // 2], dtype=torch.int32))
    q = make_q(B, 8, d, seed=5)
    ws = torch.empty(fa.fa_decode_workspace_bytes(B, 8, H, d), dtype=torch.uint8, device=DEV)
    news = torch.randn(steps, 2, B, H, d, device=DEV).to(torch.bfloat16)
    outs, lens = [], []
    torch.cuda.synchronize()
    for t in range(steps):
        c.lens += 1
        lens.append(c.lens.clone())
        fa.fa_cache_append(news[t, 0], news[t, 1], c.k, c.v, **c.args)
        outs.append(decode(c, q, ws=ws))
    ok()
    # Appends only write behind what earlier steps saw: every step can be checked now.
    for t in range(0, steps, 7):
        check_decode(*outs[t], decode_exact(c, q, 1 / math.sqrt(d), lens=lens[t].tolist()), f"step {t}")


def test_decode_scores_of_no_finite_value():
    """A row whose every score is the lowest there is (-inf from infinite keys) next to others."""
    c = Cache([200, 200], 1, 64, 16, False, seed=69)
    page, off = c.where(0, torch.tensor([3], device=DEV))
    c.k[page[0], 0, off[0], :] = 0
    c.k[page[0], 0, off[0], 0] = -float("inf")
    q = make_q(2, 2, 64).abs()  # every product with that element is -inf
    run_decode(c, q)  # the key has weight 0, as in the definition


@pytest.mark.parametrize("d", [64, 128])
def test_decode_very_low_scores(d):
    """Scores around -1e30: the maximum is far below where it starts from."""
    c = Cache([300], 1, d, 16, False, seed=70)
    r = torch.zeros(300, 1, d, device=DEV, dtype=torch.bfloat16)
    r[:, 0, 0] = -1e31
    r[150:, 0, 0] = -1e30
    c.put(c.k, c.ks, 0, torch.arange(300, device=DEV), r)
    q = torch.zeros(1, 4, d, device=DEV, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    o, L = decode(c, q, scale=1.0)
    ok()
    ref = c.rows("v", 0, 300)[0, 150:].mean(0)
    assert ((o[0].double() - ref).abs() <= BF16_HALF * ref.abs() + 2.0 ** -12).all()
    score = float(r[150, 0, 0])  # -1e30 as bf16 holds it
    assert ((L.double() - score).abs() <= 2.0 ** -22 * abs(score)).all()


# ------------------------------------------------------------------- wrapper
@pytest.mark.parametrize("e4m3", [False, True])
def test_wrapper(e4m3):
    ref = Cache([90, 0, 33], 2, 64, 16, e4m3, seed=71, fill=False)
    c = fa.KVCache(ref.num, 2, 16, 64, e4m3)
    new = torch.randn(2, 123, 2, 64, device=DEV).to(torch.bfloat16)
    cu = torch.tensor([0, 90, 90, 123], dtype=torch.int32, device=DEV)
    c.append(new[0], new[1], ref.table, ref.lens, cu)
    ref.k, ref.v, ref.ks, ref.vs = c.k, c.v, c.k_scale, c.v_scale
    q = make_q(3, 4, 64)
    o, L = c.decode(q, ref.table, ref.lens, 0.2)
    k, v = c.gather(ref.table, ref.lens, 90, rep=2)
    ok()
    check_decode(o, L, decode_exact(ref, q, 0.2))
    if not e4m3:
        assert torch.equal(k[0, 2], new[0, :90, 1]) and torch.equal(v[2, 1, :33], new[1, 90:, 0])
    assert (k[1] == 0).all() and (v[2, :, 33:] == 0).all()


# --------------------------------------------------------------- guard bands
@pytest.mark.parametrize("e4m3", [False, True])
def test_nothing_around_the_outputs_is_touched(e4m3):
    """Outputs and workspace inside larger buffers; a cache with gaps between rows, heads and pages."""
    B, H, Hq, d, page = 5, 3, 9, 64, 16
    c = Cache([40, 0, 129, 16, 700], H, d, page, e4m3, "padded", seed=72)
    q = make_q(B, Hq, d)
    ob, lb = torch.full((B * Hq * d + 64,), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((B * Hq + 8,), 7.0, device=DEV)
    size = fa.fa_decode_workspace_bytes(B, Hq, H, d)
    wb = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    o, L = ob[32:-32].view(B, Hq, d), lb[4:-4].view(B, Hq)
    fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=0.125, workspace=wb[32:-32], **c.args)
    ok()
    check_decode(o, L, decode_exact(c, q, 0.125))
    for buf, n in ((ob, 32), (lb, 4), (wb, 32)):
        edge = buf[0]
        assert (buf[:n] == edge).all() and (buf[-n:] == edge).all()
    # append: every byte of the storage but the new rows (and their factors) stays.
    bases = [x._base if x._base is not None else x for x in (c.k, c.v)]
    before = [b.clone() for b in bases]
    new = torch.randn(B, H, d, device=DEV).to(torch.bfloat16)
    fa.fa_cache_append(new, new, c.k, c.v, **c.args)
    ok()
    for x, base, was in zip((c.k, c.v), bases, before):
        now = base.clone()
        page_ids, off = zip(*[c.where(b, torch.tensor([n - 1], device=DEV)) for b, n in enumerate(c.lens.tolist()) if n])
        for pg, of in zip(page_ids, off):
            now[pg[0], :H, of[0], :d] = was[pg[0], :H, of[0], :d]
        assert same(now, was)
    # gather
    gb = torch.full((B * H * 2 * 50 * d + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = gb[32:-32].view(B, H * 2, 50, d)
    fa.fa_cache_gather(c.k, c.v, k_out=out, v_out=None, **c.args)
    ok()
    assert (gb[:32] == 7).all() and (gb[-32:] == 7).all() and torch.isfinite(out.float()).all()


# ------------------------------------- kernels that begin while the last one ends
def test_decodes_of_every_kind_in_a_row():
    """Decode calls of all instances, with one workspace and no wait in between, on one
    stream and on two at once, return the bits that they return one at a time."""
    kinds = [(G, d, e) for G in (1, 3, 8, 16, 32) for d in (64, 128) for e in (False, True)]
    work = []
    for i, (G, d, e) in enumerate(kinds):
        c = Cache([1 + 37 * i, 0, 300 - 7 * i], 2, d, 16, e, seed=80 + i)
        q = make_q(3, 2 * G, d, seed=i)
        alone = decode(c, q)
        torch.cuda.synchronize()
        work.append((c, q, alone))
    size = max(fa.fa_decode_workspace_bytes(3, q.shape[1], 2, q.shape[2]) for _, q, _ in work)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for used in ((0,), (0, 1)):
        got = []
        for r in range(4):
            for i in range(len(work)):
                for j in used:
                    c, q, alone = work[i if j == 0 else len(work) - 1 - i]
                    with torch.cuda.stream(streams[j]):
                        got.append((decode(c, q, ws=spaces[j]), alone))
        torch.cuda.synchronize()
        ok()
        for (o, L), (o1, L1) in got:
            assert torch.equal(o, o1) and torch.equal(L, L1)


def test_graph_whose_branches_meet():
    """A graph where an append waits for two branches and two decodes for it."""
    H, d = 2, 128
    n = [129, 4, 700]
    c = Cache(n, H, d, 16, True, seed=91)
    for b in range(3):  # the last position is the graph's to write
        c.put(c.k, c.ks, b, torch.tensor([n[b] - 1], device=DEV), torch.zeros(1, H, d, device=DEV))
    x = torch.zeros(2, 3, H, d, dtype=torch.bfloat16, device=DEV)
    src = torch.randn(2, 3, H, d, device=DEV).to(torch.bfloat16)
    q = [make_q(3, 8, d, seed=s) for s in (5, 6)]
    ws = [torch.empty(fa.fa_decode_workspace_bytes(3, 8, H, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    res = [decode(c, q[i], ws=ws[i]) for i in range(2)]
    old = decode_exact(c, q[1], 1 / math.sqrt(d))
    check_decode(*res[1], old)
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x[1].copy_(src[1])
            decode(c, q[1], ws=ws[1], out=res[1][0])  # the old contents: to be over before the append
        x[0].copy_(src[0])
        main.wait_stream(side)
        fa.fa_cache_append(x[0], x[1], c.k, c.v, **c.args)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            second = decode(c, q[1], ws=ws[1])
        first = decode(c, q[0], ws=ws[0])
        main.wait_stream(side)
    g.replay()
    torch.cuda.synchronize()
    ok()
    check_decode(res[1][0], res[1][1], old)
    for b in range(3):
        for which, rows, f in (("k", c.k, c.ks), ("v", c.v, c.vs)):
            want = src[0 if which == "k" else 1][b].double()
            got = c.rows(which, b, n[b])[:, -1]
            top = want.abs().amax(-1, keepdim=True)
            # half a step of e4m3: 2^-4 of the value, or 2^-10 code units below its normal numbers
            assert ((got - want).abs() <= want.abs() * 2.0**-4 + top / 448 * 2.0**-10 * (1 + 2.0**-20)).all()
    for got, qq in ((first, q[0]), (second, q[1])):
        check_decode(*got, decode_exact(c, qq, 1 / math.sqrt(d)))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[5000], [0, 3, 129, 0, 64, 1000], [100] * 200])
def test_decode_in_place(lens, e4m3):
    """o = q: sequences held by one CTA, split ones and idle ones."""
    c = Cache(lens, 2, 64, 32, e4m3, seed=95)
    for G in (2, 40):
        q = make_q(len(lens), 2 * G, 64, seed=G)
        o, L = run_decode(c, q)
        same = q.clone()
        _, L2 = decode(c, same, out=same)
        ok()
        assert torch.equal(same, o) and torch.equal(L2, L)


def test_decode_window_beyond_31_bits():
    c = Cache([300, 17], 1, 64, 16, False, seed=96)
    q = make_q(2, 4, 64)
    o, L = run_decode(c, q)
    for window in (2**31 - 1, 2**31, 2**32 + 5):
        o2, L2 = decode(c, q, window=window)
        ok()
        assert torch.equal(o, o2) and torch.equal(L, L2)
    for window in (-1, -(2**31), 5 - 2**32):
        with pytest.raises(fa.FaError) as e:
            decode(c, q, window=window)
        assert e.value.code == 1
