"""Infinities and NaN in visible rows of the cache and in queries: they reach the results
that the definition sends them to, and no others."""
from __future__ import annotations

import math

import pytest
import torch

from cache_bounds import check_tight, decode_tight, run
from cache_helpers import DEV, Cache
from io_aware_exact_23_b200 import binding as fa

pytestmark = pytest.mark.gpu


def queries(B, Hq, d, seed=0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(B, Hq, d, generator=g).to(torch.bfloat16).to(DEV)


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_gather_of_a_quantised_row_that_was_not_finite(value, d):
    """Such a row is NaN throughout, and the rows around it are what they were."""
    n = 40
    c = Cache([n], 2, d, 16, True, seed=1)
    x = torch.randn(1, 2, d, device=DEV).abs().to(torch.bfloat16)  # codes of +0 under an infinite factor
    x[0, 1, 17] = value
    fa.fa_cache_append(x, x, c.k, c.v, **c.args)  # position n - 1
    k, v = (torch.zeros(1, 4, n + 3, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fa.fa_cache_gather(c.k, c.v, k_out=k, v_out=v, **c.args)
    assert fa.fa_device_status() == 0
    for t in (k, v):
        assert torch.isnan(t[0, 2:, n - 1]).all()
        assert torch.isfinite(t[0, :2]).all() and torch.isfinite(t[0, 2:, :n - 1]).all() and (t[0, :, n:] == 0).all()


def test_gather_multiplies_every_code():
    """Zero codes under factors that are not finite; zero codes with a sign."""
    c = Cache([4], 1, 64, 16, True, seed=2)
    page, off = c.where(0, torch.arange(4, device=DEV))
    c.k[page, :, off] = 0
    c.k[page[3], 0, off[3]] = 0x80
    c.ks[page[0], 0, off[0]], c.ks[page[1], 0, off[1]] = math.inf, math.nan
    out = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    fa.fa_cache_gather(c.k, c.v, k_out=out, v_out=None, **c.args)
    assert fa.fa_device_status() == 0
    assert torch.isnan(out[0, 0, :2]).all() and (out[0, 0, 2:] == 0).all()
    assert torch.signbit(out[0, 0, 3]).all() and not torch.signbit(out[0, 0, 2]).any()


# ---------------------------------------------------- rows of the cache, in decode
@pytest.mark.parametrize("G", [1, 4, 8, 20])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_decode_of_a_quantised_row_that_was_not_finite(value, which, d, G):
    """Appended to cache head 1 of sequence 1: its query heads are NaN, all others hold."""
    lens = [300, 300, 77]
    c = Cache(lens, 2, d, 16, True, seed=3)
    q = queries(3, 2 * G, d)
    new = [torch.randn(3, 2, d, device=DEV).to(torch.bfloat16) for _ in range(2)]
    new["kv".index(which)][1, 1, 17] = value
    for n in (150, 300):  # the row in the middle of its sequence, and one at its end
        c.lens[1] = n
        fa.fa_cache_append(new[0], new[1], c.k, c.v, **c.args)
        c.lens[1] = 300
        o, L = run(fa, c, q, scale=0.2)
        assert torch.isnan(o[1, G:]).all()
        assert torch.isnan(L[1, G:]).all() if which == "k" else torch.isfinite(L[1, G:]).all()
        for b in range(3):
            ref = decode_tight(c, q[b], 0.2, b=b)
            keep = slice(0, G) if b == 1 else slice(None)
            check_tight(o[b, keep], L[b, keep], tuple(x[keep] for x in ref), f"sequence {b}")


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 100, 700, 1499])
def test_decode_of_a_factor_that_is_not_finite(at, value):
    """A visible row under such a factor, whatever its codes: NaN in every feature of its heads."""
    for where in ("ks", "vs"):
        c = Cache([1500, 300], 2, 64, 64, True, seed=4)
        page, off = c.where(0, torch.tensor([at], device=DEV))
        getattr(c, where)[page[0], 1, off[0]] = value
        c.v[page[0], 1, off[0], ::2] = 0
        q = queries(2, 8, 64)
        o, _ = run(fa, c, q, scale=0.2)
        assert torch.isnan(o[0, 4:]).all()
        assert torch.isfinite(o[0, :4]).all() and torch.isfinite(o[1]).all()
        c.lens[0] = at  # the row is no longer visible
        o, _ = run(fa, c, q, scale=0.2)
        assert torch.isfinite(o).all()


# ----------------------------------------------------------------- queries
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [2, 4, 8, 24])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_a_query_head_that_is_not_finite_is_alone(value, G, e4m3):
    for d in (64, 128):
        c = Cache([300, 40], 2, d, 16, e4m3, seed=5)
        q = queries(2, 2 * G, d)
        refs = [decode_tight(c, q[b], 0.2, b=b) for b in range(2)]
        bad = (0, G - 1), (1, G)
        for b, h in bad:
            q[b, h, 3] = value
        o, L = run(fa, c, q, scale=0.2)
        for b, h in bad:
            assert torch.isnan(o[b, h]).all() and torch.isnan(L[b, h])
            keep = [i for i in range(2 * G) if i != h]
            check_tight(o[b, keep], L[b, keep], tuple(x[keep] for x in refs[b]), f"sequence {b}")


# ------------------------------------------------------------ parts of a sequence
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B", [1, 400])
def test_a_nan_value_of_next_to_no_weight(B, e4m3):
    """0 times NaN is NaN, whether the sequence is split over CTAs or not."""
    n, d = 6000, 64
    c = Cache([n], 1, d, 64, e4m3, seed=6)
    page, off = c.where(0, torch.tensor([20, n - 30], device=DEV))
    k = torch.zeros(2, 1, d, device=DEV, dtype=torch.bfloat16)
    k[:, 0, 0] = torch.tensor([-400.0, 400.0])  # the weight of position 20 is 0 in fp32
    c.put(c.k, c.ks, 0, torch.tensor([20, n - 30], device=DEV), k)
    c.v[page[0], 0, off[0], 5] = 0x7F if e4m3 else math.nan
    q = torch.zeros(1, 4, d, dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1
    c.table, c.lens, c.B = c.table[:1].repeat(B, 1), c.lens[:1].repeat(B), B
    o, _ = run(fa, c, q.repeat(B, 1, 1))
    assert torch.isnan(o[:, :, 5]).all()
    o[:, :, 5] = 0
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("G", [1, 4, 8, 32])
@pytest.mark.parametrize("n", [50, 9000])
def test_an_infinite_value_in_bf16(n, G):
    """One infinity is an infinity of its sign in that feature, two of different signs are NaN."""
    for d in (64, 128):
        c = Cache([n, n], 1, d, 16, False, seed=7)
        for b, p, f, x in ((0, 7, 2, math.inf), (0, 30, 3, -math.inf), (0, 8, 4, math.inf), (0, 41, 4, -math.inf)):
            page, off = c.where(b, torch.tensor([p], device=DEV))
            c.v[page[0], 0, off[0], f] = x
        q = queries(2, G, d)
        o, L = run(fa, c, q, scale=0.1)
        assert (o[0, :, 2] == math.inf).all() and (o[0, :, 3] == -math.inf).all() and torch.isnan(o[0, :, 4]).all()
        assert torch.isfinite(o[0, :, 5:]).all() and torch.isfinite(o[1]).all() and torch.isfinite(L).all()
