"""fa_decode over e4m3 caches whose weights, values and queries span a wide range."""
from __future__ import annotations

import pytest
import torch

from cache_bounds import aimed, check_tight, copies, decode_tight, run
from cache_helpers import DEV, Cache
from io_aware_exact_23_b200 import binding as fa

pytestmark = pytest.mark.gpu


def rows(n, H, d, seed, mean=0.0, mult=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (mean + mult * torch.randn(n, H, d, generator=g)).to(DEV)


# --------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("nats", [9, 12, 15, 18])
@pytest.mark.parametrize("B", [1, 400])
def test_many_keys_below_one(B, nats, e4m3):
    """One key far above 100000 others whose weights count together: values with a common mean, the
    first one's own value zero.  In one CTA each (B = 400) and split over many."""
    n, d = 100000, 64
    c = Cache([n], 1, d, 64, e4m3, seed=1, fill=False)
    s = rows(n, 1, 1, 2, mult=0.2).flatten()
    s[0] = nats
    q = aimed(c, s, 8)
    v = rows(n, 1, d, 3, mean=1.0, mult=0.25)
    v[0] = 0
    c.put(c.v, c.vs, 0, torch.arange(n, device=DEV), v.to(torch.bfloat16))
    ref = decode_tight(c, q, 1.0)
    copies(c, B)
    o, L = run(fa, c, q[None].repeat(B, 1, 1))
    for b in {0, B // 2, B - 1}:
        check_tight(o[b], L[b], ref, f"{nats} nats, row {b}")


@pytest.mark.parametrize("G", [1, 2, 3, 4, 8, 16, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("times", [2.0**8, 1e4, 1e6, 1e20])
def test_one_large_value_row(times, d, G):
    """A value row `times` the others whose own weight is next to nothing."""
    n = 4096
    c = Cache([n], 2, d, 16, True, seed=4, fill=False)
    s = rows(n, 1, 1, 5).flatten()
    s[777] = -60.0
    q = aimed(c, s, G)
    v = rows(n, 2, d, 6, mean=0.5)
    v[777] *= times
    c.put(c.v, c.vs, 0, torch.arange(n, device=DEV), v.to(torch.bfloat16))
    ref = decode_tight(c, q, 1.0)
    o, L = run(fa, c, q[None])
    check_tight(o[0], L[0], ref, f"times {times}")


@pytest.mark.parametrize("G", [1, 4, 5, 12, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_factors_of_every_size(d, G):
    """Value rows between 2^-20 and 2^20 of each other, some of them zero, some factors negative,
    weights between 1 and e^-30."""
    for lens in ([1500], [100], [1]):
        n = lens[0]
        c = Cache(lens, 2, d, 32, True, seed=7, fill=False)
        g = torch.Generator(device="cpu").manual_seed(8)
        s = torch.randint(-30, 1, (n,), generator=g).float().to(DEV)
        q = aimed(c, s, G)
        v = rows(n, 2, d, 9) * torch.exp2(torch.randint(-20, 21, (n, 2, 1), generator=g).float()).to(DEV)
        v[5::9] = 0
        c.put(c.v, c.vs, 0, torch.arange(n, device=DEV), v.to(torch.bfloat16))
        c.vs[::2] = -c.vs[::2]
        ref = decode_tight(c, q, 1.0)
        o, L = run(fa, c, q[None])
        check_tight(o[0], L[0], ref, f"{n} keys")


@pytest.mark.parametrize("mult", [1e-33, 1e-20, 1e20, 1e33])
def test_values_near_the_ends_of_the_type(mult):
    n, d = 600, 64
    for e4m3 in (False, True):
        c = Cache([n], 1, d, 16, e4m3, seed=10, fill=False)
        q = aimed(c, rows(n, 1, 1, 11).flatten(), 4)
        v = (rows(n, 1, d, 12) * mult).to(torch.bfloat16)
        c.put(c.v, c.vs, 0, torch.arange(n, device=DEV), v)
        ref = decode_tight(c, q, 1.0)
        o, L = run(fa, c, q[None])
        check_tight(o[0], L[0], ref, f"{mult}")


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_climb_while_values_shrink(d, sign):
    """The largest weight and the largest product of weight and factor are different keys, and both keep moving."""
    n = 1300
    c = Cache([n], 1, d, 16, True, seed=13, fill=False)
    at = torch.arange(n, device=DEV)
    q = aimed(c, torch.floor(sign * at.float() / 8), 8)
    v = rows(n, 1, d, 14, mean=1.0) * torch.exp2(-sign * (at // 11).float())[:, None, None] * 2.0**(60 * sign)
    c.put(c.v, c.vs, 0, at, v.to(torch.bfloat16))
    ref = decode_tight(c, q, 1.0)
    o, L = run(fa, c, q[None])
    check_tight(o[0], L[0], ref)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 12, 16, 31])
@pytest.mark.parametrize("score", [-80.0, -200.0])
@pytest.mark.parametrize("value", [1e30, 3e38])
def test_a_value_row_at_the_end_of_the_type(value, score, G):
    """Hardly seen, or not at all: it leaves every head's other values alone.  First in its segment, last and between."""
    n, d = 700, 64
    for at in (0, 300, 699):
        c = Cache([n], 1, d, 16, True, seed=30, fill=False)
        s = rows(n, 1, 1, 31).flatten()
        s[at] = score
        q = aimed(c, s, G)
        v = rows(n, 1, d, 32, mean=0.5)
        v[at] = value
        c.put(c.v, c.vs, 0, torch.arange(n, device=DEV), v.to(torch.bfloat16))
        o, L = run(fa, c, q[None])
        check_tight(o[0], L[0], decode_tight(c, q, 1.0), f"at {at}")


@pytest.mark.parametrize("G", [2, 3, 8, 16])
@pytest.mark.parametrize("apart", [2.0**30, 2.0**50, 2.0**70])
@pytest.mark.parametrize("n", [200, 5000])
def test_heads_that_see_values_of_different_size(n, apart, G):
    """Even heads attend to keys with small values, odd ones to keys with values `apart` times
    those; each is as exact as if the other was not there."""
    d = 64
    c = Cache([n], 1, d, 16, True, seed=33, fill=False)
    at = torch.arange(n, device=DEV)
    odd = at % 2 == 1
    r = 0.5 * rows(n, 1, d, 34)
    r[:, 0, 0], r[:, 0, 1] = torch.where(odd, -60.0, 0.0), torch.where(odd, 0.0, -60.0)
    c.put(c.k, c.ks, 0, at, r.to(torch.bfloat16))
    v = rows(n, 1, d, 35, mean=1.0) * torch.where(odd, apart**0.5, apart**-0.5)[:, None, None]
    c.put(c.v, c.vs, 0, at, v.to(torch.bfloat16))
    g = torch.Generator(device="cpu").manual_seed(36)
    q = (0.1 * torch.randn(G, d, generator=g)).to(torch.bfloat16).to(DEV)
    q[:, 0], q[:, 1] = 0, 0
    q[0::2, 0], q[1::2, 1] = 2, 2
    o, L = run(fa, c, q[None])
    check_tight(o[0], L[0], decode_tight(c, q, 1.0))


def test_parts_whose_values_differ():
    """A split sequence whose first half has scores 34 nats below the second's and values 2^70 times
    as large, next to a head that sees both alike: the parts are joined on their own maxima."""
    n, d = 40000, 64
    c = Cache([n], 1, d, 64, True, seed=37, fill=False)
    at = torch.arange(n, device=DEV)
    first = at < n // 2
    r = torch.zeros(n, 1, d, device=DEV)
    r[:, 0, 0] = torch.where(first, -34.0, 0.0)
    r[::2, 0, 1] = -80.0  # seen by the second head alone
    c.put(c.k, c.ks, 0, at, r.to(torch.bfloat16))
    v = rows(n, 1, d, 38, mean=1.0) * torch.where(first, 2.0**35, 2.0**-35)[:, None, None]
    v[::2] *= 2.0**40
    c.put(c.v, c.vs, 0, at, v.to(torch.bfloat16))
    q = torch.zeros(4, d, dtype=torch.bfloat16, device=DEV)
    q[:, 0] = 1
    q[:3, 1] = 1
    q[3, 1] = -1
    o, L = run(fa, c, q[None])
    check_tight(o[0], L[0], decode_tight(c, q, 1.0))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_ordinary_rows(d, G, e4m3):
    """Every instance on random rows, to the bound that bf16 outputs allow."""
    lens = [1, 130, 2000, 0, 515]
    c = Cache(lens, 2, d, 64, e4m3, seed=15 + G)
    g = torch.Generator(device="cpu").manual_seed(G)
    q = torch.randn(5, 2 * G, d, generator=g).to(torch.bfloat16).to(DEV)
    o, L = run(fa, c, q, scale=0.3)
    for b, n in enumerate(lens):
        if n:
            check_tight(o[b], L[b], decode_tight(c, q[b], 0.3, b=b), f"sequence {b}")


@pytest.mark.parametrize("G", [1, 3, 8, 32])
@pytest.mark.parametrize("alike", [True, False])
@pytest.mark.parametrize("score", [1e5, 3e8, 1e30, -1e5, -3e8, -1e30])
def test_scores_far_from_zero(score, alike, G):
    """Equal scores so large that a reference a few powers of two below them is lost in their rounding,
    and ones ten times lower before and after them."""
    n, d = 500, 64
    c = Cache([n], 1, d, 16, True, seed=40, fill=False)
    at = torch.arange(n, device=DEV)
    high = (at >= 150) & (at < 400)
    lower = score / 10 if score > 0 else score * 10
    q = aimed(c, torch.where(high, score, lower), G)
    v = rows(n, 1, d, 41, mean=1.0)
    if not alike:
        v = v * torch.exp2((at % 23 - 11).float())[:, None, None]
    c.put(c.v, c.vs, 0, at, v.to(torch.bfloat16))
    o, L = run(fa, c, q[None])
    K, V = c.rows("k", 0, n)[0, :, 0], c.rows("v", 0, n)[0]
    page, off = c.where(0, at)
    ref, mag = V[high].mean(0), V[high].abs().mean(0)
    # Equal weights: their rounding (2^-15, or 2^-27 of the largest product's 448), sums and o's own.
    err = (2.0**-15 + (n / 16 + 8) * 2.0**-22) * mag + 2.0**-27 * 448 * c.vs[page, :, off].max().double()
    assert ((o[0].double() - ref).abs() <= 2.0**-8 * (ref.abs() + err) + err).all()
    want = float(K[high][0]) + float(torch.log(high.sum().double()))
    assert ((L[0].double() - want).abs() <= 2.0**-22 * abs(want)).all()


@pytest.mark.parametrize("G", [1, 4, 8, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_are_not_seen_leave_every_bit_alone(d, G):
    """Behind a sequence's end, and before its window, the pages' rows may hold anything: factors at the
    end of the type must not move a reference."""
    lens = [200, 129, 300, 17] * 100  # enough for segments of several tiles
    B = len(lens)
    for window in (0, 150):
        c = Cache(lens, 1, d, 64, True, seed=50)
        g = torch.Generator(device="cpu").manual_seed(51)
        q = (1.5 * torch.randn(B, G, d, generator=g)).to(torch.bfloat16).to(DEV)
        seen = torch.zeros_like(c.ks, dtype=torch.bool)
        for b, n in enumerate(lens):
            page, off = c.where(b, torch.arange(max(0, n - window) if window else 0, n, device=DEV))
            seen[page, :, off] = True
        want = None
        for other in (1e-3, 3.4e38, float("inf"), float("nan"), 0.0):
            for f, codes in ((c.ks, c.k), (c.vs, c.v)):
                f[~seen] = other
                codes[~seen] = 0x7E  # 448
            o, L = run(fa, c, q, scale=0.3, window=window)
            if want is None:
                want = o, L
                for b in range(8):
                    check_tight(o[b], L[b], decode_tight(c, q[b], 0.3, window, b=b), f"sequence {b}")
            assert torch.equal(o, want[0]) and torch.equal(L, want[1]), f"factors of {other}"


# ----------------------------------------------------------------- queries
@pytest.mark.parametrize("G", [2, 4, 8, 24])
@pytest.mark.parametrize("d", [64, 128])
def test_heads_of_every_size(d, G):
    """Query heads between 2^-14 and 2^6 of each other: each is as exact as if it were alone."""
    n = 700
    c = Cache([n], 2, d, 16, True, seed=20)
    g = torch.Generator(device="cpu").manual_seed(21)
    size = torch.exp2(torch.randint(-14, 7, (2 * G, 1), generator=g).float())
    q = (torch.randn(2 * G, d, generator=g) * size).to(torch.bfloat16).to(DEV)
    ref = decode_tight(c, q, 1.0)
    o, L = run(fa, c, q[None])
    check_tight(o[0], L[0], ref)
    for h in (0, G):  # the first head of either cache head, next to ones 2^20 times it
        q2 = q.clone()
        q2[h + 1] = (torch.randn(d, generator=g) * 2.0**20 * float(size[h])).to(torch.bfloat16)
        o2, L2 = run(fa, c, q2[None])
        check_tight(o2[0, h:h + 1], L2[0, h:h + 1], tuple(x[h:h + 1] for x in ref), f"head {h}")
