"""Infinities and NaN in visible rows of the cache and in queries: they reach the results
that the definition sends them to, and no others."""
from __future__ import annotations

import math

import pytest
import torch

from cache_bounds import run
from cache_helpers import DEV, Cache
from io_aware_exact_23_b200 import binding as fa

pytestmark = pytest.mark.gpu


def queries(B, Hq, d, seed=0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(B, Hq, d, generator=g).to(torch.bfloat16).to(DEV)


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
