"""Host-side tests of the sizes that include/fa_cache.h says a call takes (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

from test_cache_boundary import append, cache, decode, fa, gather  # noqa: F401  (fa: the fixture)

OK = 5  # FA_ERR_NO_DEVICE: all checks passed

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a device is present")


def work(B, H, Hq, max_pages, page):
    G = Hq // H
    return 6 * B * H * -(-G // 32) * -(-max_pages * page // 128)


CASES = [  # B, H, Hq, max_pages, page size
    (2048, 32, 32, 1 << 13, 128), (2048, 32, 32, 5461, 128), (2048, 32, 32, 5462, 128), (1, 1, 1, 1 << 20, 1024),
    (4096, 8, 256, 10922, 128), (4096, 8, 256, 10923, 128), (4096, 8, 264, 5461, 128), (4096, 8, 264, 5462, 128),
    (4096, 8, 264, 10922, 64), (4096, 8, 264, 10923, 64),
]


@no_gpu
@pytest.mark.parametrize("B,H,Hq,max_pages,page", CASES)
def test_decode_counts_the_table_s_capacity(fa, B, H, Hq, max_pages, page):  # noqa: F811
    strides = dict(k_stride=(H * page * 128, page * 128, 128), v_stride=(H * page * 128, page * 128, 128),
                   k_scale_stride=(H * page, page, 1), v_scale_stride=(H * page, page, 1))
    c = cache(fa, B=B, H=H, max_pages=max_pages, block_table_stride=max_pages, page_size=page, **strides)
    assert decode(fa, c, Hq=Hq) == (OK if work(B, H, Hq, max_pages, page) < 2**31 else 2)


@no_gpu
@pytest.mark.parametrize("T,want", [(2**28 - 1, OK), (2**28, 2)])
def test_append_counts_its_rows(fa, T, want):  # noqa: F811
    assert append(fa, cache(fa), T=T, cu=4096) == want  # 4 heads


@no_gpu
@pytest.mark.parametrize("N,want", [(2**31 // (3 * 4 * 2 * 128), OK), (2**31 // (3 * 4 * 2 * 128) + 1, 2)])
def test_gather_counts_its_elements(fa, N, want):  # noqa: F811
    assert gather(fa, cache(fa), rep=2, N=N) == want
