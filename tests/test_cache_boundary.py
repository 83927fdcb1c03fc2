"""Host-side tests of the key/value cache's C ABI and binding (no GPU needed): the
library exports what include/fa_cache.h declares, and refuses bad arguments with
the documented status codes before touching any device."""
from __future__ import annotations

import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fa_cache.h")
P = 4096  # 16-byte aligned dummy address: never dereferenced on error paths


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_23_b200 import build
    build.build()
    from io_aware_exact_23_b200 import binding
    return binding


def cache(fa, **kw):
    """A valid description: 10 pages of 64 tokens, 4 heads, d = 128, [pages, H, page, d]."""
    c = dict(k=P, v=P, k_scale=P, v_scale=P, k_stride=(4 * 64 * 128, 64 * 128, 128),
             v_stride=(4 * 64 * 128, 64 * 128, 128), k_scale_stride=(256, 64, 1), v_scale_stride=(256, 64, 1),
             block_table=P, seq_lens=P, block_table_stride=7, type=1, num_pages=10, H=4, page_size=64, d=128, B=3,
             max_pages=7)
    c.update(kw)
    return Packed(fa, c)


class Packed(bytes):
    """fa_paged_cache as bytes, in the header's field order, with the fields at hand."""
    ORDER = ("k", "v", "k_scale", "v_scale", "k_stride", "v_stride", "k_scale_stride", "v_scale_stride", "block_table",
             "seq_lens", "block_table_stride", "type", "num_pages", "H", "page_size", "d", "B", "max_pages")

    def __new__(cls, fa, c):
        vals = []
        for nm in cls.ORDER:
            vals += c[nm] if isinstance(c[nm], tuple) else [c[nm] or 0]
        self = super().__new__(cls, fa._PAGED_CACHE.pack(*vals))
        self.B, self.H = c["B"], c["H"]
        return self


def append(fa, c, k=P, v=P, ks=(512, 128), vs=(512, 128), T=3, cu=None):
    return fa.lib().fa_cache_append(c, k, v, fa._STRIDES2.pack(*ks), fa._STRIDES2.pack(*vs), T, cu, None)


def gather(fa, c, k=P, v=P, rep=2, N=100):
    return fa.lib().fa_cache_gather(c, k, v, rep, N, None)


def decode(fa, c, q=P, o=P, lse=P, Hq=8, scale=0.1, window=0, ws=P, ws_bytes=1 << 30):
    return fa.lib().fa_decode(c, q, o, lse, Hq, scale, window, ws, ws_bytes, None)


def test_library_exports_every_declared_symbol(fa):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", src))
    assert {"fa_cache_append", "fa_cache_gather", "fa_decode", "fa_decode_workspace_bytes"} <= names
    for nm in names:
        assert hasattr(fa.lib(), nm)


def test_status_string(fa):
    src = open(HEADER).read()
    code = int(re.search(r"#define FA_ERR_DEVICE_CACHE (\d+)", src).group(1))
    assert code == 9 and fa.STATUS_NAMES[code] == "FA_ERR_DEVICE_CACHE"
    assert fa.lib().fa_status_string(code).decode().startswith("FA_ERR_DEVICE_CACHE")


BAD_CACHE = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(block_table=None), 1), (dict(seq_lens=None), 1),
    (dict(type=2), 1), (dict(type=-1), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(page_size=0), 1),
    (dict(block_table_stride=6), 1), (dict(d=96), 2), (dict(d=256), 2), (dict(d=0), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=96), 2), (dict(page_size=192), 2),
    (dict(max_pages=1 << 25, block_table_stride=1 << 25), 2),
    (dict(k=P + 8), 3), (dict(v=P + 4), 3), (dict(block_table=P + 2), 3), (dict(seq_lens=P + 1), 3),
    (dict(k_scale=P + 2), 3), (dict(v_stride=(4 * 64 * 128, 64 * 128, 136)), 3),
    (dict(k_stride=(4 * 64 * 128, 64, 128)), 2), (dict(k_stride=(0, 64 * 128, 128)), 2),
    (dict(v_stride=(1 << 40, 64 * 128, 128)), 2), (dict(k_scale_stride=(256, 64, 0)), 2),
    (dict(type=0, k_stride=(4 * 64 * 128, 64 * 128, 132)), 3),
]


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_every_call_refuses_a_bad_cache(fa, kw, code):
    c = cache(fa, **kw)
    T = c.B
    assert append(fa, c, T=T) == code
    assert gather(fa, c) == code
    assert decode(fa, c, Hq=8 * max(c.H, 1)) == code


def test_packed_description_is_the_header_s_struct(fa, tmp_path):
    """Size and field offsets of fa_paged_cache, from a C compiler."""
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "fa_cache.h"\nint main(void) { fa_paged_cache c; (void)c; printf("%zu", sizeof(c));'
                   + "".join(f' printf(" %zu", offsetof(fa_paged_cache, {nm}));' for nm in Packed.ORDER) + " return 0; }\n")
    exe = tmp_path / "t"
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    want, at = [], 0
    for nm in Packed.ORDER:
        want.append(at)
        at += 24 if nm.endswith("_stride") and nm != "block_table_stride" else 4 if nm in Packed.ORDER[11:] else 8
    assert got[1:] == want
    assert got[0] == fa._PAGED_CACHE.size


def test_null_cache(fa):
    assert append(fa, None) == 1 and gather(fa, None) == 1 and decode(fa, None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(T=-1), 1), (dict(T=2), 1), (dict(T=4), 1),
    (dict(k=P + 8), 3), (dict(cu=P + 2), 3), (dict(ks=(516, 128)), 3), (dict(vs=(512, 4)), 3), (dict(vs=(-512, 128)), 2),
])
def test_append_argument_errors(fa, kw, code):
    assert append(fa, cache(fa), **kw) == code


def test_append_of_no_tokens_is_a_no_op(fa):
    assert append(fa, cache(fa), k=None, v=None, T=0, cu=P) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(k=None, v=None), 1), (dict(rep=0), 1), (dict(N=0), 1), (dict(k=P + 8), 3), (dict(v=P + 2), 3),
    (dict(N=1 << 20, rep=2), 2),
])
def test_gather_argument_errors(fa, kw, code):
    assert gather(fa, cache(fa), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(Hq=0), 1), (dict(Hq=6), 1), (dict(Hq=-4), 1), (dict(window=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1),
    (dict(ws=None), 4), (dict(ws_bytes=8), 4), (dict(q=P + 8), 3), (dict(o=P + 2), 3), (dict(lse=P + 2), 3),
    (dict(ws=P + 8), 3), (dict(Hq=1 << 23), 2),
])
def test_decode_argument_errors(fa, kw, code):
    assert decode(fa, cache(fa), **kw) == code


def test_decode_workspace_of_invalid_shapes(fa):
    f = fa.fa_decode_workspace_bytes
    assert f(1, 8, 2, 64) > 0 and f(300, 32, 1, 128) > 0
    for bad in ((0, 8, 2, 64), (1, 8, 0, 64), (1, 7, 2, 64), (1, 0, 2, 64), (1, 8, 2, 96), (1, -8, 2, 64)):
        assert f(*bad) == 0


def test_valid_arguments_without_a_device(fa):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    c = cache(fa)
    assert append(fa, c) == 5 and gather(fa, c) == 5 and decode(fa, c) == 5
    # A stride along an axis of one element is never used.
    one = cache(fa, num_pages=1, H=1, k_stride=(0, -5, 128), v_stride=(3, 0, 128), k_scale_stride=(0, 0, 1))
    assert decode(fa, one, lse=None) == 5 and gather(fa, one, k=None) == 5


def test_binding_refuses_wrong_tensors(fa):
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(4, 2, 16, 64, dtype=bf)
    table, lens = torch.zeros(1, 2, dtype=i32), torch.ones(1, dtype=i32)
    q = torch.zeros(1, 4, 64, dtype=bf)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):  # there is no CPU path
        fa.fa_decode(q, k, k, table, lens, q, None, 0.1, ws)
    with pytest.raises(TypeError):
        fa.fa_decode(q, k.float(), k.float(), table, lens, q, None, 0.1, ws)
    with pytest.raises(TypeError):
        fa.fa_cache_append(q, q, None, k, table, lens)
    m = torch.device("meta")  # tensors that pass for another device's
    with pytest.raises(ValueError):
        fa.fa_cache_gather(k.to(m), k.to(m), table.to(m), lens.to(m), k.to(m), k.to(m))
