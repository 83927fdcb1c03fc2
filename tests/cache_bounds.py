"""Bounds on fa_decode's results that follow the weights that are there: each key's
error counts in proportion to its own weight, so a kernel that loses the small weights,
or lets one key or head set the precision of another's, is over them."""
from __future__ import annotations

import math

import torch

from cache_helpers import DEV, Cache


def decode_tight(c: Cache, q, scale, window=0, b=0, n=None):
    """(o, lse, do, dl) of sequence b's rows q [Hq, d], in 64 bits.  From the kernel's arithmetic:

    * a score is a sum of d products in fp32, 2 (d + 2) 2^-24 scale sum|q k| with room for an
      accumulator that truncates; it is rounded by two factors and by the maximum that
      is taken off, 2^-22 |s| + 2^-24 |max s|; for e4m3 keys an element of q is off by at most
      2^-22 of the largest of its own head;
    * in e4m3 a score is taken relative to a reference that may lie below the head's largest one, by as
      many powers of two as V's visible factors differ (80 at most): 2^-24 of those;
    * the exponential adds 2^-21.  A key's weight is then off by its own score's error e_j
      and by the normaliser's, E = log sum_j p_j exp(e_j);
    * a weight (e4m3: times V's factor) goes into the product with an error of at most 2^-15
      of itself (bf16 hi + lo: 2^-16; e4m3: fp16 and an e5m2 remainder), or 2^-29 units where the largest
      product of weight and factor has a code of at least 2^-2, times V's 448;
    * the product adds 16 or 32 keys at a time to an fp32 accumulator that may truncate, and
      within those aligns them to the largest: 2^-22 of sum p|v| for each time.
    """
    Hq, d = q.shape
    G = Hq // c.H
    n = int(c.lens[b]) if n is None else n
    lo = max(0, n - window) if window else 0
    K, V = c.rows("k", b, n)[:, lo:], c.rows("v", b, n)[:, lo:]
    m = n - lo
    qb = q.double().view(c.H, G, d)
    s = torch.matmul(qb, K.transpose(1, 2)) * scale
    z = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - z)
    e = 2 * (d + 2) * 2.0**-24 * scale * torch.matmul(qb.abs(), K.abs().transpose(1, 2))
    if c.e4m3:
        e += 2.0**-22 * scale * qb.abs().amax(-1, keepdim=True) * K.abs().sum(-1)[:, None]
        page, off = c.where(b, torch.arange(lo, n, device=DEV))
        f = c.vs[page, :, off].double().abs().t()  # [H, m]
        apart = (torch.log2(f.amax(1) / f.amin(1)) + 2).clamp_max(80)
        e += 2.0**-24 * apart[:, None, None]
    e += 2.0**-22 * s.abs() + 2.0**-24 * s.abs().amax(-1, keepdim=True) + 2.0**-21
    E = torch.log((p * torch.exp(e)).sum(-1, keepdim=True))
    sums = (m / 16 + 8) * 2.0**-22
    o = torch.matmul(p, V)
    do = torch.matmul(p * (torch.expm1(e + E) + (2.0**-15 if c.e4m3 else 2.0**-16) + sums), V.abs())
    if c.e4m3:
        do += m * 2.0**-27 * 448 * (p * f[:, None]).amax(-1, keepdim=True)
    dl = E + sums + 2.0**-22 * z.abs()
    return o.reshape(Hq, d), z.reshape(Hq), do.reshape(Hq, d), dl.reshape(Hq)


def check_tight(o, lse, ref, label=""):
    ro, rl, do, dl = ref
    half = torch.finfo(torch.bfloat16).eps / 2
    assert torch.isfinite(o.double()).all(), f"{label}: non-finite output"
    over = (o.double() - ro).abs() - (half * (ro.abs() + do) + do + 1e-38)
    assert over.max() <= 0, f"{label}: o over its bound by {over.max():.3e} ({ro.flatten()[over.argmax()]:.3e})"
    over = ((lse.double() - rl).abs() - dl).max()
    assert over <= 0, f"{label}: lse over its bound by {over:.3e}"


def copies(c: Cache, B: int) -> None:
    """The cache's first sequence B times over (they share its pages)."""
    c.table = c.table[:1].repeat(B, 1)
    c.lens = c.lens[:1].repeat(B)
    c.B = B


def aimed(c: Cache, scores, G, scale=1.0):
    """Keys whose scores are `scores` [n] for every head (to K's rounding), and the queries."""
    n, d = len(scores), c.d
    r = torch.zeros(n, c.H, d, device=DEV)
    r[:, :, 0] = scores[:, None] / scale
    c.put(c.k, c.ks, 0, torch.arange(n, device=DEV), r.to(torch.bfloat16))
    q = torch.zeros(c.H * G, d, dtype=torch.bfloat16, device=DEV)
    q[:, 0] = 1
    return q


def run(fa, c: Cache, q, scale=1.0, window=0):
    """fa_decode with queries q [B, Hq, d]."""
    B, Hq, d = q.shape
    o, L = torch.full_like(q, math.nan), torch.full((B, Hq), math.nan, device=DEV)
    ws = torch.full((fa.fa_decode_workspace_bytes(B, Hq, c.H, d),), 0xFF, dtype=torch.uint8, device=DEV)
    fa.fa_decode(q, c.k, c.v, o=o, lse=L, scale=scale, workspace=ws, window=window, **c.args)
    st, info = fa.fa_device_status(info=True)
    assert st == 0, f"device status {st} {info}"
    return o, L
