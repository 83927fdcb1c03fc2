"""Shared by the key/value cache's GPU tests: random paged caches, the operators'
definitions in 64 bits, and the error bounds the results are held to."""
from __future__ import annotations

import math

import torch

DEV = "cuda"
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2  # rounding to bf16, relative


class Cache:
    """A paged cache of random rows whose unused rows hold NaN.

    ``layout``: "hnd" ([pages, H, page, d]), "nhd" ([pages, page, H, d]), "joint" (K and V
    as slices of one [pages, 2, H, page, d] tensor) or "padded" (rows and pages further
    apart than they need to be).
    """

    def __init__(self, lens, H, d, page, e4m3, layout="hnd", seed=0, mult=1.0, fill=True, spare=2, vmult=1.0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.H, self.d, self.page, self.e4m3, self.B = H, d, page, e4m3, len(lens)
        self.per = max(1, max(-(-n // page) for n in lens)) + 1
        used = [-(-n // page) for n in lens]
        self.num = P = max(1, sum(used)) + spare
        ids = torch.randperm(P, generator=g)
        table = torch.full((self.B, self.per + 3), -7, dtype=torch.int32)  # rows further apart than max_pages
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = ids[at:at + u].int()
            at += u
        self.table = table.to(DEV)[:, :self.per]
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        dt = torch.uint8 if e4m3 else torch.bfloat16
        bad = 0x7F if e4m3 else float("nan")

        def empty():
            if layout == "nhd":
                return torch.full((P, page, H, d), bad, dtype=dt, device=DEV).permute(0, 2, 1, 3)
            if layout == "padded":
                return torch.full((P, H + 1, page + 3, d + 16), bad, dtype=dt, device=DEV)[:, :H, :page, :d]
            return torch.full((P, H, page, d), bad, dtype=dt, device=DEV)

        if layout == "joint":
            kv = torch.full((P, 2, H, page, d), bad, dtype=dt, device=DEV)
            self.k, self.v = kv[:, 0], kv[:, 1]
        else:
            self.k, self.v = empty(), empty()
        self.ks = self.vs = None
        if e4m3:
            shape = (P, page, H) if layout == "nhd" else (P, H, page)
            self.ks, self.vs = (torch.full(shape, float("nan"), device=DEV) for _ in range(2))
            if layout == "nhd":
                self.ks, self.vs = self.ks.permute(0, 2, 1), self.vs.permute(0, 2, 1)
        if fill:
            gg = torch.Generator(device=DEV).manual_seed(seed + 1)
            for b, n in enumerate(lens):
                if n:
                    for x, f, m in ((self.k, self.ks, mult), (self.v, self.vs, vmult)):
                        r = torch.randn(n, H, d, generator=gg, device=DEV).to(torch.bfloat16) * m
                        self.put(x, f, b, torch.arange(n, device=DEV), r)

    def where(self, b, pos):
        return self.table[b].long()[pos // self.page], pos % self.page

    def put(self, x, f, b, pos, rows):
        """Rows [n, H, d] (bf16) into sequence b's positions, quantised where the cache is."""
        page, off = self.where(b, pos)
        if self.e4m3:
            # In 64 bits, then fp32: the correctly rounded fp32 quotients (torch divides a CUDA
            # tensor by a constant through the constant's rounded reciprocal).
            rows = rows.double()
            s = (rows.abs().amax(-1).float().clamp_min(1e-30).double() / 448).float()
            f[page, :, off] = s
            rows = (rows / s[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
        x[page, :, off] = rows

    def rows(self, which, b, n):
        """The values of sequence b's first n rows in 64 bits, [H, n, d]."""
        x, f = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        page, off = self.where(b, torch.arange(n, device=DEV))
        r = x[page, :, off]
        r = r.view(torch.float8_e4m3fn).double() * f[page, :, off].double()[..., None] if self.e4m3 else r.double()
        return r.transpose(0, 1)

    @property
    def args(self):
        return dict(block_table=self.table, seq_lens=self.lens, k_scale=self.ks, v_scale=self.vs)


def decode_exact(c: Cache, q, scale, window=0, lens=None):
    """(o, lse, and bounds on their errors before o's last rounding), in 64 bits.

    The bounds, from the kernel's arithmetic:
    * s sums d products in fp32: |ds| <= g * scale * sum|q k|, g = 2 (d + 2) 2^-24 with
      room for an accumulator that truncates; e4m3 keys take q in two parts whose
      remainder is at most 2^-20 max|q| per element, the maximum over the heads that
      share a cache head (they may share a scale);
    * a weight exp(s - lse) then moves by a factor within exp(+-2 max|ds|); the hardware
      exponential adds 2^-21, q's scale in the log2 domain 2^-22 |s|;
    * weights go into the product with 16 significant bits (2^-16); for e4m3 values with
      fp16's 11 (2^-11, and 2^-12 for the remainder of three e4m3 parts: 2^-10 holds both)
      and not below 2^-20 of the largest value; the sums over n keys are in fp32.
    """
    B, Hq, d = q.shape
    G = Hq // c.H
    lens = c.lens.tolist() if lens is None else lens
    o = torch.zeros(B, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    do, dl = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        lo = max(0, n - window) if window else 0
        K, V = c.rows("k", b, n)[:, lo:], c.rows("v", b, n)[:, lo:]
        m = n - lo
        qb = q[b].double().view(c.H, G, d)
        s = torch.matmul(qb, K.transpose(1, 2)) * scale
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[..., None])
        o[b] = torch.matmul(p, V).reshape(Hq, d)
        lse[b] = z.reshape(Hq)
        ds = 2 * (d + 2) * 2.0 ** -24 * scale * torch.matmul(qb.abs(), K.abs().transpose(1, 2))
        if c.e4m3:
            ds = ds + 2.0 ** -20 * scale * qb.abs().amax((1, 2), keepdim=True) * K.abs().sum(-1)[:, None]
        e = ds.amax(-1) + 2.0 ** -22 * s.abs().amax(-1) + 2.0 ** -21
        sums = m * 2.0 ** -23
        do[b] = ((torch.expm1(2 * e) + 2.0 ** (-10 if c.e4m3 else -16) + sums)[..., None] * torch.matmul(p, V.abs())).reshape(Hq, d)
        if c.e4m3:
            do[b] += (m * 2.0 ** -20 * V.abs().amax((1, 2))[:, None]).expand(c.H, G).reshape(Hq, 1)
        dl[b] = (e + sums + 2.0 ** -22 * z.abs()).reshape(Hq)
    return o, lse, do, dl


def check_decode(o, lse, ref, label=""):
    ro, rl, do, dl = ref
    assert torch.isfinite(o.double()).all(), f"{label}: non-finite output"
    bad = (o.double() - ro).abs() - (BF16_HALF * (ro.abs() + do) + do + 1e-38)
    assert bad.max() <= 0, f"{label}: o over its bound by {bad.max():.3e} at {bad.argmax()} (of {o.shape})"
    if lse is not None:
        f = torch.isfinite(rl)
        assert torch.equal(f, torch.isfinite(lse)) and (lse[~f] == -math.inf).all(), f"{label}: empty rows"
        if f.any():
            over = ((lse.double() - rl).abs() - dl)[f].max()
            assert over <= 0, f"{label}: lse over its bound by {over:.3e}"
