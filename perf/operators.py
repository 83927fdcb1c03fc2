"""What is measured of the paged key/value cache and the attention that reads it.

Three operators, each with a plain form in elementary torch operations (``own``
false) and the call that a user makes of the framework (``own`` true):

* ``append``: new keys and values [T, H, d] written to their sequences' places in a
  paged cache, as bf16 or as e4m3 codes with one fp32 factor per token and head;
* ``decode``: attention of one new token per sequence over its pages, with query
  heads sharing key/value heads, an optional window, and the log-sum-exp;
* ``gather``: a cache read back as [B, H * rep, N, d] bf16, each head repeated
  ``rep`` times, zeros behind a sequence's end.

The cache is [pages, H, page, d] (or the same memory as [pages, page, H, d], layout
"nhd"); ``block_table`` [B, pages a sequence] int32 names each sequence's pages.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
LARGEST = 131072 * 16 * 128  # elements of K in the largest listed decode


def listed():
    return [
        # One user's conversation on a small server: one token, a short odd length; latency counts.
        dict(name="decode_one_short", op="decode", B=1, Hq=32, H=8, d=128, kind="bf16", page=16, n=777, spread="equal",
             window=0, layout="hnd"),
        # An ordinary serving batch with ragged lengths and one idle slot, tokens outermost in a page.
        dict(name="decode_batch_ragged", op="decode", B=16, Hq=32, H=8, d=128, kind="bf16", page=64, n=4096,
             spread="ragged", window=0, layout="nhd"),
        # A loaded server that holds its cache in 8 bits.
        dict(name="decode_batch_e4m3", op="decode", B=64, Hq=32, H=8, d=128, kind="e4m3", page=64, n=8192,
             spread="ragged", window=0, layout="hnd"),
        # One very long document, a key/value head for each query head.
        dict(name="decode_long_heads", op="decode", B=1, Hq=16, H=16, d=128, kind="bf16", page=128, n=131072,
             spread="equal", window=0, layout="hnd"),
        # Many short chats of a small model, 8 bits.
        dict(name="decode_many_short", op="decode", B=256, Hq=16, H=16, d=64, kind="e4m3", page=16, n=512,
             spread="ragged", window=0, layout="nhd"),
        # One key/value head for all query heads, and a window over a long cache.
        dict(name="decode_shared_window", op="decode", B=8, Hq=32, H=1, d=64, kind="bf16", page=256, n=32768,
             spread="ragged", window=8191, layout="hnd"),
        # The write that goes before each serving step: one token a sequence.
        dict(name="append_tokens", op="append", B=64, H=8, d=128, kind="bf16", page=16, n=4096, spread="ragged", new=1,
             layout="nhd"),
        # The same into 8 bits, a large batch of a small model.
        dict(name="append_tokens_e4m3", op="append", B=256, H=16, d=64, kind="e4m3", page=16, n=512, spread="ragged",
             new=1, layout="hnd"),
        # Whole prompts of odd lengths written at once into 8 bits.
        dict(name="append_prompts_e4m3", op="append", B=5, H=8, d=128, kind="e4m3", page=64, n=4096, spread="ragged",
             new=0, layout="hnd"),
        # A stored prefix read back for a few hundred tokens.
        dict(name="gather_short_e4m3", op="gather", B=1, H=8, d=128, kind="e4m3", page=64, n=300, spread="equal", rep=4,
             layout="hnd"),
        # Stored prompts read back for the fused forward, heads repeated for their query heads.
        dict(name="gather_repeat", op="gather", B=4, H=8, d=128, kind="bf16", page=64, n=4096, spread="equal", rep=4,
             layout="nhd"),
        # A ragged batch read back from 8 bits.
        dict(name="gather_ragged_e4m3", op="gather", B=32, H=16, d=64, kind="e4m3", page=16, n=2048, spread="ragged",
             rep=1, layout="nhd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "gather"])
    c = dict(op=op, d=rng.choice([64, 128]), kind=rng.choice(["bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128, 256]),
             spread=rng.choice(["equal", "ragged"]), layout=rng.choice(["hnd", "nhd"]))
    if op == "decode":
        c["H"] = rng.choice([1, 2, 3, 4, 8, 16])
        c["Hq"] = c["H"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 24, 32])
        c["B"] = _log(rng, 1, 256)
        # Scores of all query heads are held in the plain form, so they bound a case too.
        most = min(LARGEST // (c["B"] * c["H"] * c["d"]), LARGEST // (c["B"] * c["Hq"]), 131072)
        c["n"] = _log(rng, 1, most)
        c["window"] = _log(rng, 1, c["n"]) if rng.random() < 0.25 else 0
    elif op == "append":
        c["H"] = rng.choice([1, 2, 3, 4, 8, 16])
        c["B"] = _log(rng, 1, 256)
        c["new"] = rng.choice([0, 1])
        c["n"] = _log(rng, 1, max(1, min(8192, (1 << 25) // (c["B"] * c["H"] * c["d"]))))
    else:
        c["H"] = rng.choice([1, 2, 3, 4, 8, 16])
        c["rep"] = rng.choice([1, 1, 2, 3, 4, 8])
        c["B"] = _log(rng, 1, 64)
        c["n"] = _log(rng, 1, max(1, min(16384, (1 << 26) // (c["B"] * c["H"] * c["rep"] * c["d"]))))
    return c


def _lengths(case):
    """The batch's lengths: all n, or spread over 0 .. n with an idle slot, a single token and a full one among them."""
    B, n = case["B"], case["n"]
    if case["spread"] == "equal":
        return [n] * B
    r = random.Random(B * 1000003 + n)
    got = [r.randint(0, n) for _ in range(B)]
    for at, v in ((B - 1, n), (B // 2, 0), (B // 3, 1)):
        got[at] = v if B > 2 else n
    return got


def _new_counts(case):
    """How many of each sequence's tokens an append brings: the last one (none for an idle slot), or all."""
    return _lengths(case) if case["new"] == 0 else [1] * case["B"]


def _e4m3(x):
    """e4m3 codes of x with one factor per last-dimension vector."""
    # The factor is divided out in 64 bits (the rounded quotient is fp32's): a CUDA tensor over a
    # constant is a product with the constant's rounded reciprocal, which moves codes next to a border.
    f = (x.abs().amax(-1).clamp_min(1e-30).double() / E4M3_MAX).float()
    return (x / f[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), f


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 17)
    B, H, d, page, lens = case["B"], case["H"], case["d"], case["page"], _lengths(case)
    per = max(1, -(-max(lens) // page))
    used = [-(-v // page) for v in lens]
    pages = max(1, sum(used)) + 3
    # Pages in no order, as a server that took and gave back pages has them; -1 behind a sequence's last.
    ids = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
    first = torch.tensor([sum(used[:b]) for b in range(B)], device=dev)
    col = torch.arange(per, device=dev)
    table = ids[(first[:, None] + col).clamp_max(pages - 1)]
    table = torch.where(col < torch.tensor(used, device=dev)[:, None], table, -1).contiguous()

    def cache(mult):
        shape = (pages, H, page, d) if case["layout"] == "hnd" else (pages, page, H, d)
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g) * mult
        f = None
        if case["kind"] == "e4m3":
            parts = [_e4m3(p.float()) for p in x.split(max(1, (1 << 26) // (H * page * d)))]
            x = torch.cat([p[0] for p in parts])
            f = torch.cat([p[1] for p in parts])
            f = f if case["layout"] == "hnd" else f.permute(0, 2, 1)
        return (x if case["layout"] == "hnd" else x.permute(0, 2, 1, 3)), f

    s = dict(case, scale=1.0 / math.sqrt(d), table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             ks=None, vs=None)
    s["k"], s["ks"] = cache(1.5)
    s["v"], s["vs"] = cache(1.0)
    if case["op"] == "decode":
        s["q"] = torch.empty((B, case["Hq"], d), dtype=torch.bfloat16, device=dev).normal_(generator=g) * 1.5
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, case["Hq"]), dtype=torch.float32, device=dev)
        if own:
            from io_aware_exact_23_b200 import binding as fa
            size = fa.fa_decode_workspace_bytes(B, case["Hq"], H, d)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=dev)
    elif case["op"] == "append":
        counts = _new_counts(case)
        T = sum(counts)
        s["cu"] = None
        if case["new"] == 0:
            s["cu"] = torch.tensor([sum(counts[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
        # The keys and values of a fused projection: slices of one wider row.
        qkv = torch.empty((max(1, T), 3, H, d), dtype=torch.bfloat16, device=dev).normal_(generator=g)
        s["k_new"], s["v_new"] = qkv[:T, 1], qkv[:T, 2]
    else:
        shape = (B, H * case["rep"], case["n"], d)
        s["k_out"] = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    return s


def _values(s, name):
    """Every sequence's cache rows in fp32, [B, H, pages a sequence * page, d]."""
    x, f = s[name], s[name + "s"]
    at = s["table"].clamp_min(0).long()
    got = x[at]
    got = got.float() if f is None else got.view(torch.float8_e4m3fn).float() * f[at][..., None]
    return got.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_decode(s):
    B, Hq, H, d = s["B"], s["Hq"], s["H"], s["d"]
    K, V = _values(s, "k"), _values(s, "v")
    at, lens = torch.arange(K.shape[2], device=K.device), s["lens"][:, None]
    seen = at < lens
    if s["window"]:
        seen &= at >= lens - s["window"]
    q = s["q"].float().view(B, H, Hq // H, d) * s["scale"]
    S = torch.matmul(q, K.transpose(2, 3))
    S = torch.where(seen[:, None, None], S, -math.inf)
    top = S.amax(-1, keepdim=True)
    P = torch.exp(S - torch.where(top == -math.inf, 0.0, top))
    total = P.sum(-1, keepdim=True)
    V = torch.where(seen[:, None, :, None], V, 0.0)
    O = torch.matmul(P, V) / torch.where(total == 0, 1.0, total)
    lse = top + torch.log(total)
    s["o"].copy_(O.reshape(B, Hq, d))
    s["lse"].copy_(lse.reshape(B, Hq))


def _plain_append(s):
    T, dev = s["k_new"].shape[0], s["k_new"].device
    t = torch.arange(T, device=dev)
    lens = s["lens"].long()
    if s["cu"] is None:
        b, pos = t, lens - 1
    else:
        cu = s["cu"].long()
        b = torch.searchsorted(cu, t, right=True) - 1
        pos = lens[b] - (cu[b + 1] - t)
    keep = pos >= 0
    b, pos = b[keep], pos[keep]
    page, off = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    for name in ("k", "v"):
        x = s[name + "_new"][keep]
        if s["kind"] == "e4m3":
            x, f = _e4m3(x.float())
            s[name + "s"][page, :, off] = f
        s[name][page, :, off] = x


def _plain_gather(s):
    n = s["n"]
    seen = (torch.arange(n, device=s["lens"].device) < s["lens"][:, None])[:, None, :, None]
    for name in ("k", "v"):
        x = torch.where(seen, _values(s, name)[:, :, :n], 0.0)
        s[name + "_out"].copy_(x.repeat_interleave(s["rep"], dim=1))


def run(s):
    if own:
        from io_aware_exact_23_b200 import binding as fa
        if s["op"] == "decode":
            fa.fa_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], s["o"], s["lse"], s["scale"], s["workspace"],
                         k_scale=s["ks"], v_scale=s["vs"], window=s["window"])
        elif s["op"] == "append":
            fa.fa_cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], cu_new=s["cu"],
                               k_scale=s["ks"], v_scale=s["vs"])
        else:
            fa.fa_cache_gather(s["k"], s["v"], s["table"], s["lens"], s["k_out"], s["v_out"], k_scale=s["ks"],
                               v_scale=s["vs"])
    else:
        {"decode": _plain_decode, "append": _plain_append, "gather": _plain_gather}[s["op"]](s)
    if s["op"] == "decode":
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "append":
        if s["kind"] == "bf16":
            return {"k": s["k"], "v": s["v"]}
        return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "ks": s["ks"], "vs": s["vs"]}
    return {"k": s["k_out"], "v": s["v_out"]}


def work(case):
    B, H, d, page, lens = case["B"], case["H"], case["d"], case["page"], _lengths(case)
    row = 2 * d * 2 if case["kind"] == "bf16" else 2 * d + 8  # K and V of one token and head in the cache
    if case["op"] == "decode":
        seen = sum(min(v, case["window"]) if case["window"] else v for v in lens)
        # K and V once, q and o, the log-sum-exp, the page ids and the lengths.
        io = B * case["Hq"] * (4 * d + 4) + 4 * B + 4 * sum(-(-v // page) for v in lens)
        return {"bytes": seen * H * row + io, "flops": 4 * d * (case["Hq"] // H) * H * seen}
    if case["op"] == "append":
        T = sum(min(a, b) for a, b in zip(_new_counts(case), lens))
        return {"bytes": T * H * (2 * d * 2 + row) + 8 * B, "flops": 4 * T * H * d}
    out = B * H * case["rep"] * case["n"] * d * 2 * 2
    return {"bytes": sum(lens) * H * row + out + 4 * B, "flops": 2 * sum(lens) * H * d}


def _exact_rows(s, name, b, n):
    """The first n rows of sequence b in 64 bits, [H, n, d]."""
    at = torch.div(torch.arange(n, device=s["table"].device), s["page"], rounding_mode="floor")
    off = torch.arange(n, device=s["table"].device) % s["page"]
    ids = s["table"][b].long()[at]
    x = s[name][ids, :, off]
    if s["kind"] == "e4m3":
        x = x.view(torch.float8_e4m3fn).double() * s[name + "s"][ids, :, off].double().unsqueeze(-1)
    return x.double().transpose(0, 1)


def _exact_decode(s, lens):
    G = s["Hq"] // s["H"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device=o.device)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        lo = max(0, n - s["window"]) if s["window"] else 0
        K, V = _exact_rows(s, "k", b, n)[:, lo:], _exact_rows(s, "v", b, n)[:, lo:]
        logits = torch.einsum("hgd,hnd->hgn", s["q"][b].double().unflatten(0, (s["H"], G)), K) / math.sqrt(s["d"])
        z = torch.logsumexp(logits, -1)
        o[b] = torch.einsum("hgn,hnd->hgd", (logits - z[..., None]).exp(), V).flatten(0, 1)
        lse[b] = z.flatten()
    return {"o": o, "lse": lse}


def _exact_append(s, lens, counts):
    e4m3 = s["kind"] == "e4m3"
    out = {}
    for name in ("k", "v"):
        x = s[name].view(torch.float8_e4m3fn).double() if e4m3 else s[name].double()
        f = s[name + "s"].double() if e4m3 else None
        at = 0
        for b, (n, m) in enumerate(zip(lens, counts)):
            new = s[name + "_new"][at:at + m].double()
            at += m
            m = min(m, n)
            if m == 0:
                continue
            pos = torch.arange(n - m, n, device=x.device)
            ids, off = s["table"][b].long()[torch.div(pos, s["page"], rounding_mode="floor")], pos % s["page"]
            if e4m3:
                big = new.abs().amax(-1).clamp_min(1e-30) / E4M3_MAX
                f[ids, :, off] = big
                new = new / big[..., None]
            x[ids, :, off] = new
        out[name] = x
        if e4m3:
            out[name + "s"] = f
    return out


def _exact_gather(s, lens):
    out = {}
    for name in ("k", "v"):
        x = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device=s["lens"].device)
        for b, n in enumerate(lens):
            if n:
                x[b, :, :n] = _exact_rows(s, name, b, n).unsqueeze(1).expand(-1, s["rep"], -1, -1).flatten(0, 1)
        out[name] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    lens = _lengths(case)
    if case["op"] == "decode":
        return _exact_decode(s, lens)
    if case["op"] == "append":
        return _exact_append(s, lens, _new_counts(case))
    return _exact_gather(s, lens)
