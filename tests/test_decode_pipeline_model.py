"""Host-side model of fa_decode_kernel's pipeline (csrc/fa_decode.cuh) under random
interleavings (engine: tests/pipeline_model.py).

A CTA's share is a list of segments (runs of tiles with one Q).  Roles, as in the kernel:
  * producer: K_0 V_0 K_1 V_1 ... through a ring of single-tile slots;
  * issuer: S(n+1) ahead of O += V_n P_n, across segments; slots, Q, P and O are handed
    back by commits;
  * Q warp: the rows of segment i into buffer i % 2;
  * scales warp (e4m3): the keys' factors of tile n into a 4-slot ring;
  * softmax, groups of four warps with a vote per tile and group: read S(n), rewrite the masked rows of V(n)
    in a segment's last tile, rescale O when the reference moves (any tile but a
    segment's first), write P(n); the segment's statistics;
  * epilogue, four warps: O and the statistics of a segment.
Tensor memory lanes: softmax warp w of a group works on the lanes that epilogue warp w reads.
Checked: no deadlock or phase aliasing; every MMA reads the tiles, the Q, the masked V
and the P it should; O holds the segment's tiles in order when it is rescaled and when the
epilogue reads it; no load or write lands in a buffer that is still in use.
"""
from __future__ import annotations

import os
import random
import re

import pytest

from pipeline_model import Bar, Machine

GROUP, SCALES = 4, 4


def decode_model(runs, slots: int, seed: int, e4m3: bool, groups: int = 1, skip: str = "") -> None:
    M = Machine(seed)
    WARPS = GROUP * groups
    rnd = random.Random(seed * 7 + 1)
    total = sum(runs)
    segs, n = [], 0  # (segment, first tile, run)
    for i, r in enumerate(runs):
        segs.append((i, n, r))
        n += r
    seg_of = [i for i, _, r in segs for _ in range(r)]
    first = {n0 for _, n0, _ in segs}
    last = {n0 + r - 1 for _, n0, r in segs}
    partial = {t for t in last if rnd.random() < 0.7} | {t for t in first if rnd.random() < 0.2}
    moves = [{t for t in range(total) if t not in first and rnd.random() < 0.3} for _ in range(groups)]

    full = [Bar(f"full{s}", 1) for s in range(slots)]
    empty = [Bar(f"empty{s}", 1) for s in range(slots)]
    pair = lambda nm, c: [Bar(f"{nm}{b}", c) for b in range(2)]  # noqa: E731
    q, q_empty = pair("q", 1), pair("q_empty", 1 + (WARPS if e4m3 else 0))
    s_full = pair("s", 1)
    p_full, pv_done = pair("p", WARPS), pair("pv", 1)
    pv_bar = slots < 5
    o_full, o_empty, stat = pair("o", 1), pair("o_empty", 4), pair("stat", WARPS)
    sc = [Bar(f"sc{s}", 1) for s in range(SCALES)]
    sc_empty = [Bar(f"sc_empty{s}", WARPS) for s in range(SCALES)]
    vote = [Bar(f"vote{g}", GROUP) for g in range(groups)]  # bar.red among a group's warps, one phase per use

    def slot(kv, t):
        g = 2 * t + kv
        return g % slots, g // slots

    def v_tag(t):
        return ("Vz" if t in partial else "V", t)

    def producer():
        for t in range(total):
            for kv in (0, 1):
                s, r = slot(kv, t)
                if r > 0:
                    yield lambda s=s, r=r: empty[s].ready(r - 1)
                M.load(("slot", s), ("KV"[kv], t), full[s])
                yield lambda: True

    def issuer():
        def pv(t):
            i, ob, b = seg_of[t], seg_of[t] & 1, t & 1
            s, r = slot(1, t)
            if t in first and i >= 2 and skip != "o_empty":
                yield lambda: o_empty[ob].ready((i >> 1) - 1)
            yield lambda: full[s].ready(r)
            if skip != "p":
                yield lambda: p_full[b].ready(t >> 1)
            reads = {("slot", s): v_tag(t), **{("P", b, w): ("P", t) for w in range(WARPS)}}
            if t not in first:
                reads.update({("O", ob, w): ("O", i, t) for w in range(WARPS)})
            M.mma("mma", reads, {("O", ob, w): ("O", i, t + 1) for w in range(WARPS)})
            M.commit("mma", empty[s])
            if pv_bar:
                M.commit("mma", pv_done[b])
            if t in last:
                M.commit("mma", o_full[ob])

        prev = None
        for i, n0, r in segs:
            yield lambda: q[i & 1].ready(i >> 1)
            for t in range(n0, n0 + r):
                s, ph = slot(0, t)
                yield lambda s=s, ph=ph: full[s].ready(ph)
                M.mma("mma", {("slot", s): ("K", t), ("Q", i & 1): ("Q", i)},
                      {("S", t & 1, w): ("S", t) for w in range(WARPS)})
                M.commit("mma", empty[s])
                M.commit("mma", s_full[t & 1])
                if t == n0 + r - 1:
                    M.commit("mma", q_empty[i & 1])
                if prev is not None:
                    yield from pv(prev)
                prev = t
        yield from pv(prev)

    def q_warp():
        for i, _, _ in segs:
            if i >= 2:
                yield lambda i=i: q_empty[i & 1].ready((i >> 1) - 1)
            M.write(("Q", i & 1), ("Q", i))
            yield lambda: True
            q[i & 1].arrive()

    def scales():
        for t in range(total if e4m3 else 0):
            s = t % SCALES
            if t >= SCALES:
                yield lambda t=t, s=s: sc_empty[s].ready(t // SCALES - 1)
            M.load(("sc", s), ("sc", t), sc[s])
        yield lambda: True

    def softmax(w):
        votes, grp = 0, w // GROUP

        def agree():
            nonlocal votes
            vote[grp].arrive()
            k = votes
            votes += 1
            yield lambda: vote[grp].done >= k + 1

        for i, n0, r in segs:
            ob = i & 1
            if e4m3:
                yield lambda: q[i & 1].ready(i >> 1)
            for t in range(n0, n0 + r):
                b = t & 1
                yield lambda t=t, b=b: s_full[b].ready(t >> 1)
                if e4m3:
                    yield lambda t=t: sc[t % SCALES].ready(t // SCALES)
                    M.read(("sc", t % SCALES), ("sc", t))
                    sc_empty[t % SCALES].arrive()
                if t in partial and grp == 0:
                    s, ph = slot(1, t)
                    yield lambda s=s, ph=ph: full[s].ready(ph)
                    M.write(("slot", s), v_tag(t))  # each warp its own rows
                M.read(("S", b, w), ("S", t))
                yield lambda: True
                if t not in first:
                    yield from agree()
                if t in first or t in moves[grp]:
                    M.write(("x", (votes >> 1) & 3, w), t)
                    yield from agree()
                if t in moves[grp]:
                    if skip != "rescale" and (pv_bar):
                        yield lambda t=t: pv_done[(t - 1) & 1].ready((t - 1) >> 1)
                    elif skip != "rescale":
                        s, ph = slot(1, t - 1)
                        yield lambda s=s, ph=ph: empty[s].ready(ph)
                    M.read(("O", ob, w), ("O", i, t))
                    M.write(("O", ob, w), ("O", i, t))
                M.write(("P", b, w), ("P", t))
                yield lambda: True
                p_full[b].arrive()
            if i >= 2:
                yield lambda i=i, ob=ob: o_empty[ob].ready((i >> 1) - 1)
            M.write(("stat", ob, w), ("stat", i))
            stat[ob].arrive()
            if e4m3:
                q_empty[i & 1].arrive()

    def epilogue(w):
        for i, n0, r in segs:
            ob = i & 1
            yield lambda: stat[ob].ready(i >> 1)
            yield lambda: o_full[ob].ready(i >> 1)
            for x in range(WARPS):
                M.read(("stat", ob, x), ("stat", i))
            for g in range(groups):
                M.read(("O", ob, w + GROUP * g), ("O", i, n0 + r))
            yield lambda: True
            o_empty[ob].arrive()

    M.run([producer(), issuer(), q_warp(), scales(), *(softmax(w) for w in range(WARPS)),
           *(epilogue(w) for w in range(4))])
    assert all(o_empty[b].done == (len(runs) + 1 - b) // 2 for b in range(2))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("slots,groups", [(3, 1), (6, 1), (12, 1), (5, 2), (6, 2), (11, 4)])
@pytest.mark.parametrize("runs", [[1], [2], [9], [1, 1, 1, 1, 1], [3, 1, 2], [1, 4, 1, 1, 2, 5]])
def test_pipeline_under_random_interleavings(runs, slots, groups, e4m3):
    for seed in range(40 // (groups + 1)):
        decode_model(runs, slots, seed, e4m3, groups)


@pytest.mark.parametrize("skip", ["p", "o_empty", "rescale"])
def test_model_detects_a_missing_wait(skip):
    failures = 0
    for seed in range(60):
        try:
            decode_model([3, 1, 2, 1, 4], 6, seed, False, skip=skip)
        except AssertionError:
            failures += 1
    assert failures > 0


def test_model_matches_the_kernel():
    """The rings this model runs are the kernel's (read from its source)."""
    src = open(os.path.join(os.path.dirname(__file__), "..", "io_aware_exact_23_b200", "csrc", "fa_decode.cuh")).read()
    assert int(re.search(r"kScStages = (\d+);", src).group(1)) == SCALES
    assert "kSlots >= 3" in src and "> 24 ? 24" in src and "kPvBar = kSlots < 5" in src
