"""The barrier protocols of rows_splitk_kernel and rows_weigh_tc_kernel (the
tensor-core kernels behind gqa_decode_tree and gqa_decode_scored), restated
role by role and run in a simulator that knows what is ordered and what may
run out.  A change to the waits, arrivals or named barriers of a kernel
belongs here too.

Held: no two conflicting accesses to TMEM or shared memory are unordered; and
a wait that runs out anywhere ends every role, none stays at a named barrier.
Each rule that the kernels keep for this can be taken away here (never on a
GPU), and the simulator then finds what it prevents."""
import itertools
import random

import pytest

from protocol_sim import Hang, Race, Sim, Waiter

STAGES = 3


class Seg:
    """A run of one lane group's tiles in the CTA's range: `tiles` of them, `nx`
    row tiles with rows, kind "whole", "early" (its part is counted by warp 3)
    or "part"; `odd`: value rows that are not finite."""

    def __init__(self, tiles, nx=1, kind="whole", odd=False):
        self.tiles, self.nx, self.kind, self.odd = tiles, nx, kind, odd

    def __repr__(self):
        return f"{self.kind}:{self.tiles}x{self.nx}{'!' if self.odd else ''}"


def s_buffer(NT, kx, x):
    return kx & 1 if NT == 1 else x


def s_phase(NT, kx):
    return (kx >> 1) & 1 if NT == 1 else kx & 1


def splitk(NT, segs, seed=0, lost=None, rush=0.0, second_waits=True, walks_on=True, own_barrier=True):
    """lost: (copy, number) of a TMA load that never arrives, such as ("k", 2).
    second_waits: the MMA lane waits for the previous segment's softmax before
    the S that overwrites the columns of its (m, l).  walks_on: a softmax warp
    whose wait ran out still takes part in the named barriers.  own_barrier:
    a segment of one warpgroup has a barrier of its own."""
    bars = {"q_full": 1, "q_empty": 1, "mma_fin": 1, "early_full": 8, "early_done": 1}
    for st in range(STAGES):
        for b in ("k_full", "k_empty", "v_full", "v_empty"):
            bars[b, st] = 1
    for s in range(2):
        bars["s_full", s] = bars["o_done", s] = 1
        bars["p_full", s, 0] = bars["p_full", s, 1] = 4
        bars["o_free", s] = 8 if NT == 1 else 4
    sim = Sim(bars, seed, rush)

    def load(kind, number, bar, cells):
        for c in cells:
            yield ("write", c)
        if lost != (kind, number):
            yield ("arrive", bar)

    def producer():
        w = Waiter()
        jj = nq = nk = nv = 0
        ok = True

        def load_q():
            if nq > 0 and not (yield from w.wait("q_empty", nq - 1)):
                return False
            yield from load("q", nq, "q_full", ["Q"])
            return True

        for seg in segs:
            if nq == 0:
                ok = yield from load_q()
                nq += ok
            due = jj > 0
            for j in range(seg.tiles):
                if not ok:
                    break
                st, par = jj % STAGES, jj // STAGES - 1
                if jj >= STAGES and not (yield from w.wait(("k_empty", st), par)):
                    ok = False
                    break
                yield from load("k", nk, ("k_full", st), [("K", st)])
                nk += 1
                if jj >= STAGES and not (yield from w.wait(("v_empty", st), par)):
                    ok = False
                    break
                yield from load("v", nv, ("v_full", st), [("V", st, q) for q in range(4)])
                nv += 1
                if j == 0 and due:
                    ok = yield from load_q()
                    nq += ok
                jj += 1
            if not ok:
                break
        # every copy in flight, each with a limit of its own
        if nq:
            yield from Waiter().wait("q_full", nq - 1)
        for k in range(max(0, nk - STAGES), nk):
            yield from Waiter().wait(("k_full", k % STAGES), k // STAGES)
        for k in range(max(0, nv - STAGES), nv):
            yield from Waiter().wait(("v_full", k % STAGES), k // STAGES)
        yield ("named", 0, 384, False)

    def s_cells(buf):
        return [("S", buf, h, q, r) for h in range(2) for q in range(4) for r in ("P", "X")]

    def mma():
        w = Waiter()
        jj = seg_no = 0
        jx, sx = [0] * NT, [0] * NT
        ok = True

        def issue_pv(k, x, kx, first, last_x):
            st, sb = k % STAGES, s_buffer(NT, kx, x)
            if not (yield from w.wait(("v_full", st), k // STAGES)):
                return False
            if first and sx[x] > 0 and not (yield from w.wait(("o_free", x), sx[x] - 1)):
                return False
            for h in range(2):
                if not (yield from w.wait(("p_full", sb, h), s_phase(NT, kx))):
                    return False
                if NT == 1:
                    reads = [("S", sb, h, q, "P") for q in range(4)] + [("V", st, q) for q in (2 * h, 2 * h + 1)]
                else:
                    reads = [("S", sb, 0, q, "PX"[h]) for q in range(4)] + [("V", st, q) for q in (2 * h, 2 * h + 1)]
                yield ("mma", reads, [("O", h if NT == 1 else x, q) for q in range(4)])
            yield ("commit", ("o_done", sb))
            if last_x:
                yield ("commit", ("v_empty", st))
            return True

        for seg in segs:
            if not ok or not (yield from w.wait("q_full", seg_no)):
                break
            for j in range(seg.tiles):
                st = jj % STAGES
                if not (yield from w.wait(("k_full", st), jj // STAGES)):
                    ok = False
                    break
                if NT == 1 and second_waits and j == 1 and sx[0] > 0:
                    if not (yield from w.wait(("o_free", 0), sx[0] - 1)):
                        ok = False
                        break
                for x in range(seg.nx):
                    if NT == 2 and j > 0 and ok:
                        ok = yield from issue_pv(jj - 1, x, jx[x] - 1, j == 1, x == seg.nx - 1)
                    if not ok:
                        break
                    sb = s_buffer(NT, jx[x], x)
                    yield ("mma", ["Q", ("K", st)], s_cells(sb))
                    yield ("commit", ("s_full", sb))
                    jx[x] += 1
                if not ok:
                    break
                yield ("commit", ("k_empty", st))
                if j + 1 == seg.tiles:
                    yield ("commit", "q_empty")
                if NT == 1 and j > 0:
                    ok = yield from issue_pv(jj - 1, 0, jx[0] - 2, j == 1, True)
                    if not ok:
                        break
                jj += 1
            for x in range(seg.nx):
                if ok:
                    ok = yield from issue_pv(jj - 1, x, jx[x] - 1, seg.tiles == 1, x == seg.nx - 1)
                    sx[x] += 1
            seg_no += 1
            if not ok:
                break
        yield ("commit", "mma_fin")
        yield from Waiter().wait("mma_fin", 0)
        yield ("named", 0, 384, False)

    def softmax(warp):
        w = Waiter()
        wg, q4 = warp >> 2, warp & 3
        x = 0 if NT == 1 else wg
        jj = jx = 0
        ok = True
        for seg in segs:
            if not ok and not walks_on:
                break
            if x >= seg.nx:
                jj += seg.tiles
                if seg.kind == "early":
                    yield ("arrive", "early_full")
                continue
            yield ("named", 1 + wg, 128, False)  # the sequence's parents
            yield ("named", 1 + wg, 128, False)
            end_jj, end_jx = jj + seg.tiles, jx + seg.tiles
            half = wg if NT == 1 else 0
            cells = [("S", 0, half, q4, r) for r in "PX"] if NT == 1 else \
                [("S", 0, h, q4, r) for h in range(2) for r in "PX"]
            for j in range(seg.tiles):
                if not ok:
                    break
                sb = s_buffer(NT, jx, x)
                if not (yield from w.wait(("s_full", sb), s_phase(NT, jx))):
                    ok = False
                    break
                if j == seg.tiles - 1 and ((q4 >> 1) == wg if NT == 1 else wg == 0):  # an edge tile
                    st = jj % STAGES
                    if not (yield from w.wait(("v_full", st), jj // STAGES)):
                        ok = False
                        break
                    yield ("write", ("V", st, q4))
                for c in cells:
                    yield ("read", (c[0], sb) + c[2:])
                if j > 0 and (j + q4) % 2:  # O is rescaled
                    if not (yield from w.wait(("o_done", s_buffer(NT, jx - 1, x)), s_phase(NT, jx - 1))):
                        ok = False
                        break
                    yield ("write", ("O", wg, q4))
                if NT == 1:
                    yield ("write", ("S", sb, wg, q4, "P"))
                    yield ("arrive", ("p_full", sb, wg))
                else:
                    for h in range(2):
                        yield ("write", ("S", sb, 0, q4, "PX"[h]))
                        yield ("arrive", ("p_full", sb, h))
                jj, jx = jj + 1, jx + 1
            if not ok and not walks_on:
                break
            jj, jx = end_jj, end_jx
            if ok and not (yield from w.wait(("o_done", s_buffer(NT, jx - 1, x)), s_phase(NT, jx - 1))):
                ok = False
                if not walks_on:
                    break
            parties = 256 if NT == 1 else 128 * seg.nx
            bar = 1 if parties == 128 and own_barrier else 3
            if (yield ("named", bar, parties, ok and seg.odd and warp == 0)):
                if ok:
                    yield ("write", ("O", wg, q4))
                yield ("named", bar, parties, False)
                yield ("named", bar, parties, False)
            if NT == 1:
                sb = s_buffer(NT, jx - 1, 0)
                if ok:
                    yield ("write", ("S", sb, wg, q4, "X"))
                yield ("named", bar, parties, False)
                if ok:
                    for h in range(2):
                        yield ("read", ("S", sb, h, q4, "X"))
            if seg.kind == "part":
                yield ("named", bar, parties, False)   # have all others been counted?
            if ok:
                for h in range(2) if NT == 1 else (wg,):
                    yield ("read", ("O", h, q4))
            if seg.kind == "early":
                if ok:
                    yield ("arrive", "early_full")
            elif seg.kind == "part":
                yield ("named", bar, parties, False)   # the part is written
                yield ("named", bar, parties, False)   # was it the last?
            if ok:
                yield ("arrive", ("o_free", x))
        yield ("named", 4, 256, False)
        if segs[0].kind == "early":
            yield from w.wait("early_done", 0)
            yield ("named", 4, 256, False)
        yield ("named", 0, 384, False)

    def early():
        if segs[0].kind == "early":
            yield from Waiter().wait("early_full", 0)
            yield ("arrive", "early_done")
        yield ("named", 0, 384, False)

    def idle():
        yield ("named", 0, 384, False)

    sim.add("producer", producer())
    sim.add("mma", mma())
    sim.add("zeros", idle())
    sim.add("early", early())
    for k in range(8):
        sim.add(f"softmax{k}", softmax(k))
    sim.run()
    return sim


def weigh(runs, seed=0, lost=None, rush=0.0, walks_on=True):
    """runs: tiles of each run of the CTA (a lane's tiles, for 128 rows each)."""
    bars = {"mma_fin": 1}
    for s in range(2):
        bars["q_full", s] = bars["q_empty", s] = 1
    for s in range(4):
        bars["k_full", s] = bars["k_empty", s] = bars["s_full", s] = 1
        bars["s_empty", s] = 4
    sim = Sim(bars, seed, rush)

    def producer():
        w = Waiter()
        nq = nk = 0
        ok = True
        for tiles in runs:
            if not ok or (nq >= 2 and not (yield from w.wait(("q_empty", nq & 1), (nq >> 1) - 1))):
                break
            yield ("write", ("Q", nq & 1))
            if lost != ("q", nq):
                yield ("arrive", ("q_full", nq & 1))
            nq += 1
            for _ in range(tiles):
                st = nk & 3
                if nk >= 4 and not (yield from w.wait(("k_empty", st), (nk >> 2) - 1)):
                    ok = False
                    break
                yield ("write", ("K", st))
                if lost != ("k", nk):
                    yield ("arrive", ("k_full", st))
                nk += 1
        for k in range(max(0, nq - 2), nq):
            yield from Waiter().wait(("q_full", k & 1), k >> 1)
        for k in range(max(0, nk - 4), nk):
            yield from Waiter().wait(("k_full", k & 3), k >> 2)
        yield ("named", 0, 384, False)

    def mma():
        w = Waiter()
        nq = step = 0
        ok = True
        for tiles in runs:
            if not ok or not (yield from w.wait(("q_full", nq & 1), nq >> 1)):
                break
            for _ in range(tiles):
                sb = step & 3
                if not (yield from w.wait(("k_full", sb), step >> 2)) or \
                        (step >= 4 and not (yield from w.wait(("s_empty", sb), (step >> 2) - 1))):
                    ok = False
                    break
                yield ("mma", [("Q", nq & 1), ("K", sb)], [("S", sb, q) for q in range(4)])
                yield ("commit", ("s_full", sb))
                yield ("commit", ("k_empty", sb))
                step += 1
            yield ("commit", ("q_empty", nq & 1))
            nq += 1
        yield ("commit", "mma_fin")
        yield from Waiter().wait("mma_fin", 0)
        yield ("named", 0, 384, False)

    def softmax(warp):
        w = Waiter()
        wg, q4 = warp >> 2, warp & 3
        step = 0
        ok = True
        for run, tiles in enumerate(runs):
            if not ok and not walks_on:
                break
            if wg == 0:
                yield ("write", ("stats", run & 1, q4))
            yield ("named", 3, 256, False)
            for j in range(tiles):
                s = step + j
                if not ok or (s & 1) != wg:
                    continue
                yield ("read", ("w", j, q4))
                if not (yield from w.wait(("s_full", s & 3), s >> 2)):
                    ok = False
                    break
                yield ("read", ("S", s & 3, q4))
                for q in range(4):
                    yield ("read", ("stats", run & 1, q))
                yield ("arrive", ("s_empty", s & 3))
                yield ("write", ("w", j, q4))
            step += tiles
        yield ("named", 0, 384, False)

    def idle():
        yield ("named", 0, 384, False)

    sim.add("producer", producer())
    sim.add("mma", mma())
    for k in range(2):
        sim.add(f"idle{k}", idle())
    for k in range(8):
        sim.add(f"softmax{k}", softmax(k))
    sim.run()
    return sim


def plans(NT):
    """Segments of 1 to 5 tiles, one to four of them, every kind of ends."""
    rng = random.Random(NT)
    for n in range(1, 5):
        for tiles in itertools.product((1, 2, 3, 5), repeat=n):
            if n > 2 and rng.random() > 0.25:
                continue
            segs = [Seg(k, rng.randint(1, NT), odd=rng.random() < 0.3) for k in tiles]
            if n > 1 and rng.random() < 0.5:
                segs[0].kind = "early"
            if rng.random() < 0.5:
                segs[-1].kind = "part"
            yield segs


@pytest.mark.parametrize("NT", [1, 2])
def test_nothing_is_unordered_and_nobody_gives_up(NT):
    for k, segs in enumerate(plans(NT)):
        assert not splitk(NT, segs, seed=k).gave_up, segs


def test_the_second_tile_waits_for_the_exchanged_maxima():
    """Without that wait S of a later segment's second tile meets the (m, l)
    that the warpgroups exchange through its columns."""
    with pytest.raises(Race, match="'X'"):
        splitk(1, [Seg(2), Seg(2)], second_waits=False)
    with pytest.raises(Race, match="'X'"):
        splitk(1, [Seg(1, kind="early"), Seg(5), Seg(3, kind="part")], second_waits=False)
    splitk(1, [Seg(4)], second_waits=False)             # one segment: nothing to wait for
    splitk(1, [Seg(4), Seg(1)], second_waits=False)     # one tile: the other buffer


def lost_copies(segs):
    tiles = sum(s.tiles for s in segs)
    return [("q", k) for k in range(len(segs))] + [(c, k) for c in "kv" for k in range(tiles)]


@pytest.mark.parametrize("NT", [1, 2])
def test_a_wait_that_runs_out_ends_every_role(NT):
    """A copy that never comes, and waits that give up on one that is late."""
    rng = random.Random(7)
    for segs in plans(NT):
        for lost in rng.sample(lost_copies(segs), 2):
            assert splitk(NT, segs, seed=rng.random(), lost=lost).gave_up, (segs, lost)
        for rush in (0.002, 0.02):
            splitk(NT, segs, seed=rng.random(), rush=rush)


def hangs(runs, of, *args, **kw):
    n = 0
    for seed in range(runs):
        try:
            of(*args, seed=seed, **kw)
        except Hang:
            n += 1
    return n


def test_what_the_rules_for_it_prevent():
    two = [Seg(3), Seg(2, kind="part")]
    assert hangs(300, splitk, 1, two, rush=0.01, walks_on=False) > 0
    assert hangs(300, splitk, 1, two, rush=0.01) == 0
    mixed = [Seg(2, 1), Seg(2, 2), Seg(1, 1), Seg(3, 2)]
    assert hangs(300, splitk, 2, mixed, rush=0.01, own_barrier=False) > 0
    assert hangs(300, splitk, 2, mixed, rush=0.01) == 0


def test_weights_from_the_keys():
    for seed, runs in enumerate(itertools.product((1, 2, 3, 6), repeat=3)):
        assert not weigh(runs, seed=seed).gave_up
        for lost in [("q", 1), ("q", 2), ("k", 0), ("k", sum(runs) - 1), ("k", runs[0])]:
            assert weigh(runs, seed=seed, lost=lost).gave_up, (runs, lost)
    assert hangs(100, weigh, (3, 2, 2), rush=0.01, walks_on=False) > 0
    assert hangs(100, weigh, (3, 2, 2), rush=0.01) == 0
