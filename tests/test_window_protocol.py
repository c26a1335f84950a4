"""Host model of the window attention kernel (gdn_window.cu): which key tiles a CTA's two query tiles
visit, and the mbarrier protocol between its copying thread, its issuing thread and the four softmax
groups (query tile x half of the keys), under random interleavings.

The plan's arithmetic is checked against the set of visible keys; the protocol must end in every
order, find each barrier one phase on, and touch no buffer early (as in test_barrier_protocols.py,
whose scheduler it uses).  The plans include query tiles that skip tiles only the other one sees.
"""

import random

import pytest

from test_barrier_protocols import _World

BM = BN = 128
KS, VS = 3, 2


class Plan:
    """make_plan of the kernel: rows of (row0, head) pairs for the two query tiles."""

    def __init__(self, row0, Tq, Tk, window, sinks, n_keys):
        off = Tk - Tq
        self.lo = [off + r for r in row0]
        self.hi = [min(off + min(r + BM, Tq), n_keys) - 1 for r in row0]
        live = [h >= l for l, h in zip(self.lo, self.hi)]
        self.n = 0
        self.first_end, self.near, self.end = [0, 0], [0, 0], [0, 0]
        if not any(live):
            return
        lo = min(l for l, a in zip(self.lo, live) if a)
        hi = max(h for h, a in zip(self.hi, live) if a)
        w_lo = max(0, lo - window + 1)
        self.sink = min(sinks, n_keys)
        split = w_lo > self.sink
        self.nA = -(-self.sink // BN) if split else 0
        self.startB = w_lo if split else 0
        self.n = self.nA + -(-(hi + 1 - self.startB) // BN)
        for q in range(2):
            if live[q]:
                w = max(0, self.lo[q] - window + 1)
                self.end[q] = self.nA + (self.hi[q] - self.startB) // BN + 1
                self.near[q] = self.nA + (w - self.startB) // BN
                self.first_end[q] = min(self.nA if split else -(-self.sink // BN), self.end[q])
        self.split = split

    def start(self, j):
        return BN * j if j < self.nA else self.startB + BN * (j - self.nA)

    def active(self, q, j):
        return 0 <= j < self.n and (j < self.first_end[q] or self.near[q] <= j < self.end[q])

    def tiles(self, q):
        return [j for j in range(self.n) if self.active(q, j)]


def visible(t, window, sinks):
    return {s for s in range(t + 1) if s > t - window or s < sinks}


@pytest.mark.parametrize("seed", range(12))
def test_plan_visits_every_visible_key_once(seed):
    r = random.Random(seed)
    for _ in range(25):
        Tk = r.choice([1, 100, 128, 129, 300, 700, 1000])
        Tq = r.randint(1, Tk)
        window, sinks = min(Tk, r.choice([1, 2, 64, 128, 150, 300, 2000])), min(Tk, r.choice([0, 0, 1, 5, 130, 400]))
        n_keys = r.choice([Tk, r.randint(0, Tk)])
        r0 = BM * r.randint(0, (Tq - 1) // BM)
        row0 = r.choice([(r0, r0), (r0, r0 + BM)])
        p = Plan(row0, Tq, Tk, window, sinks, n_keys)
        for j in range(p.n):
            assert p.active(0, j) or p.active(1, j), "a tile that no query tile sees"
        for q in range(2):
            for t in range(p.lo[q], p.hi[q] + 1):
                seen = []
                for j in p.tiles(q):
                    s0 = p.start(j)
                    sink_tile = j < p.nA
                    hi = -1 if sink_tile else min(t, n_keys - 1) - s0
                    lo = max(0, t - window + 1) - s0
                    split = p.startB > 0 or p.nA > 0
                    sk = 0 if split and not sink_tile else min(p.sink, t + 1) - s0
                    seen += [s0 + e for e in range(BN) if lo <= e <= hi or e < sk]
                assert len(seen) == len(set(seen)) and set(seen) == visible(t, window, sinks)


def run(p, seed, mutation=None, warps=2):
    live = [q for q in range(2) if p.end[q]]
    w = _World(lambda name: warps if name[0] in "PL" else 1, random.Random(seed))
    rnd = random.Random(seed + 1)
    ref, used = {}, {}                       # a warp's rows: moves of their reference; the one behind its P

    def loader():
        w.async_op("dma", "Q", ["Q"])
        for j in range(p.n):
            if j >= KS:
                yield from w.wait(f"KFree{j % KS}", j // KS - 1)
                w.need(*((("S", q, j - KS, h)) for q in range(2) if p.active(q, j - KS) for h in range(2)))
            w.async_op("dma", ("K", j), [f"KFull{j % KS}"])
            if j >= VS:
                yield from w.wait(f"VFree{j % VS}", j // VS - 1)
                w.need(*((("PV", q, j - VS, h)) for q in range(2) if p.active(q, j - VS) for h in range(2)))
            w.async_op("dma", ("V", j), [f"VFull{j % VS}"])
            yield

    def issue():
        yield from w.wait("Q", 0)
        steps = [0, 0]
        for j in range(p.n + 1):
            pv = [p.active(q, j - 1) for q in range(2)]
            qk = [p.active(q, j) for q in range(2)]
            if j >= 1:
                yield from w.wait(f"VFull{(j - 1) % VS}", (j - 1) // VS)
            if j < p.n:
                yield from w.wait(f"KFull{j % KS}", j // KS)
            for h in range(2):
                for q in range(2):
                    if pv[q]:
                        yield from w.wait(f"P{q}{h}", steps[q])
                        w.need(("V", j - 1), *(("P", q, j - 1, h, k) for k in range(warps)))
                        assert all(used[q, j - 1, h, k] == ref.get((q, k), 0) for k in range(warps)), \
                            "hazard: weights of a reference that O has left"
                        arrivals = [f"H{q}{h}"]
                        if h == 1:
                            steps[q] += 1
                            if q == 1 or not pv[1]:
                                arrivals.append(f"VFree{(j - 1) % VS}")
                            if j == p.end[q]:
                                arrivals.append(f"O{q}")
                        w.async_op("mma", ("PV", q, j - 1, h), arrivals)
                    if qk[q]:
                        w.need("Q", ("K", j))
                        arrivals = [f"S{q}{h}"]
                        if h == 1 and (q == 1 or not qk[1]):
                            arrivals.append(f"KFree{j % KS}")
                        w.async_op("mma", ("S", q, j, h), arrivals)
                    yield

    def softmax(q, h, k):
        tiles = p.tiles(q)
        other = f"P{q}{h ^ 1}"
        known = 0

        def swap(phase):
            if h == 1:
                yield from w.wait(f"L{q}0", phase)
            w.arrive(f"L{q}{h}")
            if h == 0:
                yield from w.wait(f"L{q}1", phase)

        for i, j in enumerate(tiles):
            if not (mutation == "scores asked for before the weights are stored" and i > 0):
                yield from w.wait(f"S{q}{h}", i)
            w.need(("S", q, j, h))
            if i == 0:
                yield from swap(0)
            yield
            if (h == 1 or i > 0) and mutation != "no look at the other thread":
                yield from w.wait(other, i if h else i - 1)
                known = ref.get((q, k), 0)
            if (h == 1 or i > 0) and rnd.random() < 0.3:         # the reference moves: O is rescaled
                yield from w.wait(f"H{q}{h ^ 1}", i if h else i - 1)
                w.need(*(("PV", q, t, e) for t in tiles[:i] for e in range(2)), *([("PV", q, j, 0)] if h else []))
                known = ref[q, k] = ref.get((q, k), 0) + 1
            if i > 0:
                w.need(("PV", q, tiles[i - 1], h))               # P written over a buffer whose P V is done
            if mutation == "scores asked for before the weights are stored" and i + 1 < len(tiles):
                yield from w.wait(f"S{q}{h ^ 1}" if h == 0 else f"S{q}0", i if h == 0 else i + 1)
            yield
            w.done.add(("P", q, j, h, k))
            used[q, j, h, k] = known
            w.arrive(f"P{q}{h}")
        yield from w.wait(f"O{q}", 0)
        if h == 0:
            yield from w.wait(other, len(tiles) - 1)
        yield from swap(1)

    w.run([loader(), issue()] + [softmax(q, h, k) for q in live for h in range(2) for k in range(warps)])


PLANS = [
    Plan((0, 0), 100, 100, 100, 0, 100), Plan((0, 128), 200, 200, 50, 0, 200), Plan((256, 256), 400, 400, 130, 5, 400),
    Plan((256, 384), 600, 600, 100, 5, 600), Plan((384, 512), 700, 700, 1, 130, 700), Plan((0, 128), 256, 256, 256, 300, 100),
    Plan((640, 768), 1000, 1000, 400, 260, 1000), Plan((512, 640), 700, 700, 700, 0, 650),
]


@pytest.mark.parametrize("plan", range(len(PLANS)))
def test_window_attention_protocol(plan):
    for seed in range(40):
        run(PLANS[plan], seed)


@pytest.mark.parametrize("mutation", ["scores asked for before the weights are stored", "no look at the other thread"])
def test_window_protocol_model_catches_planted_mistakes(mutation):
    """The first is a form the kernel had: a query tile that waits for scores beyond tiles that only the
    other query tile sees, before its own weights are stored, waits for good."""
    caught = 0
    for seed in range(40):
        try:
            run(PLANS[4], seed, mutation)
        except AssertionError:
            caught += 1
    assert caught > 0, f"the model missed: {mutation}"
