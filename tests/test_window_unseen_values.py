"""Host model of what the window attention kernel (gdn_window.cu) does about values that a query does not
see.  Rows of V that no query of a visited tile sees are zeroed by the softmax threads, which wait for the
copy of that tile: in the protocol model of test_window_protocol.py with that wait added, every order still
ends and finds its barriers.  The tokens that a row visits and does not see, as the rows that are done again
look for them, are all there and few.
"""

import random

import pytest

import test_window_protocol as base
from test_window_protocol import BM, BN, VS, Plan, visible


def seen_end(p, j, Tk, n_keys):
    """The key from which no query of tile j sees any, where its rows of V are zeroed; None: they are not."""
    sink_tile = j < p.nA
    end = p.sink if sink_tile else n_keys
    return end if end - p.start(j) < BN and (sink_tile or n_keys < Tk) else None


CASES = [  # row0, Tq, Tk, window, sinks, n_keys
    ((256, 384), 600, 600, 100, 5, 600), ((384, 512), 700, 700, 1, 130, 700), ((768, 896), 1000, 1000, 400, 260, 930),
    ((512, 640), 700, 700, 700, 0, 650), ((512, 512), 640, 900, 64, 3, 900), ((0, 0), 100, 400, 40, 128, 390),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_protocol_with_the_wait_for_v(case, monkeypatch):
    row0, Tq, Tk, window, sinks, n_keys = CASES[case]
    p = Plan(*CASES[case])
    waits = 0

    class World(base._World):
        def wait(self, name, phase):
            nonlocal waits
            yield from super().wait(name, phase)
            if name[0] == "S" and name[2] == "0":                 # scores of half 0 of query tile name[1]
                j = p.tiles(int(name[1]))[phase]
                if seen_end(p, j, Tk, n_keys) is not None:
                    yield from super().wait(f"VFull{j % VS}", j // VS)
                    self.need(("V", j))
                    waits += 1

    monkeypatch.setattr(base, "_World", World)
    for seed in range(40):
        base.run(p, seed)
    assert waits


@pytest.mark.parametrize("seed", range(12))
def test_rows_look_for_all_they_visit_and_do_not_see(seed):
    r = random.Random(100 + seed)
    for _ in range(25):
        Tk = r.choice([1, 100, 128, 129, 300, 700, 1000])
        Tq = r.randint(1, Tk)
        window, sinks = min(Tk, r.choice([1, 2, 64, 128, 150, 300, 2000])), min(Tk, r.choice([0, 0, 1, 5, 130, 400]))
        n_keys = r.choice([Tk, r.randint(0, Tk)])
        r0 = BM * r.randint(0, (Tq - 1) // BM)
        p = Plan(r.choice([(r0, r0), (r0, r0 + BM)]), Tq, Tk, window, sinks, n_keys)
        for q in range(2):
            if not p.end[q]:
                continue
            near_key = p.start(p.near[q]) if p.split else 0
            end = min(n_keys, p.start(p.end[q] - 1) + BN)
            visited = set()
            for j in p.tiles(q):
                z = seen_end(p, j, Tk, n_keys)
                visited |= set(range(p.start(j), p.start(j) + BN if z is None else z))
            for t in range(p.lo[q], p.hi[q] + 1):
                ws = max(0, t - window + 1)
                look = set(range(max(min(p.sink, t + 1), near_key), ws)) | set(range(t + 1, end))
                see = visible(t, window, sinks)
                assert {s for s in visited if s < n_keys} - see <= look and not look & see
                assert all(0 <= s < n_keys for s in look) and len(look) <= 4 * BM
                assert see == set(range(min(p.sink, ws))) | set(range(ws, t + 1))
