"""The ring of key and value tiles of prompt_attention as its warps' waits and
arrivals make it, played through on the host: whatever warp is late, every wait
ends and nobody takes one lap's tile for another's.

An arrival completes a barrier's phase; a wait asks by parity whether the phase
before the present one is its own.  Whether copies wait for the cleaning warp is
read from the kernel's source."""
import itertools
import os

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_top_gb300", "csrc", "gbtopk_prompt.cu")


def copies_wait_for_cleaning():
    src = open(SOURCE).read()
    part = lambda a, b: src[src.index(a):src.index(b)]  # noqa: E731
    copies = part("if (warp == kCopy) {", "} else if (warp == kIssue) {")
    cleaning = part("} else if (warp == kClean) {", "// ------------------------------------------------ softmax, output")
    assert all(f"bar_init(&sh.{name}[i], 1);" in src for name in ("full", "empty", "clean"))
    if "sh.seen" not in src:
        return False
    assert "bar_init(&sh.seen[i], 1);" in src and "warp_wait(&sh.seen[stage], (lap - 1) & 1, abort)" in copies
    assert cleaning.count("bar_arrive(&sh.seen[") == 3      # of a key tile, a whole value tile, a cleaned one
    return True


class Barrier:
    def __init__(self):
        self.phase = 0

    def arrive(self):
        self.phase += 1

    def passes(self, parity):
        return self.phase & 1 != parity


def play(stages, units, order, waits):
    """Roles as generators that yield the waits they stand at; the first of
    `order` that can go goes, so the last is as late as the others let it be."""
    full, empty, clean, seen = ([Barrier() for _ in range(stages)] for _ in range(4))
    holds = [None] * stages           # the item in a stage

    def items():
        """Items in order, and whether each is a value tile that has to be cleaned."""
        n = itertools.count()
        for count, whole in units:
            for t in range(count):
                yield next(n), False
                yield next(n), t >= whole

    def copies():
        for n, _ in items():
            s, lap = n % stages, n // stages
            if lap:
                yield empty[s], (lap - 1) & 1
            if lap and waits:
                yield seen[s], (lap - 1) & 1
            holds[s] = n
            full[s].arrive()

    def products():
        cleaned = [0] * stages
        for n, dirty in items():
            s = n % stages
            yield full[s], (n // stages) & 1
            if dirty:
                yield clean[s], cleaned[s]
                cleaned[s] ^= 1
            assert holds[s] == n, "another lap's tile is multiplied"
            empty[s].arrive()

    def cleaning():
        for n, dirty in items():
            s = n % stages
            yield full[s], (n // stages) & 1
            if dirty:
                assert holds[s] == n, "another lap's tile is cleaned"
                clean[s].arrive()
            seen[s].arrive()

    roles = {"copies": copies(), "products": products(), "cleaning": cleaning()}
    at = {}
    for name, role in roles.items():
        at[name] = next(role, None)
    while any(w is not None for w in at.values()):
        for name in order:
            w = at[name]
            if w is not None and w[0].passes(w[1]):
                at[name] = next(roles[name], None)
                break
        else:
            return sorted(name for name, w in at.items() if w is not None)
    return []


UNITS = [
    [(40, 40)],                             # one row whose keys are whole tiles
    [(40, 39)], [(40, 38), (3, 0), (41, 40), (1, 1), (2, 1)],
    [(1, 0)] * 9, [(7, 7), (1, 0), (30, 30), (8, 6)],
]


@pytest.mark.parametrize("stages", [4, 5, 7, 10])
@pytest.mark.parametrize("units", UNITS)
def test_every_wait_ends_whoever_is_late(stages, units):
    waits = copies_wait_for_cleaning()
    for order in itertools.permutations(("copies", "products", "cleaning")):
        assert play(stages, units, order, waits) == [], order
