"""The ring of e4m3 codes in prompt attention, as a model on the CPU: one warp copies quarter tiles into slots, three pairs
of warps convert them in turn, and every wait looks at an mbarrier's phase by its parity alone. Copies land in any order.

The waits of a converting warp are those that the kernel's source has, in its order.
"""

import random
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "quantized_kv_decode_partial_gb300" / "csrc"


def the_kernel():
    """Barriers that a converting warp waits for before it reads unit n's codes, in order; and the numbers of slots that shapes of
    heads can get."""
    text = (CSRC / "pkv_prefill.cuh").read_text()
    part = text[text.index("for (int n = group; n < 8 * nt; n += "):text.index("convert_quarter<D, FMT, KT>(smem_k")]
    rule = re.search(r"kRawSlots = !kCodes \? 0 : (.*);", text).group(1)
    most = int(re.search(r"kRawFit > (\d+) \? \1 : kRawFit", rule).group(1))
    by = int(re.search(r"kPairs = (\d+);", text).group(1)) if rule.endswith("/ kPairs * kPairs") else 1
    assert by in (1, 3)  # the model's pairs
    return (re.findall(r"mbar_wait_close\((?:is_k \? )?(\w+)\(", part),
            sorted({min(fit, most) // by * by for fit in range(6, 30)}))


class Barrier:
    """An mbarrier: phases completed so far, arrivals (and copies) that the current one waits for."""

    def __init__(self, arrivals):
        self.arrivals, self.phase, self.pending = arrivals, 0, arrivals

    def arrive(self, n=1):
        self.pending -= n
        assert self.pending >= 0, "an arrival in a phase that is not its own"
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.arrivals

    def passes(self, parity):
        return self.phase & 1 != parity


def tile_of(x, nt):
    """Plane tile x in the order K(0), K(1), V(0), K(2), V(1), ...: (is K, which)."""
    order = [(True, 0)]
    for j in range(nt):
        if j + 1 < nt:
            order.append((True, j + 1))
        order.append((False, j))
    return order[x]


class Ring:
    def __init__(self, slots, stages, nt, waits, late, rng):
        self.slots, self.stages, self.nt, self.waits, self.rng = slots, stages, nt, waits, rng
        self.units, self.late = 8 * nt, late
        self.raw_full = [Barrier(2) for _ in range(slots)]  # the copying warp's arrival, and the copy
        self.raw_empty = [Barrier(2) for _ in range(slots)]
        self.full = {k: [Barrier(8) for _ in range(stages)] for k in (True, False)}
        self.empty = {k: [Barrier(1) for _ in range(stages)] for k in (True, False)}
        self.held = [None] * slots  # unit whose codes lie in the slot; None while a copy is on its way
        self.flying = []
        self.asked = 0
        self.at = {(g, w): (g, 0) for g in range(3) for w in range(2)}  # a warp's unit, and which wait comes next
        self.product = 0

    def copy(self):
        n = self.asked
        if n >= self.units or (n >= self.slots and not self.raw_empty[n % self.slots].passes((n // self.slots - 1) & 1)):
            return None

        def go():
            self.held[n % self.slots] = None
            self.raw_full[n % self.slots].arrive()
            self.flying.append(n)
            self.asked += 1
        return go

    def land(self, n):
        def go():
            self.flying.remove(n)
            self.held[n % self.slots] = n
            self.raw_full[n % self.slots].arrive()
        return go

    def convert(self, who):
        n, k = self.at[who]
        if n >= self.units:
            return None
        s, (is_k, j) = n % self.slots, tile_of(n // 4, self.nt)
        if k == len(self.waits):
            def read():
                assert self.held[s] == n, f"unit {n} read while slot {s} holds {self.held[s]}"
                self.full[is_k][j % self.stages].arrive()
                self.raw_empty[s].arrive()
                self.at[who] = (n + 3, 0)
            return read
        name = self.waits[k]
        if name == "k_empty":  # or v_empty
            ready = j < self.stages or self.empty[is_k][j % self.stages].passes((j // self.stages - 1) & 1)
        elif name == "raw_empty":
            ready = n < self.slots or self.raw_empty[s].passes((n // self.slots - 1) & 1)
        else:
            assert name == "raw_full"
            ready = self.raw_full[s].passes((n // self.slots) & 1)

        def go():
            self.at[who] = (n, k + 1)
        return go if ready else None

    def products(self):
        if self.product >= 2 * self.nt:
            return None
        is_k, j = tile_of(self.product, self.nt)
        if not self.full[is_k][j % self.stages].passes((j // self.stages) & 1):
            return None

        def go():
            self.empty[is_k][j % self.stages].arrive()
            self.product += 1
        return go

    def run(self):
        while True:
            moves = [self.copy(), self.products()] + [self.convert(who) for who in self.at]
            moves += [self.land(n) for n in self.flying if n != self.late]
            moves = [m for m in moves if m]
            if not moves:  # nothing else can move: the late copy lands
                moves = [self.land(n) for n in self.flying]
            if not moves:
                break
            self.rng.choice(moves)()
        assert self.asked == self.units and self.product == 2 * self.nt, "stalled"
        assert all(n >= self.units for n, _ in self.at.values())


def runs(slots, waits):
    for stages in (2, 3, 4):
        for nt in (1, 2, 3, 7):
            for late in [None] + list(range(min(8 * nt, 3 * slots))):
                yield Ring(slots, stages, nt, waits, late, random.Random(1000 * slots + 100 * stages + nt))


def test_no_unit_is_read_before_its_copy_landed():
    waits, counts = the_kernel()
    assert waits[-1] == "raw_full" and min(counts) >= 6
    for slots in counts:
        for ring in runs(slots, waits):
            ring.run()


def test_the_model_sees_a_parity_that_is_a_phase_behind():
    """Slots that several pairs take in turn, and no other wait: each mistake that one copy's delay can make is one of these two. A
    wait for the slot's release before rules them out, as do slots that are one pair's alone."""
    for slots in (7, 8):
        with pytest.raises(AssertionError, match="read while slot|not its own"):
            for ring in runs(slots, ["k_empty", "raw_full"]):
                ring.run()
        for ring in runs(slots, ["k_empty", "raw_empty", "raw_full"]):
            ring.run()
