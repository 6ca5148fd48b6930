"""The barriers between the warps of the layer for few tokens, as a model: every warp's
waits and arrivals in its own order, the arrival counts as the kernels set them, and
schedules in which one warp is held back until nobody else can go on.

A wait goes by the parity of a phase.  Whoever waits for a slot and is not waited for
in turn can be overtaken by a whole turn of the ring: the phase it asks for is then the
one in progress, and the call ends in a timeout.  (No GPU needed.)"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_get_dispatch_gb300", "csrc")


def arrivals(source):
    """{barrier: arrivals of a phase} as the kernel's mbar_init lines say."""
    with open(os.path.join(CSRC, source)) as f:
        text = f.read()
    names = {n: int(v) for n, v in re.findall(r"\b(k\w+) = (\d+)[,;]", text)}
    names.update(kTurners=names.get("kTeams", 0) * names.get("kTeam", 0))
    return {n: eval(v, {}, names) for n, v in re.findall(r"mbar_init\(&sh\.(\w+)\[\w+\], ([^)]+)\)", text)}


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def turn(self):
        assert self.pending >= 0
        if self.pending == 0 and self.tx == 0:
            self.pending = self.count
            self.phase += 1

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        self.turn()

    def landed(self):
        self.tx -= 1
        self.turn()


class Machine:
    def __init__(self, counts, slots):
        self.bars = {(n, s): Barrier(c) for n, c in counts.items() for s in range(slots.get(n, 2))}
        self.roles, self.copies, self.at = {}, [], {}

    def add(self, name, steps):
        self.roles[name] = steps
        self.step(name, first=True)

    def step(self, name, first=False):
        """One wait or action of a role further; False where it cannot go on."""
        if not first:
            kind, bar, use = self.at[name]
            if kind == "wait":
                b = self.bars[bar]
                if b.phase % 2 == use % 2:
                    return False
                assert b.phase == use + 1, f"{name} passes {bar} for its use {use} in phase {b.phase}"
            elif kind == "arrive":
                self.bars[bar].arrive(use)
            else:
                self.copies.append(bar)
        try:
            self.at[name] = next(self.roles[name])
        except StopIteration:
            del self.roles[name]
        return True

    def run(self, held, rng):
        """Until all are done; `held` moves when nothing else does.  False: stuck."""
        while self.roles or self.copies:
            moved = False
            for name in rng.sample(sorted(self.roles), len(self.roles)):
                while name in self.roles and name != held and self.step(name):
                    moved = True
            rng.shuffle(self.copies)   # they land in any order
            if self.copies:
                self.bars[self.copies.pop()].landed()
                moved = True
            if not moved and not (held in self.roles and self.step(held)):
                return False
        return True


def uses(n, ring):
    return [(i % ring, i // ring) for i in range(n)]


def e4m3(ring, units, chunks, idle=True):
    """units: (copies of each weights' warp in a stage) a unit; idle: who has nothing to do arrives all the same."""
    counts = arrivals("few.cu")
    m = Machine(counts, {"full": ring, "turned": ring, "empty": ring, "sums_full": 4, "sums_empty": 4})
    stages = [(u, c) for u in units for c in range(chunks)]
    walk = [(s, use, u, c) for (u, c), (s, use) in zip(stages, uses(len(stages), ring))]

    def weights(turn):
        for s, use, u, _ in walk:
            yield "wait", ("empty", s), use - 1
            if turn == 0:
                yield "arrive", ("full", s), sum(u) + 1   # a row of tokens besides
            elif idle:
                yield "arrive", ("full", s), 0
            for _ in range(u[turn]):
                yield "copy", ("full", s), 0

    def rows():
        for s, use, _, _ in walk:
            yield "wait", ("empty", s), use - 1
            yield "copy", ("full", s), 0

    def turner(team):
        for i, (s, use, _, _) in enumerate(walk):
            yield "wait", ("full", s), use
            if idle or i % 2 == team:
                yield "arrive", ("turned", s), 0

    def products():
        for (s, use, _, _), (b, turn) in zip(walk, uses(len(walk), 4)):
            yield "wait", ("sums_empty", b), turn - 1
            yield "wait", ("turned", s), use
            yield "arrive", ("empty", s), 0
            yield "arrive", ("sums_full", b), 0

    def sums(team):
        unit = 0
        for (_, _, _, c), (b, turn) in zip(walk, uses(len(walk), 4)):
            if c % 2 == team:
                yield "wait", ("sums_full", b), turn
                yield "arrive", ("sums_empty", b), 0
            if c == chunks - 1 and chunks > 1:
                if team == 0:
                    yield "wait", ("part_full", unit % 2), unit // 2
                    yield "arrive", ("part_empty", unit % 2), 0
                else:
                    yield "wait", ("part_empty", unit % 2), unit // 2 - 1
                    yield "arrive", ("part_full", unit % 2), 0
                unit += 1

    for turn in range(2):
        m.add(f"weights {turn}", weights(turn))
    m.add("rows", rows())
    for team in range(2):
        for member in range(2):
            m.add(f"turner {team} {member}", turner(team))
        for quarter in range(4):
            m.add(f"sums {team} {quarter}", sums(team))
    m.add("products", products())
    return m


def bf16(ring, units, chunks, idle=True):
    """units: rows of each of the two token warps, a unit."""
    counts = arrivals("few_bf16.cu")
    reds = 2
    m = Machine(counts, {"full": ring, "empty": ring, "red_full": reds, "red_empty": reds})
    walk = [(s, use, u, c) for (u, c), (s, use) in zip([(u, c) for u in units for c in range(chunks)], uses(len(units) * chunks, ring))]

    def weights():
        for s, use, u, _ in walk:
            yield "wait", ("empty", s), use - 1
            yield "arrive", ("full", s), 1 + sum(u)
            yield "copy", ("full", s), 0

    def tokens(turn):
        for s, use, u, _ in walk:
            yield "wait", ("empty", s), use - 1
            for _ in range(u[turn]):
                yield "copy", ("full", s), 0
            if idle:
                yield "arrive", ("full", s), 0

    def products():
        unit = 0
        for s, use, _, c in walk:
            yield "wait", ("full", s), use
            yield "arrive", ("empty", s), 0
            if c == chunks - 1:
                yield "wait", ("red_empty", unit % reds), unit // reds - 1
                yield "arrive", ("red_full", unit % reds), 0
                unit += 1

    def adders():
        for unit in range(len(units)):
            yield "wait", ("red_full", unit % reds), unit // reds
            yield "arrive", ("red_empty", unit % reds), 0

    m.add("weights", weights())
    for turn in range(2):
        m.add(f"tokens {turn}", tokens(turn))
    for n in range(8):
        m.add(f"products {n}", products())
    for n in range(4):
        m.add(f"adders {n}", adders())
    return m


MODELS = {"e4m3": (e4m3, [(1, 0), (2, 2), (1, 0), (1, 0), (2, 1), (1, 0)]), "bf16": (bf16, [(1, 0), (2, 1), (1, 0), (1, 0), (1, 0), (2, 2)])}


@pytest.mark.parametrize("kind", MODELS)
@pytest.mark.parametrize("ring", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("chunks", [1, 2, 3, 7])
def test_nobody_is_left_behind(kind, ring, chunks):
    build, units = MODELS[kind]
    for held in [None] + sorted(build(ring, units, chunks).roles):
        m = build(ring, units, chunks)
        assert m.run(held, random.Random(ring * 100 + chunks)), f"{held} held back: {m.at}"


@pytest.mark.parametrize("kind,held,counts", [("e4m3", "turner 0 0", dict(full=1, turned=2)), ("e4m3", "weights 1", dict(full=1, turned=2)),
                                              ("bf16", "tokens 1", dict(full=1))])
def test_the_model_knows_a_warp_left_behind(monkeypatch, kind, held, counts):
    """Without the arrivals of those who have nothing to do, the warp that is held back gets stuck or passes in another phase."""
    build, units = MODELS[kind]
    own = arrivals
    monkeypatch.setitem(globals(), "arrivals", lambda source: dict(own(source), **counts))
    try:
        done = build(2, units, 3, idle=False).run(held, random.Random(1))
    except AssertionError as wrong_phase:
        done = held not in str(wrong_phase)
    assert not done
