"""A model of the barriers between the issuing warp and the softmax warps of the tiles kernel
(csrc/common_keys_tiles.cu), with the arrivals and waits of each in the kernel's order, run under
schedules drawn at random: whatever the speed of each warp, nobody waits for a phase that has gone
by twice, and no output is overwritten before it was read.  Copies are taken as always there."""
import random

import pytest

PAIR, SINGLE = "pair", "single"
SLOTS = 4


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending = self.count
            self.phase ^= 1

    def passed(self, parity):  # the phase of that parity is complete, as far as a parity can tell
        return self.phase != parity


class Block:
    """Pieces of (form, key tiles), in the order in which a block takes them."""

    def __init__(self, pieces, done_before_free=False):
        self.pieces, self.done_before_free = pieces, done_before_free
        self.bars = {"qfull": Barrier(1), "qempty": Barrier(1), "written": Barrier(8), "read": Barrier(8)}
        for t in range(2):
            self.bars.update({("s", t): Barrier(1), ("p", t): Barrier(4), ("done", t): Barrier(1), ("free", t): Barrier(8)})
        for i in range(SLOTS):
            self.bars.update({("full", i): Barrier(1), ("empty", i): Barrier(9)})
        self.has_read = [[False] * 8 for _ in pieces]
        self.lost = []
        self.actors = {"producer": self.producer(), "issuer": self.issuer()}
        self.actors.update({w: self.softmax(w) for w in range(8)})

    def arrive(self, *name):
        self.bars[name if len(name) > 1 else name[0]].arrive()

    def producer(self):
        for i, piece in enumerate(self.pieces + [None]):
            if i >= SLOTS:
                yield ("empty", i % SLOTS), (i // SLOTS & 1) ^ 1
            self.arrive("full", i % SLOTS)
            if piece is None:
                return
            if i > 0:
                yield "qempty", (i - 1) & 1
            self.arrive("qfull")

    def issuer(self):
        weights = [0, 0]
        for i, piece in enumerate(self.pieces + [None]):
            yield ("full", i % SLOTS), i // SLOTS & 1
            if piece is None:
                return
            form, tiles = piece
            yield "qfull", i & 1

            def product(t, first):
                yield ("p", t), weights[t] & 1
                weights[t] += 1
                if first:
                    if i > 0:
                        yield ("free", t), (i - 1) & 1
                    self.overwrites(i, t)

            if form == PAIR:
                self.arrive("s", 0), self.arrive("s", 1)
                if tiles == 1:
                    self.arrive("qempty")
                for j in range(tiles):
                    for t in range(2):
                        yield from product(t, j == 0)
                        self.arrive("done" if j == tiles - 1 else "s", t)
                    if j + 2 == tiles:
                        self.arrive("qempty")
            else:
                for t in range(min(tiles, 2)):
                    self.arrive("s", t)
                if tiles <= 2:
                    self.arrive("qempty")
                for j in range(tiles):
                    yield from product(j & 1, j < 2)
                    if j + 2 < tiles:
                        self.arrive("s", j & 1)
                        if j + 3 == tiles:
                            self.arrive("qempty")
                self.arrive("done", 0)
                if self.done_before_free:
                    self.arrive("done", 1)
                if tiles == 1 and i > 0:
                    yield ("free", 1), (i - 1) & 1
                if not self.done_before_free:
                    self.arrive("done", 1)
            self.arrive("empty", i % SLOTS)

    def overwrites(self, i, t):
        for k, (form, tiles) in enumerate(self.pieces[:i]):
            for w in range(8):
                reads = w // 4 == t if form == PAIR else t == 0 or tiles > 1
                if reads and not self.has_read[k][w]:
                    self.lost.append((k, w))

    def softmax(self, w):
        t, tiles_seen, singles = w // 4, 0, 0
        for i, piece in enumerate(self.pieces + [None]):
            yield ("full", i % SLOTS), i // SLOTS & 1
            if piece is None:
                return
            form, tiles = piece
            for _ in range(tiles if form == PAIR else (tiles + 1 - t) >> 1):
                yield ("s", t), tiles_seen & 1
                tiles_seen += 1
                yield None
                self.arrive("p", t)
            yield ("done", t), i & 1
            yield None
            if form == SINGLE:
                if singles > 0:
                    yield "read", (singles - 1) & 1
                self.arrive("written")
                yield "written", singles & 1
                singles += 1
                yield None
            self.has_read[i][w] = True
            if form == SINGLE:
                self.arrive("read")
            self.arrive("free", t)
            self.arrive("free", t if form == PAIR else 1 - t)
            self.arrive("empty", i % SLOTS)

    def run(self, rng):
        """True when every actor came to its end."""
        at, slow, patience = {}, [], rng.choice((0, 0.9, 0.99, 1.0))
        moved = list(self.actors)
        while True:
            for k in moved:
                try:
                    at[k] = next(self.actors[k])
                except StopIteration:
                    del self.actors[k]
                    at.pop(k, None)
            if not self.actors:
                return True
            if rng.random() < 0.03:
                slow = rng.sample(list(self.actors), rng.randint(0, min(5, len(self.actors))))
            ready = [k for k, what in at.items() if what is None or self.bars[what[0]].passed(what[1])]
            if not ready:
                return False
            fast = [k for k in ready if k not in slow]
            moved = [rng.choice(fast if fast and rng.random() < patience else ready)]


def blocks(rng, n):
    for _ in range(n):
        yield [(rng.choice((PAIR, SINGLE)), rng.choice((1, 1, 1, 2, 3, 4, 7))) for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("seed", range(4))
def test_no_schedule_stalls_or_overwrites(seed):
    rng = random.Random(seed)
    for pieces in blocks(rng, 1500):
        block = Block(pieces)
        assert block.run(rng), pieces
        assert not block.lost, (pieces, block.lost)


def test_the_model_sees_a_phase_that_goes_by_twice():
    """With the output of half 1 told of before its last readers are known to be past the piece before."""
    rng = random.Random(5)
    assert not all(Block(pieces, done_before_free=True).run(rng) for pieces in blocks(rng, 3000))
