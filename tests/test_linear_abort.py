"""The block-FP8 product's warps and barriers (csrc/k_linear.cu), restated as coroutines under a
random schedule: a load that never lands ends every warp, and no piece of the output is stored
whose sums miss a block's products.  Waits that give up are what happens when nothing else can."""
from __future__ import annotations

import random

import pytest

STAGES, BUFS, SUMS, STORES = 3, 2, 4, 2     # (four of the eight warps that add, two that store)


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase ^ 1

    def done(self, parity):
        return self.phase != parity


class Cta:
    def __init__(self, tiles, blocks, lost, looks):
        self.tiles, self.blocks, self.lost, self.looks = tiles, blocks, lost, looks
        self.full, self.empty = [Bar(1) for _ in range(STAGES)], [Bar(1) for _ in range(STAGES)]
        self.tfull = [Bar(2) for _ in range(BUFS)]
        self.tempty = [Bar(SUMS) for _ in range(BUFS)]
        self.ofull, self.ofree = [Bar(1) for _ in range(SUMS)], [Bar(1) for _ in range(SUMS)]
        self.stage, self.product, self.scale = [None] * STAGES, [None] * BUFS, [None] * BUFS
        self.piece, self.stored, self.abort = [None] * SUMS, [], False

    def wait(self, bar, parity):
        """Yields until the phase is over (True) or the wait gives up (False)."""
        while not bar.done(parity):
            if self.abort:
                return False
            yield bar, parity
        return True

    def loads(self):
        st = ph = n = 0
        for j in range(self.tiles):
            for b in range(self.blocks):
                if not (yield from self.wait(self.empty[st], ph ^ 1)):
                    return
                self.stage[st] = (j, b)
                if n != self.lost:
                    self.full[st].arrive()
                n, st = n + 1, st + 1
                if st == STAGES:
                    st, ph = 0, ph ^ 1

    def mmas(self, tb):
        st, ph, tph, turn = tb, 0, 0, 0
        for j in range(self.tiles):
            for b in range(self.blocks):
                if turn == tb:
                    if not (yield from self.wait(self.tempty[tb], tph ^ 1)):
                        return
                    if not (yield from self.wait(self.full[st], ph)):
                        return
                    self.product[tb] = self.stage[st]
                    self.tfull[tb].arrive()
                    self.empty[st].arrive()
                    tph, st = tph ^ 1, st + 2
                    if st >= STAGES:
                        st, ph = st - STAGES, ph ^ 1
                turn ^= 1

    def scales(self):
        tb = tph = 0
        for j in range(self.tiles):
            for b in range(self.blocks):
                ok = yield from self.wait(self.tempty[tb], tph ^ 1)
                self.scale[tb] = (j, b)
                self.tfull[tb].arrive()
                tb ^= 1
                tph ^= tb == 0
                if not ok:
                    return

    def sums(self, w):
        n = 0
        for j in range(self.tiles):
            acc = []
            for b in range(self.blocks):
                tb = n & 1
                yield from self.wait(self.tfull[tb], (n >> 1) & 1)      # the result is dropped
                acc.append((self.product[tb], self.scale[tb]))
                yield None                                              # reading takes its time
                self.tempty[tb].arrive()
                n += 1
            if self.looks and self.abort:
                return
            if not (yield from self.wait(self.ofree[w], (j & 1) ^ 1)):
                return
            self.piece[w] = (j, acc)
            self.ofull[w].arrive()

    def stores(self, s):
        for j in range(self.tiles):
            for p in range(s, SUMS, STORES):
                if not (yield from self.wait(self.ofull[p], j & 1)):
                    return
                self.stored.append((p, j, *self.piece[p]))
                self.ofree[p].arrive()

    def run(self, rng):
        live = [self.loads(), self.mmas(0), self.mmas(1), self.scales(),
                *[self.sums(w) for w in range(SUMS)], *[self.stores(s) for s in range(STORES)]]
        waits = {w: None for w in live}
        for _ in range(1000000):
            if not live:
                return
            ready = [w for w in live if waits[w] is None or waits[w][0].done(waits[w][1]) or
                     self.abort]
            if not ready:
                self.abort = True      # a limit runs out
                continue
            w = rng.choice(ready)
            try:
                waits[w] = next(w)
            except StopIteration:
                live.remove(w)
        raise AssertionError("a warp did not end")

    def wrong(self):
        """Stored pieces whose sums are not their tile's, block by block."""
        return [s for s in self.stored if s[1] != s[2] or
                s[3] != [((s[1], b), (s[1], b)) for b in range(self.blocks)]]


SHAPES = [(1, 1), (1, 4), (2, 3), (3, 2), (4, 1), (2, 7)]


@pytest.mark.parametrize("tiles, blocks", SHAPES)
def test_nothing_lost(tiles, blocks):
    for seed in range(20):
        c = Cta(tiles, blocks, None, True)
        c.run(random.Random(seed))
        assert not c.abort and not c.wrong() and len(c.stored) == tiles * SUMS


@pytest.mark.parametrize("tiles, blocks", SHAPES)
def test_a_load_that_never_lands(tiles, blocks):
    for lost in range(tiles * blocks):
        for seed in range(20):
            c = Cta(tiles, blocks, lost, True)
            c.run(random.Random(seed))
            assert c.abort and not c.wrong()
            assert all(s[1] < lost // blocks + 1 for s in c.stored)


def test_the_check_sees_sums_handed_on():
    """Warps that do not look at the flag hand on what they have, and some of it is stored before
    the storing warps look at it."""
    seen = 0
    for seed in range(200):
        c = Cta(1, 1, 0, False)
        c.run(random.Random(seed))
        seen += bool(c.wrong())
    assert seen > 0
