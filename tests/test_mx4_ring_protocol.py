"""A model of the MXFP4 product's barriers, run through random interleavings (CPU).

Roles as in csrc/mx4_product.cu: TMA and the scale warps fill a stage's slot, a fence warp passes the scales on, the MMA
warp consumes the slot and frees it when its MMAs have finished (later, in order), epilogue groups of warps take
every other tile and free its accumulator. A barrier counts arrivals and flips its phase; a parity wait passes
when the phase of that parity is over, which says nothing about how many phases ago. The model checks, at every step a
wait has let through, that what the role believes is true, and that every run ends.
"""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "an arrival too many"
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return self.phase & 1 != parity & 1


class Model:
    def __init__(self, stages, accs, tiles, nk, owners=True, warps=None):
        self.S, self.A, self.tiles, self.nk, self.total = stages, accs, tiles, nk, tiles * nk
        self.full = [Barrier(2) for _ in range(stages)]      # TMA's bytes, the fence warp
        self.sf_in = [Barrier(1) for _ in range(stages)]
        self.empty = [Barrier(1) for _ in range(stages)]
        self.acc_full = [Barrier(1) for _ in range(accs)]
        self.acc_empty = [Barrier(4) for _ in range(accs)]
        self.codes, self.scales = [-1] * stages, [-1] * stages  # stage that a slot holds
        self.done = -1                                          # last stage whose MMAs have finished
        self.issued = []                                        # stages whose MMAs are under way
        self.acc = [-1] * accs                                  # tile that an accumulator holds
        self.drained = [0] * tiles                              # warps that have read a tile
        self.roles = [self.tma(), self.fence(), self.mma()]
        n = stages // 2 if owners else warps
        self.roles += [self.scale_owner(w) if owners else self.scale_in_turn(w, n) for w in range(n)]
        self.roles += [self.epilogue(who, q) for who in range(2) for q in range(4)]

    def free(self, g):  # the slot of stage g may be written: its last stage's MMAs are over
        assert self.done >= g - self.S, ("slot still read", g, self.done)

    def tma(self):
        for g in range(self.total):
            yield self.empty[g % self.S], (g // self.S + 1)
            self.free(g)
            self.codes[g % self.S] = g
            self.full[g % self.S].arrive()

    def put(self, g):
        yield self.empty[g % self.S], (g // self.S + 1)
        self.free(g)
        self.scales[g % self.S] = g
        self.sf_in[g % self.S].arrive()

    def scale_owner(self, w):  # the stages of the slots 2w and 2w + 1
        for g in range(2 * w, self.total, self.S):
            yield from self.put(g)
            if g + 1 < self.total:
                yield from self.put(g + 1)

    def scale_in_turn(self, w, n):  # every n-th pair of stages, whatever its slots
        for g in range(2 * w, self.total, 2 * n):
            yield from self.put(g)
            if g + 1 < self.total:
                yield from self.put(g + 1)

    def fence(self):
        for g in range(self.total):
            yield self.sf_in[g % self.S], g // self.S
            assert self.scales[g % self.S] == g, ("scales of another stage", g)
            self.full[g % self.S].arrive()

    def mma(self):
        for t in range(self.tiles):
            b = t % self.A
            yield self.acc_empty[b], (t // self.A + 1)
            assert t < self.A or self.drained[t - self.A] == 4, ("accumulator still read", t)
            for k in range(self.nk):
                g = t * self.nk + k
                yield self.full[g % self.S], g // self.S
                assert self.codes[g % self.S] == g and self.scales[g % self.S] == g, ("another stage's operands", g)
                self.acc[b] = t
                self.issued.append(g)

    def finish(self):  # the oldest stage's MMAs end
        g = self.issued.pop(0)
        self.done = g
        self.empty[g % self.S].arrive()
        if (g + 1) % self.nk == 0:
            self.acc_full[g // self.nk % self.A].arrive()

    def epilogue(self, who, q):
        for t in range(who, self.tiles, 2):
            b = t % self.A
            yield self.acc_full[b], t // self.A
            assert self.acc[b] == t and self.done >= (t + 1) * self.nk - 1, ("another tile's sums", t)
            self.drained[t] += 1
            self.acc_empty[b].arrive()

    def run(self, rng, bias):
        """Steps a random role whose wait has passed; `bias` weighs how eager each is."""
        waits = {}
        for i, r in enumerate(self.roles):
            waits[i] = next(r, None)
        live = {i for i, w in waits.items() if w is not None}
        while live or self.issued:
            ready = [i for i in live if waits[i][0].passed(waits[i][1])]
            moves = ready + (["mma"] if self.issued else [])
            assert moves, "nobody can go on"
            m = rng.choices(moves, [bias[i] if i != "mma" else bias[-1] for i in moves])[0]
            if m == "mma":
                self.finish()
                continue
            waits[m] = next(self.roles[m], None)
            if waits[m] is None:
                live.discard(m)
        assert self.done == self.total - 1 and all(d == 4 for d in self.drained)


@pytest.mark.parametrize("stages,accs", [(4, 2), (6, 4)])
@pytest.mark.parametrize("tiles,nk", [(1, 1), (3, 1), (2, 5), (9, 2), (7, 3), (4, 8), (1, 16)])
def test_every_wait_sees_the_phase_it_means(stages, accs, tiles, nk):
    rng = random.Random(stages * 1000 + tiles * 10 + nk)
    for _ in range(60):
        m = Model(stages, accs, tiles, nk)
        m.run(rng, [10 ** rng.uniform(-2, 2) for _ in range(len(m.roles) + 1)])


def test_scale_warps_that_skip_uses_of_a_slot_are_caught():
    """Pairs of stages dealt to four warps in turn over four slots: a warp meets a slot's barrier at every second use,
    where the parity it waits for is that of the phase before the one it needs."""
    rng = random.Random(1)
    failed = 0
    for _ in range(60):
        m = Model(4, 2, 4, 8, owners=False, warps=4)
        try:
            m.run(rng, [10 ** rng.uniform(-2, 2) for _ in range(len(m.roles) + 1)])
        except AssertionError:
            failed += 1
    assert failed > 30
