"""Host model of the few-rows gated kernel's mbarrier protocol (race detection
without a GPU).

``gated_rows_kernel`` streams a run of units through three rings: packed bytes
and scales (8 stages), X (3 to 8), decoded weights (3, one per turn of
decoders); two warps issue one half each of every unit's products; four warps
load scales and read the sums of each segment.  The roles are generators with
the kernel's own index arithmetic; an mbarrier is exact (pending arrivals,
phase bit, try_wait(parity) true once a phase of that parity has completed and
the next has not).  Random interleavings check that no stage is overwritten or
read out of turn, that every product sees the unit it is meant for, that no
barrier receives more arrivals than it counts, and that the run ends.
"""
import random

import pytest

PK, W, TURNS, SCALE, MMA, LOOK = 8, 3, 3, 4, 2, 4


class MBar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.phase ^= 1
            self.pending = self.count

    def done(self, parity):
        return self.phase != parity


def run(u0, u1, nk, weights, nx, nbuf, seed, alternate_units=False):
    """weights: units below it are weights, from it on adapters."""
    rng = random.Random(seed)
    full, empty = [MBar(1) for _ in range(W)], [MBar(MMA) for _ in range(W)]
    pfull, pempty = [MBar(2) for _ in range(PK)], [MBar(1) for _ in range(PK)]
    xfull, xempty = [MBar(1) for _ in range(nx)], [MBar(MMA) for _ in range(nx)]
    if alternate_units:
        empty, xempty = [MBar(1) for _ in range(W)], [MBar(1) for _ in range(nx)]
    tfull, tempty = [MBar(MMA) for _ in range(2)], [MBar(SCALE) for _ in range(2)]
    packed, scale, xs_, dec = [None] * PK, [None] * PK, [None] * nx, [None] * W
    acc = {}
    sums = []
    uw = min(u1, weights)

    def tma_packed():
        s, ph = 0, 1
        for u in range(u0, uw):
            while not pempty[s].done(ph):
                yield
            packed[s] = u
            yield
            pfull[s].arrive()
            s += 1
            if s == PK:
                s, ph = 0, ph ^ 1

    def tma_x():
        s, ph = 0, 1
        for u in range(u0, u1):
            while not xempty[s].done(ph):
                yield
            xs_[s] = u
            yield
            xfull[s].arrive()
            s += 1
            if s == nx:
                s, ph = 0, ph ^ 1

    def decoders(turn):
        ph, ps, pph = 1, turn, 0
        for u in range(u0 + turn, u1, TURNS):
            if u < uw:
                while not pfull[ps].done(pph):
                    yield
                assert packed[ps] == u and scale[ps] == u
                yield
            while not empty[turn].done(ph):
                yield
            dec[turn] = u
            yield
            full[turn].arrive()
            if u < uw:
                pempty[ps].arrive()
            ph ^= 1
            ps += TURNS
            if ps >= PK:
                ps, pph = ps - PK, pph ^ 1
            yield

    def segments():
        ua = u0
        while ua < u1:
            ub = min(u1, (ua // nk + 1) * nk)
            yield ua, ub
            ua = ub

    def mma(m):
        s = ph = x = xph = 0
        b, tph = 0, 1
        for ua, ub in segments():
            while not tempty[b].done(tph):
                yield
            acc[b, m] = []
            for u in range(ua, ub):
                if alternate_units and (u - u0) % 2 != m:
                    s, ph = ((s + 1) % W, ph ^ (s + 1 == W))
                    x, xph = ((x + 1) % nx, xph ^ (x + 1 == nx))
                    continue
                while not xfull[x].done(xph):
                    yield
                while not full[s].done(ph):
                    yield
                assert xs_[x] == u and dec[s] == u
                acc[b, m].append(u)
                yield
                assert xs_[x] == u and dec[s] == u     # the products read them until here
                empty[s].arrive()
                xempty[x].arrive()
                s, ph = ((s + 1) % W, ph ^ (s + 1 == W))
                x, xph = ((x + 1) % nx, xph ^ (x + 1 == nx))
                yield
            tfull[b].arrive()
            b += 1
            if b == nbuf:
                b, tph = 0, tph ^ 1

    def scales(q):
        us, ps, pph, b, tph = u0 + q, q, 1, 0, 0
        segs = list(segments())
        while True:
            if us < uw and (not segs or us < segs[0][1] + LOOK):
                while not pempty[ps].done(pph):
                    yield
                scale[ps] = us
                yield
                pfull[ps].arrive()
                us += SCALE
                ps += SCALE
                if ps >= PK:
                    ps, pph = ps - PK, pph ^ 1
            elif segs:
                ua, ub = segs.pop(0)
                while not tfull[b].done(tph):
                    yield
                if not alternate_units:
                    assert acc[b, 0] == acc[b, 1] == list(range(ua, ub))
                sums.append((q, ua, ub))
                yield
                tempty[b].arrive()
                b += 1
                if b == nbuf:
                    b, tph = 0, tph ^ 1
            else:
                return
            yield

    roles = [tma_packed(), tma_x(), *(decoders(t) for t in range(TURNS)), *(mma(m) for m in range(MMA)),
             *(scales(q) for q in range(SCALE))]
    weight = [rng.random() ** 3 + 0.01 for _ in roles]      # some agents much slower than others
    idle = 0
    while roles:
        i = rng.choices(range(len(roles)), weight)[0]
        before = [b.phase for b in full + empty + pfull + pempty + xfull + xempty + tfull + tempty]
        try:
            next(roles[i])
        except StopIteration:
            roles.pop(i)
            weight.pop(i)
        idle = 0 if before != [b.phase for b in full + empty + pfull + pempty + xfull + xempty + tfull + tempty] else idle + 1
        assert idle < 60000, "no progress"
    assert len(sums) == SCALE * len(list(segments()))


@pytest.mark.parametrize("seed", range(60))
def test_protocol(seed):
    rng = random.Random(1000 + seed)
    nk = rng.choice((1, 2, 3, 5, 9, 16))
    per = rng.choice((2, 3, 7, 20, 40))
    u0 = rng.randrange(0, 4 * nk)
    weights = rng.choice((u0, u0 + per // 2, u0 + per, u0 + 100))
    weights = -(-weights // nk) * nk                         # whole groups
    run(u0, u0 + per, nk, weights, rng.choice((3, 4, 5, 8)), rng.choice((1, 2)), seed)


def test_alternate_units_per_warp_is_caught():
    """Two issuing warps that take every other unit of a three-stage ring skip
    phases, and a parity wait lets them through early."""
    caught = 0
    for seed in range(20):
        try:
            run(0, 40, 64, 1000, 8, 2, seed, alternate_units=True)
        except AssertionError:
            caught += 1
    assert caught > 0
