"""Host model of the fused kernel's operator modes (race detection without a GPU).

``test_pipeline_model.py`` models K-steps of whole tiles.  Here a pair's work
items have what the operators' modes add: one or two LoRA steps, each two
activation stages (the rank-r product, then its weights) that no decoder takes
part in, the first of two before the last two K-steps where an item has four or
more; items that are parts of a tile's contraction, of which only the first has
LoRA steps; tiles with one accumulator only (no more than 256 rows), whose other
one the epilogue gives back at once.  Roles are generators with the kernel's own
ring and parity arithmetic, barriers are exact.  Random interleavings check that
no stage or accumulator is overwritten before it has been read, that products
meet the stages they are meant for, that every sum is complete when it is read,
and that the run ends.

The decoders' block cursor (additions, a new look-up only at the end of an item,
of the first of two weights or of the contraction) is compared with the block
that each K-step of each item stands for.
"""
import random

import pytest

A = B = 4          # stages of the activation and the decoded ring
GROUPS, DEC, EPI, ACC = 2, 2, 2, 2


class MBar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.phase ^= 1
            self.pending = self.count

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        assert self.pending >= 0
        self._check()

    def land(self, n):
        self.tx -= n
        self._check()

    def done(self, parity):
        return self.phase != parity


def lora_early(loras, nsteps):
    return loras > 1 and nsteps >= 4


def stages(item):
    """What the item's activation stages hold, in order."""
    idx, nsteps, split, loras, nh = item
    n = loras if split == 0 else 0
    early = lora_early(loras, nsteps) and split == 0
    out = []
    for kk in range(nsteps):
        if early and kk == nsteps - 2:
            out += [(idx, "z0"), (idx, "w0")]
        out.append((idx, kk))
    for l in range(1 if early else 0, n):
        out += [(idx, f"z{l}"), (idx, f"w{l}")]
    return out


def run(items, seed, producer_order=None, keep_unused=False, late_clear=False):
    """items: (index, K-steps, split, LoRA steps of the mode, accumulators).
    The faults: a producer with another order of the stages; an epilogue that
    keeps the accumulator it does not read; an issuer that waits for the
    accumulators after an item's first product instead of before it."""
    rng = random.Random(seed)
    ctas = (0, 1)
    full_a, full_b = [MBar(1) for _ in range(A)], [MBar(2 * DEC) for _ in range(B)]
    empty_a = {q: [MBar(1) for _ in range(A)] for q in ctas}
    empty_b = {q: [MBar(1) for _ in range(B)] for q in ctas}
    tfull = {q: MBar(1) for q in ctas}
    tempty = [MBar(2 * EPI) for _ in range(ACC)]
    a_slot = {q: [None] * A for q in ctas}
    b_slot = {q: [[None] * DEC for _ in range(B)] for q in ctas}
    used_a, used_b = set(), set()
    acc = {q: [None] * ACC for q in ctas}              # (item, products) of each
    reading = {q: [0] * ACC for q in ctas}             # epilogue warps that still have to read it
    ksteps = [(it[0], kk) for it in items for kk in range(it[1])]
    moved = [0]

    def until(cond):
        while not cond():
            yield
        moved[0] += 1

    def producer(q):
        i = 0
        for it in items:
            for what in (producer_order or stages)(it):
                s, ph = i % A, (i // A) & 1
                yield from until(lambda: empty_a[q][s].done(ph ^ 1))
                if q == 0:
                    full_a[s].arrive(tx=2 * it[4])     # both CTAs' bytes, by slices
                assert a_slot[q][s] is None or a_slot[q][s] in used_a, "activation stage overwritten"
                yield
                a_slot[q][s] = what
                full_a[s].land(it[4])
                moved[0] += 1
                i += 1
                yield

    def decoder(q, g, d):
        for i in range(g, len(ksteps), GROUPS):
            s, ph = i % B, (i // B) & 1
            yield from until(lambda: empty_b[q][s].done(ph ^ 1))
            old = b_slot[q][s][d]
            assert old is None or old in used_b, "decoded stage overwritten"
            yield
            b_slot[q][s][d] = ksteps[i]
            full_b[s].arrive()
            moved[0] += 1
            yield

    def issuer():
        ia = ib = 0
        for tc, it in enumerate(items):
            order, nh = stages(it), it[4]
            n = 0
            while n < len(order):
                what = order[n]
                if isinstance(what[1], str):           # a LoRA step: two stages
                    took = []
                    for k in range(2):
                        s, ph = (ia + k) % A, ((ia + k) // A) & 1
                        yield from until(lambda: full_a[s].done(ph))
                        assert all(a_slot[q][s] == order[n + k] for q in ctas), "wrong LoRA stage"
                        took.append(s)
                    ia, n = ia + 2, n + 2
                else:
                    s, ph, sb, pb = ia % A, (ia // A) & 1, ib % B, (ib // B) & 1
                    yield from until(lambda: full_a[s].done(ph))
                    yield from until(lambda: full_b[sb].done(pb))
                    assert all(a_slot[q][s] == what for q in ctas), "wrong activation stage"
                    assert all(x == what for q in ctas for x in b_slot[q][sb]), "wrong decoded stage"
                    if what[1] == 0:
                        for h in range(ACC):
                            if not late_clear:
                                yield from until(lambda: tempty[h].done((tc & 1) ^ 1))
                            if h < nh:
                                for q in ctas:
                                    assert reading[q][h] == 0, "accumulator overwritten"
                                    acc[q][h] = [it[0], 0]
                            if late_clear:
                                yield from until(lambda: tempty[h].done((tc & 1) ^ 1))
                    took = [s]
                    ia, ib, n = ia + 1, ib + 1, n + 1
                    used_b.add(what)
                for q in ctas:
                    for h in range(nh):
                        assert acc[q][h][0] == it[0]
                        acc[q][h][1] += 1
                used_a.update(a_slot[0][s] for s in took)
                for q in ctas:                          # multicast commits
                    for s in took:
                        empty_a[q][s].arrive()
                    if not isinstance(what[1], str):
                        empty_b[q][sb].arrive()
                moved[0] += 1
                yield
            for q in ctas:
                for h in range(nh):
                    reading[q][h] = EPI
                tfull[q].arrive()

    def epilogue(q, e):
        for tc, it in enumerate(items):
            idx, nsteps, split, loras, nh = it
            yield from until(lambda: tfull[q].done(tc & 1))
            for h in range(ACC):
                if h < nh:
                    want = [idx, nsteps + (loras if split == 0 else 0)]
                    assert acc[q][h] == want, "sums incomplete when read"
                    yield
                    assert acc[q][h] == want, "sums changed while read"
                    reading[q][h] -= 1
                elif keep_unused:
                    continue
                tempty[h].arrive()
                moved[0] += 1
                yield

    roles = [producer(0), producer(1), issuer(), *(decoder(q, g, d) for q in ctas for g in range(GROUPS)
                                                   for d in range(DEC)),
             *(epilogue(q, e) for q in ctas for e in range(EPI))]
    weight = [rng.random() ** 3 + 0.02 for _ in roles]     # some much slower than others
    idle = 0
    while roles:
        i = rng.choices(range(len(roles)), weight)[0]
        before = moved[0]
        try:
            next(roles[i])
        except StopIteration:
            roles.pop(i)
            weight.pop(i)
            moved[0] += 1
        idle = 0 if moved[0] != before else idle + 1
        assert idle < 20000, "no progress"


def draw(rng, loras, splits):
    """The items of one pair: tiles of one contraction, whole or in equal parts."""
    nsteps = rng.choice((1, 2, 3, 4, 5, 7))
    return [(i, nsteps, rng.randrange(splits), loras, rng.choice((1, 2))) for i in range(rng.choice((1, 2, 4)))]


# the modes: gated forward (two LoRA steps), gated dX (two, split), the loss's
# forward modes (none), its dX (none, split), the layer (one)
@pytest.mark.parametrize("loras,splits", [(2, 1), (2, 3), (0, 1), (0, 3), (1, 1)])
@pytest.mark.parametrize("seed", range(12))
def test_protocol(loras, splits, seed):
    rng = random.Random(100 * seed + 10 * loras + splits)
    run(draw(rng, loras, splits), seed)


def caught(**fault):
    n = 0
    for seed in range(10):
        try:
            run([(i, 5, 0, 2, 1 + i % 2) for i in range(4)], seed, **fault)
        except AssertionError:
            n += 1
    return n


def test_a_producer_with_another_order_is_caught():
    """Both LoRA steps at the end while the issuer takes the first one early."""
    def late(item):
        order = stages(item)
        k = [w for w in order if not isinstance(w[1], str)]
        return k + [w for w in order if isinstance(w[1], str)]
    assert caught(producer_order=late) == 10


def test_an_unused_accumulator_that_is_kept_is_caught():
    assert caught(keep_unused=True) == 10


def test_a_late_wait_for_the_accumulators_is_caught():
    assert caught(late_clear=True) > 0


# --------------------------------------------------------------------------
# the decoders' cursor
# --------------------------------------------------------------------------
class Shape:
    """The contraction of a mode that may be split: nk K-steps (of both weights with
    two), `steps` an item; a weight row has `bpr` blocks."""

    def __init__(self, nk, splits, two, m_tiles, n_tiles, rows):
        self.nk, self.splits, self.two = nk, splits, two
        self.steps = -(-nk // splits)
        self.m_tiles, self.n_tiles, self.rows = m_tiles, n_tiles, rows
        self.bpr = nk // 2 if two else nk
        self.tiles = m_tiles * n_tiles


def block(a, item, kk, R, rank):
    """(weight, block) of row R of the decoded tile at K-step kk of an item, None where
    there is none."""
    split, tile = divmod(item, a.tiles)
    row = tile // a.m_tiles * 256 + 128 * rank + R
    k = split * a.steps + kk
    if k >= a.nk or row >= a.rows:
        return None
    second = a.two and k >= a.nk // 2
    return int(second), row * a.bpr + (k - a.nk // 2 if second else k)


def seek(a, c, R, rank, num_items):
    c.update(valid=False, second=False, until=a.steps, blk=0, stride=0)
    if c["item"] >= num_items:
        return
    split, tile = divmod(c["item"], a.tiles)
    kk = c["kk"] + split * a.steps
    if kk >= a.nk:
        return
    c["until"] = min(c["until"], a.nk - split * a.steps)
    if a.two:
        half = a.nk // 2
        if kk >= half:
            c["second"] = True
            kk -= half
        elif half - split * a.steps < c["until"]:
            c["until"] = half - split * a.steps
    row = tile // a.m_tiles * 256 + 128 * rank + R
    if row >= a.rows:
        return
    c.update(valid=True, blk=row * a.bpr + kk, stride=1)


def advance(a, c, n, R, rank, num_items, stride):
    c["kk"] += n
    c["blk"] += n * c["stride"]
    if c["kk"] >= c["until"]:
        while c["kk"] >= a.steps:
            c["kk"] -= a.steps
            c["item"] += stride
        seek(a, c, R, rank, num_items)


@pytest.mark.parametrize("nk,splits", [(2, 1), (6, 1), (16, 2), (38, 4), (86, 10), (344, 4), (346, 4), (20, 7)])
@pytest.mark.parametrize("two", [True, False])
def test_cursor(nk, splits, two):
    for m_tiles, n_tiles, rows, npairs in ((1, 1, 192, 1), (1, 5, 1088, 3), (3, 2, 300, 4), (2, 3, 768, 74)):
        a = Shape(nk, splits, two, m_tiles, n_tiles, rows)
        num = a.tiles * splits
        for pair in range(min(npairs, num)):
            mine = [(i, kk) for i in range(pair, num, npairs) for kk in range(a.steps)]
            for grp in range(GROUPS):
                for R, rank in ((0, 0), (127, 0), (0, 1), (64, 1)):
                    c = {"item": pair + grp // a.steps * npairs, "kk": grp % a.steps}
                    seek(a, c, R, rank, num)
                    for i in range(grp, len(mine), GROUPS):
                        got = (int(c["second"]), c["blk"]) if c["valid"] else None
                        assert got == block(a, *mine[i], R, rank), (mine[i], R, rank)
                        advance(a, c, GROUPS, R, rank, num, npairs)
                    # past the pair's last step it loads nothing
                    assert not c["valid"]
