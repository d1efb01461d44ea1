"""The operand ring and the two overlapping accumulators of the 4-bit products, as
a model on the host: the barriers, the producers, the MMA issuer and the epilogue
warps of a CTA pair under schedules that hold one of them back.  A wait for a phase's parity is only sound while the waiter is at most
one phase behind, so every producer has to be needed for every phase, also where
it has nothing to copy (a row tile that ends in the first CTA)."""

import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_moe_gate_gb300", "csrc",
                   "ffn_fp4.cuh")


def full_arrivals():
    """What the kernel initialises a stage's full barrier with."""
    src = open(SRC).read()
    count = re.search(r"mbar_init\(&ctl->full\[s\], (\w+)\)", src).group(1)
    if not count.isdigit():
        count = re.search(rf"constexpr int {count} = (\d+);", src).group(1)
    return int(count)


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.tx, self.done = count, count, 0, 0

    def arrive(self, tx=0):
        self.left -= 1
        self.tx += tx
        self.settle()

    def complete(self, n):
        self.tx -= n
        self.settle()

    def settle(self):
        assert self.left >= 0
        if self.left == 0 and self.tx == 0:
            self.left, self.done = self.count, self.done + 1

    def passed(self, parity):   # mbarrier.try_wait.parity
        return (self.done & 1) != parity


def run_ring(rows, stages, nk, arrivals, first, rng):
    """Tiles of `rows` kept rows, nk stages each; `first`: actors in order of
    priority (the others at random).  Whether all of them finish, with every
    stage read holding the copies meant for it."""
    full = [Barrier(arrivals) for _ in range(stages)]
    tfull, tempty = [Barrier(1), Barrier(1)], Barrier(4)   # one epilogue warp per CTA and column half
    columns = {}     # 32-column chunk of TMEM -> the tile whose sums it holds
    empty = [[Barrier(1) for _ in range(stages)] for _ in range(2)]
    slots = {}       # (stage, cta, producer) -> the use its content belongs to
    copies = []      # in flight

    def boxes(r, cta, hh):   # 32-row boxes of A with kept rows
        return min(max(-(-(r - hh * 64 - cta * 128) // 32), 0), 2)

    def producer(cta, prod):
        use, is_a, hh = 0, prod % 2 == 0, prod // 2
        for r in rows:
            mine = boxes(r, cta, hh) + (hh == 0 and boxes(r, cta, 0) > 0) if is_a else 2
            both = sum(boxes(r, c, hh) + (hh == 0 and boxes(r, c, 0) > 0) for c in (0, 1)) if is_a else 4
            for _ in range(nk):
                s, ph = use % stages, use // stages & 1
                while not empty[cta][s].passed(ph ^ 1):
                    yield False
                if cta == 0:
                    full[s].arrive(both)
                elif is_a and arrivals > 4:
                    full[s].arrive()
                if mine:
                    copies.append((s, cta, prod, use, mine))
                use += 1
                yield True

    def issuer():
        use = 0
        for t, r in enumerate(rows):
            while t and not tempty.passed(t - 1 & 1):
                yield False
            columns.update({(t & 1) * 6 + c: t for c in range(8)})
            for _ in range(nk):
                s, ph = use % stages, use // stages & 1
                while not full[s].passed(ph):
                    yield False
                for cta in (0, 1):
                    for prod in range(4):
                        if prod % 2 or boxes(r, cta, prod // 2):
                            assert slots.get((s, cta, prod)) == use, "a stage read before its copies"
                for cta in (0, 1):
                    empty[cta][s].arrive()
                use += 1
                yield True
            for cta in (0, 1):
                tfull[cta].arrive()
            yield True

    def epilogue(cta, half):
        for t in range(len(rows)):
            while not tfull[cta].passed(t & 1):
                yield False
            first = half if t & 1 else 6 + half   # in the columns that the next tile shares
            for i in range(4):
                assert columns[(t & 1) * 6 + (first + 2 * i & 7)] == t, "an accumulator overwritten before it was read"
                if i == 0:
                    tempty.arrive()
                yield True

    actors = {("p", c, i): producer(c, i) for c in (0, 1) for i in range(4)}
    actors["mma"] = issuer()
    actors.update({("e", c, h): epilogue(c, h) for c in (0, 1) for h in (0, 1)})
    while actors:
        if copies and rng.random() < 0.5:
            s, cta, prod, use, n = copies.pop(rng.randrange(len(copies)))
            slots[s, cta, prod] = use
            full[s].complete(n)
            continue
        order = list(actors)
        rng.shuffle(order)
        order.sort(key=lambda a: first.index(a) if a in first else len(first))
        for a in order:
            moved = next(actors[a], None)
            if moved is None:
                del actors[a]
            if moved is None or moved:
                break
        else:
            if not copies:
                return False   # nobody can go on: on the device a bounded wait runs out
    return True


ALL = [("p", c, i) for c in (0, 1) for i in range(4)] + ["mma"] + [("e", c, h) for c in (0, 1) for h in (0, 1)]


@pytest.mark.parametrize("stages", [5, 6])
@pytest.mark.parametrize("rows", [[16] * 6, [256, 100, 100, 100, 256], [128, 129, 200, 64, 65, 1]], ids=str)
@pytest.mark.parametrize("last", ALL, ids=str)
def test_a_producer_that_is_held_back_is_waited_for(stages, rows, last):
    first = [a for a in ALL if a != last]   # `last` moves only when nothing else can
    for seed in range(4):
        assert run_ring(rows, stages, 16, full_arrivals(), first, random.Random(seed))


def test_random_schedules():
    for seed in range(30):
        rng = random.Random(seed)
        rows = [rng.randint(1, 256) for _ in range(rng.randint(1, 8))]
        assert run_ring(rows, rng.choice((5, 6)), rng.randint(1, 17), full_arrivals(), [], rng)


def test_the_model_shows_the_lap():
    """Four arrivals alone, those of the first CTA: an idle producer is lapped."""
    first = [a for a in ALL if a != ("p", 1, 0)]
    assert not run_ring([16] * 6, 5, 16, 4, first, random.Random(0))


def test_lag_hook_arguments():
    import combine_moe_gate_gb300 as M

    lib = M.load()
    assert lib.moe_debug_lag_gemms(-1) == M.MOE_ERR_INVALID_ARG
    assert lib.moe_debug_lag_gemms(2) == M.MOE_OK
    assert lib.moe_debug_lag_gemms(0) == M.MOE_OK
    with pytest.raises(M.MoEError):
        M.moe_debug_lag_gemms(-1)
