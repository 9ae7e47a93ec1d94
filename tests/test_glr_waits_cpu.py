"""The walk of the gated linear recurrence over its spans (exchange and finish in csrc/glr_walk.cuh) as a model on the CPU: what becomes of
a cluster when waits run out.

The first block of a cluster takes the next span and sends its number to the others; a block that has it goes on, and one
that sees the end leaves.  Every wait may run out (a copy or a state that does not come, a GPU that runs something else for a while),
at any place.  The model runs a cluster's blocks as coroutines in random orders and lets waits run out at random; messages land at any time after
they were sent.  It looks for a number used before it has come, for a message to a block that has left, for blocks that part (one
goes on without the other), for walks without an end.  The cluster's barrier waits for the blocks that have not left, as the hardware's does."""
import random

import pytest

SPANS, LEAVE = 12, 3                     # LEAVE: exchanges after which a block that lost a number leaves, that one included


class Block:
    def __init__(self, rank):
        self.rank, self.here, self.arrived = rank, True, 0
        self.next, self.come = [0, 0], [0, 0]              # by parity of the tile: the number, and how many have come
        self.lost, self.err, self.tiles = 0, False, []


def run(rng, p_out=0.0, form="agreed", blind=False):
    """One random order of a cluster of two; the faults met.  form: "agreed", as the kernels are; "error": a block's first error ends all its
    waits, and the number is used without a look at whether it came.  blind: that is not a fault yet, only what comes of it."""
    blocks, mail, faults, taken = [Block(0), Block(1)], [], [], [0]

    def check(ok, what):
        if not ok:
            faults.append(what)

    def barrier(b):                      # the cluster's: everyone who has not left has arrived as often
        while any(x.here and x.arrived < b.arrived for x in blocks):
            yield False

    def out():
        return rng.random() < p_out

    def walk(b):
        unit = k = 0
        b.arrived += 1
        while True:
            buf, need = k & 1, k // 2 + 1                  # need: messages of this parity so far
            check(len(b.tiles) <= SPANS + 4, "a walk without an end")
            if faults:
                return
            b.tiles.append(unit)
            if not b.err and out():      # the rows' copies
                b.err = True
            yield True
            mine = None
            if b.rank == 0:              # takes the next span
                if form == "agreed" and b.err:
                    mine = SPANS
                else:
                    mine = taken[0] = min(taken[0] + 1, SPANS)
            yield True
            yield from barrier(b)
            if b.rank == 0:
                if form == "agreed":
                    b.next[buf], b.come[buf] = mine, need
                for x in blocks[1:] if form == "agreed" else blocks:
                    mail.append((x, buf, mine))
            yield True
            before = b.lost
            while b.come[buf] < need and not (form == "agreed" and before):     # the number of the next span
                if (form == "error" and b.err) or out():
                    break
                yield False
            lost = form == "agreed" and (before > 0 or b.come[buf] < need)
            if lost:
                b.err, b.lost = True, before + 1
                if before == 0:
                    check(blocks[0].here, "an error is set in a block that has left")
                    blocks[0].err = True
                unit = SPANS if b.lost == LEAVE else None  # (None: an empty tile)
            elif form == "error" and b.come[buf] < need:
                b.err = True
            if not b.err and out():      # the state before
                b.err = True
            yield True
            b.arrived += 1
            if not lost:
                check(blind or b.come[buf] >= need, "a number is used that has not come")
                unit = b.next[buf]
            k += 1
            if unit is not None and unit >= SPANS:
                yield from finish(b)
                return

    def finish(b):
        yield from barrier(b)
        b.arrived += 1
        yield from barrier(b)
        while form == "agreed" and b.err and any(m[0] is b for m in mail):      # (what was sent lands)
            yield False
        b.here = False

    def network():
        while True:
            if mail:
                to, buf, value = mail.pop(rng.randrange(len(mail)))
                check(to.here, "a message to a block that has left")
                to.next[buf], to.come[buf] = value, to.come[buf] + 1
                yield True
            yield False

    actors = [walk(b) for b in blocks]
    net, ready = network(), list(actors)
    weight = {a: rng.choice([1.0, 1.0, 0.05]) for a in (*actors, net)}
    idle = 0
    while ready and not faults and idle < 2000:
        a = rng.choices([*ready, net], [weight[x] for x in (*ready, net)])[0]
        moved = next(a, None)
        if moved is None:
            ready.remove(a)
        idle = idle + 1 if moved is False else 0
    check(not ready or faults, "every block waits")
    while mail and not faults:
        next(net)
    if not faults:
        first, second = (b.tiles for b in blocks)
        real = [t for t in second if t is not None]
        check(real == first[:len(real)], "the blocks walk different spans")
        check(len(first) <= len(real) + LEAVE - 1, "the first block goes on without the other")
        check(any(b.err for b in blocks) or len(first) == len(second) == SPANS, "spans are left out without an error")
    return faults


@pytest.mark.parametrize("p_out", [0.0, 0.003, 0.03, 0.3])
def test_blocks_end_together(p_out):
    rng = random.Random(4)
    for _ in range(600):
        assert run(rng, p_out) == []


def test_waits_that_do_not_run_out_hide_it():
    rng = random.Random(1)
    assert not any(run(rng, form="error") for _ in range(200))


def test_model_sees_blocks_that_part():
    """One error for all of a block's waits, and the number of two tiles ago in place of one that has not come."""
    rng = random.Random(2)
    faults = {f for _ in range(600) for f in run(rng, p_out=0.03, form="error")}
    assert "a number is used that has not come" in faults
    faults = {f for _ in range(600) for f in run(rng, p_out=0.03, form="error", blind=True)}
    assert {"a message to a block that has left", "a walk without an end"} <= faults, faults


def test_model_sees_a_block_that_leaves_at_once(monkeypatch):
    monkeypatch.setitem(globals(), "LEAVE", 1)
    rng = random.Random(3)
    assert "a message to a block that has left" in {f for _ in range(2000) for f in run(rng, p_out=0.03)}
