"""The waits of the own-state kernel of decayed linear attention (dla_own_kernel, csrc/dla_tc.cu) as a model on the CPU.

An mbarrier wait tests one bit: a wait for phase n passes whenever the barrier's phase in progress has the other parity,
be it n + 1 (phase n is complete) or n - 1 (it is two completions away).  So every wait has to be for a phase whose next
one cannot complete, and whose previous one is known to be complete, before the waiter has passed.  The model runs
the kernel's warps as coroutines in random orders, with one of them often far slower than the rest, and looks at each
step whether what the wait stands for has happened: tiles read before they are overwritten, split buffers read before
they are written again, every MMA done before the sum is read and its tiles are reused."""
import random

import pytest

TILES, BUFS, MEMBERS = 3, 4, 2          # tiles, split buffers, warps of each split group (the kernel has eight)


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1

    def passes(self, phase):             # what mbarrier.test_wait.parity answers
        return (self.done & 1) != (phase & 1)


def run(nch, rng, final="end", loader="empty"):
    """One random order of a segment of nch chunks; the faults met.  final: the barrier that the split warps wait on
    before they read the sum; loader: the one that frees a tile."""
    full, empty = [Bar(1) for _ in range(TILES)], [Bar(1) for _ in range(TILES)]
    split, free = [Bar(MEMBERS) for _ in range(BUFS)], [Bar(1) for _ in range(BUFS)]
    end, faults, pipe = Bar(1), [], []
    mma_done, b_read, tile, in_flight = set(), set(), [None] * TILES, []

    def check(ok, what):
        if not ok:
            faults.append(what)

    def wait(bar, phase):
        while not bar.passes(phase):
            yield False
        check(bar.done > phase, f"phase {phase} passed with {bar.done} complete")

    def load():
        for ic in range(nch):
            s = ic % TILES
            if ic >= TILES:
                yield from (wait(empty[s], ic // TILES - 1) if loader == "empty" else wait(free[-1], ic - TILES))
                old = ic - TILES
                check(all((old, q) in mma_done for q in range(BUFS)), f"tile of chunk {old} overwritten before its MMAs")
                check(sum(x[0] == old for x in b_read) == BUFS * MEMBERS, f"tile of chunk {old} overwritten before its split")
            in_flight.append((s, ic))
            yield True

    def copies():
        for ic in range(nch):
            while not in_flight:
                yield False
            s, c = in_flight.pop(0)
            tile[s] = c
            full[s].arrive()
            yield True

    def issue():
        for ic in range(nch):
            s = ic % TILES
            yield from wait(full[s], ic // TILES)
            for q in range(BUFS):
                yield from wait(split[q], ic)
                pipe.append((ic, q))
                pipe.append(free[q])
                yield True
            if loader == "empty":
                pipe.append(empty[s])
        pipe.append(end)

    def tensor():
        for _ in range(nch * (2 * BUFS + (loader == "empty")) + 1):
            while not pipe:
                yield False
            x = pipe.pop(0)
            if isinstance(x, Bar):
                x.arrive()
            else:
                check(tile[x[0] % TILES] == x[0], f"MMA {x} reads another chunk's tile")
                mma_done.add(x)
            yield True

    def splitter(odd, member):
        for ic in range(nch):
            yield from wait(full[ic % TILES], ic // TILES)
            for q in range(odd, BUFS, 2):
                if ic > 0:
                    yield from wait(free[q], ic - 1)
                    check((ic - 1, q) in mma_done, f"split buffer {q} of chunk {ic - 1} overwritten")
                check(tile[ic % TILES] == ic, f"split of chunk {ic} reads another chunk's tile")
                b_read.add((ic, q, member))
                split[q].arrive()
                yield True
        yield from (wait(end, 0) if final == "end" else wait(free[-1], nch - 1))
        check(len(mma_done) == nch * BUFS, "the sum is read before its last MMA")
        check(len(b_read) == nch * BUFS * MEMBERS, "tiles are reused before they are split")

    actors = [load(), copies(), issue(), tensor(), *(splitter(o, m) for o in (0, 1) for m in range(MEMBERS))]
    weight = {a: rng.choice([1.0, 1.0, 0.01]) for a in actors}
    ready, idle = list(actors), []       # idle: the last poll found nothing to do
    while ready:
        a = rng.choices(ready, [weight[x] for x in ready])[0]
        moved = next(a, None)            # None: the warp is through
        if moved is False:
            idle.append(a)
            ready.remove(a)
            continue
        if moved is None:
            ready.remove(a)
        ready, idle = ready + idle, []
    check(not idle, "every warp waits")
    return faults


@pytest.mark.parametrize("nch", [1, 2, 3, 4, 5, 7, 8, 13])
def test_waits_are_sound(nch):
    rng = random.Random(nch)
    for _ in range(100):
        assert run(nch, rng) == []


@pytest.mark.parametrize("nch", [2, 3, 8])
def test_model_sees_a_final_wait_that_passes_a_phase_early(nch):
    """The final wait on the last split buffer's barrier instead, which the warps of the even steps have not waited on
    before: its parity passes while the MMAs of the chunk before are still pending."""
    rng = random.Random(nch)
    faults = [f for _ in range(200) for f in run(nch, rng, final="free")]
    assert "the sum is read before its last MMA" in faults and "tiles are reused before they are split" in faults
    assert any("passed with" in f for f in faults)


def test_one_chunk_hides_it():
    """With one chunk the last buffer's barrier has no phase before: such segments do not show the fault above."""
    rng = random.Random(0)
    assert not any(run(1, rng, final="free") for _ in range(100))


def test_a_late_loader_stays_sound_but_stalls():
    """The loader on the last buffer's barrier: never early, but two phases late it waits for the chunk after, so a
    tile's own barrier takes its place."""
    rng = random.Random(1)
    assert not any(run(9, rng, loader="free") for _ in range(100))
