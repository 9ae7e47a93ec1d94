"""The status word during a call of the gated linear recurrence (csrc/glr.cu, csrc/glr_walk.cuh) as a model on the CPU.

A call is several launches of several blocks, and another stream's call may set a shared status word at any time between their looks at
it.  What is not formed then is not to be used: a call that goes on has formed all that it reads.  The model runs a call's blocks in
random orders, sets the word before one of the looks, and names what was read without having been formed."""
import random

import pytest


class Word:
    """Set before the look number `at`."""

    def __init__(self, at):
        self.left, self.value = at, False

    def look(self):
        self.value = self.value or self.left <= 0
        self.left -= 1
        return self.value


def backward(rng, word, blocks=4, states_decide=False, setup_skips=False):
    """A backward of several spans that forms the states itself: set-up, the walk that forms the states, the walk of the gradients.
    states_decide: the states' walk, of one span, looks at the word for itself.  setup_skips: a block of the set-up that sees the word set
    leaves its share of the packets and borders as they were."""
    looks = {b: word.look() for b in rng.sample(range(blocks), blocks)}
    stopped = looks[0]                                     # what the set-up leaves the walks
    if stopped:
        return []
    formed = not (word.look() if states_decide else stopped)
    return ["packets"] * (setup_skips and any(looks.values())) + ["states"] * (not formed)


@pytest.mark.parametrize("at", range(8))
def test_the_call_goes_by_one_look(at):
    for seed in range(50):
        assert backward(random.Random(seed), Word(at)) == []


@pytest.mark.parametrize("form,read", [("states_decide", "states"), ("setup_skips", "packets")])
def test_model_sees_looks_that_differ(form, read):
    assert any(read in backward(random.Random(s), Word(at), **{form: True}) for s in range(50) for at in range(8))
