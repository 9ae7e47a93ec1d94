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


def backward(rng, word, blocks=4, states_decide=False):
    """A backward of several spans that forms the states itself: set-up, the walk that forms the states, the walk of the gradients.
    states_decide: the states' walk, of one span, looks at the word for itself."""
    looks = {b: word.look() for b in rng.sample(range(blocks), blocks)}
    stopped = looks[0]                                     # what the set-up leaves the walks
    formed = not (word.look() if states_decide else stopped)
    return [] if stopped or formed else ["states"]


@pytest.mark.parametrize("at", range(8))
def test_the_states_walk_goes_by_the_set_ups_look(at):
    for seed in range(50):
        assert backward(random.Random(seed), Word(at)) == []


def test_model_sees_a_walk_that_looks_for_itself():
    assert any(backward(random.Random(s), Word(at), states_decide=True) for s in range(50) for at in range(8))
