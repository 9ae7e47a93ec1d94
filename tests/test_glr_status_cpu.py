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


def one_span(rng, word, clusters=4, sum_by_the_first=False):
    """A backward of one span with the gradient of the rates: each cluster looks at the word and leaves the sums of its channels, a last
    launch adds them up.  sum_by_the_first: it goes by the first cluster's look alone."""
    looks = {c: word.look() for c in rng.sample(range(clusters), clusters)}
    stopped = looks[0] or not sum_by_the_first and word.look()
    return [] if stopped or not any(looks.values()) else ["sums"]


@pytest.mark.parametrize("at", range(8))
def test_sums_are_of_what_was_formed(at):
    for seed in range(50):
        assert one_span(random.Random(seed), Word(at)) == []


def test_model_sees_sums_of_what_was_not_formed():
    assert any(one_span(random.Random(s), Word(at), sum_by_the_first=True) for s in range(50) for at in range(8))


@pytest.mark.parametrize("at", range(8))
def test_the_call_goes_by_one_look(at):
    for seed in range(50):
        assert backward(random.Random(seed), Word(at)) == []


@pytest.mark.parametrize("form,read", [("states_decide", "states"), ("setup_skips", "packets")])
def test_model_sees_looks_that_differ(form, read):
    assert any(read in backward(random.Random(s), Word(at), **{form: True}) for s in range(50) for at in range(8))
