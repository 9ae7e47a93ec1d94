"""Decayed linear attention refuses a state that is written where another is read: a sequence's segments
run side by side, so one could write it before another has read it (refused before anything is enqueued)."""
import ctypes

import pytest

from test_dla_cpu import FAKE, INVALID, dla_args, gcl  # noqa: F401


@pytest.mark.parametrize("backward,states,text", [
    (False, dict(h0=FAKE, ht=FAKE), b"ht must not be h0"),
    (True, dict(dht=FAKE, dh0=FAKE), b"dh0 must not be dht"),
    (True, dict(h0=FAKE, dh0=FAKE), b"dh0 must not be h0")])
def test_state_in_place_is_refused(gcl, backward, states, text):  # noqa: F811
    lib = gcl.lib()
    call = lib.dla_chunk_bwd if backward else lib.dla_chunk_fwd
    assert call(ctypes.byref(dla_args(gcl, backward, **states)), None) == INVALID
    assert text in lib.gcl_last_error()
