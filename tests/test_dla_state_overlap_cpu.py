"""States in and out of dla_chunk_fwd and _bwd that share memory at an offset are refused like equal ones: a sequence's
segments run side by side, so one could write what another has yet to read.  States side by side are not."""
import ctypes

import pytest

from test_dla_cpu import CAPACITY, FAKE, INVALID, dla_args, gcl  # noqa: F401

BYTES = 2 * 2 * 64 * 128 * 4         # the states of dla_args: n_max = 2, H = 2, K = 64, V = 128, fp32


@pytest.mark.parametrize("apart", [-BYTES + 16, -4096, 16, BYTES - 16])
@pytest.mark.parametrize("backward,out,into", [(False, "ht", "h0"), (True, "dh0", "dht"), (True, "dh0", "h0")])
def test_overlapping_states_are_refused(gcl, backward, out, into, apart):  # noqa: F811
    lib = gcl.lib()
    call = lib.dla_chunk_bwd if backward else lib.dla_chunk_fwd
    a = dla_args(gcl, backward, **{into: FAKE, out: FAKE + apart})
    assert call(ctypes.byref(a), None) == INVALID
    assert f"{out} must not be {into}".encode() in lib.gcl_last_error()


@pytest.mark.parametrize("apart", [-BYTES // 2, BYTES // 2])
@pytest.mark.parametrize("backward,out,into", [(False, "ht", "h0"), (True, "dh0", "dht"), (True, "dh0", "h0")])
def test_states_side_by_side_are_not(gcl, backward, out, into, apart):  # noqa: F811
    """One sequence, half the states.  (The workspace that is missing stops the call after the states' check.)"""
    lib = gcl.lib()
    call = lib.dla_chunk_bwd if backward else lib.dla_chunk_fwd
    a = dla_args(gcl, backward, t_max=65536, n_max=1, **{into: FAKE, out: FAKE + apart})
    assert call(ctypes.byref(a), None) == CAPACITY and b"workspace" in lib.gcl_last_error()
