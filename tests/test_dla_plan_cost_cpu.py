"""The plan of the decayed attention is made on the host at every call, so its time is bounded: a few hundred candidate
lengths however long the sequence (the bar is a hundred times what they take)."""
import time

import pytest

from test_dla_cpu import gcl  # noqa: F401


@pytest.mark.parametrize("T", [1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("backward", [False, True])
def test_plan_takes_microseconds(gcl, T, backward):  # noqa: F811
    best = 1.0
    for _ in range(5):
        t0 = time.perf_counter()
        seg = gcl.dla_segment_tokens(T, 1, 1, backward)
        best = min(best, time.perf_counter() - t0)
    assert 0 < seg < T and best < 1e-3
