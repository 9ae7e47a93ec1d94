"""Decayed linear attention with growing states (g > 0): finite as long as exp(g n) is finite over a sequence's own n
tokens, though it is not over a whole chunk.  Tolerances of tests/dla_ref.py: exp(g n) is off by half a step of g n, 2^-18
at g n < 128 (3.8e-6), within the states' 1e-5."""
import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("torch")
from test_gpu_dla import DIMS, Case  # noqa: E402


@pytest.mark.parametrize("dims", DIMS, ids=lambda d: f"{d[0]}x{d[1]}")
@pytest.mark.parametrize("dtype,g,lens", [("bf16", 0.75, [97, 0, 33, 1]), ("f32", 1.5, [40, 0, 33, 1])], ids=["bf16", "f32"])
def test_growing_states(dtype, g, lens, dims):
    """bf16: exp(128 g) is infinite, exp(97 g) 4e31; fp32: exp(64 g) is 5e41, exp(40 g) 1e26."""
    c = Case(dtype, lens, 2, *dims, seed=14, g=[g, 0.5 * g])
    c.check_fwd(f"growing {dtype} {dims}")
    c.check_bwd(f"growing {dtype} {dims}")
