"""The decayed-attention operators in the bounds-checking debug build (libgcl_debug.so): short and ragged shapes
in every engine and plan run with their checked indices tested against their buffers; the status word stays 0
and the results match the references."""
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402
from test_gpu_dla import RAGGED, Case  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def debug_library():
    """Route every call of this module through the debug build, then restore the release one."""
    if not os.path.exists(gcl.DEBUG_LIB_PATH):
        pytest.fail("libgcl_debug.so not built (__graft_entry__.build() builds it)")
    saved = gcl._lib
    gcl._lib = gcl.load_library(gcl.DEBUG_LIB_PATH)
    yield
    gcl._lib = saved


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,H", [([1], 2), (RAGGED, 2), ([0, 0], 1), ([900, 0, 5], 1)], ids=["one", "ragged", "empty", "segments"])
def test_in_bounds(dtype, lens, H):
    for K, V in ((64, 128), (128, 128)):
        c = Case(dtype, lens, H, K, V, seed=31, t_pad=0)
        c.check_fwd(f"debug fwd {dtype}")              # asserts status 0 first
        c.check_bwd(f"debug bwd {dtype}")


def test_step_in_bounds():
    q, state = torch.ones(3, 2, 64, device="cuda:0"), torch.zeros(3, 2, 64, 128, device="cuda:0")
    v, o = torch.ones(3, 2, 128, device="cuda:0"), torch.empty(3, 2, 128, device="cuda:0")
    status = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    gcl.dla_step(q, q, v, torch.zeros(2, device="cuda:0"), state, o, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and (state == 1).all() and torch.allclose(o, torch.full_like(o, 8.0))
