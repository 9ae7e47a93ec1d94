"""The binding of the strided-row calls refuses tensors that are not on the current device, before the library is called:
it launches there and plans for its SMs.  The current device and the tensors are stand-ins; no GPU is used."""
import pytest

from test_dla_cpu import gcl  # noqa: F401


class Tensor:
    """What the binding looks at of a contiguous tensor on cuda:1."""

    def __init__(self, *shape, dtype=None):
        torch = pytest.importorskip("torch")
        self.shape, self.dtype = torch.Size(shape), dtype or torch.bfloat16
        self.device = torch.device("cuda", 1)
        self.is_cuda = True

    def get_device(self):
        return 1

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def stride(self):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st)

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return 0

    def element_size(self):
        return 1


@pytest.fixture
def cuda0(gcl, monkeypatch):  # noqa: F811
    """cuda:0 is current; a library that must not be reached."""
    class Unreached:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(gcl, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(gcl, "_devices", 2, raising=False)
    monkeypatch.setattr(gcl, "_lib", Unreached())
    return gcl


def calls(m):
    torch = pytest.importorskip("torch")
    f, i = torch.float32, torch.int32
    x, cu, g, st = Tensor(6, 2, 64), Tensor(3, dtype=i), Tensor(2, dtype=f), Tensor(6, 2, 64, 64, dtype=f)
    tab = Tensor(8, 16, dtype=f)
    return {"fwd": lambda: m.dla_chunk_fwd(x, x, x, g, cu, x, stream=0),
            "bwd": lambda: m.dla_chunk_bwd(x, x, x, g, x, cu, x, x, x, stream=0),
            "step": lambda: m.dla_step(x, x, x, g, st, x, stream=0),
            "norm": lambda: m.qk_norm_rope_fwd(x, x, x, x, stream=0),
            "norm bwd": lambda: m.qk_norm_rope_bwd(x, x, x, x, x, x, stream=0),
            "table": lambda: m.rope_table_build(tab, tab, stream=0),
            "fwd bytes": lambda: m.dla_fwd_workspace_bytes(x, x, cu),
            "bwd bytes": lambda: m.dla_bwd_workspace_bytes(x, x, cu),
            "norm bytes": lambda: m.qk_norm_rope_bwd_workspace_bytes(x, x)}


NAMES = ["fwd", "bwd", "step", "norm", "norm bwd", "table", "fwd bytes", "bwd bytes", "norm bytes"]


@pytest.mark.parametrize("name", NAMES)
def test_other_device_is_refused(cuda0, name):
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        calls(cuda0)[name]()


@pytest.mark.parametrize("name", NAMES)
def test_current_device_reaches_the_library(cuda0, monkeypatch, name):
    monkeypatch.setattr(cuda0, "_current_device", lambda: 1, raising=False)
    with pytest.raises(AssertionError, match="was called"):
        calls(cuda0)[name]()
