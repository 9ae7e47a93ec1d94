"""A position out of range that a call of qk_norm_rope finds itself: its rows are left alone, and every other row and the
weights' gradients come out as if it had been padding, whichever blocks run after the status word is set.  A word that was
set before the call stops it."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402

DEV = "cuda:0"
I32 = torch.int32
BAD_RANGE = 4


def norm(x, status, back):
    """Outputs of one call on x = (q, k, dyq, dyk, w, cos, sin, positions), NaN where nothing was written."""
    q, k, dyq, dyk, w, cos, sin, pos = x
    status = torch.tensor([status], dtype=I32, device=DEV)
    kw = dict(q_weight=w, k_weight=w, cos=cos, sin=sin, positions=pos, dev_status=status)
    out = [torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))]
    if back:
        dw = [torch.full((q.shape[2],), float("nan"), device=DEV) for _ in range(2)]
        ws = torch.empty(gcl.qk_norm_rope_bwd_workspace_bytes(q, k), dtype=torch.uint8, device=DEV)
        gcl.qk_norm_rope_bwd(q, k, dyq, dyk, *out, dq_weight=dw[0], dk_weight=dw[1], workspace=ws, **kw)
        out += dw
    else:
        gcl.qk_norm_rope_fwd(q, k, *out, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def norm_inputs(T):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    x = lambda *s: torch.randn(s, generator=gen, device=DEV).bfloat16()  # noqa: E731
    cos, sin = torch.empty(64, 32, device=DEV), torch.empty(64, 32, device=DEV)
    gcl.rope_table_build(cos, sin)
    pos = torch.randint(0, 64, (T,), generator=gen, device=DEV).to(I32)
    return [x(T, 16, 128), x(T, 2, 128), x(T, 16, 128), x(T, 2, 128), x(128), cos, sin, pos]


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("T", [5, 20000])
def test_norm_writes_every_other_row(T, back):
    x = norm_inputs(T)
    pos = x[-1]
    idle, out = pos.clone(), pos.clone()
    idle[[0, T - 2]], out[[0, T - 2]] = -1, 64
    ref, status = norm([*x[:-1], idle], 0, back)
    assert status == 0
    for _ in range(5):
        got, status = norm([*x[:-1], out], 0, back)
        assert status == BAD_RANGE
        for a, b in zip(got, ref):
            assert torch.equal(a.nan_to_num(123.0), b.nan_to_num(123.0))
        assert not any(a.isnan().any() for a in got[2:])


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("status,bad", [(BAD_RANGE, False), (3, True)])
def test_norm_with_a_set_status_does_nothing(status, bad, back):
    x = norm_inputs(50)
    if bad:
        x[-1][7] = 64
    got, st = norm(x, status, back)
    assert st == status and all(a.isnan().all() for a in got)


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
def test_norm_cannot_tell_an_earlier_bad_range_from_its_own(back):
    """The word holds GCL_DEV_BAD_RANGE and the call has a position out of range itself: as without the word."""
    x = norm_inputs(50)
    x[-1][7] = 64
    ref, got = norm(x, 0, back), norm(x, BAD_RANGE, back)
    assert ref[1] == got[1] == BAD_RANGE
    assert all(torch.equal(a.nan_to_num(123.0), b.nan_to_num(123.0)) for a, b in zip(ref[0], got[0]))
