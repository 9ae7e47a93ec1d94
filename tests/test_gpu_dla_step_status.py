"""A slot out of range that a call of dla_step finds itself: every other request comes out as if that one had been idle,
whichever blocks of the grid run before and after the one that sets the status word.  A word that was set before the call
stops it."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402

DEV = "cuda:0"
I32 = torch.int32
BAD_RANGE = 4


def step_inputs(B=256, H=16):
    """4,096 blocks: several waves on any GPU."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    q, k, v = (x(B, H, 64).bfloat16() for _ in range(3))
    return q, k, v, -x(H).abs(), x(B + 2, H, 64, 64), torch.randperm(B + 2, generator=gen, device=DEV)[:B].to(I32)


def step(q, k, v, g, pool, slots, status):
    pool, o, status = pool.clone(), torch.full_like(v, 7.0), torch.tensor([status], dtype=I32, device=DEV)
    gcl.dla_step(q, k, v, g, pool, o, slots=slots, dev_status=status)
    torch.cuda.synchronize()
    return pool, o, int(status.item())


@pytest.mark.parametrize("bad", [[0], [0, 17, 255]], ids=["first", "three"])
def test_step_advances_every_other_request(bad):
    q, k, v, g, pool, slots = step_inputs()
    idle, out = slots.clone(), slots.clone()
    idle[bad], out[bad] = -1, pool.shape[0]
    ref = step(q, k, v, g, pool, idle, 0)
    assert ref[2] == 0
    for _ in range(10):
        got = step(q, k, v, g, pool, out, 0)
        assert got[2] == BAD_RANGE
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("status,bad", [(BAD_RANGE, False), (2, False), (2, True)])
def test_step_with_a_set_status_does_nothing(status, bad):
    q, k, v, g, pool, slots = step_inputs()
    if bad:
        slots[100] = pool.shape[0]
    got = step(q, k, v, g, pool, slots, status)
    assert got[2] == status and torch.equal(got[0], pool) and (got[1] == 7).all()



def test_step_cannot_tell_an_earlier_bad_range_from_its_own():
    """The word holds GCL_DEV_BAD_RANGE and the call has a slot out of range itself: served as without the word."""
    q, k, v, g, pool, slots = step_inputs()
    slots[100] = pool.shape[0]
    ref, got = step(q, k, v, g, pool, slots, 0), step(q, k, v, g, pool, slots, BAD_RANGE)
    assert ref[2] == got[2] == BAD_RANGE and torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
