"""The operators of a gated recurrent block together (examples/gated_recurrent_block.py): a training step against torch's
gradients in fp64, decoding against the longer prefill; and the bounds-checking build on their kernels."""
import importlib.util
import os

import numpy as np
import pytest

import glr_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("gated_recurrent_block", os.path.join(ROOT, "examples", "gated_recurrent_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rms(x, w):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def plain(block, w, x, lengths, mask):
    """The block in elementary operations; w: its weights with rate."""
    z = rms(x, w["first"])
    xin, gates = z @ w["x"], z @ w["gates"]
    r, i, g = gates.chunk(3, -1)
    taps = w["conv"].shape[1]
    cs, hs, at = [], [], 0
    for n in lengths:
        s = torch.cat([xin.new_zeros(taps - 1, block.D), xin[at:at + n]])
        c = sum(s[j:j + n] * w["conv"][:, j] for j in range(taps))
        la = -w["rate"] * torch.sigmoid(r[at:at + n])
        u = torch.sqrt(-torch.expm1(2 * la)) * c * torch.sigmoid(i[at:at + n])
        h, rows = u.new_zeros(block.D), []
        for t in range(n):
            h = la[t].exp() * h + u[t]
            rows.append(h)
        hs.append(torch.stack(rows))
        at += n
    h = torch.cat(hs)
    y = rms(h.view(-1, block.H, block.dim), w["head"]).reshape(h.shape) * torch.nn.functional.silu(g)
    xo = x + block.scale * mask * rms(y @ w["out"], w["post"])
    return xo, rms(xo, w["pre"])


def test_training_step_matches_torch():
    m = example()
    lengths, width = [70, 1, 33], 96
    block = m.GatedRecurrentBlock(width, 2, 72, dropout=0.3, dtype=torch.float32, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    T = sum(lengths)
    x, dxo, dzo = (torch.randn(T, width, generator=gen, device="cuda") for _ in range(3))
    block.rng[1] = 5
    cu = m.packed(lengths, "cuda")
    xo, zo, _, saved = block.forward(x, cu)
    grads = block.backward(dxo, dzo, saved)
    torch.cuda.synchronize()
    assert int(block.status.item()) == 0
    w = {k: v.double().requires_grad_() for k, v in {**block.w, "rate": block.rate}.items()}
    xd = x.double().requires_grad_()
    mask = torch.from_numpy(ref.keep((T, width), 0.3, *block.rng.tolist())).cuda()
    xr, zr = plain(block, w, xd, lengths, mask)
    ((xr * dxo.double()).sum() + (zr * dzo.double()).sum()).backward()
    # fp32 throughout: a product of `width` or D terms and some ten operators one after the other, each with its 1e-6
    bar = 2e-5
    for name, got, want in [("xo", xo, xr), ("zo", zo, zr), ("stream", grads["stream"], xd.grad), *((k, grads[k], v.grad) for k, v in w.items())]:
        e = float((got.double() - want.detach()).norm() / want.detach().norm())
        assert e <= bar, (name, e)


def test_example_runs_and_decoding_follows_the_prefill():
    r = example().run(width=128, heads=2, dim=64, lengths=(150, 1, 40), new_tokens=3)
    assert r["decode_error"] <= 5 * 2.0 ** -8, r["decode_error"]
    assert all(bool(torch.isfinite(g).all()) and bool((g != 0).any()) for g in r["grads"].values())


@pytest.fixture
def debug_library():
    if not os.path.exists(gcl.DEBUG_LIB_PATH):
        pytest.fail("libgcl_debug.so not built (__graft_entry__.build() builds it)")
    saved = gcl._lib
    gcl._lib = gcl.load_library(gcl.DEBUG_LIB_PATH)
    yield
    gcl._lib = saved


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_bounds(debug_library, dtype):
    from test_gpu_block_norm import Case as Norm
    from test_gpu_glr import Case
    for lens in ([1], [128, 0, 256], [300, 7, 0, 61]):
        c = Case(dtype, lens, 72, "power", "root", True)
        c.fwd()
        c.check_fwd()
        c.check_bwd(c.bwd(c.save))
        c.check_bwd(c.bwd())
    for D in (72, 1000, 4104, 16384):
        Norm(5, 1, D, dtype, p=0.1, live=4).check()
    Norm(5, 6, 128, dtype, x=False, z=False).check()


def test_two_operators_on_two_streams():
    """The norm of one batch beside the recurrence of another, each with workspaces of its own."""
    from test_gpu_block_norm import Case as Norm
    from test_gpu_glr import Case
    a, b = Case("bf16", [4000, 500], 520, "sigmoid", "complement", True), Norm(3000, 1, 2048, p=0.2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(streams[0]):
            a.fwd()
            grads = a.bwd(a.save)
        with torch.cuda.stream(streams[1]):
            b.fwd()
            out = b.bwd()
    torch.cuda.synchronize()
    a.check_fwd()
    a.check_bwd(grads)
    b.check_fwd()
    b.check_bwd(out)
    assert np.isfinite(grads["dx"].float().cpu().numpy()[:4500]).all()
