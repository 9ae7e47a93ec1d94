"""The example layer end to end on the GPU: its training step against torch's own differentiation of the
same layer in fp32, and decoding against the longer prefill."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decayed_linear_layer", os.path.join(ROOT, "examples", "decayed_linear_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_decoding_continues_the_prefill(example):
    """Rows pass five bf16 roundings (projection, norm, score or state, o, output), each 2^-8 at most: 5 x 2^-8.
    States: the steps' k, v come from the same rounded projections; its rows may differ by one rounding where the
    matrix product sums in another order: 2 x 2^-8."""
    r = example.run()
    assert r["decode_error"] <= 5 * 2.0 ** -8 and r["state_error"] <= 2 * 2.0 ** -8


def test_training_step_matches_torch(example):
    """Gradients of the layer by torch in fp32 (recurrence written out).  The kernels' chain rounds to bf16 about
    eight times on the way (qkv, q', k', o, d_o, dq', dk', dqkv): 8^(1/2) x 2^-8 for independent roundings, and twice that
    as the bar."""
    layer = example.DecayedLinearLayer(96, 2, 64, 32, 64, seed=3)
    lengths = [20, 1, 33]
    cu, pos = example.packed(lengths, "cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x, dy = (torch.randn(54, 96, generator=gen, device="cuda").to(layer.dtype) for _ in range(2))
    y, _, saved = layer.forward(x, pos, cu)
    got = layer.backward(dy, saved)
    p = {n: t.float().requires_grad_() for n, t in
         dict(x=x, w_in=layer.w_in, w_out=layer.w_out, q_weight=layer.q_weight, k_weight=layer.k_weight).items()}
    qkv = (p["x"] @ p["w_in"]).view(54, 3, 2, 64)
    cos, sin = layer.cos[pos.long()][:, None], layer.sin[pos.long()][:, None]

    def norm_rope(t, w):
        z = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = z[..., :16], z[..., 16:32]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, z[..., 32:]], -1)

    q, k, v = norm_rope(qkv[:, 0], p["q_weight"]), norm_rope(qkv[:, 1], p["k_weight"]), qkv[:, 2]
    o, at = [], 0
    for n in lengths:
        S = torch.zeros(2, 64, 64, device="cuda")
        for t in range(at, at + n):
            S = torch.exp(layer.g)[:, None, None] * S + k[t][:, :, None] * v[t][:, None]
            o.append(64 ** -0.5 * torch.einsum("hk,hkv->hv", q[t], S))
        at += n
    ref = torch.stack(o).reshape(54, -1) @ p["w_out"]
    ref.backward(dy.float())
    bar = 2 * 8 ** 0.5 * 2.0 ** -8
    assert float((y.float() - ref).norm() / ref.norm()) <= bar
    for n, g in got.items():
        e = float((g.float() - p[n].grad).norm() / p[n].grad.norm())
        assert e <= bar, (n, e)
