"""The norms around a block without a GPU: the generator's published vectors, the reference's gradients against differences,
and the refusals of the C entry points and of the binding (each before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

import glr_ref as ref
from test_dla_cpu import FAKE, gcl, rows  # noqa: F401
from test_dla_device_cpu import Tensor, cuda0  # noqa: F401

INVALID, UNSUPPORTED, CAPACITY = 1, 2, 3


def test_generator_against_published_vectors():
    """The known answers that accompany the paper's generator: zeros, ones, digits of pi."""
    for ctr, key, want in (([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
                           ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
                           ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
                            [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert ref.philox(np.array(ctr), key).tolist() == want


@pytest.mark.parametrize("post", ["none", "rms", "l2"])
@pytest.mark.parametrize("pre", ["none", "rms", "l2"])
@pytest.mark.parametrize("gate", [None, "plain", "silu", "sigmoid"])
def test_reference_gradients_match_differences(post, pre, gate):
    r = np.random.default_rng(2)
    T, H, D = 3, 2, 8
    y, x, dxo, dz, g = (r.standard_normal((T, H, D)) for _ in range(5))
    w1, w2 = r.standard_normal(D), r.standard_normal(D)
    f = 0.7 * ref.keep((T, H, D), 0.3, 5, 9)
    kind = None if gate == "plain" else gate

    def loss(y, g, x, w1, w2):
        xo, z = ref.block_fwd(y, g if gate else None, x, w1, w2, f, post, pre, kind, 1e-3)
        return (xo * dxo).sum() + (z * dz).sum()

    dy, dg, dx, dw1, dw2, _, _ = ref.block_bwd(y, g if gate else None, x, dxo, dz, w1, w2, f, post, pre, kind, 1e-3)
    args = [y, g, x, w1, w2]
    for k, grad in enumerate((dy, dg, dx, dw1, dw2)):
        d, e = r.standard_normal(args[k].shape), 1e-6
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + e * d, args[k] - e * d
        assert (loss(*up) - loss(*dn)) / (2 * e) == pytest.approx((grad * d).sum(), rel=1e-6, abs=1e-7)


def args(gcl, backward, **bad):  # noqa: F811
    H, D = 2, 72
    row = lambda: rows(gcl, H, D)  # noqa: E731
    a = dict(y=row(), gate=row(), x=row(), post_weight=FAKE, pre_weight=FAKE, t_max=100, H=H, D=D, scale=1.0, eps=1e-6, post_norm=1,
             pre_norm=1, activation=1, dtype=1, stream_dtype=1)
    if backward:
        a |= dict(dxo=row(), dz=row(), dy=row(), dgate=row(), dx=row(), dpost_weight=FAKE, dpre_weight=FAKE, workspace=FAKE,
                  workspace_bytes=1 << 40)
    else:
        a |= dict(xo=row(), z=row())
    return gcl.BlockArgs(**{**a, **bad})


@pytest.mark.parametrize("backward", [False, True])
def test_refusals(gcl, backward):  # noqa: F811
    lib = gcl.lib()
    call = lib.block_norm_bwd if backward else lib.block_norm_fwd
    assert call(None, None) == INVALID
    none = rows(gcl, 2, 72, ptr=None)
    cases = [(dict(t_max=0), INVALID, b"t_max"), (dict(t_max=1 << 31), INVALID, b"t_max"), (dict(H=0), INVALID, b"H"),
             (dict(H=65536), INVALID, b"H"), (dict(D=76), UNSUPPORTED, b"D=76"), (dict(D=16392), UNSUPPORTED, b"D=16392"),
             (dict(dtype=4, stream_dtype=4), UNSUPPORTED, b"dtype"), (dict(stream_dtype=2), UNSUPPORTED, b"stream_dtype"),
             (dict(dtype=0), UNSUPPORTED, b"stream_dtype"), (dict(post_norm=3), UNSUPPORTED, b"norm"), (dict(pre_norm=-1), UNSUPPORTED, b"norm"),
             (dict(activation=3), UNSUPPORTED, b"activation"), (dict(eps=-1.0), INVALID, b"eps"), (dict(eps=float("nan")), INVALID, b"eps"),
             (dict(dropout=1.0, ), INVALID, b"dropout"), (dict(dropout=-0.1), INVALID, b"dropout"), (dict(dropout=float("nan")), INVALID, b"dropout"),
             (dict(dropout=0.999999), INVALID, b"dropout"), (dict(dropout=0.5), INVALID, b"rng"), (dict(cu_seqlens=FAKE), INVALID, b"n_max"),
             (dict(y=none), INVALID, b"y is required"), (dict(x=rows(gcl, 2, 72, ptr=FAKE + 8)), INVALID, b"x must be 16-byte"),
             (dict(gate=rows(gcl, 2, 72, sh=76)), INVALID, b"gate strides"), (dict(post_weight=FAKE + 2), INVALID, b"16-byte")]
    if backward:
        cases += [(dict(dxo=none, dz=none), INVALID, b"dxo or dz"), (dict(dy=none), INVALID, b"dy is required"),
                  (dict(dgate=none), INVALID, b"dgate is required"), (dict(x=none), INVALID, b"dx needs x"),
                  (dict(post_weight=None), INVALID, b"gradient"), (dict(dz=none), INVALID, b"gradient"),
                  (dict(workspace=None), CAPACITY, b"workspace"), (dict(workspace_bytes=16), CAPACITY, b"workspace"),
                  (dict(dy=rows(gcl, 2, 72, st=72, sh=72)), INVALID, b"rows of dy overlap")]
    else:
        cases += [(dict(xo=none, z=none), INVALID, b"xo or z"), (dict(z=rows(gcl, 2, 72, st=72, sh=72)), INVALID, b"rows of z overlap")]
    for bad, code, text in cases:
        assert call(ctypes.byref(args(gcl, backward, **bad)), None) == code, bad
        assert text in lib.gcl_last_error(), (bad, lib.gcl_last_error())


def test_convolution_still_refuses_the_sigmoid(gcl):  # noqa: F811
    a = gcl.ConvArgs(x=FAKE, weight=FAKE, y=FAKE, cu_seqlens=FAKE, chunk_indices=FAKE, t_max=64, n_max=1, D=64, W=4, bt=64,
                     activation=2, dtype=1)
    assert gcl.lib().causal_conv1d_fwd(ctypes.byref(a), None) == UNSUPPORTED


def test_workspace_sizes(gcl):  # noqa: F811
    fn = gcl.lib().gcl_block_norm_bwd_workspace_bytes
    assert fn(ctypes.byref(gcl.BlockArgs(t_max=3, H=2, D=72))) == 6 * 2 * 72 * 4
    assert fn(ctypes.byref(gcl.BlockArgs(t_max=3, H=2, D=70))) == 0 == fn(None)


def test_binding_refusals(cuda0):  # noqa: F811
    import torch
    m = cuda0
    f = torch.float32
    x = Tensor(6, 2, 64)
    for call in (lambda **k: m.block_norm_fwd(x, Tensor(6, 64), **k), lambda **k: m.block_norm_fwd(x, x, x=Tensor(6, 2, 64, dtype=f), **k),
                 lambda **k: m.block_norm_fwd(x, x, x=Tensor(6, 2, 64, dtype=torch.float16), **k),
                 lambda **k: m.block_norm_fwd(x, x, gate=Tensor(6, 2, 64, dtype=f), **k), lambda **k: m.block_norm_fwd(x, x, activation="tanh", **k),
                 lambda **k: m.block_norm_fwd(x, x, post_norm="layer", **k), lambda **k: m.block_norm_fwd(x, x, post_weight=Tensor(64, dtype=f), **k),
                 lambda **k: m.block_norm_fwd(x, x, rng=Tensor(2, dtype=f), dropout=0.1, **k), lambda **k: m.block_norm_bwd(x, x, x, gate=x, **k),
                 # the tensors are on cuda:1, cuda:0 is current
                 lambda **k: m.block_norm_fwd(x, x, **k), lambda **k: m.block_norm_bwd(x, x, x, **k)):
        with pytest.raises(ValueError):
            call(stream=0)
    with pytest.raises(ValueError):
        m.block_norm_bwd_workspace_bytes(x)
