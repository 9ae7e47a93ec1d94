"""The gated linear recurrence without a GPU: the reference's gradients against differences of its forward, workspace
sizes, and the refusals of the C entry points and of the binding (each before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

import glr_ref
from test_dla_cpu import FAKE, gcl  # noqa: F401
from test_dla_device_cpu import Tensor, cuda0  # noqa: F401

INVALID, UNSUPPORTED, CAPACITY = 1, 2, 3


@pytest.mark.parametrize("decay", ["log", "sigmoid", "power"])
@pytest.mark.parametrize("mix", ["one", "complement", "root"])
@pytest.mark.parametrize("gate", [False, True])
def test_reference_gradients_match_differences(decay, mix, gate):
    r = np.random.default_rng(0)
    T, D, cu = 9, 5, [0, 4, 4, 9]
    x, i, h0, dht, d_o = (r.standard_normal(s) for s in ((T, D), (T, D), (3, D), (3, D), (T, D)))
    rr = -np.exp(r.standard_normal((T, D)) - 1) if decay == "log" else r.standard_normal((T, D))
    rate = r.random(D) + 0.1
    if not gate:
        i = None

    def loss(x, rr, i, rate, h0):
        h, _, ht = glr_ref.fwd(x, rr, i, rate, h0, cu, decay, mix)
        return (h * d_o).sum() + (ht * dht).sum()

    dx, dr, di, drate, dh0, _ = glr_ref.bwd(x, rr, i, rate, h0, d_o, dht, cu, decay, mix)
    if decay != "power":
        drate = np.zeros(D)
    args = [x, rr, i, rate, h0]
    for k, g in enumerate((dx, dr, di, drate, dh0)):
        if args[k] is None:
            continue
        d, e = r.standard_normal(args[k].shape), 1e-6
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + e * d, args[k] - e * d
        assert (loss(*up) - loss(*dn)) / (2 * e) == pytest.approx((g * d).sum(), rel=1e-6, abs=1e-7)


def rows(gcl, D, ptr=FAKE, st=None):  # noqa: F811
    return gcl.Rows(ptr, D if st is None else st, 0)


def args(gcl, backward, **bad):  # noqa: F811
    D = 72
    a = dict(x=rows(gcl, D), r=rows(gcl, D), rate=FAKE, cu_seqlens=FAKE, workspace=FAKE, workspace_bytes=1 << 40,
             t_max=100, n_max=2, D=D, decay=2, mix=2, dtype=1)
    a |= dict(d_o=rows(gcl, D), dx=rows(gcl, D), dr=rows(gcl, D)) if backward else dict(o=rows(gcl, D))
    return gcl.GlrArgs(**{**a, **bad})


@pytest.mark.parametrize("backward", [False, True])
def test_refusals(gcl, backward):  # noqa: F811
    lib = gcl.lib()
    call = lib.glr_bwd if backward else lib.glr_fwd
    assert call(None, None) == INVALID
    none = rows(gcl, 72, ptr=None)
    cases = [(dict(cu_seqlens=None), INVALID, b"cu_seqlens"), (dict(t_max=0), INVALID, b"t_max"), (dict(t_max=1 << 31), INVALID, b"t_max"),
             (dict(n_max=0), INVALID, b"n_max"), (dict(D=68), UNSUPPORTED, b"D=68"), (dict(D=0), UNSUPPORTED, b"D=0"),
             (dict(D=(1 << 20) + 8), UNSUPPORTED, b"D="), (dict(dtype=3), UNSUPPORTED, b"dtype"), (dict(decay=3), UNSUPPORTED, b"decay"),
             (dict(mix=-1), UNSUPPORTED, b"mix"), (dict(rate=None), INVALID, b"rate"), (dict(x=none), INVALID, b"x is required"),
             (dict(r=none), INVALID, b"r is required"), (dict(x=rows(gcl, 72, ptr=FAKE + 8)), INVALID, b"x must be 16-byte"),
             (dict(r=rows(gcl, 72, st=76)), INVALID, b"r strides"), (dict(r=rows(gcl, 72, st=64)), INVALID, b"r strides"),
             (dict(h0=FAKE + 4), INVALID, b"states"), (dict(h_save=FAKE + 8), INVALID, b"states"), (dict(workspace=None), CAPACITY, b"workspace"),
             (dict(workspace_bytes=64), CAPACITY, b"workspace"), (dict(workspace=FAKE + 8), INVALID, b"workspace"),
             (dict(t_max=(1 << 31) - 1, D=1 << 20), UNSUPPORTED, b"too large")]
    if backward:
        cases += [(dict(d_o=none), INVALID, b"d_o is required"), (dict(dx=none), INVALID, b"dx is required"),
                  (dict(dr=none), INVALID, b"dr is required"), (dict(i=rows(gcl, 72)), INVALID, b"di is required"),
                  (dict(decay=0, drate=FAKE), INVALID, b"drate"), (dict(dh0=FAKE, dht=FAKE), INVALID, b"dh0 must not be dht"),
                  (dict(dh0=FAKE + 64, h0=FAKE), INVALID, b"dh0 must not be h0")]
    else:
        cases += [(dict(ht=FAKE, h0=FAKE + 16), INVALID, b"ht must not be h0")]
    for bad, code, text in cases:
        assert call(ctypes.byref(args(gcl, backward, **bad)), None) == code, bad
        assert text in lib.gcl_last_error(), (bad, lib.gcl_last_error())


def test_step_refusals(gcl):  # noqa: F811
    lib = gcl.lib()
    good = dict(x=rows(gcl, 72), r=rows(gcl, 72), o=rows(gcl, 72), rate=FAKE, state=FAKE, slots=FAKE, batch=3, n_slots=2,
                D=72, decay=2, mix=0, dtype=1)
    assert lib.glr_step(None, None) == INVALID
    none = rows(gcl, 72, ptr=None)
    for bad, code, text in ((dict(state=None), INVALID, b"state"), (dict(batch=0), INVALID, b"batch"), (dict(n_slots=0), INVALID, b"n_slots"),
                            (dict(slots=None), INVALID, b"without slots"), (dict(D=4), UNSUPPORTED, b"D=4"), (dict(rate=None), INVALID, b"rate"),
                            (dict(dtype=9), UNSUPPORTED, b"dtype"), (dict(decay=-1), UNSUPPORTED, b"decay"), (dict(mix=3), UNSUPPORTED, b"mix"),
                            (dict(x=none), INVALID, b"x is required"), (dict(o=none), INVALID, b"o is required"),
                            (dict(i=rows(gcl, 72, st=70)), INVALID, b"i strides"), (dict(state=FAKE + 4), INVALID, b"16-byte"),
                            (dict(rate=FAKE + 4), INVALID, b"16-byte"), (dict(batch=1 << 30, D=1 << 10), UNSUPPORTED, b"batch")):
        assert lib.glr_step(ctypes.byref(gcl.GlrStepArgs(**{**good, **bad})), None) == code, bad
        assert text in lib.gcl_last_error(), (bad, lib.gcl_last_error())


def test_workspace_sizes(gcl):  # noqa: F811
    lib = gcl.lib()
    for dtype in (0, 1, 2):
        a = gcl.GlrArgs(t_max=1000, n_max=3, D=72, dtype=dtype)
        fwd, bwd = lib.gcl_glr_fwd_workspace_bytes(ctypes.byref(a)), lib.gcl_glr_bwd_workspace_bytes(ctypes.byref(a))
        assert fwd > 0 and bwd > fwd
        a.h_save = FAKE
        assert lib.gcl_glr_bwd_workspace_bytes(ctypes.byref(a)) < bwd
    for bad in (dict(t_max=0), dict(n_max=0), dict(D=12), dict(dtype=7)):
        a = gcl.GlrArgs(**{**dict(t_max=1000, n_max=3, D=72, dtype=1), **bad})
        assert lib.gcl_glr_fwd_workspace_bytes(ctypes.byref(a)) == 0 == lib.gcl_glr_bwd_workspace_bytes(ctypes.byref(a))
    assert lib.gcl_glr_fwd_workspace_bytes(None) == 0


def test_binding_refusals(cuda0):  # noqa: F811
    import torch
    m = cuda0
    f, i32 = torch.float32, torch.int32
    x, cu, rate = Tensor(6, 64), Tensor(3, dtype=i32), Tensor(64, dtype=f)
    good = dict(rate=rate, stream=0)
    for call in (lambda: m.glr_fwd(x, Tensor(6, 72), cu, x, **good), lambda: m.glr_fwd(x, Tensor(6, 64, dtype=f), cu, x, **good),
                 lambda: m.glr_fwd(x, x, Tensor(3, dtype=f), x, **good), lambda: m.glr_fwd(x, x, cu, x, decay="half", **good),
                 lambda: m.glr_fwd(x, x, cu, x, mix="two", **good), lambda: m.glr_fwd(x, x, cu, x, h0=Tensor(3, 64, dtype=f), **good),
                 lambda: m.glr_fwd(x, x, cu, x, h_save=Tensor(2, 64, dtype=f), **good),
                 lambda: m.glr_bwd(x, x, x, cu, x, x, i=x, **good), lambda: m.glr_step(x, x, Tensor(9, 32, dtype=f), x, **good),
                 # the tensors are on cuda:1, cuda:0 is current
                 lambda: m.glr_fwd(x, x, cu, x, **good), lambda: m.glr_bwd(x, x, x, cu, x, x, **good),
                 lambda: m.glr_step(x, x, Tensor(9, 64, dtype=f), x, **good), lambda: m.glr_fwd_workspace_bytes(x, cu),
                 lambda: m.glr_bwd_workspace_bytes(x, cu)):
        with pytest.raises(ValueError):
            call()
