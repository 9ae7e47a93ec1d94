"""Decayed linear attention and the per-head norm with rotation without a GPU: the references'
gradients against differences of their forwards, the segment plan, and the refusals of the C entry
points and of the binding (each before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

import dla_ref


@pytest.fixture(scope="module")
def gcl():
    from chunked_gated_linear_gb300 import _build
    _build.build()
    import chunked_gated_linear_gb300 as gcl
    gcl.lib()
    return gcl


def test_reference_gradients_match_differences():
    """Central differences of <d_o, o> + <dht, ht> along random directions, in fp64; the forward is
    quadratic in (k, v) together, so the difference is exact up to rounding."""
    r = np.random.default_rng(0)
    T, H, K, V, cu = 9, 2, 3, 4, [0, 5, 5, 9]
    q, k, v = r.standard_normal((T, H, K)), r.standard_normal((T, H, K)), r.standard_normal((T, H, V))
    h0, dht, d_o = (r.standard_normal((3, H, K, V)), r.standard_normal((3, H, K, V)), r.standard_normal((T, H, V)))
    g, scale = np.array([-0.3, -2.0]), 0.7

    def loss(q, k, v, h0):
        o, ht = dla_ref.fwd(q, k, v, g, h0, cu, scale)
        return (o * d_o).sum() + (ht * dht).sum()

    grads = dla_ref.bwd(q, k, v, g, h0, d_o, dht, cu, scale)
    x = [q, k, v, h0]
    for i, gr in enumerate(grads):
        d = r.standard_normal(x[i].shape)
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + 0.5 * d, x[i] - 0.5 * d
        assert loss(*up) - loss(*dn) == pytest.approx((gr * d).sum(), rel=1e-10)


@pytest.mark.parametrize("norm", ["none", "rms", "l2"])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_norm_rope_reference_gradients_match_differences(norm, pairing):
    r = np.random.default_rng(1)
    T, H, D, R, eps = 3, 2, 8, 4, 1e-3
    x, w, dy = r.standard_normal((T, H, D)), r.standard_normal(D), r.standard_normal((T, H, D))
    a = r.standard_normal((T, R // 2))
    f = lambda x, w: (dla_ref.norm_rope(x, w, np.cos(a), np.sin(a), R, norm, eps, pairing) * dy).sum()  # noqa: E731
    dx, dw = dla_ref.norm_rope_bwd(x, w, dy, np.cos(a), np.sin(a), R, norm, eps, pairing)
    e = 1e-5
    d, dd = r.standard_normal(x.shape), r.standard_normal(D)
    assert (f(x + e * d, w) - f(x - e * d, w)) / (2 * e) == pytest.approx((dx * d).sum(), rel=1e-7)
    assert (f(x, w + e * dd) - f(x, w - e * dd)) / (2 * e) == pytest.approx((dw * dd).sum(), rel=1e-7)


def test_segment_plan_from_sizes_alone(gcl):
    """Many units: whole sequences, no workspace.  One long sequence of one head: segments of a
    multiple of 128 tokens whose states fit the workspace.  A few tokens stay whole."""
    assert gcl.dla_segment_tokens(65536, 128, 16) >= 65536
    seg = gcl.dla_segment_tokens(65536, 1, 1)
    assert 0 < seg < 65536 and seg % 128 == 0
    assert gcl.dla_segment_tokens(200, 1, 1) >= 200
    assert gcl.dla_segment_tokens(0, 1, 1) == 0 and gcl.dla_segment_tokens(5, 0, 1) == 0
    for T, N, H in ((65536, 1, 1), (8192, 3, 4), (777, 2, 1)):
        for back in (False, True):
            seg = gcl.dla_segment_tokens(T, N, H, back)
            a = gcl.DlaArgs(t_max=T, n_max=N, H=H, K=64, V=128, dtype=1)
            fn = gcl.lib().gcl_dla_bwd_workspace_bytes if back else gcl.lib().gcl_dla_fwd_workspace_bytes
            rows = gcl.nt_max(T, N, seg) if seg < T else 0
            assert fn(ctypes.byref(a)) == rows * H * 64 * 128 * 4 * (2 if back else 1)


FAKE = 1 << 20      # a 16-byte aligned non-null value; never dereferenced on these paths


def rows(gcl, H, D, ptr=FAKE, st=None, sh=None):
    return gcl.Rows(ptr, H * D if st is None else st, D if sh is None else sh)


def dla_args(gcl, backward, **bad):
    H, K, V = 2, 64, 128
    a = dict(q=rows(gcl, H, K), k=rows(gcl, H, K), v=rows(gcl, H, V), g=FAKE, cu_seqlens=FAKE, t_max=100,
             n_max=2, H=H, K=K, V=V, scale=1.0, dtype=1)
    if backward:
        a |= dict(d_o=rows(gcl, H, V), dq=rows(gcl, H, K), dk=rows(gcl, H, K), dv=rows(gcl, H, V))
    else:
        a |= dict(o=rows(gcl, H, V))
    return gcl.DlaArgs(**{**a, **bad})


INVALID, UNSUPPORTED, CAPACITY = 1, 2, 3


@pytest.mark.parametrize("backward", [False, True])
def test_dla_chunk_refusals(gcl, backward):
    lib = gcl.lib()
    call = lib.dla_chunk_bwd if backward else lib.dla_chunk_fwd
    assert call(None, None) == INVALID
    cases = [(dict(g=None), INVALID, b"g and cu"), (dict(cu_seqlens=None), INVALID, b"g and cu"),
             (dict(t_max=0), INVALID, b"t_max"), (dict(t_max=1 << 31), INVALID, b"t_max"), (dict(n_max=0), INVALID, b"n_max"),
             (dict(H=0), INVALID, b"H=0"), (dict(K=96), UNSUPPORTED, b"K=96"), (dict(V=256), UNSUPPORTED, b"V=256"),
             (dict(dtype=5), UNSUPPORTED, b"dtype"), (dict(q=rows(gcl, 2, 64, ptr=None)), INVALID, b"q is required"),
             (dict(v=rows(gcl, 2, 128, ptr=FAKE + 8)), INVALID, b"v must be 16-byte"),
             (dict(k=rows(gcl, 2, 64, st=60)), INVALID, b"k strides"), (dict(k=rows(gcl, 2, 64, sh=68)), INVALID, b"k strides"),
             (dict(h0=FAKE + 4), INVALID, b"states"),
             # a plan with segments and no workspace, and one too small
             (dict(t_max=65536, n_max=1), CAPACITY, b"workspace"),
             (dict(t_max=65536, n_max=1, workspace=FAKE, workspace_bytes=64), CAPACITY, b"workspace")]
    if backward:
        cases += [(dict(d_o=rows(gcl, 2, 128, ptr=None)), INVALID, b"d_o is required"),
                  (dict(dk=rows(gcl, 2, 64, st=64, sh=64)), INVALID, b"rows of dk overlap")]
    else:
        cases += [(dict(o=rows(gcl, 2, 128, st=128, sh=128)), INVALID, b"rows of o overlap")]
    for bad, code, text in cases:
        assert call(ctypes.byref(dla_args(gcl, backward, **bad)), None) == code, bad
        assert text in lib.gcl_last_error(), (bad, lib.gcl_last_error())


def test_dla_step_refusals(gcl):
    lib = gcl.lib()
    good = dict(q=rows(gcl, 2, 64), k=rows(gcl, 2, 64), v=rows(gcl, 2, 64), o=rows(gcl, 2, 64), g=FAKE, state=FAKE,
                batch=3, n_slots=2, H=2, K=64, V=64, scale=1.0, dtype=1)
    assert lib.dla_step(None, None) == INVALID
    for bad, code, text in ((dict(g=None), INVALID, b"required"), (dict(state=None), INVALID, b"required"),
                            (dict(batch=0), INVALID, b"batch"), (dict(n_slots=0), INVALID, b"n_slots"),
                            (dict(), INVALID, b"without slots"), (dict(slots=FAKE, K=32), UNSUPPORTED, b"K=32"),
                            (dict(slots=FAKE, dtype=9), UNSUPPORTED, b"dtype"),
                            (dict(slots=FAKE, state=FAKE + 4), INVALID, b"state"),
                            (dict(slots=FAKE, o=rows(gcl, 2, 64, ptr=None)), INVALID, b"o is required"),
                            (dict(slots=FAKE, o=rows(gcl, 2, 64, st=64, sh=64)), INVALID, b"overlap")):
        assert lib.dla_step(ctypes.byref(gcl.DlaStepArgs(**{**good, **bad})), None) == code, bad
        assert text in lib.gcl_last_error(), (bad, lib.gcl_last_error())


@pytest.mark.parametrize("backward", [False, True])
def test_qk_norm_rope_refusals(gcl, backward):
    lib = gcl.lib()
    call = lib.qk_norm_rope_bwd if backward else lib.qk_norm_rope_fwd
    r = lambda H, **kw: rows(gcl, H, 128, **kw)  # noqa: E731
    good = dict(q=r(4), k=r(2), cos_table=FAKE, sin_table=FAKE, positions=FAKE, t_max=10, n_positions=64, HQ=4, HK=2,
                D=128, R=32, eps=1e-6, norm=1, pair=0, dtype=1)
    good |= dict(dyq=r(4), dyk=r(2), dq=r(4), dk=r(2)) if backward else dict(yq=r(4), yk=r(2))
    assert call(None, None) == INVALID
    cases = [(dict(t_max=0), INVALID, b"t_max"), (dict(HQ=0), INVALID, b"HQ"), (dict(HK=-1), INVALID, b"HK"),
             (dict(D=96), UNSUPPORTED, b"D=96"), (dict(R=24), UNSUPPORTED, b"R=24"), (dict(R=144), UNSUPPORTED, b"R=144"),
             (dict(dtype=3), UNSUPPORTED, b"dtype"), (dict(norm=3), UNSUPPORTED, b"norm"), (dict(pair=2), UNSUPPORTED, b"pair"),
             (dict(eps=-1.0), INVALID, b"eps"), (dict(eps=float("nan")), INVALID, b"eps"),
             (dict(cos_table=None), INVALID, b"needs cos"), (dict(positions=None), INVALID, b"positions"),
             (dict(n_positions=0), INVALID, b"n_positions"), (dict(k=r(2, ptr=None)), INVALID, b"k is required"),
             (dict(q=r(4, ptr=FAKE + 2)), INVALID, b"q must be"), (dict(q_weight=FAKE + 2), INVALID, b"weights"),
             (dict(sin_table=FAKE + 4), INVALID, b"tables")]
    if backward:
        cases += [(dict(dq_weight=FAKE), INVALID, b"needs the weight"),
                  (dict(q_weight=FAKE, dq_weight=FAKE), CAPACITY, b"workspace"),
                  (dict(dq=r(4, st=128, sh=128)), INVALID, b"rows of dq overlap")]
    else:
        cases += [(dict(yk=r(2, st=128, sh=128)), INVALID, b"rows of yk overlap")]
    for bad, code, text in cases:
        assert call(ctypes.byref(gcl.QkArgs(**{**good, **bad})), None) == code, bad
        assert text in lib.gcl_last_error(), (bad, lib.gcl_last_error())


def test_rope_table_refusals(gcl):
    lib = gcl.lib()
    for args in ((None, FAKE, 4, 64, 1e4), (FAKE, None, 4, 64, 1e4), (FAKE, FAKE, 0, 64, 1e4), (FAKE, FAKE, 4, 63, 1e4),
                 (FAKE, FAKE, 4, 0, 1e4), (FAKE, FAKE, 4, 64, 0.0), (FAKE, FAKE, 4, 64, float("nan"))):
        assert lib.rope_table_build(*args, None) == INVALID, args


def test_binding_refuses_host_tensors_and_shapes(gcl):
    """The binding's checks come before the library is called: host tensors are refused by name."""
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    cu = torch.tensor([0, 4], dtype=torch.int32)
    q, v, g = z(4, 2, 64), z(4, 2, 64), z(2, dt=torch.float32)
    for call in (lambda: gcl.dla_chunk_fwd(q, q, v, g, cu, v),
                 lambda: gcl.dla_chunk_bwd(q, q, v, g, v, cu, q, q, v),
                 lambda: gcl.dla_step(q, q, v, g, z(4, 2, 64, 64, dt=torch.float32), v),
                 lambda: gcl.qk_norm_rope_fwd(q, q, q, q),
                 lambda: gcl.qk_norm_rope_bwd(q, q, q, q, q, q),
                 lambda: gcl.rope_table_build(z(4, 16, dt=torch.float32), z(4, 16, dt=torch.float32))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="norm"):
        gcl.qk_norm_rope_fwd(q, q, q, q, norm="layer")


def test_packed_structs_match_the_declared_ones(gcl):
    """The packed argument layouts have the size and the field offsets of the ctypes structs."""
    for pack, cls in ((gcl._DLA_PACK, gcl.DlaArgs), (gcl._STEP_PACK, gcl.DlaStepArgs), (gcl._QK_PACK, gcl.QkArgs)):
        assert pack.size == ctypes.sizeof(cls)
        kinds = []
        for _, t in cls._fields_:
            kinds += [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64] if t is gcl.Rows else [t]
        values = [float(i) if t is ctypes.c_float else i for i, t in enumerate(kinds, start=1)]
        a = cls.from_buffer_copy(pack.pack(*values))
        got = []
        for name, t in cls._fields_:
            x = getattr(a, name)
            got += [x.ptr, x.token_stride, x.head_stride] if t is gcl.Rows else [x]
        assert got == values
