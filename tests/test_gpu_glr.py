"""The gated linear recurrence on the GPU against its definition in fp64 (tests/glr_ref.py, where the tolerances stand)."""
import numpy as np
import pytest

import glr_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402

DEV = "cuda:0"
F32, I32 = torch.float32, torch.int32
DT = {"f32": F32, "bf16": torch.bfloat16, "f16": torch.float16}
CANARY = 1536.0
KINDS = [("power", "root", True), ("power", "complement", False), ("sigmoid", "complement", False), ("sigmoid", "root", True),
         ("log", "one", False), ("log", "root", True)]
LENS = {"one": [1], "short": [3, 0, 1, 5], "tile": [128], "edges": [127, 1, 0, 0, 129, 64, 63, 2], "ragged": [300, 0, 17, 1, 641, 0],
        "ones": [1] * 150, "empty": [0, 0], "long": [3001]}


def np64(t):
    return t.double().cpu().numpy()


class Case:
    """Inputs of one call; rows are slices of one wider buffer (strided tokens), with `pad` rows behind the last sequence."""

    def __init__(self, dtype, lens, D, decay, mix, gate, seed=0, pad=5, strided=True, h0=True, n_more=0):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        self.dtype, self.decay, self.mix, self.D = dtype, decay, mix, D
        self.live, self.T, self.N = sum(lens), max(sum(lens) + pad, 1), len(lens) + n_more
        dt = DT[dtype]
        rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
        buf = rnd(self.T, 3 * D + 16).to(dt)
        cut = [buf[:, k * D + 8:(k + 1) * D + 8] if strided else buf[:, k * D + 8:(k + 1) * D + 8].contiguous() for k in range(3)]
        self.x, self.r, self.i = cut[0], cut[1], cut[2] if gate else None
        if decay == "log":
            self.r.copy_(-torch.exp(self.r.float() - 2))
        elif decay == "sigmoid":
            self.r.add_(2)
        self.rate = torch.rand(D, generator=gen, device=DEV) * 0.8 + 0.01 if decay == "power" else None
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens + [0] * n_more)]), dtype=I32, device=DEV)
        self.h0 = rnd(self.N, D) if h0 else None
        self.d_o, self.dht = rnd(self.T, D).to(dt), rnd(self.N, D) if h0 else None
        self.status = torch.zeros(1, dtype=I32, device=DEV)
        self.kw = dict(i=self.i, rate=self.rate, decay=decay, mix=mix, dev_status=self.status)

    def full(self, *shape, dtype=F32):
        return torch.full(shape, CANARY, dtype=dtype, device=DEV)

    def fwd(self, save=True, o=True, stream=None):
        self.o = self.full(self.T, self.D + 8, dtype=DT[self.dtype])[:, :self.D] if o else None
        self.ht, self.save = self.full(self.N, self.D), self.full(-(-self.T // 64), self.D) if save else None
        ws = torch.full((gcl.glr_fwd_workspace_bytes(self.x, self.cu),), 0xFF, dtype=torch.uint8, device=DEV)
        gcl.glr_fwd(self.x, self.r, self.cu, self.o, h0=self.h0, ht=self.ht, h_save=self.save, workspace=ws, stream=stream, **self.kw)
        return self.o, self.ht, self.save

    def bwd(self, save=None):
        dt = DT[self.dtype]
        out = dict(dx=self.full(self.T, self.D, dtype=dt), dr=self.full(self.T, 2 * self.D, dtype=dt)[:, self.D:],
                   di=None if self.i is None else self.full(self.T, self.D, dtype=dt),
                   drate=self.full(self.D) if self.decay == "power" else None, dh0=self.full(self.N, self.D))
        ws = torch.full((gcl.glr_bwd_workspace_bytes(self.x, self.cu, h_save=save, drate=out["drate"]),), 0xFF, dtype=torch.uint8, device=DEV)
        gcl.glr_bwd(self.x, self.r, self.d_o, self.cu, h0=self.h0, dht=self.dht, h_save=save, workspace=ws, **out, **self.kw)
        return out

    def ref_args(self):
        z = lambda t: None if t is None else np64(t)  # noqa: E731
        return z(self.x), z(self.r), z(self.i), z(self.rate), z(self.h0)

    def e32(self):
        _, r, _, rate, _ = self.ref_args()
        return 10 * ref.E32 * ref.memory(r[:max(self.live, 1)], rate, self.decay, self.T)

    def check_fwd(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        x, r, i, rate, h0 = self.ref_args()
        h, prev, ht = ref.fwd(x, r, i, rate, h0, self.cu.tolist(), self.decay, self.mix)
        e, L = self.e32(), self.live
        top = max(np.abs(h[:L]).max() if L else 0, np.abs(ht).max())
        ref.check("ht", np64(self.ht), ht, "f32", e, top)
        if self.o is not None:
            ref.check("o", np64(self.o)[:L], h[:L], self.dtype, e)
            assert (np64(self.o)[L:] == CANARY).all(), "rows behind the last sequence were written"
        if self.save is not None:
            n = -(-L // 64)
            ref.check("h_save", np64(self.save)[:n], prev[:L:64], "f32", e, top)
            assert (np64(self.save)[n:] == CANARY).all()

    def check_bwd(self, out):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        x, r, i, rate, h0 = self.ref_args()
        dx, dr, di, drate, dh0, size = ref.bwd(x, r, i, rate, h0, np64(self.d_o), None if self.dht is None else np64(self.dht),
                                               self.cu.tolist(), self.decay, self.mix)
        e, L = 4 * self.e32(), self.live
        rows = {"dx": dx, "dr": dr} | ({"di": di} if self.i is not None else {})
        for n, v in rows.items():
            ref.check(n, np64(out[n])[:L], v[:L], self.dtype, e)
            assert (np64(out[n])[L:] == CANARY).all(), f"{n}: rows behind the last sequence were written"
        ref.check("dh0", np64(out["dh0"]), dh0, "f32", e, max(np.abs(dh0).max(), 1.0))
        if out["drate"] is not None:
            ref.check("drate", np64(out["drate"]), drate, "f32", e, size.max())


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_forward_layouts(dtype, lens):
    c = Case(dtype, LENS[lens], 72, "power", "root", True, seed=len(lens))
    c.fwd()
    c.check_fwd()


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_backward_layouts(dtype, lens):
    c = Case(dtype, LENS[lens], 72, "power", "root", True, seed=len(lens))
    c.fwd()
    with_save, without = c.bwd(c.save), c.bwd()
    c.check_bwd(with_save)
    c.check_bwd(without)


@pytest.mark.parametrize("decay,mix,gate", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [8, 200])
def test_kinds(dtype, D, decay, mix, gate):
    c = Case(dtype, [70, 0, 200, 1], D, decay, mix, gate, seed=D, n_more=3)
    c.fwd()
    c.check_fwd()
    c.check_bwd(c.bwd(c.save))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_states(dtype):
    """h0, dht NULL; o NULL; contiguous rows without padding."""
    c = Case(dtype, [65, 200], 64, "sigmoid", "complement", False, pad=0, strided=False, h0=False)
    c.fwd(save=False)
    c.check_fwd()
    c.check_bwd(c.bwd())
    c.fwd(o=False)
    c.check_fwd()


def test_wide_and_many_tiles():
    """Many tiles and blocks of channels in flight: several waves of the GPU."""
    c = Case("bf16", [5000, 1, 0, 2500, 700], 4104, "power", "root", True, strided=False)
    c.fwd()
    c.check_fwd()
    c.check_bwd(c.bwd(c.save))


@pytest.mark.parametrize("dtype,D", [("f32", 8), ("bf16", 72), ("f16", 264)])
def test_borders_anywhere(dtype, D):
    """Thousands of tokens in sequences of 0 to 400: starts and ends at every place of tiles, spans and warps, many spans in flight
    of few channels."""
    r = np.random.default_rng(D)
    lens = [int(n) for n in r.integers(0, 401, 60)] + [1] * 40 + [0] * 3 + [5000]
    c = Case(dtype, lens, D, "power", "root", True, seed=D, pad=200)
    c.fwd()
    c.check_fwd()
    c.check_bwd(c.bwd(c.save))
    c.check_bwd(c.bwd())


def test_results_repeat():
    c = Case("bf16", [3000, 77, 4000], 1000, "power", "root", True)
    first = [t.clone() for t in c.fwd()]
    grads = {n: v.clone() for n, v in c.bwd(c.save).items()}
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(c.fwd(), first))
        assert all(torch.equal(v, grads[n]) for n, v in c.bwd(c.save).items())


def test_saved_states_do_not_change_the_gradients():
    c = Case("f32", [300, 500], 136, "power", "root", True)
    c.fwd()
    a, b = c.bwd(c.save), c.bwd()
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_rows(dtype):
    """Token strides that put the last rows past 2^31 elements."""
    T, D, stride = 140, 64, 1 << 24
    c = Case(dtype, [100, 40], D, "power", "root", False, pad=0, strided=False)
    far = torch.empty((T - 1) * stride + D, dtype=DT[dtype], device=DEV).as_strided((T, D), (stride, 1))
    far.copy_(c.x)
    c.x = far
    c.fwd()
    c.check_fwd()
    c.check_bwd(c.bwd(c.save))


def test_values_that_are_not_finite_stay_in_their_sequence_and_channel():
    lens = [50, 100, 200]
    for dtype in ("f32", "bf16"):
        c = Case(dtype, lens, 64, "log", "one", True, pad=3)
        clean = [t.clone() for t in c.fwd()]
        for t, d, v in ((60, 5, float("nan")), (70, 9, float("inf")), (149, 3, float("-inf"))):
            c.x[t, d] = v
        c.x[c.live:] = float("nan")
        c.r[c.live:] = float("nan")
        c.h0[0, 40] = float("nan")
        o, ht, save = c.fwd()
        bad = torch.zeros_like(clean[0], dtype=torch.bool)
        for t, d in ((60, 5), (70, 9), (149, 3)):
            bad[t:150, d] = True
        bad[:50, 40] = True
        assert not o[bad].isfinite().any()
        assert torch.equal(o[~bad], clean[0][~bad])
        assert not ht[1, [3, 5, 9]].isfinite().any() and torch.equal(ht[2], clean[1][2])
        # d_o that is not finite: earlier tokens of its sequence and channel
        c = Case(dtype, lens, 64, "log", "one", True, pad=3)
        c.fwd()
        clean = {n: v.clone() for n, v in c.bwd(c.save).items() if v is not None}
        c.d_o[100, 7] = float("nan")
        c.d_o[c.live:] = float("inf")
        got = c.bwd(c.save)
        bad = torch.zeros_like(clean["dx"], dtype=torch.bool)
        bad[50:101, 7] = True
        for n in ("dx", "dr", "di"):
            assert not got[n][bad].isfinite().any() and torch.equal(got[n][~bad], clean[n][~bad])
        assert not got["dh0"][1, 7].isfinite() and torch.equal(got["dh0"][[0, 2]], clean["dh0"][[0, 2]])


def test_extreme_decays():
    """a = 0 (r = -inf), a = 1 (r = 0: m = 0 with the root mix) and far gates."""
    c = Case("f32", [90, 130], 64, "log", "root", False)
    c.r[10], c.r[100:104], c.r[40:60] = float("-inf"), float("-inf"), 0.0
    c.fwd()
    x, r, i, rate, h0 = c.ref_args()
    h, prev, ht = ref.fwd(x, r, i, rate, h0, c.cu.tolist(), c.decay, c.mix)
    e = 10 * ref.E32 * 140
    ref.check("o", np64(c.o)[:220], h[:220], "f32", e)
    assert torch.equal(c.o[10], c.x[10])                   # a = 0, m = 1: the input alone
    out = c.bwd(c.save)
    g = ref.bwd(x, np.where(np.isinf(r), -200.0, r), i, rate, h0, np64(c.d_o), np64(c.dht), c.cu.tolist(), c.decay, c.mix)
    for n, v in zip(("dx", "dr"), g):
        ref.check(n, np64(out[n])[:220], v[:220], "f32", 4 * e)
    for decay in ("sigmoid", "power"):
        c = Case("bf16", [40], 64, decay, "root", True, pad=0)
        c.r[3], c.r[4], c.i[5], c.i[6] = 100.0, -100.0, 100.0, -100.0
        c.fwd()
        c.check_fwd()
        c.check_bwd(c.bwd(c.save))


# ---------------------------------------------------------------- single tokens
@pytest.mark.parametrize("decay,mix,gate", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_step(dtype, decay, mix, gate):
    B, D, pool = 9, 200, 14
    c = Case(dtype, [B], D, decay, mix, gate, pad=0)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    state = torch.randn(pool, D, generator=gen, device=DEV)
    slots = torch.tensor([3, -1, 13, 0, 5, -7, 6, 1, 12], dtype=I32, device=DEV)
    before, o = state.clone(), c.full(B, D + 8, dtype=DT[dtype])[:, :D]
    gcl.glr_step(c.x, c.r, state, o, slots=slots, **c.kw)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    x, r, i, rate, _ = c.ref_args()
    on = [b for b in range(B) if slots[b] >= 0]
    at = slots[on].long().cpu().numpy()
    want = np64(before)
    _, a, m, _ = ref.gates(r, rate, decay, mix)
    u = x if i is None else x * ref.sigmoid(i)
    h = a[on] * want[at] + (m * u)[on]
    want[at] = h
    ref.check("state", np64(state), want, "f32", 10 * ref.E32)
    ref.check("o", np64(o)[on], h, dtype, 10 * ref.E32)
    assert (o[[1, 5]] == 0).all()
    idle = [s for s in range(pool) if s not in at]
    assert torch.equal(state[idle], before[idle])


def test_steps_continue_a_prefill():
    """Single tokens after a prefill give the rows of the longer prefill."""
    lens, more, D = [40, 130], 6, 136
    for dtype in ("f32", "bf16"):
        c = Case(dtype, [n + more for n in lens], D, "power", "root", True, pad=0)
        o, ht, _ = c.fwd()
        starts = c.cu[:-1].tolist()
        head = Case(dtype, lens, D, "power", "root", True, pad=0)
        pick = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lens)]).to(DEV)
        head.x, head.r, head.i, head.rate, head.h0 = c.x[pick], c.r[pick], c.i[pick], c.rate, c.h0
        head.kw |= dict(i=head.i, rate=head.rate)
        state = head.fwd()[1].clone()
        for k in range(more):
            at = torch.tensor([s + n + k for s, n in zip(starts, lens)], device=DEV)
            step = torch.empty(2, D, dtype=DT[dtype], device=DEV)
            gcl.glr_step(c.x[at], c.r[at], state, step, i=c.i[at], rate=c.rate, decay="power", mix="root")
            ref.check("o", np64(step), np64(o[at]), dtype, ref.U[dtype] + 3e-6)    # both rounded: twice the rounding
        ref.check("state", np64(state), np64(ht), "f32", 3e-6)


def test_step_bad_slots():
    B, D = 600, 264
    c = Case("bf16", [B], D, "power", "root", False, pad=0)
    slots = torch.arange(B, dtype=I32, device=DEV)
    idle = slots.clone()
    slots[[0, 300, B - 1]], idle[[0, 300, B - 1]] = B, -1
    results = []
    for s in (idle, slots):
        state, o = torch.ones(B, D, device=DEV), c.full(B, D, dtype=torch.bfloat16)
        c.status.zero_()
        gcl.glr_step(c.x, c.r, state, o, slots=s, **c.kw)
        torch.cuda.synchronize()
        results.append((state, o, int(c.status.item())))
    assert results[0][2] == 0 and results[1][2] == 4
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    c.status.fill_(3)
    state, o = torch.ones(B, D, device=DEV), c.full(B, D, dtype=torch.bfloat16)
    gcl.glr_step(c.x, c.r, state, o, slots=slots, **c.kw)
    torch.cuda.synchronize()
    assert (state == 1).all() and (o == CANARY).all()


# ---------------------------------------------------------------- status, streams, graphs
@pytest.mark.parametrize("cu", [[0, 60, 50, 100], [5, 50, 100], [0, 50, 200], [0, -4, 100]])
def test_invalid_sequences_write_nothing(cu):
    c = Case("bf16", [100], 64, "power", "root", False, pad=0)
    c.cu = torch.tensor(cu, dtype=I32, device=DEV)
    c.N = len(cu) - 1
    c.h0 = c.dht = None
    o, ht, save = c.fwd()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4
    assert all((t == CANARY).all() for t in (o, ht, save))
    c.status.zero_()
    out = c.bwd()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4
    assert all((t == CANARY).all() for t in out.values() if t is not None)


def test_a_set_status_word_stops_the_call():
    c = Case("bf16", [100, 0], 64, "power", "root", False)
    c.status.fill_(3)
    o, ht, save = c.fwd()
    out = c.bwd(save)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 3
    assert all((t == CANARY).all() for t in (o, ht, save, *(v for v in out.values() if v is not None)))


def test_captured_calls_follow_their_buffers():
    """One graph of forward and backward, replayed as lengths and inputs change; two graphs share a workspace."""
    T, D, N = 700, 200, 4
    c = Case("bf16", [300, 100, 0, 250], D, "power", "root", True, pad=50)
    ws = torch.full((max(gcl.glr_fwd_workspace_bytes(c.x, c.cu), gcl.glr_bwd_workspace_bytes(c.x, c.cu)),), 0xFF, dtype=torch.uint8, device=DEV)
    out = [(c.full(T, D, dtype=torch.bfloat16), c.full(N, D)) for _ in range(2)]
    dx, dr, di, drate, dh0 = (c.full(T, D, dtype=torch.bfloat16) for _ in range(3)), None, None, c.full(D), c.full(N, D)
    dx, dr, di = dx

    def fwd(k):
        gcl.glr_fwd(c.x, c.r, c.cu, out[k][0], h0=c.h0, ht=out[k][1], workspace=ws, **c.kw)

    def bwd():
        gcl.glr_bwd(c.x, c.r, c.d_o, c.cu, dx, dr, di=di, drate=drate, h0=c.h0, dht=c.dht, dh0=dh0, workspace=ws, **c.kw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fwd(0)
        bwd()
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        fwd(0)
        bwd()
    with torch.cuda.graph(graphs[1]):
        fwd(1)
    for lens in ([300, 100, 0, 250], [1, 0, 698, 1], [0, 0, 0, 5], [700, 0, 0, 0]):
        c.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=I32))
        c.live = sum(lens)
        for t in (*out[0], *out[1], dx, dr, di, drate, dh0):
            t.fill_(CANARY)
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        c.save = None
        for k in range(2):
            c.o, c.ht = out[k]
            c.check_fwd()
        c.check_bwd(dict(dx=dx, dr=dr, di=di, drate=drate, dh0=dh0))


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own run side by side."""
    cs = [Case("bf16", [6000, 3000], 512, "power", "root", True, seed=k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                c.fwd()
                c.out = c.bwd(c.save)
    torch.cuda.synchronize()
    for c in cs:
        c.check_fwd()
        c.check_bwd(c.out)


# ---------------------------------------------------------------- gates that are not numbers
@pytest.mark.parametrize("lens", [[50, 100, 200], [20, 40]])
@pytest.mark.parametrize("decay,mix,gate", KINDS + [("power", "one", True)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gates_that_are_not_numbers_are_passed_on(dtype, decay, mix, gate, lens):
    """NaN in r and in i: NaN wherever the definition has it, numbers everywhere else (in other channels the same bits)."""
    c, at = Case(dtype, lens, 72, decay, mix, gate), lens[0] + 10
    e = c.e32()
    clean, grads = [t.clone() for t in c.fwd()], c.bwd(c.save)
    c.r[at, 5] = float("nan")
    if gate:
        c.i[at + 8, 9] = float("nan")
    got, out = c.fwd(), c.bwd(c.save)
    torch.cuda.synchronize()
    x, r, i, rate, h0 = c.ref_args()
    with np.errstate(invalid="ignore"):
        h, prev, ht = ref.fwd(x, r, i, rate, h0, c.cu.tolist(), decay, mix)
        dx, dr, di, drate, dh0, _ = ref.bwd(x, r, i, rate, h0, np64(c.d_o), np64(c.dht), c.cu.tolist(), decay, mix)
    if gate and mix == "one":
        dr[at + 8, 9] = np64(grads["dr"])[at + 8, 9]       # (m is a constant: the input has no part in its decay's gradient)
    L, n = c.live, -(-c.live // 64)
    rows = [("o", got[0][:L], clean[0][:L], h[:L], dtype), ("ht", got[1], clean[1], ht, "f32"), ("h_save", got[2][:n], clean[2][:n], prev[:L:64], "f32")]
    rows += [(k, out[k][:L], grads[k][:L], v[:L], dtype) for k, v in (("dx", dx), ("dr", dr), ("di", di)) if out[k] is not None]
    rows += [("dh0", out["dh0"], grads["dh0"], dh0, "f32")] + ([("drate", out["drate"], grads["drate"], drate, "f32")] if decay == "power" else [])
    for name, a, b, want, dt in rows:
        bad = np.isnan(want)
        assert np.isnan(np64(a)[bad]).all(), name
        same = [k for k in range(72) if k not in (5, 9)]
        assert torch.equal(a[..., same], b[..., same]), name
        if name != "drate":
            ref.check(name, np64(a)[~bad], want[~bad], dt, 4 * e, max(np.abs(want[~bad]).max(), 1.0))


@pytest.mark.parametrize("decay,mix,gate", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_step_passes_on_gates_that_are_not_numbers(dtype, decay, mix, gate):
    c = Case(dtype, [4], 200, decay, mix, gate, pad=0)
    states = [torch.ones(4, 200, device=DEV) for _ in range(2)]
    outs = [c.full(4, 200, dtype=DT[dtype]) for _ in range(2)]
    gcl.glr_step(c.x, c.r, states[0], outs[0], **c.kw)
    bad = torch.zeros(4, 200, dtype=torch.bool, device=DEV)
    c.r[1, 3], bad[1, 3] = float("nan"), True
    if gate:
        c.i[2, 150], bad[2, 150] = float("nan"), True
    gcl.glr_step(c.x, c.r, states[1], outs[1], **c.kw)
    for a, b in ((states[1], states[0]), (outs[1], outs[0])):
        assert a[bad].isnan().all() and torch.equal(a[~bad], b[~bad])


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sigmoid_decay_near_one(dtype, gate):
    """The decay itself: with x = 0 and a state of 1 the state after a token is a, unrounded (a 1 + 0).  Where a >= 1/2 it is 1 - c with
    c = sigmoid(-r): one rounding of at most 2^-25, and c's own error.  c's (a's where a < 1/2) is relative: the exponent's product and
    its constant are off by 2^-24 of it each, 2 |r| in all, and exponential, sum, reciprocal and product by at most 10 more."""
    n = 4096
    c = Case(dtype, [1], n, "sigmoid", "complement", gate, pad=0)
    c.r.copy_(torch.linspace(-12, 12, n, device=DEV).view(1, n))
    c.x.zero_()
    state, o = torch.ones(1, n, device=DEV), c.full(1, n, dtype=DT[dtype])
    gcl.glr_step(c.x, c.r, state, o, **c.kw)
    r = np64(c.r)[0]
    a, small = ref.sigmoid(r), ref.sigmoid(-np.abs(r))
    bound = np.where(r > 0, 2.0 ** -25, 0) + (2 * np.abs(r) + 10) * ref.E32 * small
    err = np.abs(np64(state)[0] - a)
    assert (err <= bound).all(), (float(r[(err - bound).argmax()]), float((err / bound).max()))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_memory(dtype, gate):
    """Sigmoid decays of 0.998 to 0.9999 over thousands of tokens."""
    c = Case(dtype, [3001, 500], 72, "sigmoid", "complement", gate)
    c.r.copy_(6.2 + 3 * torch.rand(c.T, 72, device=DEV))
    c.fwd()
    c.check_fwd()
    c.check_bwd(c.bwd(c.save))


@pytest.mark.parametrize("mix,gate", [("root", True), ("complement", False), ("one", True)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rates_on_both_sides_of_the_near_range(dtype, mix, gate):
    """Rates of 0.01 to 8 in every warp's channels, and of one warp's channels alone: the exponential beside the polynomial."""
    for lens, D in (([70, 0, 200, 1], 200), ([100], 72), ([900, 2100], 136)):
        c = Case(dtype, lens, D, "power", mix, gate, seed=D)
        c.rate.copy_(torch.logspace(-2, 0.9, D, device=DEV)[torch.randperm(D, device=DEV)])
        if D == 136:
            c.rate[64:].mul_(0.1)
        c.fwd()
        c.check_fwd()
        c.check_bwd(c.bwd(c.save))
        c.check_bwd(c.bwd())
        state, o = torch.ones(c.T, D, device=DEV), c.full(c.T, D, dtype=DT[dtype])
        gcl.glr_step(c.x, c.r, state, o, **c.kw)
        x, r, i, rate, _ = c.ref_args()
        _, a, m, _ = ref.gates(r, rate, "power", mix)
        h = a + m * (x if i is None else x * ref.sigmoid(i))
        ref.check("state", np64(state), h, "f32", 10 * ref.E32)
        ref.check("o", np64(o), h, dtype, 10 * ref.E32)
