"""Decayed linear attention on the GPU (dla_chunk_fwd, dla_chunk_bwd, dla_step) against the fp64
recurrence of tests/dla_ref.py, at the tolerances derived there."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402
import dla_ref  # noqa: E402
from parity import check  # noqa: E402

DEV = "cuda:0"
CANARY = 1536.0
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def strided(x, layout):
    """The same values as a device view: contiguous, as a slice of a wider buffer, or head-major."""
    if layout == "packed":
        T, H, D = x.shape
        wide = torch.full((T, H * D + 48 + 64), float("nan"), dtype=x.dtype, device=DEV)
        view = wide[:, 48:48 + H * D].view(T, H, D)
        view.copy_(x)
        return view
    if layout == "head_major":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    return x.contiguous()


class Case:
    """Random inputs of one layout; rows past the last sequence hold NaN."""

    def __init__(self, dtype, lens, H, K, V, seed=0, g=None, h0=True, t_pad=17, layout="contiguous"):
        r = np.random.default_rng(seed)
        self.dt, self.H, self.K, self.V, self.N = DT[dtype], H, K, V, len(lens)
        self.dtype, self.live = dtype, sum(lens)
        self.T = max(self.live, 1) + t_pad
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.scale = K ** -0.5
        g = -(2.0 ** (-8.0 * (np.arange(H) + 1) / H)) if g is None else g
        self.g = torch.tensor(np.asarray(g), dtype=torch.float32, device=DEV)

        def rows(D):
            x = torch.full((self.T, H, D), float("nan"))
            x[:self.live] = torch.from_numpy(r.standard_normal((self.live, H, D)).astype(np.float32))
            return strided(x.to(self.dt).to(DEV), layout)

        self.q, self.k, self.v, self.d_o = rows(K), rows(K), rows(V), rows(V)
        state = lambda: torch.from_numpy(r.standard_normal((self.N, H, K, V)).astype(np.float32)).to(DEV)  # noqa: E731
        self.h0, self.dht = (state(), state()) if h0 else (None, None)
        self.cud = torch.from_numpy(self.cu).to(DEV)
        self.order = torch.argsort(torch.tensor(lens), descending=True, stable=True).to(torch.int32).to(DEV)
        self.layout = layout

    def out(self, D):
        return strided(torch.full((self.T, self.H, D), CANARY, dtype=self.dt, device=DEV), self.layout)

    def states(self):
        return torch.full((self.N, self.H, self.K, self.V), CANARY, device=DEV)

    def host(self, *names):
        f = lambda x: None if x is None else x.float().cpu().numpy()  # noqa: E731
        return [f(getattr(self, n)) for n in names]

    def fwd(self, status=None, order=True, stream=None):
        o, ht = self.out(self.V), self.states()
        status = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
        nb = gcl.dla_fwd_workspace_bytes(self.q, self.v, self.cud)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV) if nb else None
        gcl.dla_chunk_fwd(self.q, self.k, self.v, self.g, self.cud, o, h0=self.h0, ht=ht, dev_status=status,
                          seq_order=self.order if order else None, workspace=ws, stream=stream)
        return o, ht, status

    def bwd(self, status=None):
        dq, dk, dv, dh0 = self.out(self.K), self.out(self.K), self.out(self.V), self.states()
        status = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
        nb = gcl.dla_bwd_workspace_bytes(self.q, self.v, self.cud)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV) if nb else None
        gcl.dla_chunk_bwd(self.q, self.k, self.v, self.g, self.d_o, self.cud, dq, dk, dv, h0=self.h0, dht=self.dht,
                          dh0=dh0, dev_status=status, workspace=ws)
        return dq, dk, dv, dh0, status

    def check_rows(self, name, got, ref):
        got = got.float().cpu().numpy()
        assert (got[self.live:] == CANARY).all(), name + ": padding was written"
        if self.live:
            check(name, got[:self.live], ref[:self.live], dla_ref.TOL[self.dtype], cu=self.cu, reduction=False)

    def check_fwd(self, label, **kw):
        o, ht, status = self.fwd(**kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        q, k, v, g, h0 = self.host("q", "k", "v", "g", "h0")
        ro, rh = dla_ref.fwd(q, k, v, g, h0, self.cu, self.scale)
        self.check_rows(label + " o", o, ro)
        check(label + " ht", ht.cpu().numpy(), rh, dla_ref.TOL_STATE)

    def check_bwd(self, label):
        *grads, dh0, status = self.bwd()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        q, k, v, g, h0, d_o, dht = self.host("q", "k", "v", "g", "h0", "d_o", "dht")
        *ref, rh = dla_ref.bwd(q, k, v, g, h0, d_o, dht, self.cu, self.scale)
        for name, got, r in zip(("dq", "dk", "dv"), grads, ref):
            self.check_rows(f"{label} {name}", got, r)
        check(label + " dh0", dh0.cpu().numpy(), rh, dla_ref.TOL_STATE)


RAGGED = [1, 0, 2, 63, 64, 65, 127, 128, 129, 0, 200, 257]
DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]
# (lens, H): whole sequences (many units), and segments (few units; the plan is asserted below)
LAYOUTS = {"one": ([1], 3), "ragged": (RAGGED, 3), "empty": ([0, 0], 2), "segments": ([700, 0, 1, 1900], 1)}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("dims", DIMS, ids=lambda d: f"{d[0]}x{d[1]}")
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_forward(dtype, dims, layout):
    lens, H = LAYOUTS[layout]
    c = Case(dtype, lens, H, *dims, seed=1, layout={"one": "packed", "ragged": "packed"}.get(layout, "contiguous"))
    assert (gcl.dla_segment_tokens(c.T, c.N, H) < c.T) == (layout == "segments")
    c.check_fwd(f"fwd {dtype} {dims} {layout}")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("dims", DIMS, ids=lambda d: f"{d[0]}x{d[1]}")
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_backward(dtype, dims, layout):
    lens, H = LAYOUTS[layout]
    c = Case(dtype, lens, H, *dims, seed=2, layout={"one": "head_major", "ragged": "packed"}.get(layout, "contiguous"))
    assert (gcl.dla_segment_tokens(c.T, c.N, H, True) < c.T) == (layout == "segments")
    c.check_bwd(f"bwd {dtype} {dims} {layout}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [RAGGED, [1500]], ids=["ragged", "segments"])
@pytest.mark.parametrize("h0", [True, False], ids=["h0", "zero"])
def test_extreme_decays(dtype, lens, h0):
    """gamma = 0 (only the token itself counts), a decay that underflows within a chunk, none at all."""
    for g in (-np.inf, -30.0, -0.7, -1e-4, 0.0):
        c = Case(dtype, lens, 1, 64, 128, seed=3, g=[g], h0=h0)
        c.check_fwd(f"decay {g} {dtype}")
        c.check_bwd(f"decay {g} {dtype}")


def test_forward_order_and_missing_outputs():
    """Index order, o alone and ht alone: the same bits as everything together."""
    c = Case("bf16", RAGGED, 4, 128, 128, seed=4, layout="head_major")
    o, ht, _ = c.fwd()
    o2, ht2, _ = c.fwd(order=False)
    assert torch.equal(o, o2) and torch.equal(ht, ht2)
    o3, ht3 = c.out(128), c.states()
    gcl.dla_chunk_fwd(c.q, c.k, c.v, c.g, c.cud, o3, h0=c.h0)
    gcl.dla_chunk_fwd(c.q, c.k, c.v, c.g, c.cud, None, h0=c.h0, ht=ht3)
    assert torch.equal(o, o3) and torch.equal(ht, ht3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_match_differences(dtype):
    """o and ht are linear in each of q, k, v and h0 alone, so the change of <d_o, o> + <dht, ht> along a
    direction x' is the forward with x' in x's place (minus, for h0-free terms, what does not depend on
    it); with the kernels' own forward.  Accumulated in fp64 on the host; the bars are the outputs'."""
    c = Case(dtype, [130, 1, 77], 3, 128, 128, seed=5)
    *grads, dh0, _ = c.bwd()
    L = c.live
    dots = lambda o, ht: float((o[:L].double() * c.d_o[:L].double()).sum() + (ht.double() * c.dht.double()).sum())  # noqa: E731
    size = lambda a, b: float(a.double().norm() * b.double().norm())  # noqa: E731
    o, ht, _ = c.fwd()
    full, tol = dots(o, ht), dla_ref.TOL[dtype]
    zero, c.h0 = c.h0, torch.zeros_like(c.h0)
    o, ht, _ = c.fwd()
    free = dots(o, ht)                                  # bilinear in (k, v), the h0 part left out
    c.h0 = zero
    bar = tol * (size(o[:L], c.d_o[:L]) + size(ht, c.dht))
    dq, dk, dv = (x[:L].double() for x in grads)
    # d/dv along v itself, d/dk along k itself: the bilinear part; d/dh0 along h0: the rest
    assert abs(float((dv * c.v[:L].double()).sum()) - free) <= bar
    assert abs(float((dk * c.k[:L].double()).sum()) - free) <= bar
    assert abs(float((dh0.double() * c.h0.double()).sum()) - (full - free)) <= bar
    # d/dq along q: <d_o, o> alone (ht does not depend on q)
    o, ht, _ = c.fwd()
    assert abs(float((dq * c.q[:L].double()).sum()) - float((o[:L].double() * c.d_o[:L].double()).sum())) <= bar


def test_sequences_do_not_mix():
    """A sequence of NaN leaves its neighbours' bits alone, forward and backward."""
    a, b = Case("bf16", [100, 40, 300], 2, 128, 128, seed=6), Case("bf16", [100, 40, 300], 2, 128, 128, seed=6)
    for x in (b.q, b.k, b.v, b.d_o):
        x[100:140] = float("nan")
    for run in ("fwd", "bwd"):
        for x, y in zip(getattr(a, run)()[:-1], getattr(b, run)()[:-1]):
            if x.shape[0] == a.T:
                assert torch.equal(x[:100], y[:100]) and torch.equal(x[140:440], y[140:440])
                assert y[100:140].isnan().any()
            else:
                assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])


@pytest.mark.parametrize("lens,H", [([500, 80], 3), ([3000], 1)], ids=["whole", "segments"])
def test_repeated_calls_are_bitwise_equal(lens, H):
    for dtype in ("bf16", "f32"):
        c = Case(dtype, lens, H, 128, 64, seed=7)
        for run in ("fwd", "bwd"):
            for x, y in zip(getattr(c, run)()[:-1], getattr(c, run)()[:-1]):
                assert torch.equal(x, y)


@pytest.mark.parametrize("cu", [[0, 50, 40, 60], [0, 20, 40, 500], [-4, 20, 40, 60]], ids=["decreasing", "over", "negative"])
@pytest.mark.parametrize("H", [80, 1], ids=["whole", "segments"])
def test_bad_ranges_set_the_status(cu, H):
    """The kernels check every range before they use it; nothing outside the buffers is touched."""
    c = Case("bf16", [2000, 700, 300], H, 64, 64, seed=8) if H == 1 else Case("bf16", [20, 20, 20], H, 64, 64, seed=8)
    if H == 1:
        cu = [0 if x == 0 else x if x > 400 or x < 0 else x for x in cu]
        cu[3] = cu[3] if cu[3] != 500 else c.T + 400
    c.cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    for run in ("fwd", "bwd"):
        status = getattr(c, run)()[-1]
        torch.cuda.synchronize()
        assert int(status.item()) == 4


def test_set_status_stops_the_work():
    c = Case("bf16", [200, 30], 2, 64, 64, seed=9)
    for run in ("fwd", "bwd"):
        *out, status = getattr(c, run)(status=torch.tensor([3], dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        assert int(status.item()) == 3
        for x in out:
            assert (x == CANARY).all()


@pytest.mark.parametrize("lens,H", [([300, 45], 3), ([2500], 1)], ids=["whole", "segments"])
def test_graph_replay_with_new_inputs(lens, H):
    """Forward and backward captured once on a side stream; replayed after the inputs and the lengths
    change in place: the same bits as eager calls."""
    c = Case("bf16", lens, H, 128, 128, seed=10)
    o, ht = c.out(128), c.states()
    dq, dk, dv, dh0 = c.out(128), c.out(128), c.out(128), c.states()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(gcl.dla_bwd_workspace_bytes(c.q, c.v, c.cud), 16), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def both():
        gcl.dla_chunk_fwd(c.q, c.k, c.v, c.g, c.cud, o, h0=c.h0, ht=ht, dev_status=status, workspace=ws)
        gcl.dla_chunk_bwd(c.q, c.k, c.v, c.g, c.d_o, c.cud, dq, dk, dv, h0=c.h0, dht=c.dht, dh0=dh0,
                          dev_status=status, workspace=ws)

    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    d = Case("bf16", [x - 7 for x in lens], H, 128, 128, seed=11, t_pad=17 + 7 * len(lens))
    for n in ("q", "k", "v", "d_o", "h0", "dht", "cud"):
        getattr(c, n).copy_(getattr(d, n))
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    live = sum(lens) - 7 * len(lens)
    eo, eht, _ = c.fwd()
    edq, edk, edv, edh0, _ = c.bwd()
    for x, y in ((o, eo), (dq, edq), (dk, edk), (dv, edv)):
        assert torch.equal(x[:live], y[:live])
    assert torch.equal(ht, eht) and torch.equal(dh0, edh0)


def test_offsets_past_32_bits():
    """Token rows 16 MiB apart: the last lies 4.8 GB (2.4 G elements) into the buffer."""
    T, H, D, stride = 300, 1, 64, 1 << 23
    big = torch.empty((T - 1) * stride + 4 * D, dtype=torch.bfloat16, device=DEV)
    view = lambda i: big[i * D:].as_strided((T, H, D), (stride, D, 1))  # noqa: E731
    c = Case("bf16", [300], H, D, D, seed=12, t_pad=0)
    o, ht, _ = c.fwd()
    q, k, v, out = (view(i) for i in range(4))
    for x, y in ((q, c.q), (k, c.k), (v, c.v)):
        x.copy_(y)
    ht2 = c.states()
    gcl.dla_chunk_fwd(q, k, v, c.g, c.cud, out, h0=c.h0, ht=ht2)
    assert torch.equal(out, o) and torch.equal(ht, ht2)


# ---------------------------------------------------------------- single tokens
def step_ref(q, k, v, g, state, slots, scale):
    o = np.zeros(v.shape)
    state = state.astype(np.float64)
    for b in range(q.shape[0]):
        if 0 <= slots[b] < state.shape[0]:
            S = dla_ref.decay(g)[:, None, None] * state[slots[b]] + k[b][:, :, None] * v[b][:, None, :].astype(np.float64)
            state[slots[b]] = S
            o[b] = scale * np.einsum("hk,hkv->hv", q[b].astype(np.float64), S)
    return o, state


# the result is fp32 arithmetic rounded once: half a step of the type, plus the fp32 bar
STEP_TOL = {"f32": 1e-5, "f16": 2.0 ** -11 + 1e-5, "bf16": 2.0 ** -8 + 1e-5}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("dims", DIMS, ids=lambda d: f"{d[0]}x{d[1]}")
@pytest.mark.parametrize("B,H", [(1, 1), (5, 3), (110, 3)])
def test_step(dtype, dims, B, H):
    K, V = dims
    r = np.random.default_rng(20)
    n_slots = B + 3
    x = lambda *s: strided(torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(DT[dtype]).to(DEV), "packed")  # noqa: E731
    q, k, v, o = x(B, H, K), x(B, H, K), x(B, H, V), x(B, H, V)
    state = torch.from_numpy(r.standard_normal((n_slots, H, K, V)).astype(np.float32)).to(DEV)
    slots = r.permutation(n_slots)[:B].astype(np.int32)
    if B > 1:
        slots[1] = -1
    g = np.array([-0.5, -np.inf, 0.0][:H], dtype=np.float32)
    ref_o, ref_s = step_ref(*(t.float().cpu().numpy() for t in (q, k, v)), g, state.cpu().numpy(), slots, K ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gcl.dla_step(q, k, v, torch.from_numpy(g).to(DEV), state, o, slots=torch.from_numpy(slots).to(DEV), dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check("step o", o.float().cpu().numpy().reshape(1, B * H, 1, V), ref_o.reshape(1, B * H, 1, V), STEP_TOL[dtype], reduction=False)
    check("step state", state.cpu().numpy(), ref_s, dla_ref.TOL_STATE)
    idle = [s for s in range(n_slots) if s not in slots]
    assert idle and np.array_equal(state.cpu().numpy()[idle], ref_s.astype(np.float32)[idle])


def test_step_slot_out_of_range_is_idle():
    q, state = torch.ones(3, 2, 64, device=DEV), torch.ones(2, 2, 64, 64, device=DEV)
    o, g = torch.full((3, 2, 64), CANARY, device=DEV), torch.zeros(2, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gcl.dla_step(q, q, q, g, state, o, slots=torch.tensor([2, -7, 0], dtype=torch.int32, device=DEV), dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 4 and (o[:2] == 0).all() and (o[2] != 0).all()
    assert (state[1] == 1).all() and (state[0] == 2).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_then_steps_continue_the_sequence(dtype):
    """ht of a prompt, advanced token by token, gives the rows and the state of the longer prompt."""
    c = Case(dtype, [150], 3, 128, 64, seed=21, t_pad=0)
    o, ht, _ = c.fwd()
    full = c.cud
    c.cud = torch.tensor([0, 143], dtype=torch.int32, device=DEV)
    _, state, _ = c.fwd()
    for t in range(143, 150):
        row = torch.empty(1, 3, 64, dtype=c.dt, device=DEV)
        gcl.dla_step(c.q[t:t + 1], c.k[t:t + 1], c.v[t:t + 1], c.g, state, row)
        tol = dla_ref.TOL[dtype] + STEP_TOL[dtype]
        check("step row", row.float().cpu().numpy()[None], o[t:t + 1].float().cpu().numpy()[None], tol, reduction=False)
    check("state", state.cpu().numpy(), ht.cpu().numpy(), 2 * dla_ref.TOL_STATE)
    c.cud = full


def test_step_states_past_32_bits():
    """A pool of 9 GB: the last state starts past element 2^31."""
    n = (1 << 31) // (128 * 128) + 2
    state = torch.empty(n, 1, 128, 128, device=DEV)
    state[n - 1] = 1.0
    state[0] = 5.0
    q = torch.ones(1, 1, 128, device=DEV)
    o = torch.empty(1, 1, 128, device=DEV)
    gcl.dla_step(q, q, q, torch.zeros(1, device=DEV), state, o, slots=torch.tensor([n - 1], dtype=torch.int32, device=DEV))
    assert (state[n - 1] == 2).all() and (state[0] == 5).all()
    assert torch.allclose(o, torch.full_like(o, 256 * 128 ** -0.5), rtol=1e-6)


def test_step_graph_replay():
    q = torch.randn(4, 2, 64, device=DEV)
    state, g = torch.randn(6, 2, 64, 64, device=DEV), torch.tensor([-0.1, -1.0], device=DEV)
    slots, o = torch.tensor([3, 0, 5, 1], dtype=torch.int32, device=DEV), torch.empty(4, 2, 64, device=DEV)
    eager_state, eager_o = state.clone(), torch.empty_like(o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gcl.dla_step(q, q, q, g, state, o, slots=slots)
    for s in ([3, 0, 5, 1], [-1, 2, 4, 0]):
        slots.copy_(torch.tensor(s, dtype=torch.int32))
        graph.replay()
        gcl.dla_step(q, q, q, g, eager_state, eager_o, slots=slots)
        torch.cuda.synchronize()
        assert torch.equal(state, eager_state) and torch.equal(o, eager_o)
