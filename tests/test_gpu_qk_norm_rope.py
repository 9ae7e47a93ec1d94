"""The per-head norm with rotation on the GPU against fp64 (tests/dla_ref.py).

Tolerances: arithmetic is fp32 over a row of D <= 256 values, the result is rounded once.  A value may
be off by u of itself (u = eps / 2 of the type) and by the fp32 arithmetic, a few roundings of the
row's largest value: 8 x 2^-24 of it for the sums of squares, the inverse root (2 ulp), the products
and the rotation; 16 x 2^-24 in the backward, which has one more sum.  A weight's gradient is an fp32
sum over n rows in a fixed order of partial sums: 1e-5 of its norm, the fp32 bar."""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402
import dla_ref  # noqa: E402

DEV = "cuda:0"
CANARY = 1536.0
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
EPS = 1e-6
P = 500


def host(x):
    return x.float().cpu().numpy()


def near(name, got, ref, dtype, fp32_steps):
    got, big = host(got).astype(np.float64), np.abs(ref).max(-1, keepdims=True)
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0            # half a step of fp16's smallest values
    bar = U[dtype] * np.abs(ref) * (1 + 1e-3) + fp32_steps * 2.0 ** -24 * big + tiny
    worst = np.max(np.abs(got - ref) - bar)
    assert worst <= 0, f"{name}: over its bar by {worst:.3e}"


class Case:
    def __init__(self, dtype, T, HQ, HK, D, R, norm, weight, pairing, seed=0):
        r = np.random.default_rng(seed)
        self.dtype, self.R, self.D, self.norm, self.pairing = dtype, R, D, norm, pairing
        dt = DT[dtype]
        dev = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(dt).to(DEV)  # noqa: E731
        wide = dev(r.standard_normal((T, (HQ + 2 * HK) * D)))
        self.q = wide[:, :HQ * D].view(T, HQ, D)
        self.k = wide[:, HQ * D:(HQ + HK) * D].view(T, HK, D) if HK else None
        self.dyq, self.dyk = dev(r.standard_normal((T, HQ, D))), dev(r.standard_normal((T, HK, D))) if HK else None
        self.wq = dev(r.standard_normal(D)) if weight else None
        self.wk = dev(r.standard_normal(D)) if weight and HK else None
        self.pos = torch.from_numpy(r.integers(0, P, T).astype(np.int32)).to(DEV)
        if R:
            self.cos, self.sin = torch.empty(P, R // 2, device=DEV), torch.empty(P, R // 2, device=DEV)
            gcl.rope_table_build(self.cos, self.sin)
        else:
            self.cos = self.sin = None
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def kw(self):
        return dict(q_weight=self.wq, k_weight=self.wk, cos=self.cos, sin=self.sin, positions=self.pos, norm=self.norm,
                    eps=EPS, pairing=self.pairing, dev_status=self.status)

    def table(self):
        if not self.R:
            return None, None
        at = self.pos.cpu().numpy()
        return self.cos.cpu().numpy().astype(np.float64)[at], self.sin.cpu().numpy().astype(np.float64)[at]

    def fwd(self):
        yq, yk = torch.full_like(self.dyq, CANARY), None if self.k is None else torch.full_like(self.dyk, CANARY)
        gcl.qk_norm_rope_fwd(self.q, self.k, yq, yk, **self.kw())
        return yq, yk

    def bwd(self):
        dq, dk = torch.full_like(self.dyq, CANARY), None if self.k is None else torch.full_like(self.dyk, CANARY)
        dw = [None if w is None else torch.full((self.D,), CANARY, device=DEV) for w in (self.wq, self.wk)]
        ws = torch.full((gcl.qk_norm_rope_bwd_workspace_bytes(self.q, self.k),), 0xFF, dtype=torch.uint8, device=DEV)
        gcl.qk_norm_rope_bwd(self.q, self.k, self.dyq, self.dyk, dq, dk, dq_weight=dw[0], dk_weight=dw[1],
                             workspace=ws, **self.kw())
        return dq, dk, *dw

    def check(self, label):
        cos, sin = self.table()
        args = (cos, sin, self.R, self.norm, EPS, self.pairing)
        y, d = self.fwd(), self.bwd()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        for i, (x, w, dy) in enumerate(((self.q, self.wq, self.dyq), (self.k, self.wk, self.dyk))):
            if x is None:
                continue
            x, w, dy = host(x), None if w is None else host(w), host(dy)
            near(f"{label} y{i}", y[i], dla_ref.norm_rope(x, w, *args), self.dtype, 8)
            dx, dw = dla_ref.norm_rope_bwd(x, w, dy, *args)
            # the cancelling sum u - x (u x): its fp32 error is of the terms, at most 2 r max|u| a row
            near(f"{label} dx{i}", d[i], dx, self.dtype, 64)
            if w is not None:
                e = np.linalg.norm(host(d[2 + i]) - dw) / np.linalg.norm(dw)
                assert e <= 1e-5, f"{label} dw{i}: {e:.2e}"


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_values_and_gradients(dtype, D, pairing):
    for (norm, weight), R in itertools.product((("rms", True), ("l2", False), ("none", True), ("rms", False)),
                                               (0, 16, D // 2, D)):
        Case(dtype, 37, 3, 2, D, R, norm, weight, pairing, seed=D + R).check(f"{dtype} D{D} R{R} {norm} {pairing}")


@pytest.mark.parametrize("T,HQ,HK", [(1, 1, 1), (1, 5, 0), (700, 9, 3), (6000, 16, 7)])
def test_shapes(T, HQ, HK):
    """One row, queries alone, and sizes where a lane group takes several heads (the last group short)."""
    for dtype in DT:
        Case(dtype, T, HQ, HK, 128, 64, "rms", True, "half", seed=T).check(f"{dtype} {T}x{HQ}x{HK}")


def test_zero_rows_and_eps():
    """A row of zeros: finite with eps > 0, forward and backward."""
    c = Case("f32", 4, 2, 1, 64, 32, "l2", True, "half")
    c.q[2] = 0
    c.check("zero rows")


def test_padding_and_bad_positions():
    """Tokens with a negative position are neither read nor written and add nothing to the weights'
    gradients (also with eps = 0); a position past the table sets the status and skips its rows."""
    c = Case("bf16", 9, 2, 2, 64, 32, "rms", True, "adjacent")
    ref = c.fwd()
    live = [0, 1, 2, 5, 6, 8]
    pad = [3, 4, 7]
    c.pos[pad] = torch.tensor([-1, -5, -2147483648], dtype=torch.int32, device=DEV)
    for x in (c.q, c.k, c.dyq, c.dyk):
        x[pad] = float("nan")
    y, d = c.fwd(), c.bwd()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    for a, b in zip(y, ref):
        assert torch.equal(a[live], b[live]) and (a[pad] == CANARY).all()
    assert (d[0][pad] == CANARY).all() and (d[1][pad] == CANARY).all()
    assert all(torch.isfinite(x).all() for x in d)
    c.pos[0] = P
    y = c.fwd()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 4 and (y[0][0] == CANARY).all()


def test_in_place_forward_and_strided_outputs():
    """In place, and into slices of one buffer: the same bits."""
    c = Case("bf16", 50, 4, 2, 128, 128, "rms", True, "half", seed=3)
    y = c.fwd()
    wide = torch.full((50, 8 * 128), CANARY, dtype=torch.bfloat16, device=DEV)
    a, b = wide[:, 128:5 * 128].view(50, 4, 128), wide[:, 6 * 128:].view(50, 2, 128)
    gcl.qk_norm_rope_fwd(c.q, c.k, a, b, **c.kw())
    assert torch.equal(a, y[0]) and torch.equal(b, y[1]) and (wide[:, :128] == CANARY).all()
    gcl.qk_norm_rope_fwd(c.q, c.k, c.q, c.k, **c.kw())
    assert torch.equal(c.q, y[0]) and torch.equal(c.k, y[1])


def test_repeats_and_graph_replay_are_bitwise_equal():
    c = Case("bf16", 5000, 8, 4, 128, 64, "rms", True, "half", seed=4)
    first = [*c.fwd(), *c.bwd()]
    assert all(torch.equal(x, y) for x, y in zip(first, [*c.fwd(), *c.bwd()]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = [*c.fwd(), *c.bwd()]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, out))


def test_set_status_stops_the_work():
    c = Case("bf16", 20, 2, 1, 64, 32, "rms", True, "half")
    c.status.fill_(2)
    for x in (*c.fwd(), *c.bwd()):
        assert (x == CANARY).all()


@pytest.mark.parametrize("base", [10000.0, 1e6])
def test_rope_table(base):
    """Angles in fp64: each entry is the correctly rounded fp32 value, up to fp64's own error."""
    n, R = 150000, 64
    cos, sin = torch.empty(n, R // 2, device=DEV), torch.empty(n, R // 2, device=DEV)
    gcl.rope_table_build(cos, sin, base=base)
    at = np.r_[0:50, 100000:100050, n - 50:n]
    a = at[:, None] * base ** (-2.0 * np.arange(R // 2) / R)
    for got, ref in ((cos, np.cos(a)), (sin, np.sin(a))):
        assert np.abs(got.cpu().numpy()[at] - ref).max() <= 2.0 ** -24 + 1e-9
