"""The norms around a block on the GPU against their definition in fp64 (tests/glr_ref.py, where the tolerances stand)."""
import itertools
import sys

import numpy as np
import pytest

import glr_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402

DEV = "cuda:0"
F32, I32, I64 = torch.float32, torch.int32, torch.int64
DT = {"f32": F32, "bf16": torch.bfloat16, "f16": torch.float16}
CANARY = 1536.0
EPS = 1e-5
SEED, OFFSET = -7_000_000_000_123, 5_000_000_017


def np64(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, T, H, D, dtype="bf16", stream=None, gate="silu", x=True, z=True, weights=True, post="rms", pre="rms", p=0.0,
                 scale=0.7, live=None, strided=True, seed=0):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        self.dtype, self.stream = dtype, stream or dtype
        self.T, self.H, self.D, self.live = T, H, D, T if live is None else live
        rnd = lambda n, dt: [self.rows(dt, strided and k % 2 == 0).copy_(torch.randn(T, H, D, generator=gen, device=DEV)) for k in range(n)]  # noqa: E731
        dt, st = DT[dtype], DT[self.stream]
        self.y, self.gate, self.dz = rnd(3, dt)
        self.x, self.dxo = rnd(2, st)
        self.act = gate if gate != "plain" else None
        if gate is None:
            self.gate = None
        self.x = self.x if x else None
        self.has_z, self.post, self.pre, self.p, self.scale = z, post, pre, p, scale
        w = lambda: (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt) if weights else None  # noqa: E731
        self.w_post, self.w_pre = w(), w()
        self.rng = torch.tensor([SEED, OFFSET], dtype=I64, device=DEV) if p else None
        self.cu = None if live is None else torch.tensor([0, live // 2, live // 2, live], dtype=I32, device=DEV)
        self.status = torch.zeros(1, dtype=I32, device=DEV)
        self.kw = dict(post_norm=post, pre_norm=pre, activation=self.act, scale=scale, eps=EPS, dropout=p, rng=self.rng,
                       cu_seqlens=self.cu, dev_status=self.status)

    def rows(self, dt, strided=True):
        """Canaries [T, H, D], head-major with wider rows where strided."""
        if not strided:
            return torch.full((self.T, self.H, self.D), CANARY, dtype=dt, device=DEV)
        return torch.full((self.H, self.T, self.D + 8), CANARY, dtype=dt, device=DEV)[:, :, 8:].transpose(0, 1) if 8 * dt.itemsize % 16 == 0 else None

    def fwd(self, xo=True):
        self.xo = self.rows(DT[self.stream]) if xo else None
        self.z = self.rows(DT[self.dtype], False) if self.has_z else None
        gcl.block_norm_fwd(self.y, self.xo, x=self.x, z=self.z, gate=self.gate, post_weight=self.w_post,
                           pre_weight=self.w_pre if self.has_z else None, **self.kw)
        return self.xo, self.z

    def bwd(self, dxo=True, dz=True, dx=True):
        dz = dz and self.has_z
        out = dict(dy=self.rows(DT[self.dtype]), dgate=self.rows(DT[self.dtype], False) if self.gate is not None else None,
                   dx=self.rows(DT[self.stream], False) if dx and self.x is not None else None,
                   dpost_weight=torch.full((self.D,), CANARY, device=DEV) if self.w_post is not None else None,
                   dpre_weight=torch.full((self.D,), CANARY, device=DEV) if self.w_pre is not None and dz else None)
        ws = torch.full((gcl.block_norm_bwd_workspace_bytes(self.y),), 0xFF, dtype=torch.uint8, device=DEV)
        gcl.block_norm_bwd(self.y, self.dxo if dxo else None, x=self.x, dz=self.dz if dz else None, gate=self.gate,
                           post_weight=self.w_post, pre_weight=self.w_pre if dz else None, workspace=ws, **out, **self.kw)
        return out

    def plain(self):
        f = float(np.float32(self.scale)) * ref.keep((self.T, self.H, self.D), self.p, SEED, OFFSET)
        return [np64(t) for t in (self.y, self.gate, self.x)], [np64(self.w_post), np64(self.w_pre), f, self.post, self.pre, self.act, EPS]

    def check_rows(self, name, got, want, dtype):
        if got is None:
            return
        L = self.live
        ref.check(name, np64(got)[:L], want[:L], dtype, ref.E_NORM)
        assert (np64(got)[L:] == CANARY).all(), f"{name}: rows behind the last sequence were written"

    def check_fwd(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        rows, rest = self.plain()
        xo, z = ref.block_fwd(*rows, *rest)
        self.check_rows("xo", self.xo, xo, self.stream)
        self.check_rows("z", self.z, z, self.dtype)

    def check_bwd(self, out, dxo=True, dz=True):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        rows, rest = self.plain()
        L = self.live
        rows = [None if r is None else r[:L] for r in rows]
        rest[2] = rest[2][:L]
        want = ref.block_bwd(*rows, np64(self.dxo)[:L] if dxo else None, np64(self.dz)[:L] if dz and self.has_z else None, *rest)
        for n, v, dt in (("dy", want[0], self.dtype), ("dgate", want[1], self.dtype), ("dx", want[2], self.stream)):
            self.check_rows(n, out[n], np.concatenate([v, np.zeros((self.T - L,) + v.shape[1:])]), dt)
        for n, v, s in (("dpost_weight", want[3], want[5]), ("dpre_weight", want[4], want[6])):
            if out[n] is not None:
                ref.check(n, np64(out[n]), v, "f32", ref.E_NORM, s)

    def check(self):
        self.fwd()
        self.check_fwd()
        self.check_bwd(self.bwd())


WIDTHS = [8, 64, 72, 128, 136, 256, 264, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,stream", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_widths(dtype, stream, D):
    Case(37, 1, D, dtype, stream, p=0.1, live=33, seed=D).check()


@pytest.mark.parametrize("post,pre", list(itertools.product(["rms", "l2", "none"], repeat=2)))
@pytest.mark.parametrize("gate", [None, "plain", "silu", "sigmoid"])
def test_norms_and_gates(gate, post, pre):
    Case(50, 2, 72, "f32", gate=gate, post=post, pre=pre, weights=gate is not None, seed=3).check()
    Case(9, 1, 1160, "bf16", "f32", gate=gate, post=post, pre=pre, weights=gate is None, p=0.5, seed=4).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H,D", [(1, 1, 8), (1, 16, 128), (5, 1, 2048), (200, 16, 128), (33, 7, 64), (3, 3, 256)])
def test_parts_left_out(dtype, T, H, D):
    Case(T, H, D, dtype, x=False, z=False).check()                          # gated norm of each head
    Case(T, H, D, dtype, gate=None, post="none", weights=False).check()     # residual sum and the next norm
    Case(T, H, D, dtype, gate=None, x=False, post="none", p=0.25).check()   # no residual
    c = Case(T, H, D, dtype, gate=None, x=False, scale=1.0, post="none", weights=False)
    c.fwd(xo=False)                                                         # a norm alone
    c.check_fwd()
    c = Case(T, H, D, dtype)
    for dxo, dz in ((True, False), (False, True)):
        c.check_bwd(c.bwd(dxo, dz, dx=dz), dxo, dz)


def test_many_rows():
    """More rows than resident blocks hold at once, and their gradients' sums."""
    for args in ((30000, 1, 136), (3000, 16, 128), (4000, 1, 2048), (1500, 1, 4096)):
        c = Case(*args, "bf16", p=0.1, live=args[0] - 3)
        c.check()
        a, b = c.bwd(), c.bwd()
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_in_place():
    for D in (72, 2048):
        c = Case(40, 1, D, "bf16", "f32", p=0.1, strided=False)
        xo, z = (t.clone() for t in c.fwd())
        want = c.bwd()
        x, d = c.x.clone(), c.dxo.clone()
        z2, dy, dg = torch.empty_like(z), torch.empty_like(c.y), torch.empty_like(c.y)
        gcl.block_norm_bwd(c.y, d, dy, x=c.x, dx=d, dz=c.dz, gate=c.gate, dgate=dg, post_weight=c.w_post, pre_weight=c.w_pre, **c.kw)
        assert torch.equal(d, want["dx"]) and torch.equal(dy, want["dy"]) and torch.equal(dg, want["dgate"])
        gcl.block_norm_fwd(c.y, x, x=x, z=z2, gate=c.gate, post_weight=c.w_post, pre_weight=c.w_pre, **c.kw)
        assert torch.equal(x, xo) and torch.equal(z2, z)


@pytest.mark.parametrize("p", [0.1, 0.5, 0.999])
def test_dropout_share_and_scale(p):
    """The share that is kept, within six deviations; kept values carry scale / (1 - p), and the mask is the generator's."""
    c = Case(400, 1, 1000, "f32", gate=None, x=False, z=False, weights=False, post="none", p=p, scale=1.0, strided=False)
    c.fwd()
    c.check_fwd()
    cut = round(p * 65536)
    n, q = c.y.numel(), 1 - cut / 65536
    share = float((c.xo != 0).double().mean())
    assert abs(share - q) <= 6 * (q * (1 - q) / n) ** 0.5
    first = c.xo.clone()
    c.rng[1] += 1
    c.fwd()
    assert not torch.equal(c.xo != 0, first != 0)


def test_two_dimensional_rows():
    y, x = (torch.randn(30, 200, device=DEV).bfloat16()[:, :136] for _ in range(2))
    xo, z = torch.empty(30, 136, device=DEV, dtype=torch.bfloat16), torch.empty(30, 136, device=DEV, dtype=torch.bfloat16)
    gcl.block_norm_fwd(y, xo, x=x, z=z)
    want = ref.block_fwd(np64(y), None, np64(x), None, None, 1.0, "rms", "rms", None, 1e-6)
    for n, a, b in zip(("xo", "z"), (xo, z), want):
        ref.check(n, np64(a), b, "bf16", ref.E_NORM)


def test_values_that_are_not_finite_stay_in_their_row():
    for D, H in ((128, 4), (2048, 1)):
        c = Case(20, H, D, "bf16", live=15)
        clean = [t.clone() for t in c.fwd()]
        grads = {n: v.clone() for n, v in c.bwd().items()}
        c.y[3, 0, 5], c.x[7, H - 1, 2], c.gate[9, 0, 1] = float("nan"), float("inf"), float("nan")
        for t in (c.y, c.gate, c.x, c.dxo, c.dz):
            t[15:] = float("nan")
        got = c.fwd()
        ok = torch.ones(20, H, dtype=torch.bool, device=DEV)
        ok[3, 0] = ok[7, H - 1] = ok[9, 0] = False
        for a, b in zip(got, clean):
            assert torch.equal(a[ok], b[ok])
        assert not got[1][3, 0].isfinite().any()
        out = c.bwd()
        for n in ("dy", "dgate", "dx"):
            assert torch.equal(out[n][ok], grads[n][ok]), n


def test_far_rows():
    """Token strides that put the last rows past 2^31 elements."""
    T, D, stride = 140, 64, 1 << 24
    c = Case(T, 1, D, "bf16", strided=False)
    far = torch.empty((T - 1) * stride + D, dtype=torch.bfloat16, device=DEV).as_strided((T, 1, D), (stride, D, 1))
    far.copy_(c.y)
    c.y = far
    c.check()


def test_status():
    c = Case(40, 1, 136, live=30)
    c.status.fill_(3)
    xo, z = c.fwd()
    out = c.bwd()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 3
    assert all((t == CANARY).all() for t in (xo, z, *out.values()))
    for bad in (-1, 41):
        c.status.zero_()
        c.cu[-1] = bad
        xo, z = c.fwd()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 4
        c.status.zero_()
        out = c.bwd()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 4
        assert all((t == CANARY).all() for t in (xo, z, *out.values()))
    c.status.zero_()
    c.cu.zero_()                                             # no live rows: nothing but zero gradients of the weights
    out = c.bwd()
    torch.cuda.synchronize()
    assert all((out[n] == CANARY).all() for n in ("dy", "dgate", "dx")) and all((out[n] == 0).all() for n in ("dpost_weight", "dpre_weight"))


def test_captured_calls_read_their_buffers():
    """A graph of forward and backward follows the live rows, the inputs and the generator's offset."""
    c = Case(60, 1, 264, "bf16", p=0.3, live=50)
    out = dict(dy=c.rows(DT["bf16"]), dgate=c.rows(DT["bf16"]), dx=c.rows(DT["bf16"]), dpost_weight=torch.empty(264, device=DEV),
               dpre_weight=torch.empty(264, device=DEV))
    c.xo, c.z = c.rows(DT["bf16"]), c.rows(DT["bf16"])
    ws = torch.full((gcl.block_norm_bwd_workspace_bytes(c.y),), 0xFF, dtype=torch.uint8, device=DEV)

    def call():
        gcl.block_norm_fwd(c.y, c.xo, x=c.x, z=c.z, gate=c.gate, post_weight=c.w_post, pre_weight=c.w_pre, **c.kw)
        gcl.block_norm_bwd(c.y, c.dxo, x=c.x, dz=c.dz, gate=c.gate, post_weight=c.w_post, pre_weight=c.w_pre, workspace=ws, **out, **c.kw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    global OFFSET
    was = OFFSET
    try:
        for k, live in enumerate((50, 1, 60, 17)):
            c.live, OFFSET = live, was + k
            c.cu.copy_(torch.tensor([0, live // 2, live // 2, live]))
            c.rng[1] = OFFSET
            c.y.mul_(-0.5)
            for t in (c.xo, c.z, *out.values()):
                t.fill_(CANARY)
            graph.replay()
            c.check_fwd()
            c.check_bwd(out)
    finally:
        OFFSET = was


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_no_eps(norm, monkeypatch):
    """eps = 0: rows that a block holds no more of add nothing to the weights' gradients (not 0 times infinity)."""
    monkeypatch.setattr(sys.modules[__name__], "EPS", 0.0)
    for T, live in ((5, None), (37, 30)):
        Case(T, 1, 64, "bf16", post=norm, pre=norm, live=live).check()


@pytest.mark.parametrize("gate", ["plain", "silu", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gates_that_are_not_numbers_are_passed_on(dtype, gate):
    """A NaN of the gate: NaN in its value of xo, in its row of z and in its row of every gradient; other rows as without."""
    for D, H in ((128, 4), (2048, 1)):
        c = Case(12, H, D, dtype, gate=gate)
        clean, grads = [t.clone() for t in c.fwd()], c.bwd()
        c.gate[9, 0, 1] = float("nan")
        (xo, z), out = c.fwd(), c.bwd()
        bad = torch.zeros(12, H, D, dtype=torch.bool, device=DEV)
        bad[9, 0, 1] = True
        assert xo[bad].isnan().all() and torch.equal(xo[~bad], clean[0][~bad])
        bad[9, 0] = True
        for a, b in ((z, clean[1]), *((out[n], grads[n]) for n in ("dy", "dgate", "dx"))):
            assert a[bad].isnan().all() and torch.equal(a[~bad], b[~bad])
        assert out["dpost_weight"].isnan().all() and out["dpre_weight"].isnan().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_far_gates(dtype):
    """Gates whose exponential overflows: SiLU, the sigmoid and their slopes are 0 there, not the gate times the least sigmoid."""
    top = float(torch.finfo(DT[dtype]).max)
    for gate in ("silu", "sigmoid"):
        c = Case(3, 1, 72, dtype, gate=gate)
        c.gate[1, 0, :11] = torch.tensor([-top, -top / 1e3, -1e4, -150.0, -100.0, -90.0, -88.0, -87.0, -60.0, 100.0, 60.0])
        c.check()


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("size", [1e-16, 1e-13, 1e14, 1e17])
def test_rows_of_extreme_length(norm, size, monkeypatch):
    """Rows whose inverse length has a cube outside fp32's range: the gradients themselves are inside it."""
    monkeypatch.setattr(sys.modules[__name__], "EPS", 0.0)
    for D in (64, 1024):
        c = Case(7, 1, D, "f32", post=norm, pre=norm, scale=size)
        c.x.mul_(size)
        c.fwd()
        c.check_fwd()
        c.check_bwd(c.bwd(dxo=False), dxo=False)
        if size < 1:
            c.check_bwd(c.bwd())
