"""Timed cases of the operators of a gated recurrent block.

Two families, each in every direction that a block needs:

* the gated linear recurrence, per channel and per sequence
      h_t = a_t h_{t-1} + m(a_t) u_t,   u_t = x_t sigmoid(i_t)   (x_t without an input gate)
  with a_t = exp(r_t), sigmoid(r_t) or exp(-rate sigmoid(r_t)) and m(a) = 1, 1 - a or sqrt(1 - a^2):
  over packed sequences, its backward pass, and the single-token form on a pool of states;
* the norms after and before a block, with its gate, dropout, residual scale and residual sum,
      xo = x + scale drop(act(gate) norm(y) w_post),   z = norm(xo) w_pre,
  and its backward pass; dropout's mask is a function of a seed, an offset and the element's index
  (Philox4x32-10, Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
  2011) and is never stored.

``own`` chooses the side: False computes the plain form (elementary torch operations, fp32), True
calls the library.  ``exact`` evaluates the definitions in fp64, the recurrence token by token, apart
from both.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SAVE = 64                        # tokens between the states that a training forward saves
EPS = 1e-6


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # prefill of one long prompt: few channels beside the tokens, so that time itself has to be split
        dict(name="recurrence long prompt", op="fwd", dtype="bf16", T=65536, N=1, slots=1, D=2048, decay="power", mix="root", gate=True, packed=True, save=False),
        # serving prefill of a mixed batch: 32 prompts of 1 to some thousand tokens in 64 slots
        dict(name="recurrence mixed prompts", op="fwd", dtype="bf16", T=33000, N=32, slots=64, D=2048, decay="power", mix="root", gate=True, packed=True, save=False),
        # the smallest prefill: a handful of short odd prompts of a small model, fp16
        dict(name="recurrence short fp16", op="fwd", dtype="f16", T=777, N=3, slots=3, D=512, decay="sigmoid", mix="complement", gate=False, packed=False, save=False),
        # the training step's backward: 4 sequences of 8,192 tokens, with the states that the forward saved
        dict(name="recurrence backward training", op="bwd", dtype="bf16", T=32768, N=4, slots=4, D=2048, decay="power", mix="root", gate=True, packed=True, save=True),
        # fp32 gradients of a small model with log decays, states not saved
        dict(name="recurrence backward fp32", op="bwd", dtype="f32", T=1000, N=2, slots=3, D=200, decay="log", mix="one", gate=False, packed=False, save=False),
        # decoding with a full batch: one token of each of 256 requests
        dict(name="recurrence step 256 requests", op="step", dtype="bf16", B=256, pool=300, D=2048, decay="power", mix="root", gate=True),
        # decoding for a single small request, where latency counts
        dict(name="recurrence step one request", op="step", dtype="f16", B=1, pool=4, D=512, decay="sigmoid", mix="complement", gate=False),
        # training forward between two blocks: gated post-norm, dropout, residual, the next block's pre-norm
        dict(name="norms training", op="norm_fwd", dtype="bf16", stream="bf16", T=32768, H=1, D=2048, post="rms", pre="rms", weights=True, act="silu", gate=True, residual=True, p=0.1),
        # its backward
        dict(name="norms backward training", op="norm_bwd", dtype="bf16", stream="bf16", T=32768, H=1, D=2048, post="rms", pre="rms", weights=True, act="silu", gate=True, residual=True, p=0.1),
        # serving: the norm of each head's output with its gate, before the output projection
        dict(name="norms gated heads", op="norm_fwd", dtype="bf16", stream="bf16", T=33000, H=16, D=128, post="rms", pre=None, weights=True, act="silu", gate=True, residual=False, p=0.0),
        # one decoding step of a few requests: residual sum and pre-norm
        dict(name="norms decode", op="norm_fwd", dtype="f16", stream="f16", T=5, H=1, D=2048, post="none", pre="rms", weights=True, act=None, gate=False, residual=True, p=0.0),
        # fp32 gradients of an odd batch with dropout
        dict(name="norms backward fp32", op="norm_bwd", dtype="f32", stream="f32", T=1001, H=1, D=1000, post="l2", pre="rms", weights=True, act="sigmoid", gate=True, residual=True, p=0.25),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if op in ("fwd", "bwd", "step"):
        kind = dict(decay=rng.choice(["power", "power", "sigmoid", "log"]), mix=rng.choice(["root", "complement", "one"]),
                    gate=rng.choice([False, True]))
        D = 8 * _log_int(rng, 1, 512)
        if op == "step":
            B = _log_int(rng, 1, min(256, 524288 // D))
            return dict(op=op, dtype=dtype, B=B, pool=B + rng.randrange(0, 40), D=D, **kind)
        most = (1 << (27 if op == "fwd" else 26)) // (2 if dtype == "f32" else 1)
        T = _log_int(rng, 1, min(65536, most // D))
        N = min(T, _log_int(rng, 1, 40))
        return dict(op=op, dtype=dtype, T=T, N=N, slots=N + rng.choice([0, 0, 1, 9]), D=D, packed=rng.choice([False, True]),
                    save=rng.choice([False, True]), **kind)
    H = rng.choice([1, 1, 1, 2, 6, 16])
    D = 8 * _log_int(rng, 1, 1024 if H == 1 else 32)
    residual = rng.choice([False, True, True]) if H == 1 else False
    gate = rng.choice([False, True])
    post, pre = rng.choice(["rms", "rms", "l2", "none"]), rng.choice(["rms", "l2", None]) if residual else None
    most = (1 << 26) // (H * D) // (2 if dtype == "f32" else 1)
    return dict(op=op, dtype=dtype, stream=rng.choice([dtype, "f32"]) if residual else dtype, T=_log_int(rng, 1, min(33000, most)), H=H, D=D,
                post=post, pre=pre, weights=rng.choice([False, True]), act=rng.choice(["silu", "sigmoid", None]) if gate else None,
                gate=gate, residual=residual, p=rng.choice([0.0, 0.1, 0.5]))


def _lengths(case):
    """The case's sequence lengths: N >= 1 live lengths that sum to T (log-normal spread), then empty slots."""
    T, N = case["T"], case["N"]
    gen = torch.Generator()
    gen.manual_seed(T * 131 + N)
    w = torch.ones(N, dtype=torch.float64)
    if T % (N * 64):
        w = torch.exp(0.8 * torch.randn(N, generator=gen, dtype=torch.float64))
    cut = torch.floor(w.cumsum(0) / w.sum() * (T - N)).long()
    lens = (torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)) + 1).tolist()
    lens[-1] += T - sum(lens)
    return lens + [0] * (case["slots"] - N)


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dt, gen = DTYPES[case["dtype"]], torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rnd(*shape, dtype=dt, mul=1.0, add=0.0):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
        return x.mul_(mul).add_(add).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(shape, device=DEV, dtype=dtype)

    f32 = torch.float32
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        T, H, D, st = case["T"], case["H"], case["D"], DTYPES[case["stream"]]
        s["y"] = rnd(T, H, D, mul=1.5)
        s["gate"] = rnd(T, H, D) if case["gate"] else None
        s["x"] = rnd(T, H, D, dtype=st, mul=2.0) if case["residual"] else None
        s["w_post"] = rnd(D, mul=0.1, add=1.0) if case["weights"] else None
        s["w_pre"] = rnd(D, mul=0.1, add=1.0) if case["weights"] and case["pre"] else None
        s["scale"] = 0.5 if case["residual"] else 1.0        # the residual scale of the branch
        s["rng"] = torch.tensor([seed * 7919 + 13, seed + 1], dtype=torch.int64, device=DEV)
        if op == "norm_fwd":
            s["xo"], s["z"] = empty(T, H, D, dtype=st), empty(T, H, D) if case["pre"] else None
        else:
            s["dxo"], s["dz"] = rnd(T, H, D, dtype=st), rnd(T, H, D) if case["pre"] else None
            s["dy"], s["dgate"] = empty(T, H, D), empty(T, H, D) if case["gate"] else None
            s["dx"] = empty(T, H, D, dtype=st) if case["residual"] else None
            for n in ("post", "pre"):
                s["dw_" + n] = empty(D, dtype=f32) if s["w_" + n] is not None else None
        return s
    D, R = case["D"], case["B"] if op == "step" else case["T"]
    bias = {"power": 0.0, "sigmoid": 3.0, "log": 0.0}[case["decay"]]
    if case.get("packed"):                               # x, r and the input gate as slices of one projection's output
        rows = rnd(R, 3 * D)
        s["x"], s["r"] = rows[:, :D], rows[:, D:2 * D].add_(bias)
        s["i"] = rows[:, 2 * D:] if case["gate"] else None
    else:
        s["x"], s["r"] = rnd(R, D), rnd(R, D, add=bias)
        s["i"] = rnd(R, D) if case["gate"] else None
    if case["decay"] == "log":
        s["r"].copy_(-torch.exp(s["r"].float() - 3.0))
    # per channel: a decay of 0.9 to 0.999 to the eighth power where the gate is open
    s["rate"] = -8.0 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device=DEV)) if case["decay"] == "power" else None
    s["o"] = empty(R, D)
    if op == "step":
        s["state"] = rnd(case["pool"], D, dtype=f32)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=DEV)[:R].to(torch.int32)
        return s
    lens = torch.tensor(_lengths(case))
    s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).to(torch.int32).to(DEV)
    N, saved = case["slots"], -(-R // SAVE)
    s["h0"] = rnd(N, D, dtype=f32)
    s["save"] = empty(saved, D, dtype=f32) if case["save"] else None
    if op == "fwd":
        s["ht"] = empty(N, D, dtype=f32)
        return s
    s["do"], s["dht"] = rnd(R, D), rnd(N, D, dtype=f32)
    s["dx"], s["dr"], s["di"] = empty(R, D), empty(R, D), empty(R, D) if case["gate"] else None
    s["dh0"] = empty(N, D, dtype=f32)
    s["drate"] = empty(D, dtype=f32) if case["decay"] == "power" else None
    if case["save"]:                                     # what the training forward left
        s["save"].copy_(_plain_states(s)[3][::SAVE])
    return s


# --------------------------------------------------------------------------- the library's calls
def _run_own(s):
    import chunked_gated_linear_gb300 as gcl
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        gcl.block_norm_fwd(s["y"], s["xo"], x=s["x"], z=s["z"], gate=s["gate"], post_weight=s["w_post"], pre_weight=s["w_pre"],
                           post_norm=c["post"], pre_norm=c["pre"], activation=c["act"], scale=s["scale"], eps=EPS,
                           dropout=c["p"], rng=s["rng"], dev_status=s["status"])
        return {n: s[n] for n in ("xo", "z") if s[n] is not None}
    if op == "norm_bwd":
        if "ws" not in s:                        # the workspace, kept by the program
            s["ws"] = torch.empty(gcl.block_norm_bwd_workspace_bytes(s["y"]), dtype=torch.uint8, device=DEV)
        gcl.block_norm_bwd(s["y"], s["dxo"], s["dy"], x=s["x"], dx=s["dx"], dz=s["dz"], gate=s["gate"], dgate=s["dgate"],
                           post_weight=s["w_post"], pre_weight=s["w_pre"], dpost_weight=s["dw_post"], dpre_weight=s["dw_pre"],
                           post_norm=c["post"], pre_norm=c["pre"], activation=c["act"], scale=s["scale"], eps=EPS,
                           dropout=c["p"], rng=s["rng"], dev_status=s["status"], workspace=s["ws"])
        return {n: s[n] for n in ("dy", "dgate", "dx", "dw_post", "dw_pre") if s[n] is not None}
    kind = dict(i=s["i"], rate=s["rate"], decay=c["decay"], mix=c["mix"], dev_status=s["status"])
    if op == "step":
        gcl.glr_step(s["x"], s["r"], s["state"], s["o"], slots=s["slots"], **kind)
        return {"o": s["o"], "state": s["state"]}
    if op == "fwd":
        if "ws" not in s:
            s["ws"] = torch.empty(gcl.glr_fwd_workspace_bytes(s["x"], s["cu"]), dtype=torch.uint8, device=DEV)
        gcl.glr_fwd(s["x"], s["r"], s["cu"], s["o"], h0=s["h0"], ht=s["ht"], h_save=s["save"], workspace=s["ws"], **kind)
        return {n: s[n] for n in ("o", "ht", "save") if s[n] is not None}
    if "ws" not in s:
        s["ws"] = torch.empty(gcl.glr_bwd_workspace_bytes(s["x"], s["cu"], h_save=s["save"]), dtype=torch.uint8, device=DEV)
    gcl.glr_bwd(s["x"], s["r"], s["do"], s["cu"], s["dx"], s["dr"], di=s["di"], drate=s["drate"], h0=s["h0"], dht=s["dht"],
                dh0=s["dh0"], h_save=s["save"], workspace=s["ws"], **kind)
    return {n: s[n] for n in ("dx", "dr", "di", "drate", "dh0") if s[n] is not None}


# --------------------------------------------------------------------------- the plain forms
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _gates(s):
    """log a, a, m(a), u and the input gate's value, fp32."""
    c, r = s["case"], s["r"].float()
    if c["decay"] == "log":
        la, a = r, torch.exp(r)
    elif c["decay"] == "sigmoid":
        la, a = -(torch.log1p(torch.exp(-r.abs())) + (-r).clamp(min=0)), _sigmoid(r)
    else:
        la = -s["rate"] * _sigmoid(r)
        a = torch.exp(la)
    m = {"one": lambda: torch.ones_like(a), "complement": lambda: -torch.expm1(la),
         "root": lambda: torch.sqrt((-torch.expm1(2 * la)).clamp(min=0))}[c["mix"]]()
    u, gate = s["x"].float(), None
    if s["i"] is not None:
        gate = _sigmoid(s["i"].float())
        u = u * gate
    return la, a, m, u, gate


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis from zero, by doubling within runs of 64 and over the runs' ends."""
    T, D = a.shape
    C = 64
    pad = -T % C
    if pad:
        a, b = torch.cat([a, a.new_ones(pad, D)]), torch.cat([b, b.new_zeros(pad, D)])
    A, B = a.view(-1, C, D).clone(), b.view(-1, C, D).clone()
    step = 1
    while step < C:
        B[:, step:] += A[:, step:] * B[:, :-step].clone()
        A[:, step:] *= A[:, :-step].clone()
        step *= 2
    if len(A) > 1:
        ends = _scan(A[:, -1], B[:, -1])
        B[1:] += A[1:] * ends[:-1, None]
    return B.view(-1, D)[:T]


def _ranges(s):
    """First and last tokens of the sequences that have some, and which they are."""
    cu = s["cu"].long()
    some = torch.nonzero(cu[1:] > cu[:-1])[:, 0]
    return cu[some], cu[some + 1] - 1, some


def _plain_states(s):
    """a, b and the states after and before each token."""
    _, a, m, u, _ = _gates(s)
    first, _, some = _ranges(s)
    A, B = a.clone(), m * u
    B[first] += a[first] * s["h0"][some]
    A[first] = 0
    h = _scan(A, B)
    before = torch.cat([h.new_zeros(1, h.shape[1]), h[:-1]])
    before[first] = s["h0"][some]
    return a, B, h, before


def _plain_fwd(s):
    _, _, h, before = _plain_states(s)
    _, last, some = _ranges(s)
    ht = s["h0"].clone()
    ht[some] = h[last]
    out = {"o": h.to(s["x"].dtype), "ht": ht}
    if s["case"]["save"]:
        out["save"] = before[::SAVE].contiguous()
    return out


def _plain_bwd(s):
    c, dt = s["case"], s["x"].dtype
    before = _plain_states(s)[3]
    la, a, m, u, gate = _gates(s)
    first, last, some = _ranges(s)
    nxt = torch.cat([a[1:], a.new_zeros(1, a.shape[1])])     # G_t = do_t + a_{t+1} G_{t+1} within a sequence
    nxt[last] = 0
    g = s["do"].float().clone()                              # (fp32 rows would be changed in place)
    g[last] += s["dht"][some]
    G = _scan(nxt.flip(0), g.flip(0)).flip(0)
    dh0 = s["dht"].clone()
    dh0[some] = a[first] * G[first]
    dla = a * G * before
    if c["mix"] == "complement":
        dla = dla - G * u * a
    elif c["mix"] == "root":
        dla = dla - G * u * torch.where(m > 0, a * a / m, torch.zeros_like(m))
    r, x = s["r"].float(), s["x"].float()
    out = {"dx": (G * m if gate is None else G * m * gate).to(dt)}
    if c["decay"] == "log":
        dr = dla
    elif c["decay"] == "sigmoid":
        dr = dla * _sigmoid(-r)
    else:
        dr = dla * la * _sigmoid(-r)
        out["drate"] = -(dla * _sigmoid(r)).double().sum(0).float()
    out["dr"] = dr.to(dt)
    if gate is not None:
        out["di"] = (G * m * x * gate * _sigmoid(-s["i"].float())).to(dt)
    out["dh0"] = dh0
    return out


def _plain_step(s):
    _, a, m, u, _ = _gates(s)
    at = s["slots"].long()
    h = a * s["state"][at] + m * u
    s["state"][at] = h
    return {"o": h.to(s["x"].dtype), "state": s["state"]}


def _keep(s, shape):
    """Dropout's factors: element e of the whole tensor takes half-word e % 8 of block e / 8 of the generator."""
    p = s["case"]["p"]
    cut = round(p * 65536)
    n = math.prod(shape)
    low = 0xFFFFFFFF
    blocks = torch.arange(-(-n // 8), dtype=torch.int64, device=DEV)
    seed, offset = s["rng"][0], s["rng"][1]
    ctr = [blocks & low, blocks >> 32, (offset & low).expand_as(blocks), ((offset >> 32) & low).expand_as(blocks)]
    key = [seed & low, (seed >> 32) & low]
    for _ in range(10):
        p0, p1 = ctr[0] * 0xD2511F53, ctr[2] * 0xCD9E8D57        # (they wrap; the bits of both halves are right)
        ctr = [((p1 >> 32) & low) ^ ctr[1] ^ key[0], p1 & low, ((p0 >> 32) & low) ^ ctr[3] ^ key[1], p0 & low]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    halves = torch.stack([h for w in ctr for h in (w & 0xFFFF, w >> 16)], -1).reshape(-1)[:n]
    return (halves >= cut).view(shape).float() * (65536.0 / (65536 - cut))


def _length(x, norm):
    """1 / the norm's length of each row."""
    if norm == "none":
        return torch.ones_like(x[..., :1])
    ss = x.square()
    return 1.0 / torch.sqrt((ss.mean(-1, keepdim=True) if norm == "rms" else ss.sum(-1, keepdim=True)) + EPS)


def _branch(s):
    """y's scale, w_post and scale times the dropout factors, the gate's value and its slope (fp32)."""
    c, y = s["case"], s["y"].float()
    ry = _length(y, c["post"])
    w = s["w_post"].float() if s["w_post"] is not None else torch.ones(c["D"], device=DEV)
    f = torch.full((), s["scale"], device=DEV)
    if c["p"] > 0:
        f = f * _keep(s, y.shape)
    act = slope = None
    if s["gate"] is not None:
        g = s["gate"].float()
        sg = _sigmoid(g)
        act, slope = {None: lambda: (g, torch.ones_like(g)), "sigmoid": lambda: (sg, sg * _sigmoid(-g)),
                      "silu": lambda: (g * sg, sg * (1 + g * _sigmoid(-g)))}[c["act"]]()
    return y, ry, w, f, act, slope


def _plain_norm_fwd(s):
    c, dt = s["case"], s["y"].dtype
    y, ry, w, f, act, _ = _branch(s)
    xo = y * ry * w * f
    if act is not None:
        xo = xo * act
    if s["x"] is not None:
        xo = xo + s["x"].float()
    out = {"xo": xo.to(DTYPES[c["stream"]])}
    if c["pre"]:
        z = xo * _length(xo, c["pre"])
        out["z"] = (z if s["w_pre"] is None else z * s["w_pre"].float()).to(dt)
    return out


def _norm_back(du, x, r, norm):
    """The gradient of x r(x) from that of the normed row."""
    if norm == "none":
        return du
    m = (du * x * r).sum(-1, keepdim=True) / (x.shape[-1] if norm == "rms" else 1)
    return r * (du - x * r * m)


def _plain_norm_bwd(s):
    c, dt, st = s["case"], s["y"].dtype, DTYPES[s["case"]["stream"]]
    y, ry, w, f, act, slope = _branch(s)
    n = y * ry
    d = s["dxo"].float()
    out = {}
    if c["pre"]:
        xo = n * w * f if act is None else n * w * f * act
        if s["x"] is not None:
            xo = xo + s["x"].float()
        r, dz = _length(xo, c["pre"]), s["dz"].float()
        if s["w_pre"] is not None:
            out["dw_pre"] = (dz * xo * r).double().sum((0, 1)).float()
            dz = dz * s["w_pre"].float()
        d = d + _norm_back(dz, xo, r, c["pre"])
    if s["x"] is not None:
        out["dx"] = d.to(st)
    d = d * f
    if act is not None:
        out["dgate"] = (d * n * w * slope).to(dt)
        d = d * act
    if s["w_post"] is not None:
        out["dw_post"] = (d * n).double().sum((0, 1)).float()
    out["dy"] = _norm_back(d * w, y, ry, c["post"]).to(dt)
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm_fwd": _plain_norm_fwd,
            "norm_bwd": _plain_norm_bwd}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- floors
def work(case):
    e = {"bf16": 2, "f16": 2, "f32": 4}
    op, b, D = case["op"], e[case["dtype"]], case["D"]
    if op in ("norm_fwd", "norm_bwd"):
        n, st, gate, res, pre = case["T"] * case["H"] * D, e[case["stream"]], case["gate"], case["residual"], bool(case["pre"])
        if op == "norm_fwd":                     # y, the gate, x; xo, z
            return {"bytes": n * (b * (1 + gate + pre) + st * (1 + res)), "flops": n * 16}
        need_x = res and pre                     # y, the gate, x, dxo, dz; dy, dgate, dx
        return {"bytes": n * (b * (2 + 2 * gate + pre) + st * (1 + need_x + res)), "flops": n * 40}
    gate = case["gate"]
    if op == "step":
        return {"bytes": case["B"] * D * (8 + b * (3 + gate)), "flops": case["B"] * D * 20}
    n, states = case["T"] * D, 2 * case["slots"] * D * 4
    saved = -(-case["T"] // SAVE) * D * 4 if case["save"] else 0
    if op == "fwd":
        return {"bytes": n * b * (3 + gate) + states + saved, "flops": n * 20}
    return {"bytes": n * b * (5 + 2 * gate) + states + case["slots"] * D * 4 + saved, "flops": n * 40}


# --------------------------------------------------------------------------- the definitions in fp64
def _walk(a, b, h, starts, h0):
    """Token by token, h <- a_t h + b_t, with h = h0[n] before the first token of sequence n; every state after its token."""
    out = torch.empty_like(b)
    for t in range(b.shape[0]):
        n = starts.get(t)
        if n is not None:
            h = h0[n]
        h = torch.addcmul(b[t], a[t], h, out=out[t])
    return out


def _exact_recurrence(case, s):
    op = case["op"]
    r, x = s["r"].double(), s["x"].double()
    sig = torch.special.expit
    if case["decay"] == "power":
        la = -s["rate"].double() * sig(r)
    else:
        la = r if case["decay"] == "log" else -torch.nn.functional.softplus(-r)
    a = la.exp()
    gate = sig(s["i"].double()) if s["i"] is not None else torch.ones((), dtype=torch.float64, device=DEV)
    m = {"one": torch.ones_like, "complement": lambda v: -torch.expm1(v), "root": lambda v: torch.sqrt(torch.relu(-torch.expm1(2 * v)))}[case["mix"]](la)
    if op == "step":
        at, state = s["slots"].long(), s["state"].double()
        h = torch.addcmul(m * gate * x, a, state[at])
        state[at] = h
        return {"o": h, "state": state}
    cu = s["cu"].tolist()
    live = [n for n in range(len(cu) - 1) if cu[n + 1] > cu[n]]
    h0 = s["h0"].double()
    h = _walk(a, m * gate * x, None, {cu[n]: n for n in live}, h0)
    prev = h.roll(1, 0)
    for n in live:
        prev[cu[n]] = h0[n]
    if op == "fwd":
        ht = h0.clone()
        for n in live:
            ht[n] = h[cu[n + 1] - 1]
        out = {"o": h, "ht": ht}
        if case["save"]:
            out["save"] = prev[::SAVE].clone()
        return out
    # backwards: lam_t is the gradient of h_t with its decay a_{t+1} from the token after; the last token's comes from dht
    T, dht = r.shape[0], s["dht"].double()
    ahead = torch.cat([a[1:], torch.ones_like(a[:1])])
    for n in live:
        ahead[cu[n + 1] - 1] = 1.0
    G = _walk(ahead.flip(0), s["do"].double().flip(0), None, {T - cu[n + 1]: n for n in live}, dht).flip(0)
    del ahead, h
    dh0 = dht.clone()
    for n in live:
        dh0[n] = a[cu[n]] * G[cu[n]]
    back = prev * a
    if case["mix"] == "complement":
        back = back - gate * x * a
    elif case["mix"] == "root":
        back = back - gate * x * torch.nan_to_num(a.square() / m, posinf=0.0, nan=0.0)
    dla = G * back
    out = {"dx": G * m * gate, "dh0": dh0}
    if case["decay"] == "log":
        out["dr"] = dla
    elif case["decay"] == "sigmoid":
        out["dr"] = dla * sig(-r)
    else:
        out["dr"] = dla * la * sig(-r)
        out["drate"] = -torch.einsum("td,td->d", dla, sig(r))
    if case["gate"]:
        out["di"] = G * m * x * gate * sig(-s["i"].double())
    return {n: out[n] for n in ("dx", "dr", "di", "drate", "dh0") if n in out}


def _generator(n, seed, offset):
    """n half-words of the counter generator, from 16-bit halves of its words (no product passes 2^49)."""
    dev, mask = DEV, 0xFFFFFFFF
    at = torch.arange((n + 7) // 8, dtype=torch.int64, device=dev)
    c0, c1 = at.remainder(1 << 32), at.div(1 << 32, rounding_mode="floor")
    c2, c3 = torch.full_like(at, offset % (1 << 32)), torch.full_like(at, (offset >> 32) % (1 << 32))
    k0, k1 = seed % (1 << 32), (seed >> 32) % (1 << 32)

    def product(k, v):
        low, high = (v % 65536) * k, v.div(65536, rounding_mode="floor") * k
        high = high + low.div(65536, rounding_mode="floor")
        return high.div(65536, rounding_mode="floor"), ((high % 65536) * 65536 + low % 65536) & mask

    for i in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ ((k0 + i * 0x9E3779B9) & mask), l1, h0 ^ c3 ^ ((k1 + i * 0xBB67AE85) & mask), l0
    words = torch.stack([c0, c1, c2, c3], 1)
    return torch.stack([words % 65536, words.div(65536, rounding_mode="floor")], 2).flatten()[:n]


def _exact_norm(case, s):
    D = case["D"]
    y = s["y"].double()
    one = torch.ones((), dtype=torch.float64, device=DEV)
    wp = s["w_post"].double() if s["w_post"] is not None else one
    wn = s["w_pre"].double() if s["w_pre"] is not None else one
    size = {"rms": 1.0 / D, "l2": 1.0, "none": None, None: None}

    def length(v, norm):
        return one if size[norm] is None else torch.linalg.vector_norm(v, dim=-1, keepdim=True).square().mul(size[norm]).add(EPS).sqrt()

    def back(g, v, ln, norm):                            # d(v / ln(v))
        return g if size[norm] is None else g / ln - v * ((g * v).sum(-1, keepdim=True) * size[norm] / ln ** 3)

    gate, slope = one, None
    if case["gate"]:
        g = s["gate"].double()
        p = torch.special.expit(g)
        gate = {None: g, "sigmoid": p, "silu": g * p}[case["act"]]
        slope = {None: torch.ones_like(g), "sigmoid": p - p * p, "silu": p + g * (p - p * p)}[case["act"]]
    factor = one * s["scale"]
    if case["p"]:
        cut = round(case["p"] * 65536)
        kept = (_generator(y.numel(), *s["rng"].tolist()) >= cut).view(y.shape)
        factor = kept.double() * (s["scale"] / (1 - cut / 65536))
    ly = length(y, case["post"])
    n = y / ly
    xo = n * wp * gate * factor
    if case["residual"]:
        xo = xo + s["x"].double()
    if case["op"] == "norm_fwd":
        out = {"xo": xo}
        if case["pre"]:
            out["z"] = xo / length(xo, case["pre"]) * wn
        return out
    dxo = s["dxo"].double()
    out = {}
    if case["pre"]:
        lx, dz = length(xo, case["pre"]), s["dz"].double()
        if case["weights"]:
            out["dw_pre"] = torch.einsum("thd,thd->d", dz, xo / lx)
        dxo = dxo + back(dz * wn, xo, lx, case["pre"])
    if case["residual"]:
        out["dx"] = dxo
    if case["gate"]:
        out["dgate"] = dxo * factor * n * wp * slope
    dn = dxo * factor * gate
    if case["weights"]:
        out["dw_post"] = torch.einsum("thd,thd->d", dn, n)
    out["dy"] = back(dn * wp, y, ly, case["post"])
    return {k: out[k] for k in ("dy", "dgate", "dx", "dw_post", "dw_pre") if k in out}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"].startswith("norm") else _exact_recurrence(case, s)
