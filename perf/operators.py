"""Timed cases of the linear-attention operators with a fixed decay for each head.

Two operators, each in every direction that a layer needs:

* decayed linear attention, gamma_h = exp(g_h), per sequence and head
      S_t = gamma S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
  as the chunked forward over packed sequences, its backward pass, and the single-token form on
  a pool of states;
* the norm of queries and keys for each head with the position rotation in the same pass, and
  its backward pass.

``own`` chooses the side: False computes the plain form (elementary torch operations, fp32, angles
and decay exponents in fp64), True calls the library.  ``exact`` evaluates the definitions token by
token in fp64, apart from both.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
CHUNK = 64                       # chunk of the plain form
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # serving prefill of a mixed batch: 32 prompts of 1 to 2,048 tokens in 64 slots
        dict(name="fwd mixed prompts", op="fwd", dtype="bf16", T=33000, N=32, slots=64, H=16, K=128, V=128, packed=True),
        # one long prompt of few heads: the sequence itself has to be split to fill the GPU
        dict(name="fwd one long prompt", op="fwd", dtype="bf16", T=65536, N=1, slots=1, H=4, K=128, V=128, packed=False),
        # the smallest prefill: a handful of short odd prompts of a small model, fp16, 64-wide heads
        dict(name="fwd short fp16", op="fwd", dtype="f16", T=777, N=3, slots=3, H=4, K=64, V=64, packed=False),
        # fp32 runs: the reference precision of a small model
        dict(name="fwd fp32", op="fwd", dtype="f32", T=4096, N=2, slots=2, H=8, K=64, V=64, packed=False),
        # the training step: 4 sequences of 8,192 tokens, 16 heads
        dict(name="bwd training batch", op="bwd", dtype="bf16", T=32768, N=4, slots=4, H=16, K=128, V=128, packed=False),
        # a ragged fine-tuning batch with narrow keys
        dict(name="bwd ragged narrow keys", op="bwd", dtype="bf16", T=5003, N=7, slots=8, H=6, K=64, V=128, packed=True),
        # fp32 gradients of a small model
        dict(name="bwd fp32", op="bwd", dtype="f32", T=1000, N=2, slots=2, H=4, K=128, V=64, packed=False),
        # decoding with a full batch: one token of each of 256 requests
        dict(name="step 256 requests", op="step", dtype="bf16", B=256, pool=300, H=16, K=128, V=128),
        # decoding for a single small request, where latency counts
        dict(name="step one request", op="step", dtype="f16", B=1, pool=4, H=4, K=64, V=64),
        # norm and rotation of a packed prefill batch
        dict(name="norm_rope prefill", op="nr_fwd", dtype="bf16", T=32768, HQ=16, HK=16, D=128, R=128, norm="rms", weight=True, pair="half"),
        # norm and rotation of the tokens of one decoding step
        dict(name="norm_rope decode", op="nr_fwd", dtype="f16", T=5, HQ=4, HK=4, D=64, R=32, norm="l2", weight=False, pair="adjacent"),
        # its gradient in training, with shared key heads
        dict(name="norm_rope backward", op="nr_bwd", dtype="bf16", T=16384, HQ=16, HK=2, D=128, R=64, norm="rms", weight=True, pair="half"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "nr_fwd", "nr_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if op in ("fwd", "bwd"):
        H = rng.choice([1, 2, 3, 4, 6, 10, 20])
        most = 65536 if dtype == "bf16" else 4096
        T = _log_int(rng, 1, min(most, (262144 if op == "fwd" else 131072) // H))
        N = min(T, _log_int(rng, 1, 40))
        return dict(op=op, dtype=dtype, T=T, N=N, slots=N + rng.choice([0, 0, 1, 9]), H=H, K=rng.choice([64, 128, 128]),
                    V=rng.choice([64, 128, 128]), packed=rng.choice([False, True]))
    if op == "step":
        B = _log_int(rng, 1, 256)
        return dict(op=op, dtype=dtype, B=B, pool=B + rng.randrange(0, 40), H=rng.choice([1, 2, 4, 5, 8, 16]),
                    K=rng.choice([64, 128, 128]), V=rng.choice([64, 128, 128]))
    D = rng.choice([64, 128, 128, 256])
    HK = rng.choice([1, 2, 5, 7, 10])
    return dict(op=op, dtype=dtype, T=_log_int(rng, 1, 16384), HQ=HK * rng.choice([1, 1, 2]), HK=HK, D=D,
                R=rng.choice([0, D // 4, D // 2, D]), norm=rng.choice(["rms", "rms", "l2", "none"]),
                weight=rng.choice([False, True]), pair=rng.choice(["half", "adjacent"]))


def _lengths(case):
    """The case's sequence lengths: N >= 1 live lengths that sum to T (log-normal spread), then empty slots."""
    T, N = case["T"], case["N"]
    r = np.random.Generator(np.random.PCG64(T * 131 + N))
    w = np.ones(N) if case["H"] >= 16 and T % (N * 64) == 0 else np.exp(0.8 * r.standard_normal(N))
    cut = np.floor(np.cumsum(w) / w.sum() * (T - N)).astype(np.int64)
    lens = np.diff(np.concatenate([[0], cut])) + 1
    lens[-1] += T - lens.sum()
    return lens.tolist() + [0] * (case["slots"] - N)


def _decay(H):
    """Log decays: a geometric ladder from fast to slow heads."""
    return torch.tensor([-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)], dtype=torch.float32)


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dt, gen = DTYPES[case["dtype"]], torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rnd(*shape, dtype=dt, mul=1.0):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
        return (x if mul == 1.0 else x * mul).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(shape, device=DEV, dtype=dtype)

    s = {"case": case}
    op = case["op"]
    if op in ("fwd", "bwd"):
        T, H, K, V, N = case["T"], case["H"], case["K"], case["V"], case["slots"]
        lens = _lengths(case)
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
        s["order"] = torch.argsort(torch.tensor(lens), descending=True, stable=True).to(torch.int32).to(DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if case["packed"]:                       # q, k, v as slices of one projection's output
            qkv = rnd(T, H * (2 * K + V))
            s["q"] = qkv[:, :H * K].view(T, H, K)
            s["k"] = qkv[:, H * K:2 * H * K].view(T, H, K)
            s["v"] = qkv[:, 2 * H * K:].view(T, H, V)
        else:
            s["q"], s["k"], s["v"] = rnd(T, H, K), rnd(T, H, K), rnd(T, H, V)
        s["g"] = _decay(H).to(DEV)
        s["h0"] = rnd(N, H, K, V, dtype=torch.float32)
        if op == "fwd":
            s["o"], s["ht"] = empty(T, H, V), empty(N, H, K, V, dtype=torch.float32)
        else:
            s["do"], s["dht"] = rnd(T, H, V), rnd(N, H, K, V, dtype=torch.float32)
            s["dq"], s["dk"], s["dv"] = empty(T, H, K), empty(T, H, K), empty(T, H, V)
            s["dh0"] = empty(N, H, K, V, dtype=torch.float32)
    elif op == "step":
        B, H, K, V = case["B"], case["H"], case["K"], case["V"]
        s["q"], s["k"], s["v"] = rnd(B, H, K), rnd(B, H, K), rnd(B, H, V)
        s["g"] = _decay(H).to(DEV)
        s["state"] = rnd(case["pool"], H, K, V, dtype=torch.float32)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=DEV)[:B].to(torch.int32)
        s["o"] = empty(B, H, V)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    else:
        T, HQ, HK, D, R = case["T"], case["HQ"], case["HK"], case["D"], case["R"]
        qkv = rnd(T, (HQ + 2 * HK) * D)          # the projection's output; the values are not touched
        s["q"], s["k"] = qkv[:, :HQ * D].view(T, HQ, D), qkv[:, HQ * D:(HQ + HK) * D].view(T, HK, D)
        far = 131072                             # positions of a long context
        s["positions"] = torch.randint(0, far, (T,), generator=gen, device=DEV, dtype=torch.int32)
        if R:
            i = torch.arange(R // 2, dtype=torch.float64, device=DEV)
            a = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (-2.0 * i / R)
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        else:
            s["cos"] = s["sin"] = None
        s["wq"] = 1 + rnd(D, mul=0.1) if case["weight"] else None
        s["wk"] = 1 + rnd(D, mul=0.1) if case["weight"] else None
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["yq"], s["yk"] = empty(T, HQ, D), empty(T, HK, D)
        if op == "nr_bwd":
            s["dyq"], s["dyk"] = rnd(T, HQ, D), rnd(T, HK, D)
            s["dwq"] = empty(D, dtype=torch.float32) if case["weight"] else None
            s["dwk"] = empty(D, dtype=torch.float32) if case["weight"] else None
    return s


EPS = 1e-6


# --------------------------------------------------------------------------- the library's calls
def _run_own(s):
    import chunked_gated_linear_gb300 as gcl
    c = s["case"]
    op = c["op"]
    if op == "fwd":
        if "ws" not in s:                        # the workspace, kept by the program
            s["ws"] = torch.empty(gcl.dla_fwd_workspace_bytes(s["q"], s["v"], s["cu"]), dtype=torch.uint8, device=DEV)
        gcl.dla_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["cu"], s["o"], h0=s["h0"], ht=s["ht"],
                          seq_order=s["order"], dev_status=s["status"], workspace=s["ws"])
        return {"o": s["o"], "ht": s["ht"]}
    if op == "bwd":
        if "ws" not in s:
            s["ws"] = torch.empty(gcl.dla_bwd_workspace_bytes(s["q"], s["v"], s["cu"]), dtype=torch.uint8, device=DEV)
        gcl.dla_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["cu"], s["dq"], s["dk"], s["dv"], h0=s["h0"],
                          dht=s["dht"], dh0=s["dh0"], seq_order=s["order"], dev_status=s["status"], workspace=s["ws"])
        return {n: s[n] for n in ("dq", "dk", "dv", "dh0")}
    if op == "step":
        gcl.dla_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["o"], slots=s["slots"], dev_status=s["status"])
        return {"o": s["o"], "state": s["state"]}
    kw = dict(q_weight=s["wq"], k_weight=s["wk"], cos=s["cos"], sin=s["sin"], positions=s["positions"],
              norm=c["norm"], eps=EPS, pairing=c["pair"], dev_status=s["status"])
    if op == "nr_fwd":
        gcl.qk_norm_rope_fwd(s["q"], s["k"], s["yq"], s["yk"], **kw)
        return {"q": s["yq"], "k": s["yk"]}
    if "ws" not in s:
        s["ws"] = torch.empty(gcl.qk_norm_rope_bwd_workspace_bytes(s["q"], s["k"]), dtype=torch.uint8, device=DEV)
    gcl.qk_norm_rope_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["yq"], s["yk"], dq_weight=s["dwq"], dk_weight=s["dwk"],
                         workspace=s["ws"], **kw)
    out = {"dq": s["yq"], "dk": s["yk"]}
    if c["weight"]:
        out |= {"dwq": s["dwq"], "dwk": s["dwk"]}
    return out


# --------------------------------------------------------------------------- the plain forms
def _pow(g64, n):
    """exp(g n) for every head: g64 [H], n of any shape -> [H, *n.shape] fp32 (1 where n is 0)."""
    e = torch.exp(g64.view(-1, *([1] * n.dim())) * n.double())
    return torch.where(n == 0, torch.ones_like(e), e).float()


def _table(cu, T, N):
    """Chunk rows of the packed sequences: token index (T where empty) [R, C], sequence, start in it, live tokens."""
    lens = (cu[1:] - cu[:-1]).long()
    per = (lens + CHUNK - 1) // CHUNK
    ends = torch.cumsum(per, 0)
    R = -(-T // CHUNK) + N - 1
    r = torch.arange(R, device=cu.device)
    n = torch.searchsorted(ends, r, right=True).clamp(max=N - 1)
    start = (r - (ends - per)[n]) * CHUNK
    count = torch.where(r < ends[-1], (lens[n] - start).clamp(0, CHUNK), torch.zeros_like(r))
    j = torch.arange(CHUNK, device=cu.device)
    tok = torch.where(j[None] < count[:, None], cu[:-1].long()[n][:, None] + start[:, None] + j, torch.full_like(j, T)[None])
    return tok, n, start, count, lens


def _chunks(x, tok):
    """[T, H, D] -> [H, R, C, D] fp32 with zero rows where a chunk has no token."""
    x = torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:], dtype=torch.float32)])
    return x[tok].permute(2, 0, 1, 3)


def _tokens(x, tok, T):
    """[H, R, C, D] -> [T, H, D]."""
    out = x.new_empty((T + 1, x.shape[0], x.shape[3]))
    out[tok.reshape(-1)] = x.permute(1, 2, 0, 3).reshape(-1, x.shape[0], x.shape[3])
    return out[:T]


def _states(a, b, g64, first, tab, reverse):
    """State before (after, in reverse) every chunk and the sequences' last states:
    sums of gamma^(distance) a_j b_j^T over the earlier (later) tokens and the decayed `first`."""
    tok, n, start, count, lens = tab
    H, R, C, K = a.shape
    V = b.shape[3]
    j = torch.arange(C, device=a.device)
    away = (j + 1)[None] if reverse else (count[:, None] - 1 - j[None]).clamp(min=0)
    loc = (a * _pow(g64, away)[..., None]).transpose(2, 3) @ b                # [H, R, K, V]
    end = start + count
    same = n[:, None] == n[None]
    if reverse:
        gap, link = start[None] - end[:, None], same & (start[None] > start[:, None])
        seed = lens[n] - end
        gap_n, seed_n = start[None].expand(len(lens), R), lens
    else:
        gap, link = start[:, None] - end[None], same & (start[None] < start[:, None])
        seed = start
        gap_n, seed_n = lens[:, None] - end[None], lens
    link_n = torch.arange(len(lens), device=a.device)[:, None] == n[None]
    w = _pow(g64, gap.clamp(min=0)) * (link & (count > 0)[None])
    w_n = _pow(g64, gap_n.clamp(min=0)) * (link_n & (count > 0)[None])
    flat = loc.reshape(H, R, K * V)
    f = first.float().transpose(0, 1)                                          # [H, N, K, V]
    before = (w @ flat).view(H, R, K, V) + _pow(g64, seed)[..., None, None] * f[:, n]
    last = (w_n @ flat).view(H, len(lens), K, V) + _pow(g64, seed_n)[..., None, None] * f
    return before, last.transpose(0, 1)


def _inside(g64, device, reverse):
    j = torch.arange(CHUNK, device=device)
    d = j[None] - j[:, None] if reverse else j[:, None] - j[None]
    return _pow(g64, d.clamp(min=0)) * (d >= 0)                               # [H, C, C]


def _plain_fwd(s):
    c = s["case"]
    T, K = c["T"], c["K"]
    g64, scale = s["g"].double(), K ** -0.5
    tab = _table(s["cu"], T, c["slots"])
    tok = tab[0]
    q, k, v = (_chunks(s[n], tok) for n in "qkv")
    S, last = _states(k, v, g64, s["h0"], tab, False)
    near = (q @ k.transpose(2, 3)) * _inside(g64, q.device, False)[:, None] @ v
    j = torch.arange(CHUNK, device=q.device)
    far = _pow(g64, j + 1)[:, None, :, None] * (q @ S)
    o = _tokens(scale * (near + far), tok, T)
    return {"o": o.to(s["q"].dtype), "ht": last.contiguous()}


def _plain_bwd(s):
    c = s["case"]
    T, K = c["T"], c["K"]
    g64, scale, dt = s["g"].double(), K ** -0.5, s["q"].dtype
    tab = _table(s["cu"], T, c["slots"])
    tok, count = tab[0], tab[3]
    q, k, v, do = (_chunks(s[n], tok) for n in ("q", "k", "v", "do"))
    q = q * scale
    j = torch.arange(CHUNK, device=q.device)
    S, _ = _states(k, v, g64, s["h0"], tab, False)
    down, up = _inside(g64, q.device, False)[:, None], _inside(g64, q.device, True)[:, None]
    lead = _pow(g64, j + 1)[:, None, :, None]
    dq = scale * (((do @ v.transpose(2, 3)) * down) @ k + lead * (do @ S.transpose(2, 3)))
    G, first = _states(q, do, g64, s["dht"], tab, True)                        # gradient of the states, one decay ahead
    tail = _pow(g64, (count[:, None] - 1 - j[None]).clamp(min=0))[..., None]
    dk = ((v @ do.transpose(2, 3)) * up) @ q + tail * (v @ G.transpose(2, 3))
    dv = ((k @ q.transpose(2, 3)) * up) @ do + tail * (k @ G)
    return {"dq": _tokens(dq, tok, T).to(dt), "dk": _tokens(dk, tok, T).to(dt), "dv": _tokens(dv, tok, T).to(dt),
            "dh0": first.contiguous()}


def _plain_step(s):
    K = s["case"]["K"]
    at = s["slots"].long()
    S = s["state"][at] * torch.exp(s["g"])[:, None, None] + s["k"].float()[..., None] * s["v"].float()[..., None, :]
    s["state"][at] = S
    o = K ** -0.5 * (s["q"].float()[..., None] * S).sum(-2)
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _rotate(x, cos, sin, R, pair, back=False):
    """The rotation of the first R channels (its transpose with `back`)."""
    if R == 0:
        return x
    sin = -sin if back else sin
    if pair == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _inv_norm(x, norm):
    if norm == "none":
        return torch.ones_like(x[..., :1])
    ss = x.square()
    return torch.rsqrt((ss.mean(-1, keepdim=True) if norm == "rms" else ss.sum(-1, keepdim=True)) + EPS)


def _plain_nr(s, backward):
    c = s["case"]
    R, dt = c["R"], s["q"].dtype
    cos = sin = None
    if R:
        at = s["positions"].long()
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    out = {}
    for n in "qk":
        x = s[n].float()
        w = s["w" + n]
        w = torch.ones(c["D"], device=x.device) if w is None else w.float()
        r = _inv_norm(x, c["norm"])
        if not backward:
            out[n] = _rotate(x * r * w, cos, sin, R, c["pair"]).to(dt)
            continue
        dy = _rotate(s["dy" + n].float(), cos, sin, R, c["pair"], back=True)
        u = dy * w
        if c["norm"] == "none":
            dx = u
        else:
            m = (u * x * r).sum(-1, keepdim=True) / (c["D"] if c["norm"] == "rms" else 1)
            dx = r * (u - x * r * m)
        out["d" + n] = dx.to(dt)
        if c["weight"]:
            out["dw" + n] = (dy * x * r).sum((0, 1))
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "fwd":
        return _plain_fwd(state)
    if op == "bwd":
        return _plain_bwd(state)
    if op == "step":
        return _plain_step(state)
    return _plain_nr(state, op == "nr_bwd")


# --------------------------------------------------------------------------- floors
def work(case):
    e = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    op = case["op"]
    if op in ("fwd", "bwd"):
        T, H, K, V = case["T"], case["H"], case["K"], case["V"]
        states = 2 * case["slots"] * H * K * V * 4
        if op == "fwd":                          # q k^T, the product with v, q S and the state update, at a chunk of 64
            return {"bytes": T * H * (2 * K + 2 * V) * e + states, "flops": 2 * T * H * (CHUNK / 2 * (K + V) + 2 * K * V)}
        return {"bytes": T * H * (4 * K + 3 * V) * e + states + case["slots"] * H * K * V * 4,
                "flops": 2 * T * H * (CHUNK / 2 * (3 * K + 3 * V) + 5 * K * V)}
    if op == "step":
        B, H, K, V = case["B"], case["H"], case["K"], case["V"]
        return {"bytes": B * H * (8 * K * V + (2 * K + 2 * V) * e), "flops": B * H * K * V * 5}
    n = case["T"] * (case["HQ"] + case["HK"]) * case["D"]
    return {"bytes": n * e * (2 if op == "nr_fwd" else 3), "flops": n * (8 if op == "nr_fwd" else 16)}


# --------------------------------------------------------------------------- the definitions in fp64
def _walk(a, b, c, decay, first, lens, cu, backwards):
    """Per token and head in fp64, from first to last token of each sequence (or back): M <- decay M + a_t b_t^T, then
    M c_t.  Backwards the state is met before its decay, so `first` is taken undecayed.  Sequences go side by side."""
    N, H = first.shape[:2]
    M = first.clone()
    lens_h = lens.tolist()
    order = sorted(range(N), key=lambda n: -lens_h[n])
    M = M[order]
    at = cu[:-1].long()[order]
    ln = lens.long()[order]
    out = torch.zeros(a.shape[0], H, M.shape[2], dtype=torch.float64, device=a.device)
    live = N
    top = lens_h[order[0]]
    t = 0
    while t < top:
        while lens_h[order[live - 1]] <= t:
            live -= 1
        tok = (at[:live] + ln[:live] - 1 - t) if backwards else (at[:live] + t)
        m = M[:live]
        if not (backwards and t == 0):
            m.mul_(decay)
        x = a[tok]
        m.addcmul_(x[..., None], b[tok][..., None, :])
        out[tok] = (m @ c[tok][..., None])[..., 0]
        t += 1
    undo = torch.empty(N, dtype=torch.long, device=a.device)
    undo[torch.tensor(order, device=a.device)] = torch.arange(N, device=a.device)
    return out, M[undo]


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("fwd", "bwd"):
        lens = torch.tensor(_lengths(case), device=DEV)
        longest = int(lens.max())
        cost = longest * (40e-6 + 4e-12 * case["slots"] * case["H"] * case["K"] * case["V"]) * (1 if op == "fwd" else 3)
        if cost > 15:
            return None
        q, k, v = (s[n].double() for n in "qkv")
        q = q / math.sqrt(case["K"])
        decay = torch.exp(s["g"].double())[:, None, None]
        h0 = s["h0"].double()
        if op == "fwd":
            o, last = _walk(v, k, q, decay, h0.transpose(2, 3).contiguous(), lens, s["cu"], False)
            return {"o": o, "ht": last.transpose(2, 3).contiguous()}
        do, dht = s["do"].double(), s["dht"].double()
        dq, _ = _walk(k, v, do, decay, h0, lens, s["cu"], False)
        # the gradient of the state after token t: decay times that after t + 1, plus q_t do_t^T
        dk, G = _walk(q, do, v, decay, dht, lens, s["cu"], True)
        dv, _ = _walk(do, q, k, decay, dht.transpose(2, 3).contiguous(), lens, s["cu"], True)
        some = (lens > 0)[:, None, None, None]
        return {"dq": dq / math.sqrt(case["K"]), "dk": dk, "dv": dv, "dh0": torch.where(some, G * decay, G)}
    if op == "step":
        at = s["slots"].long()
        state = s["state"].double()
        S = torch.einsum("bhk,bhv->bhkv", s["k"].double(), s["v"].double())
        S = S + state[at] * s["g"].double().exp()[:, None, None]
        state[at] = S
        return {"o": torch.einsum("bhk,bhkv->bhv", s["q"].double(), S) / math.sqrt(case["K"]), "state": state}
    D, R = case["D"], case["R"]
    out = {}
    phase = None
    if R:                                        # the rotation as a product with exp(i angle), from the stored table
        at = s["positions"].long()
        phase = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]

    def turned(y, sign):
        if not R:
            return y
        a, b = (y[..., :R // 2], y[..., R // 2:R]) if case["pair"] == "half" else (y[..., 0:R:2], y[..., 1:R:2])
        z = torch.complex(a, b) * (phase if sign > 0 else phase.conj())
        y = y.clone()
        if case["pair"] == "half":
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        else:
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        return y

    for n in "qk":
        x = s[n].double()
        w = s["w" + n].double() if case["weight"] else torch.ones(D, dtype=torch.float64, device=DEV)
        size = {"rms": 1.0 / D, "l2": 1.0, "none": 0.0}[case["norm"]]
        length = torch.sqrt((x * x).sum(-1, keepdim=True) * size + EPS) if size else torch.ones_like(x[..., :1])
        if op == "nr_fwd":
            out[n] = turned(x / length * w, +1)
            continue
        dy = turned(s["dy" + n].double(), -1)
        dx = dy * w / length
        if size:
            dx = dx - x * size * (dy * w * x).sum(-1, keepdim=True) / length ** 3
        out["d" + n] = dx
        if case["weight"]:
            out["dw" + n] = torch.einsum("thd,thd->d", dy, x / length)
    return out
