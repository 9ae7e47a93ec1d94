"""A gated recurrent block, as a model uses its operators: a training step on packed sequences, then serving -- a prefill
and a captured single-token step.

    z = norm(x)  ->  x', r, i, g (projections)  ->  short convolution of x'  ->  gated linear recurrence (decay gate r, input gate i)
      ->  norm of each head with the gate silu(g)  ->  output projection
      ->  norm, dropout, residual scale and sum, and the next block's norm, in one pass

The projections are torch matrix products; everything between them is this library.  Run it on a GB300:

    python examples/gated_recurrent_block.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_linear_gb300 as gcl  # noqa: E402

F32, I32, I64 = torch.float32, torch.int32, torch.int64


class GatedRecurrentBlock:
    """Weights of one block between two residual streams; D = heads * dim channels recur."""

    def __init__(self, width, heads, dim, taps=4, dropout=0.1, scale=0.5, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        D = heads * dim
        self.H, self.dim, self.D, self.dtype, self.device = heads, dim, D, dtype, device
        self.p, self.scale = dropout, scale
        self.w = {"x": rnd(width, D) / math.sqrt(width), "gates": rnd(width, 3 * D) / math.sqrt(width), "conv": rnd(D, taps) / 2,
                  "out": rnd(D, width) / math.sqrt(D), "head": 1 + 0.1 * rnd(dim), "first": 1 + 0.1 * rnd(width),
                  "post": 1 + 0.1 * rnd(width), "pre": 1 + 0.1 * rnd(width)}
        self.w = {k: v.to(dtype) for k, v in self.w.items()}
        self.rate = -8 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device=device))
        self.rng = torch.tensor([seed + 17, 0], dtype=I64, device=device)      # seed and offset of dropout
        self.status = torch.zeros(1, dtype=I32, device=device)

    def empty(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def head_kw(self, gate):
        return dict(gate=gate, post_weight=self.w["head"], post_norm="rms", activation="silu", dev_status=self.status)

    def join_kw(self, p):
        return dict(post_weight=self.w["post"], pre_weight=self.w["pre"], post_norm="rms", pre_norm="rms", scale=self.scale, dropout=p,
                    rng=self.rng, dev_status=self.status)

    def glr_kw(self, i):
        return dict(i=i, rate=self.rate, decay="power", mix="root", dev_status=self.status)

    def chunks(self, cu, T):
        """Chunk metadata of the convolution."""
        N = cu.shape[0] - 1
        idx, off = self.empty(gcl.nt_max(T, N), 2, dtype=I32), self.empty(N + 1, dtype=I32)
        gcl.chunk_meta_build(cu, T, idx, off, self.status)
        return idx

    def forward(self, x, cu, states=None, train=True):
        """Packed sequences x [T, width]: the stream behind the block, the next block's input, the last states (convolution,
        recurrence) and what the backward needs."""
        T, N, D, w = x.shape[0], cu.shape[0] - 1, self.D, self.w
        z = torch.empty_like(x)
        gcl.block_norm_fwd(x, None, z=z, pre_weight=w["first"], post_norm=None, pre_norm="rms", dev_status=self.status)
        xin, gates = z @ w["x"], z @ w["gates"]
        r, i, g = (gates[:, k * D:(k + 1) * D] for k in range(3))
        idx = self.chunks(cu, T)
        c0, h0 = (None, None) if states is None else states
        c, cT = self.empty(T, D), self.empty(N, D, w["conv"].shape[1] - 1)
        gcl.causal_conv1d_fwd(xin, w["conv"], cu, idx, h0=c0, y=c, ht=cT, dev_status=self.status)
        h, hT = self.empty(T, D), self.empty(N, D, dtype=F32)
        save = self.empty(-(-T // 64), D, dtype=F32) if train else None
        ws = self.empty(gcl.glr_fwd_workspace_bytes(c, cu), dtype=torch.uint8)
        gcl.glr_fwd(c, r, cu, h, h0=h0, ht=hT, h_save=save, workspace=ws, **self.glr_kw(i))
        u = self.empty(T, D)
        heads = lambda t: t.view(T, self.H, self.dim)  # noqa: E731
        gcl.block_norm_fwd(heads(h), heads(u), **self.head_kw(g.view(T, self.H, self.dim)))
        b, xo, zo = u @ w["out"], torch.empty_like(x), torch.empty_like(x)
        gcl.block_norm_fwd(b, xo, x=x, z=zo, **self.join_kw(self.p if train else 0.0))
        return xo, zo, (cT, hT), (x, z, cu, idx, xin, r, i, g, c, h, save, u, b)

    def backward(self, dxo, dzo, saved):
        """Gradients of the stream x and of every weight, from those of both outputs."""
        x, z, cu, idx, xin, r, i, g, c, h, save, u, b = saved
        T, D, w = x.shape[0], self.D, self.w
        grads = {k: torch.empty(v.shape, dtype=F32, device=self.device) for k, v in w.items() if k in ("head", "first", "post", "pre", "conv")}
        scratch = lambda n: self.empty(n, dtype=torch.uint8)  # noqa: E731
        db, dx = torch.empty_like(b), torch.empty_like(x)
        gcl.block_norm_bwd(b, dxo, db, x=x, dx=dx, dz=dzo, dpost_weight=grads["post"], dpre_weight=grads["pre"],
                           workspace=scratch(gcl.block_norm_bwd_workspace_bytes(b)), **self.join_kw(self.p))
        grads["out"], du = u.T @ db, db @ w["out"].T
        dgates = self.empty(T, 3 * D)                                         # the gates' gradients land in its slices
        dr, di, dg = (dgates[:, k * D:(k + 1) * D] for k in range(3))
        dh, heads = self.empty(T, D), lambda t: t.view(T, self.H, self.dim)  # noqa: E731
        gcl.block_norm_bwd(heads(h), heads(du), heads(dh), dgate=heads(dg), dpost_weight=grads["head"],
                           workspace=scratch(gcl.block_norm_bwd_workspace_bytes(heads(h))), **self.head_kw(heads(g)))
        dc, grads["rate"] = self.empty(T, D), self.empty(D, dtype=F32)
        gcl.glr_bwd(c, r, dh, cu, dc, dr, di=di, drate=grads["rate"], h_save=save,
                    workspace=scratch(gcl.glr_bwd_workspace_bytes(c, cu, h_save=save)), **self.glr_kw(i))
        dxin = self.empty(T, D, dtype=F32)
        kw = dict(dy=dc, dx=dxin, dweight=grads["conv"], dev_status=self.status)
        gcl.causal_conv1d_bwd(xin, w["conv"], cu, idx,
                              workspace=scratch(gcl.causal_conv1d_bwd_workspace_bytes(xin, w["conv"], cu, idx, **kw)), **kw)
        dxin = dxin.to(self.dtype)
        grads["x"], grads["gates"] = z.T @ dxin, z.T @ dgates
        dz, dfirst = dxin @ w["x"].T + dgates @ w["gates"].T, torch.empty_like(x)
        gcl.block_norm_bwd(x, None, dfirst, dz=dz, pre_weight=w["first"], dpre_weight=grads["first"], post_norm=None, pre_norm="rms",
                           workspace=scratch(gcl.block_norm_bwd_workspace_bytes(x)), dev_status=self.status)
        grads["stream"] = dx + dfirst
        return grads

    def step(self, x, cu, idx, conv, conv_next, pool, slots):
        """One token of each request, x [B, width]: the requests' convolution states conv [B, D, taps - 1] and their slots of the
        pool [slots, D] advance."""
        B, D, w = x.shape[0], self.D, self.w
        z = torch.empty_like(x)
        gcl.block_norm_fwd(x, None, z=z, pre_weight=w["first"], post_norm=None, pre_norm="rms", dev_status=self.status)
        xin, gates = z @ w["x"], z @ w["gates"]
        r, i, g = (gates[:, k * D:(k + 1) * D] for k in range(3))
        c, h, u = (self.empty(B, D) for _ in range(3))
        gcl.causal_conv1d_fwd(xin, w["conv"], cu, idx, h0=conv, y=c, ht=conv_next, dev_status=self.status)
        conv.copy_(conv_next)
        gcl.glr_step(c, r, pool, h, slots=slots, **self.glr_kw(i))
        heads = lambda t: t.view(B, self.H, self.dim)  # noqa: E731
        gcl.block_norm_fwd(heads(h), heads(u), **self.head_kw(heads(g)))
        b, xo, zo = u @ w["out"], torch.empty_like(x), torch.empty_like(x)
        gcl.block_norm_fwd(b, xo, x=x, z=zo, **self.join_kw(0.0))
        return xo, zo


def packed(lengths, device):
    return torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=I32, device=device)


def run(width=512, heads=4, dim=128, lengths=(300, 1, 77, 640), new_tokens=5, seed=0):
    """A training step, then serving; returns the gradients and how far decoding is from the longer prefill."""
    block = GatedRecurrentBlock(width, heads, dim, seed=seed)
    dev = block.device
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed + 1)
    rows = lambda n: torch.randn(n, width, generator=gen, device=dev).to(block.dtype)  # noqa: E731

    cu, T = packed(lengths, dev), sum(lengths)
    x, target = rows(T), rows(T)
    block.rng[1] = 1                                        # the step's number: another mask every step
    xo, zo, _, saved = block.forward(x, cu)
    loss = (zo.float() - target.float()).square().mean()
    dz = (2 / zo.numel() * (zo.float() - target.float())).to(block.dtype)
    grads = block.backward(torch.zeros_like(xo), dz, saved)

    # serving: prefill all but the last tokens of each prompt, decode the rest
    prompts = [n + new_tokens for n in lengths]
    cu_all, x_all = packed(prompts, dev), rows(sum(prompts))
    xo_all, _, _, _ = block.forward(x_all, cu_all, train=False)
    starts, B = cu_all[:-1].long(), len(lengths)
    head = torch.cat([x_all[s:s + n] for s, n in zip(starts.tolist(), lengths)])
    _, _, (conv, hT), _ = block.forward(head, cu, train=False)
    pool, slots = torch.zeros(B + 2, block.D, device=dev), torch.arange(B, 0, -1, dtype=I32, device=dev)
    pool[slots.long()] = hT
    one = torch.arange(B + 1, dtype=I32, device=dev)        # B sequences of one token
    idx, conv_next, tok = block.chunks(one, B), torch.empty_like(conv), torch.zeros(B, width, dtype=block.dtype, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                           # a first call outside the capture; idle slots leave the pool alone
        block.step(tok, one, idx, torch.zeros_like(conv), conv_next, pool, torch.full_like(slots, -1))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block.step(tok, one, idx, conv, conv_next, pool, slots)
    far = 0.0
    for t in range(new_tokens):
        at = starts + torch.tensor(lengths, device=dev) + t
        tok.copy_(x_all[at])
        graph.replay()
        ref = xo_all[at].float()
        far = max(far, float((out.float() - ref).norm() / ref.norm()))
    torch.cuda.synchronize()
    assert int(block.status.item()) == 0
    return {"loss": float(loss), "grads": grads, "decode_error": far}


if __name__ == "__main__":
    r = run()
    print(f"loss {r['loss']:.4f}; gradient norms " + ", ".join(f"{k} {float(v.float().norm()):.3e}" for k, v in r["grads"].items()))
    print(f"decoding against the longer prefill: {r['decode_error']:.2e}")
