"""One layer of decayed linear attention, as a model uses its operators: a training step on packed
sequences, then serving -- a prefill and a captured single-token step.

    x -> q, k, v (one projection) -> norm and rotation of q, k -> decayed linear attention -> output projection

The projections are torch matrix products; everything between them is this library.  Run it on a GB300:

    python examples/decayed_linear_layer.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_linear_gb300 as gcl  # noqa: E402

F32, I32 = torch.float32, torch.int32


class DecayedLinearLayer:
    """Weights, the rotation table and the decays of one layer; q, k and v are slices of one projection."""

    def __init__(self, width, heads, dim, rotary, max_positions, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.H, self.D, self.dtype, self.device = heads, dim, dtype, device
        self.w_in = (rnd(width, 3 * heads * dim) / math.sqrt(width)).to(dtype)
        self.w_out = (rnd(heads * dim, width) / math.sqrt(heads * dim)).to(dtype)
        self.q_weight, self.k_weight = torch.ones(dim, device=device, dtype=dtype), torch.ones(dim, device=device, dtype=dtype)
        self.g = -(2.0 ** (-8.0 * (torch.arange(heads, device=device, dtype=F32) + 1) / heads))    # log decays
        self.cos, self.sin = (torch.empty(max_positions, rotary // 2, device=device) for _ in range(2))
        gcl.rope_table_build(self.cos, self.sin)
        self.status = torch.zeros(1, dtype=I32, device=device)

    def project(self, x):
        """q, k, v as views [T, H, D] of one buffer."""
        n = self.H * self.D
        qkv = x @ self.w_in
        return qkv, *(qkv[:, i * n:(i + 1) * n].view(-1, self.H, self.D) for i in range(3))

    def norm_kw(self, positions):
        return dict(q_weight=self.q_weight, k_weight=self.k_weight, cos=self.cos, sin=self.sin, positions=positions,
                    norm="rms", dev_status=self.status)

    def forward(self, x, positions, cu_seqlens, h0=None):
        """Packed sequences x [T, width]; returns y, the last states and what the backward needs."""
        T, N = x.shape[0], cu_seqlens.shape[0] - 1
        _, q, k, v = self.project(x)
        qn, kn, o = (torch.empty(T, self.H, self.D, dtype=self.dtype, device=self.device) for _ in range(3))
        gcl.qk_norm_rope_fwd(q, k, qn, kn, **self.norm_kw(positions))
        ht = torch.empty(N, self.H, self.D, self.D, device=self.device)
        ws = torch.empty(gcl.dla_fwd_workspace_bytes(qn, v, cu_seqlens), dtype=torch.uint8, device=self.device)
        gcl.dla_chunk_fwd(qn, kn, v, self.g, cu_seqlens, o, h0=h0, ht=ht, dev_status=self.status, workspace=ws)
        return o.view(T, -1) @ self.w_out, ht, (x, q, k, v, qn, kn, o, positions, cu_seqlens, h0)

    def backward(self, dy, saved):
        """Gradients of the input and the weights from dy [T, width]."""
        x, q, k, v, qn, kn, o, positions, cu_seqlens, h0 = saved
        T, n = x.shape[0], self.H * self.D
        d_o = (dy @ self.w_out.T).view(T, self.H, self.D)
        dqkv = torch.empty(T, 3 * n, dtype=self.dtype, device=self.device)      # gradients land in its slices
        dq, dk, dv = (dqkv[:, i * n:(i + 1) * n].view(T, self.H, self.D) for i in range(3))
        dqn, dkn = torch.empty_like(qn), torch.empty_like(kn)
        ws = torch.empty(gcl.dla_bwd_workspace_bytes(qn, v, cu_seqlens), dtype=torch.uint8, device=self.device)
        gcl.dla_chunk_bwd(qn, kn, v, self.g, d_o, cu_seqlens, dqn, dkn, dv, h0=h0, dev_status=self.status, workspace=ws)
        dwq, dwk = torch.empty(self.D, device=self.device), torch.empty(self.D, device=self.device)
        ws = torch.empty(gcl.qk_norm_rope_bwd_workspace_bytes(q, k), dtype=torch.uint8, device=self.device)
        gcl.qk_norm_rope_bwd(q, k, dqn, dkn, dq, dk, dq_weight=dwq, dk_weight=dwk, workspace=ws, **self.norm_kw(positions))
        return {"x": dqkv @ self.w_in.T, "w_in": x.T @ dqkv, "w_out": o.view(T, -1).T @ dy, "q_weight": dwq, "k_weight": dwk}

    def step(self, x, positions, state, slots):
        """One token of each request, x [B, width]; the requests' states in the pool advance in place."""
        B = x.shape[0]
        _, q, k, v = self.project(x)
        qn, kn, o = (torch.empty(B, self.H, self.D, dtype=self.dtype, device=self.device) for _ in range(3))
        gcl.qk_norm_rope_fwd(q, k, qn, kn, **self.norm_kw(positions))
        gcl.dla_step(qn, kn, v, self.g, state, o, slots=slots, dev_status=self.status)
        return o.view(B, -1) @ self.w_out


def packed(lengths, device):
    """cu_seqlens and each token's position in its sequence."""
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=I32, device=device)
    return cu, torch.cat([torch.arange(n) for n in lengths]).to(I32).to(device)


def run(width=512, heads=4, dim=128, rotary=64, lengths=(300, 1, 77, 640), new_tokens=5, seed=0):
    """A training step, then serving; returns the gradients and how far decoding is from the longer prefill."""
    layer = DecayedLinearLayer(width, heads, dim, rotary, max(lengths) + 64, seed=seed)
    dev = layer.device
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed + 1)
    rows = lambda n: torch.randn(n, width, generator=gen, device=dev).to(layer.dtype)  # noqa: E731

    cu, positions = packed(lengths, dev)
    x, target = rows(sum(lengths)), rows(sum(lengths))
    y, _, saved = layer.forward(x, positions, cu)
    loss = (y.float() - target.float()).square().mean()
    grads = layer.backward((2 / y.numel() * (y.float() - target.float())).to(layer.dtype), saved)

    # serving: prefill all but the last tokens of each prompt, put the states into a pool, decode the rest
    prompts = [n + new_tokens for n in lengths]
    cu_all, pos_all = packed(prompts, dev)
    x_all = rows(sum(prompts))
    y_all, h_all, _ = layer.forward(x_all, pos_all, cu_all)
    starts = cu_all[:-1].long()
    head = torch.cat([x_all[s:s + n] for s, n in zip(starts.tolist(), lengths)])
    _, ht, _ = layer.forward(head, positions, cu)
    pool = torch.zeros(len(lengths) + 2, heads, dim, dim, device=dev)
    slots = torch.arange(len(lengths), 0, -1, dtype=I32, device=dev)
    pool[slots.long()] = ht
    tok, pos = torch.empty(len(lengths), width, dtype=layer.dtype, device=dev), torch.zeros(len(lengths), dtype=I32, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                       # a first call outside the capture; idle slots leave the pool alone
        layer.step(tok.zero_(), pos, pool, torch.full_like(slots, -1))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(tok, pos, pool, slots)
    far = 0.0
    for t in range(new_tokens):
        at = starts + torch.tensor(lengths, device=dev) + t
        tok.copy_(x_all[at])
        pos.copy_(pos_all[at])
        graph.replay()
        ref = y_all[at].float()
        far = max(far, float((out.float() - ref).norm() / ref.norm()))
    state_far = float((pool[slots.long()] - h_all).norm() / h_all.norm())
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    return {"loss": float(loss), "grads": grads, "decode_error": far, "state_error": state_far}


if __name__ == "__main__":
    r = run()
    print(f"loss {r['loss']:.4f}; gradient norms " + ", ".join(f"{k} {float(v.float().norm()):.3e}" for k, v in r["grads"].items()))
    print(f"decoding against the longer prefill: rows {r['decode_error']:.2e}, states {r['state_error']:.2e}")
