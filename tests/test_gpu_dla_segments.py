"""Decayed linear attention in plans whose segments are several chunks long, and in whole sequences of many chunks: the
rings of tiles, split buffers and barriers turn several times.  Sizes are looked up in the plan of the case's own dtype and
dims, and the plan is asserted.  References and tolerances as in tests/dla_ref.py; heads are independent, so some of
them are compared."""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import chunked_gated_linear_gb300 as gcl  # noqa: E402
import dla_ref  # noqa: E402
from parity import check  # noqa: E402
from test_gpu_dla import DIMS, Case  # noqa: E402

CODE = {"f32": gcl.GCL_F32, "bf16": gcl.GCL_BF16, "f16": gcl.GCL_F16}
CHUNK = {"f32": 64, "bf16": 128, "f16": 64}


def find(dtype, K, V, back, chunks):
    """The smallest capacities (tokens, sequences, heads) whose plan has segments of so many chunks, and two of them
    at least with a short one at the end."""
    sizes = itertools.product(range(300, 6400, 128), (1, 2, 3), (1, 2, 3, 4, 6, 8, 12, 16, 24, 32))
    for T, N, H in sorted(sizes, key=lambda s: s[0] * s[2]):
        seg = gcl.dla_segment_tokens(T, N, H, back, CODE[dtype], K, V)
        if seg == chunks * CHUNK[dtype] and T - 23 > seg + 1:
            return T, N, H
    pytest.fail(f"no plan of {chunks} chunks a segment")


def make(dtype, T, N, H, K, V, seed):
    """Capacity T, five rows of padding; nearly all tokens in the first sequence, then an empty one and short ones."""
    live = T - 5
    lens = {1: [live], 2: [live - 18, 18], 3: [live - 1, 0, 1]}[N]
    return Case(dtype, lens, H, K, V, seed=seed, t_pad=5)


def verify(c, back, label):
    """The case against fp64 on its first, middle and last head."""
    hs = sorted({0, c.H // 2, c.H - 1})
    f = lambda x: None if x is None else x.float().cpu().numpy()  # noqa: E731
    q, k, v, d_o = (f(x[:, hs]) for x in (c.q, c.k, c.v, c.d_o))
    h0, dht = (f(x[:, hs]) for x in (c.h0, c.dht))
    g = f(c.g[hs])
    if back:
        *rows, state, status = c.bwd()
        ref = dla_ref.bwd(q, k, v, g, h0, d_o, dht, c.cu, c.scale)
    else:
        *rows, state, status = c.fwd()
        ref = dla_ref.fwd(q, k, v, g, h0, c.cu, c.scale)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for i, (got, r) in enumerate(zip(rows, ref)):
        check(f"{label} rows {i}", f(got[:c.live, hs]), r[:c.live], dla_ref.TOL[c.dtype], cu=c.cu, reduction=False)
    check(f"{label} state", f(state[:, hs]), ref[-1], dla_ref.TOL_STATE)
    return [*rows, state]


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("dims", DIMS, ids=lambda d: f"{d[0]}x{d[1]}")
@pytest.mark.parametrize("chunks", [2, 3, 4, 8])
def test_segments_of_several_chunks(chunks, dims, back):
    """bf16: against fp64, then again with the same bits (a wait that passes early would show in some of the runs)."""
    T, N, H = find("bf16", *dims, back, chunks)
    c = make("bf16", T, N, H, *dims, seed=chunks)
    first = verify(c, back, f"{chunks} chunks {dims}")
    for _ in range(20):
        *again, _ = c.bwd() if back else c.fwd()
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_segments_of_two_chunks_on_the_cuda_cores(dtype, back):
    T, N, H = find(dtype, 64, 64, back, 2)
    verify(make(dtype, T, N, H, 64, 64, seed=5), back, f"{dtype} two chunks")


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("dims", DIMS, ids=lambda d: f"{d[0]}x{d[1]}")
def test_whole_sequences_of_many_chunks(dims, back):
    """bf16, one CTA per sequence: 14 chunks, so the five tile slots go round nearly three times."""
    T = 1700
    H = next(h for h in range(140, 1300) if gcl.dla_segment_tokens(T, 1, h, back, gcl.GCL_BF16, *dims) >= T)
    verify(make("bf16", T, 1, H, *dims, seed=9), back, f"whole {dims}")


def test_more_sequences_than_a_block_has_threads():
    """fp32 in a cut plan of 310 sequences: the blocks of the CUDA-core engine and of the scan (256 threads) add up the
    sequences' borders in two rounds.  The long sequences come late; empty and short ones lie between."""
    N, K, V = 310, 64, 64
    lens = [0, 3, 1] * 103 + [0]
    lens[270], lens[309] = 1500, 900
    live = sum(lens)
    c = Case("f32", lens, 1, K, V, seed=11, t_pad=N * 700 - live)
    assert gcl.dla_segment_tokens(c.T, N, 1, False, gcl.GCL_F32, K, V) < 900
    verify(c, False, "many sequences")


def test_segments_in_the_bounds_checking_build():
    """The tensor-core engine's cut plan in libgcl_debug.so: every checked index in its buffer, status 0."""
    saved = gcl._lib
    gcl._lib = gcl.load_library(gcl.DEBUG_LIB_PATH)
    try:
        for back in (False, True):
            T, N, H = find("bf16", 64, 128, back, 2)
            verify(make("bf16", T, N, H, 64, 128, seed=13), back, "debug build")
    finally:
        gcl._lib = saved
