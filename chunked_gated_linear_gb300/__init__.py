"""Python binding of libgcl, the GB300 chunked gated linear attention library.

Argument marshalling only: every entry point forwards torch tensors' device
pointers and the current CUDA stream to the C ABI declared in
``include/gcl.h``; all computation happens in the library's CUDA kernels.  The
library must have been built (``python -m chunked_gated_linear_gb300._build``
or ``__graft_entry__.build()``); importing this package fails loudly otherwise,
and there is no other implementation to fall back on.

The library sees raw pointers only, so before each launch the binding checks what a
pointer cannot carry: every tensor is a contiguous CUDA tensor on the call's device, of the
dtype and at least the size ``include/gcl.h`` gives it.  A host tensor or a too-small buffer
would otherwise be read or written out of bounds on the device.
"""
from __future__ import annotations

import ctypes
import inspect
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgcl.so")
# the bounds-checking debug build (GCL_DEBUG_BOUNDS), for tests: load_library(DEBUG_LIB_PATH)
DEBUG_LIB_PATH = os.path.join(PKG, "libgcl_debug.so")

GCL_F32, GCL_BF16, GCL_F16 = 0, 1, 2
DEV_STATUS = {0: "ok", 1: "cu_seqlens decreasing", 2: "cu_seqlens[0] != 0",
              3: "cu_seqlens[N_max] > T_max", 4: "invalid sequence range"}
CHUNK = 64


class GclError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


class FwdArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("h0", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("chunk_indices", ctypes.c_void_p),
                ("chunk_offsets", ctypes.c_void_p),
                ("seq_order", ctypes.c_void_p), ("o", ctypes.c_void_p), ("ht", ctypes.c_void_p),
                ("h_save", ctypes.c_void_p), ("dev_status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("t_max", ctypes.c_int64), ("n_max", ctypes.c_int32), ("H", ctypes.c_int32),
                ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("bt", ctypes.c_int32),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class BwdArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("h0", ctypes.c_void_p),
                ("d_o", ctypes.c_void_p), ("dht", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("chunk_indices", ctypes.c_void_p),
                ("chunk_offsets", ctypes.c_void_p), ("h_save", ctypes.c_void_p),
                ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
                ("dg", ctypes.c_void_p), ("dbeta", ctypes.c_void_p), ("dh0", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("dev_status", ctypes.c_void_p), ("t_max", ctypes.c_int64),
                ("n_max", ctypes.c_int32), ("H", ctypes.c_int32), ("K", ctypes.c_int32),
                ("V", ctypes.c_int32), ("bt", ctypes.c_int32), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("fwd_workspace", ctypes.c_void_p),
                ("fwd_workspace_bytes", ctypes.c_size_t)]


class ConvArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("ht", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("dht", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("dh0", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("chunk_indices", ctypes.c_void_p), ("dev_status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("t_max", ctypes.c_int64), ("n_max", ctypes.c_int32), ("D", ctypes.c_int32),
                ("W", ctypes.c_int32), ("bt", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class DlaArgs(ctypes.Structure):
    _fields_ = [("q", Rows), ("k", Rows), ("v", Rows), ("o", Rows), ("d_o", Rows), ("dq", Rows),
                ("dk", Rows), ("dv", Rows), ("g", ctypes.c_void_p), ("h0", ctypes.c_void_p),
                ("ht", ctypes.c_void_p), ("dht", ctypes.c_void_p), ("dh0", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("seq_order", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("t_max", ctypes.c_int64),
                ("n_max", ctypes.c_int32), ("H", ctypes.c_int32), ("K", ctypes.c_int32),
                ("V", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class DlaStepArgs(ctypes.Structure):
    _fields_ = [("q", Rows), ("k", Rows), ("v", Rows), ("o", Rows), ("g", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("n_slots", ctypes.c_int32), ("H", ctypes.c_int32), ("K", ctypes.c_int32),
                ("V", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class QkArgs(ctypes.Structure):
    _fields_ = [("q", Rows), ("k", Rows), ("yq", Rows), ("yk", Rows), ("dyq", Rows), ("dyk", Rows),
                ("dq", Rows), ("dk", Rows), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("dq_weight", ctypes.c_void_p),
                ("dk_weight", ctypes.c_void_p), ("cos_table", ctypes.c_void_p),
                ("sin_table", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("t_max", ctypes.c_int64),
                ("n_positions", ctypes.c_int64), ("HQ", ctypes.c_int32), ("HK", ctypes.c_int32),
                ("D", ctypes.c_int32), ("R", ctypes.c_int32), ("eps", ctypes.c_float),
                ("norm", ctypes.c_int32), ("pair", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class GlrArgs(ctypes.Structure):
    _fields_ = [("x", Rows), ("r", Rows), ("i", Rows), ("o", Rows), ("d_o", Rows), ("dx", Rows),
                ("dr", Rows), ("di", Rows), ("rate", ctypes.c_void_p), ("h0", ctypes.c_void_p),
                ("ht", ctypes.c_void_p), ("dht", ctypes.c_void_p), ("dh0", ctypes.c_void_p),
                ("drate", ctypes.c_void_p), ("h_save", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("dev_status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("t_max", ctypes.c_int64), ("n_max", ctypes.c_int32), ("D", ctypes.c_int32),
                ("decay", ctypes.c_int32), ("mix", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class GlrStepArgs(ctypes.Structure):
    _fields_ = [("x", Rows), ("r", Rows), ("i", Rows), ("o", Rows), ("rate", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("n_slots", ctypes.c_int32), ("D", ctypes.c_int32), ("decay", ctypes.c_int32),
                ("mix", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class BlockArgs(ctypes.Structure):
    _fields_ = [("y", Rows), ("gate", Rows), ("x", Rows), ("xo", Rows), ("z", Rows), ("dxo", Rows),
                ("dz", Rows), ("dy", Rows), ("dgate", Rows), ("dx", Rows),
                ("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
                ("dpost_weight", ctypes.c_void_p), ("dpre_weight", ctypes.c_void_p),
                ("rng", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("t_max", ctypes.c_int64),
                ("n_max", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("dropout", ctypes.c_float),
                ("post_norm", ctypes.c_int32), ("pre_norm", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("stream_dtype", ctypes.c_int32)]


def load_library(path: str = LIB_PATH):
    """Load libgcl.so and declare its C signatures."""
    if not os.path.exists(path):
        raise ImportError(f"libgcl.so not built at {path}; run chunked_gated_linear_gb300._build")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.gcl_last_error.restype = ctypes.c_char_p
    lib.gcl_status_string.restype = ctypes.c_char_p
    lib.gcl_status_string.argtypes = [i32]
    lib.gcl_nt_max.restype = i64
    lib.gcl_nt_max.argtypes = [i64, i64, i32]
    lib.gcl_fwd_chain_segments.restype = i32
    lib.gcl_fwd_chain_segments.argtypes = [i64, i32, i32, i32]
    lib.gcl_selftest_wait_timeout.restype = ctypes.c_int
    lib.gcl_selftest_wait_timeout.argtypes = [vp, vp]
    lib.chunk_meta_build.restype = ctypes.c_int
    lib.chunk_meta_build.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp, vp, vp]
    lib.chunk_meta_build_i64.restype = ctypes.c_int
    lib.chunk_meta_build_i64.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp, vp, vp, vp]
    for fn in ("gdn_chunk_fwd", "kda_chunk_fwd"):
        getattr(lib, fn).restype = ctypes.c_int
        getattr(lib, fn).argtypes = [ctypes.POINTER(FwdArgs), vp]
    lib.gdn_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.gdn_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(FwdArgs), vp]
    lib.gcl_noalloc_scratch_bytes.restype = ctypes.c_size_t
    lib.gcl_noalloc_scratch_bytes.argtypes = []
    for fn in ("gcl_fwd_workspace_bytes", "gcl_fwd_workspace_min_bytes", "gcl_kda_fwd_workspace_bytes"):
        getattr(lib, fn).restype = ctypes.c_size_t
        getattr(lib, fn).argtypes = [ctypes.POINTER(FwdArgs)]
    for fn in ("gcl_fwd_plan", "gcl_kda_fwd_plan"):
        getattr(lib, fn).restype = i32
        getattr(lib, fn).argtypes = [ctypes.POINTER(FwdArgs)]
    for fn in ("gdn_chunk_bwd", "kda_chunk_bwd"):
        getattr(lib, fn).restype = ctypes.c_int
        getattr(lib, fn).argtypes = [ctypes.POINTER(BwdArgs), vp]
    for fn in ("gcl_bwd_workspace_bytes", "gcl_kda_bwd_workspace_bytes"):
        getattr(lib, fn).restype = ctypes.c_size_t
        getattr(lib, fn).argtypes = [ctypes.POINTER(BwdArgs)]
    for fn in ("causal_conv1d_fwd", "causal_conv1d_bwd"):
        getattr(lib, fn).restype = ctypes.c_int
        getattr(lib, fn).argtypes = [ctypes.POINTER(ConvArgs), vp]
    lib.gcl_causal_conv1d_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.gcl_causal_conv1d_bwd_workspace_bytes.argtypes = [ctypes.POINTER(ConvArgs)]
    for fn, args in (("dla_chunk_fwd", DlaArgs), ("dla_chunk_bwd", DlaArgs),
                     ("dla_step", DlaStepArgs), ("qk_norm_rope_fwd", QkArgs),
                     ("qk_norm_rope_bwd", QkArgs), ("glr_fwd", GlrArgs), ("glr_bwd", GlrArgs),
                     ("glr_step", GlrStepArgs), ("block_norm_fwd", BlockArgs),
                     ("block_norm_bwd", BlockArgs)):
        getattr(lib, fn).restype = ctypes.c_int
        getattr(lib, fn).argtypes = [ctypes.POINTER(args), vp]
    for fn, args in (("gcl_dla_fwd_workspace_bytes", DlaArgs),
                     ("gcl_dla_bwd_workspace_bytes", DlaArgs),
                     ("gcl_qk_norm_rope_bwd_workspace_bytes", QkArgs),
                     ("gcl_glr_fwd_workspace_bytes", GlrArgs),
                     ("gcl_glr_bwd_workspace_bytes", GlrArgs),
                     ("gcl_block_norm_bwd_workspace_bytes", BlockArgs)):
        getattr(lib, fn).restype = ctypes.c_size_t
        getattr(lib, fn).argtypes = [ctypes.POINTER(args)]
    lib.gcl_dla_segment_tokens.restype = i64
    lib.gcl_dla_segment_tokens.argtypes = [i64, i32, i32, i32, i32, i32, i32]
    lib.rope_table_build.restype = ctypes.c_int
    lib.rope_table_build.argtypes = [vp, vp, i64, i32, ctypes.c_double, vp]
    return lib


_lib = None


def lib():
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


def _p(t):
    """Device pointer of a tensor (or None)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libgcl must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(fn, st):
    if st != 0:
        raise GclError(fn, st, lib().gcl_last_error().decode())


def _dtype_of(t):
    import torch
    if t.dtype == torch.float32:
        return GCL_F32
    if t.dtype == torch.bfloat16:
        return GCL_BF16
    if t.dtype == torch.float16:
        return GCL_F16
    raise ValueError(f"unsupported dtype {t.dtype}")


class _Layout:
    """Checks one call's tensors against their layouts in include/gcl.h: a CUDA tensor on the
    call's device (when require_cuda), contiguous, of the given dtype(s), with the given
    trailing dimensions and at least the given number of rows."""

    def __init__(self, fn: str, require_cuda: bool = True):
        self.fn, self.require_cuda, self.device = fn, require_cuda, None

    def __call__(self, name, t, dtypes=None, shape=None):
        if t is None:
            return
        if self.require_cuda:
            dev = t.get_device()                         # -1 for a host tensor
            if dev < 0:
                raise ValueError(f"{self.fn}: {name} must be a CUDA tensor (got {t.device})")
            if self.device is None:
                self.device = dev
            elif dev != self.device:
                raise ValueError(f"{self.fn}: {name} is on cuda:{dev}, other tensors on "
                                 f"cuda:{self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{self.fn}: {name} must be contiguous")
        if dtypes is not None:
            dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
            if t.dtype not in dtypes:
                raise ValueError(f"{self.fn}: {name} has dtype {t.dtype}, expected "
                                 + " or ".join(str(d) for d in dtypes))
        if shape is not None:
            got = t.shape
            if len(got) != len(shape) or tuple(got[1:]) != tuple(shape[1:]) or got[0] < shape[0]:
                raise ValueError(f"{self.fn}: {name} has shape {tuple(got)}, expected "
                                 f"{tuple(shape)} (more rows are allowed)")


_SIGNATURES = {}


def _named(builder, args, kw):
    """The arguments of a call of `builder` (fwd_args, bwd_args, conv_args) by name."""
    sig = _SIGNATURES.get(builder)
    if sig is None:
        sig = _SIGNATURES[builder] = inspect.signature(builder)
    b = sig.bind(*args, **kw)
    b.apply_defaults()
    return b.arguments


def validate_fwd(fn, a, kda, require_cuda=True):
    """Layouts of a forward call's tensors (a: fwd_args' arguments by name)."""
    import torch
    L = _Layout(fn, require_cuda)
    q, cu = a["q"], a["cu_seqlens"]
    T, H, K = q.shape
    V = a["v"].shape[-1]
    N = cu.shape[0] - 1
    ntm = nt_max(T, N, a["bt"])
    dt, f32, i32 = q.dtype, torch.float32, torch.int32
    for name, shp in (("q", (T, H, K)), ("k", (T, H, K)), ("v", (T, H, V)), ("beta", (T, H)),
                      ("o", (T, H, V))):
        L(name, a[name], dt, shp)
    L("g", a["g"], f32, (T, H, K) if kda else (T, H))
    L("cu_seqlens", cu, i32, (N + 1,))
    for name in ("h0", "ht"):
        L(name, a[name], f32, (N, H, K, V))
    L("h_save", a["h_save"], f32, (ntm, H, K, V))
    L("chunk_indices", a["chunk_indices"], i32, (ntm, 2))
    L("chunk_offsets", a["chunk_offsets"], i32, (N + 1,))
    L("seq_order", a["seq_order"], i32, (N,))
    L("dev_status", a["dev_status"], i32, (1,))
    L("workspace", a["workspace"])


def validate_bwd(fn, a, kda, require_cuda=True):
    """Layouts of a backward call's tensors (a: bwd_args' arguments by name)."""
    import torch
    L = _Layout(fn, require_cuda)
    q, cu = a["q"], a["cu_seqlens"]
    T, H, K = q.shape
    V = a["v"].shape[-1]
    N = cu.shape[0] - 1
    ntm = nt_max(T, N, a["bt"])
    dt, f32, i32 = q.dtype, torch.float32, torch.int32
    gshape = (T, H, K) if kda else (T, H)
    for name, shp in (("q", (T, H, K)), ("k", (T, H, K)), ("v", (T, H, V)), ("beta", (T, H)),
                      ("d_o", (T, H, V))):
        L(name, a[name], dt, shp)
    for name, shp in (("g", gshape), ("dg", gshape), ("dq", (T, H, K)), ("dk", (T, H, K)),
                      ("dv", (T, H, V)), ("dbeta", (T, H)), ("h0", (N, H, K, V)),
                      ("dht", (N, H, K, V)), ("dh0", (N, H, K, V)), ("h_save", (ntm, H, K, V))):
        L(name, a[name], f32, shp)
    L("cu_seqlens", cu, i32, (N + 1,))
    L("chunk_indices", a["chunk_indices"], i32, (ntm, 2))
    L("chunk_offsets", a["chunk_offsets"], i32, (N + 1,))
    L("dev_status", a["dev_status"], i32, (1,))
    L("workspace", a["workspace"])
    L("fwd_workspace", a["fwd_workspace"])


def validate_conv(fn, a, require_cuda=True):
    """Layouts of a causal_conv1d call's tensors (a: conv_args' arguments by name)."""
    import torch
    L = _Layout(fn, require_cuda)
    x, w, cu = a["x"], a["weight"], a["cu_seqlens"]
    T, D = x.shape
    W = w.shape[1]
    N = cu.shape[0] - 1
    dt, f32, i32 = x.dtype, torch.float32, torch.int32
    for name, shp in (("x", (T, D)), ("weight", (D, W)), ("bias", (D,)), ("residual", (T, D)),
                      ("h0", (N, D, W - 1)), ("y", (T, D)), ("ht", (N, D, W - 1)),
                      ("dy", (T, D))):
        L(name, a[name], dt, shp)
    for name, shp in (("dht", (N, D, W - 1)), ("dx", (T, D)), ("dweight", (D, W)),
                      ("dbias", (D,)), ("dh0", (N, D, W - 1))):
        L(name, a[name], f32, shp)
    L("cu_seqlens", cu, i32, (N + 1,))
    L("chunk_indices", a["chunk_indices"], i32, (nt_max(T, N, a["bt"]), 2))
    L("dev_status", a["dev_status"], i32, (1,))
    L("workspace", a["workspace"])


def nt_max(t_max: int, n_max: int, bt: int = CHUNK) -> int:
    return int(lib().gcl_nt_max(t_max, n_max, bt))


def selftest_wait_timeout(dev_status, stream=None):
    """One CTA waits on an mbarrier nothing arrives at; after the time limit dev_status holds
    GCL_DEV_WAIT_TIMEOUT (the bounded-wait path of every tensor-core kernel)."""
    import torch
    _Layout("gcl_selftest_wait_timeout")("dev_status", dev_status, torch.int32, (1,))
    _check("gcl_selftest_wait_timeout", lib().gcl_selftest_wait_timeout(_p(dev_status), _stream(stream)))


def fwd_chain_segments(t_max: int, n_max: int, H: int, bt: int = CHUNK) -> int:
    """Segments per sequence of the fastest tensor-core forward plan (0: the plain chain)."""
    return int(lib().gcl_fwd_chain_segments(t_max, n_max, H, bt))


def chunk_meta_build(cu_seqlens, t_max, chunk_indices, chunk_offsets, dev_status,
                     seq_order=None, bt: int = CHUNK, stream=None, cu_seqlens32=None):
    """Chunk metadata from cu_seqlens (int32, or int64 with an int32 copy written to
    cu_seqlens32 for the compute calls)."""
    import torch
    n_max = cu_seqlens.shape[0] - 1
    L = _Layout("chunk_meta_build")
    L("cu_seqlens", cu_seqlens, (torch.int32, torch.int64), (n_max + 1,))
    L("chunk_indices", chunk_indices, torch.int32, (chunk_indices.shape[0], 2))
    L("chunk_offsets", chunk_offsets, torch.int32, (n_max + 1,))
    L("seq_order", seq_order, torch.int32, (n_max,))
    L("dev_status", dev_status, torch.int32, (1,))
    L("cu_seqlens32", cu_seqlens32, torch.int32, (n_max + 1,))
    if cu_seqlens.element_size() == 8:
        if cu_seqlens32 is None:
            raise ValueError("an int64 cu_seqlens needs cu_seqlens32 (int32 [n_max + 1]) for its copy")
        _check("chunk_meta_build_i64",
               lib().chunk_meta_build_i64(_p(cu_seqlens), n_max, t_max, bt, chunk_indices.shape[0],
                                          _p(cu_seqlens32), _p(chunk_indices), _p(chunk_offsets),
                                          _p(seq_order), _p(dev_status), _stream(stream)))
        return
    _check("chunk_meta_build",
           lib().chunk_meta_build(_p(cu_seqlens), n_max, t_max, bt, chunk_indices.shape[0],
                                  _p(chunk_indices), _p(chunk_offsets), _p(seq_order),
                                  _p(dev_status), _stream(stream)))


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def fwd_args(q, k, v, g, beta, cu_seqlens, o, h0=None, ht=None, h_save=None,
             chunk_indices=None, chunk_offsets=None, seq_order=None, dev_status=None,
             workspace=None, scale=None, bt=CHUNK):
    T, H, K = q.shape
    V = v.shape[-1]
    a = FwdArgs(q=_p(q), k=_p(k), v=_p(v), g=_p(g), beta=_p(beta), h0=_p(h0),
                cu_seqlens=_p(cu_seqlens), chunk_indices=_p(chunk_indices),
                chunk_offsets=_p(chunk_offsets), seq_order=_p(seq_order), o=_p(o), ht=_p(ht),
                h_save=_p(h_save), dev_status=_p(dev_status), workspace=_p(workspace),
                workspace_bytes=_nbytes(workspace), t_max=T, n_max=cu_seqlens.shape[0] - 1,
                H=H, K=K, V=V, bt=bt, scale=float(K ** -0.5 if scale is None else scale),
                dtype=_dtype_of(q))
    return a


def fwd_workspace_bytes(*args, **kw) -> int:
    """Workspace of the fastest launch plan for these sizes."""
    a = fwd_args(*args, **kw)
    return int(lib().gcl_fwd_workspace_bytes(ctypes.byref(a)))


def fwd_workspace_min_bytes(*args, **kw) -> int:
    """Least workspace the forward accepts (it then runs the W-form plan; 0 where the fused
    plan runs)."""
    a = fwd_args(*args, **kw)
    return int(lib().gcl_fwd_workspace_min_bytes(ctypes.byref(a)))


def kda_fwd_workspace_bytes(*args, **kw) -> int:
    """Workspace kda_chunk_fwd needs (its one tensor-core plan; 0 on the CUDA-core path)."""
    a = fwd_args(*args, **kw)
    return int(lib().gcl_kda_fwd_workspace_bytes(ctypes.byref(a)))


PLANS = {0: "cuda_cores", 1: "fused", 2: "w_form", 3: "transition", 4: "segmented",
         5: "cuda_cores_split"}


def fwd_plan(*args, kda=False, **kw) -> str:
    """Name of the launch plan the forward runs with these arguments (workspace included):
    cuda_cores, fused, w_form, transition or segmented (include/gcl.h, gcl_fwd_plan)."""
    a = fwd_args(*args, **kw)
    code = int((lib().gcl_kda_fwd_plan if kda else lib().gcl_fwd_plan)(ctypes.byref(a)))
    if code < 0:
        raise GclError("gcl_fwd_plan", code, lib().gcl_last_error().decode())
    return PLANS[code]


def gdn_chunk_fwd(*args, stream=None, **kw):
    validate_fwd("gdn_chunk_fwd", _named(fwd_args, args, kw), kda=False)
    a = fwd_args(*args, **kw)
    _check("gdn_chunk_fwd", lib().gdn_chunk_fwd(ctypes.byref(a), _stream(stream)))


def gdn_chunk_fwd_noalloc(*args, stream=None, **kw):
    """gdn_chunk_fwd without a workspace argument: the library's static scratch is used
    (for callers that cannot allocate device memory; see include/gcl.h)."""
    kw.pop("workspace", None)
    validate_fwd("gdn_chunk_fwd_noalloc", _named(fwd_args, args, kw), kda=False)
    a = fwd_args(*args, **kw)
    _check("gdn_chunk_fwd_noalloc", lib().gdn_chunk_fwd_noalloc(ctypes.byref(a), _stream(stream)))


def noalloc_scratch_bytes() -> int:
    return int(lib().gcl_noalloc_scratch_bytes())


def kda_chunk_fwd(*args, stream=None, **kw):
    validate_fwd("kda_chunk_fwd", _named(fwd_args, args, kw), kda=True)
    a = fwd_args(*args, **kw)
    _check("kda_chunk_fwd", lib().kda_chunk_fwd(ctypes.byref(a), _stream(stream)))


def bwd_args(q, k, v, g, beta, d_o, cu_seqlens, chunk_indices, chunk_offsets, dq, dk, dv, dg,
             dbeta, h0=None, dht=None, dh0=None, h_save=None, workspace=None,
             dev_status=None, scale=None, bt=CHUNK, fwd_workspace=None):
    T, H, K = q.shape
    V = v.shape[-1]
    return BwdArgs(q=_p(q), k=_p(k), v=_p(v), g=_p(g), beta=_p(beta), h0=_p(h0), d_o=_p(d_o),
                   dht=_p(dht), cu_seqlens=_p(cu_seqlens), chunk_indices=_p(chunk_indices),
                   chunk_offsets=_p(chunk_offsets), h_save=_p(h_save), dq=_p(dq), dk=_p(dk),
                   dv=_p(dv), dg=_p(dg), dbeta=_p(dbeta), dh0=_p(dh0),
                   workspace=_p(workspace), workspace_bytes=_nbytes(workspace),
                   dev_status=_p(dev_status), t_max=T, n_max=cu_seqlens.shape[0] - 1, H=H, K=K,
                   V=V, bt=bt, scale=float(K ** -0.5 if scale is None else scale),
                   dtype=_dtype_of(q), fwd_workspace=_p(fwd_workspace),
                   fwd_workspace_bytes=_nbytes(fwd_workspace))


def bwd_workspace_bytes(*args, **kw) -> int:
    a = bwd_args(*args, **kw)
    return int(lib().gcl_bwd_workspace_bytes(ctypes.byref(a)))


def gdn_chunk_bwd(*args, stream=None, **kw):
    validate_bwd("gdn_chunk_bwd", _named(bwd_args, args, kw), kda=False)
    a = bwd_args(*args, **kw)
    _check("gdn_chunk_bwd", lib().gdn_chunk_bwd(ctypes.byref(a), _stream(stream)))


def kda_bwd_workspace_bytes(*args, **kw) -> int:
    a = bwd_args(*args, **kw)
    return int(lib().gcl_kda_bwd_workspace_bytes(ctypes.byref(a)))


def kda_chunk_bwd(*args, stream=None, **kw):
    """The KDA backward; dg has the shape of g, [T, H, K]."""
    validate_bwd("kda_chunk_bwd", _named(bwd_args, args, kw), kda=True)
    a = bwd_args(*args, **kw)
    _check("kda_chunk_bwd", lib().kda_chunk_bwd(ctypes.byref(a), _stream(stream)))


# ---------------------------------------------------------------- causal_conv1d
ACTIVATIONS = {None: 0, "silu": 1}


def conv_args(x, weight, cu_seqlens, chunk_indices, bias=None, residual=None, h0=None, y=None,
              ht=None, dy=None, dht=None, dx=None, dweight=None, dbias=None, dh0=None,
              workspace=None, dev_status=None, activation=None, bt=CHUNK):
    """gcl_conv_args for x [T, D], weight [D, W]; see include/gcl.h (causal_conv1d)."""
    T, D = x.shape
    return ConvArgs(x=_p(x), weight=_p(weight), bias=_p(bias), residual=_p(residual), h0=_p(h0),
                    y=_p(y), ht=_p(ht), dy=_p(dy), dht=_p(dht), dx=_p(dx), dweight=_p(dweight),
                    dbias=_p(dbias), dh0=_p(dh0), cu_seqlens=_p(cu_seqlens),
                    chunk_indices=_p(chunk_indices), dev_status=_p(dev_status),
                    workspace=_p(workspace), workspace_bytes=_nbytes(workspace), t_max=T,
                    n_max=cu_seqlens.shape[0] - 1, D=D, W=weight.shape[1], bt=bt,
                    activation=ACTIVATIONS[activation], dtype=_dtype_of(x))


def causal_conv1d_fwd(*args, stream=None, **kw):
    validate_conv("causal_conv1d_fwd", _named(conv_args, args, kw))
    a = conv_args(*args, **kw)
    _check("causal_conv1d_fwd", lib().causal_conv1d_fwd(ctypes.byref(a), _stream(stream)))


def causal_conv1d_bwd_workspace_bytes(*args, **kw) -> int:
    a = conv_args(*args, **kw)
    return int(lib().gcl_causal_conv1d_bwd_workspace_bytes(ctypes.byref(a)))


def causal_conv1d_bwd(*args, stream=None, **kw):
    validate_conv("causal_conv1d_bwd", _named(conv_args, args, kw))
    a = conv_args(*args, **kw)
    _check("causal_conv1d_bwd", lib().causal_conv1d_bwd(ctypes.byref(a), _stream(stream)))


# ------------------------------------------------- decayed linear attention, norm and rotation
# These calls take strided rows and are also made for single tokens, where the host's time counts:
# each tensor is checked by plain comparisons, and the argument struct is packed in one go (the
# layouts of DlaArgs, DlaStepArgs and QkArgs above, which the C structs share).
_ROWS_FMT = "Pqq"
_DLA_PACK = struct.Struct("@" + _ROWS_FMT * 8 + "PPPPPPPPPNqiiiifi0q")
_STEP_PACK = struct.Struct("@" + _ROWS_FMT * 4 + "PPPPiiiiifi0q")
_QK_PACK = struct.Struct("@" + _ROWS_FMT * 8 + "PPPPPPPPPNqqiiiifiii0q")
_NO_ROWS = (0, 0, 0)


_devices = 0                             # visible devices, counted at the first call


def _current_device():
    global _devices
    import torch
    _devices = torch.cuda.device_count()
    return torch._C._cuda_getDevice()


def _on_device(fn, device):
    """The library launches on the current device and plans for it, so the tensors have to live there.  (A pointer of
    another device would be used on this one.)"""
    if device != _current_device():
        raise ValueError(f"{fn}: the tensors are on cuda:{device}, the current device is cuda:{_current_device()}; make "
                         f"theirs current (torch.cuda.device)")


def _raw_stream(device):
    """The current stream; after the first call torch's own function."""
    global _raw_stream
    import torch
    _raw_stream = torch._C._cuda_getCurrentRawStream
    return _raw_stream(device)


def _packed_call(fn, packed, stream, device):
    """Calls entry point `fn` of the loaded library with a packed argument struct."""
    if _devices != 1:                    # (with one device there is no other; the look at it takes 0.4 us a call)
        _on_device(fn, device)
    handle = lib()
    entry = handle.__dict__.get("_packed_" + fn)
    if entry is None:
        entry = handle._FuncPtr((fn, handle))
        entry.restype, entry.argtypes = ctypes.c_int, [ctypes.c_char_p, ctypes.c_void_p]
        handle.__dict__["_packed_" + fn] = entry
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    st = entry(packed, stream)
    if st != 0:
        _check(fn, st)


def _rows(fn, name, t, shape, dtype, device):
    """gcl_rows of a tensor [tokens, heads, D] with contiguous D and any token and head strides."""
    if t.get_device() != device or device < 0:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor on the call's device (got {t.device})")
    if t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {shape}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{fn}: {name} must have contiguous rows (strides {t.stride()})")
    if shape[1] == 1:                        # the stride of an extent of one is free: one that fits
        sh = shape[2]
    if shape[0] == 1:
        st = shape[1] * sh
    if st < 0 or sh < 0:
        raise ValueError(f"{fn}: {name} has negative strides {t.stride()}")
    return t.data_ptr(), st, sh


def _flat(fn, name, t, shape, dtype, device):
    """Pointer of a contiguous tensor of exactly this shape; 0 for None."""
    if t is None:
        return 0
    if t.get_device() != device or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous CUDA tensor {shape} of {dtype} on the "
                         f"call's device (got {tuple(t.shape)}, {t.dtype}, {t.device})")
    return t.data_ptr()


def _scratch(fn, t, device):
    if t is None:
        return 0, 0
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{fn}: workspace must be a contiguous CUDA tensor on the call's device")
    return t.data_ptr(), t.numel() * t.element_size()


def _dla_sizes(fn, q, v, cu_seqlens):
    if q.get_device() >= 0:                                # (the plan is for the current device's SMs)
        _on_device(fn, q.get_device())
    T, H, K = q.shape
    return DlaArgs(t_max=T, n_max=cu_seqlens.shape[0] - 1, H=H, K=K, V=v.shape[2], dtype=_dtype_of(q))


def dla_segment_tokens(t_max: int, n_max: int, H: int, backward: bool = False, dtype: int = GCL_BF16,
                       K: int = 128, V: int = 128) -> int:
    """Tokens per segment of the plan for these capacities on the current device (t_max or more: sequences stay whole)."""
    return int(lib().gcl_dla_segment_tokens(t_max, n_max, H, int(backward), dtype, K, V))


def dla_fwd_workspace_bytes(q, v, cu_seqlens) -> int:
    """Workspace of dla_chunk_fwd for these sizes (0: none)."""
    a = _dla_sizes("dla_fwd_workspace_bytes", q, v, cu_seqlens)
    return int(lib().gcl_dla_fwd_workspace_bytes(ctypes.byref(a)))


def dla_bwd_workspace_bytes(q, v, cu_seqlens) -> int:
    """Workspace of dla_chunk_bwd for these sizes (0: none)."""
    a = _dla_sizes("dla_bwd_workspace_bytes", q, v, cu_seqlens)
    return int(lib().gcl_dla_bwd_workspace_bytes(ctypes.byref(a)))


def dla_chunk_fwd(q, k, v, g, cu_seqlens, o, h0=None, ht=None, seq_order=None, dev_status=None,
                  workspace=None, scale=None, stream=None):
    """Linear attention with the fixed log decay g [H] over packed sequences (include/gcl.h, dla):
    o [T, H, V] (None: only ht) and ht from q, k [T, H, K], v [T, H, V] and h0.  q, k, v and o may
    have strided tokens and heads."""
    from torch import float32 as f32, int32 as i32
    fn = "dla_chunk_fwd"
    sk = tuple(q.shape)
    T, H, K = sk
    V, N, dt, dev = v.shape[2], cu_seqlens.shape[0] - 1, q.dtype, q.get_device()
    sv, ss = (T, H, V), (N, H, K, V)
    packed = _DLA_PACK.pack(
        *_rows(fn, "q", q, sk, dt, dev), *_rows(fn, "k", k, sk, dt, dev), *_rows(fn, "v", v, sv, dt, dev),
        *(_NO_ROWS if o is None else _rows(fn, "o", o, sv, dt, dev)), *_NO_ROWS, *_NO_ROWS, *_NO_ROWS, *_NO_ROWS,
        _flat(fn, "g", g, (H,), f32, dev), _flat(fn, "h0", h0, ss, f32, dev), _flat(fn, "ht", ht, ss, f32, dev), 0, 0,
        _flat(fn, "cu_seqlens", cu_seqlens, (N + 1,), i32, dev), _flat(fn, "seq_order", seq_order, (N,), i32, dev),
        _flat(fn, "dev_status", dev_status, (1,), i32, dev), *_scratch(fn, workspace, dev), T, N, H, K, V,
        K ** -0.5 if scale is None else scale, _dtype_of(q))
    _packed_call(fn, packed, stream, dev)


def dla_chunk_bwd(q, k, v, g, d_o, cu_seqlens, dq, dk, dv, h0=None, dht=None, dh0=None,
                  seq_order=None, dev_status=None, workspace=None, scale=None, stream=None):
    """The backward of dla_chunk_fwd: dq, dk, dv (of q's dtype) and dh0 from d_o and dht."""
    from torch import float32 as f32, int32 as i32
    fn = "dla_chunk_bwd"
    sk = tuple(q.shape)
    T, H, K = sk
    V, N, dt, dev = v.shape[2], cu_seqlens.shape[0] - 1, q.dtype, q.get_device()
    sv, ss = (T, H, V), (N, H, K, V)
    packed = _DLA_PACK.pack(
        *_rows(fn, "q", q, sk, dt, dev), *_rows(fn, "k", k, sk, dt, dev), *_rows(fn, "v", v, sv, dt, dev), *_NO_ROWS,
        *_rows(fn, "d_o", d_o, sv, dt, dev), *_rows(fn, "dq", dq, sk, dt, dev), *_rows(fn, "dk", dk, sk, dt, dev),
        *_rows(fn, "dv", dv, sv, dt, dev), _flat(fn, "g", g, (H,), f32, dev), _flat(fn, "h0", h0, ss, f32, dev), 0,
        _flat(fn, "dht", dht, ss, f32, dev), _flat(fn, "dh0", dh0, ss, f32, dev),
        _flat(fn, "cu_seqlens", cu_seqlens, (N + 1,), i32, dev), _flat(fn, "seq_order", seq_order, (N,), i32, dev),
        _flat(fn, "dev_status", dev_status, (1,), i32, dev), *_scratch(fn, workspace, dev), T, N, H, K, V,
        K ** -0.5 if scale is None else scale, _dtype_of(q))
    _packed_call(fn, packed, stream, dev)


def dla_step(q, k, v, g, state, o, slots=None, dev_status=None, scale=None, stream=None):
    """One token of each request: the states [n_slots, H, K, V] of the requests' slots are updated
    in place and o [B, H, V] is written (include/gcl.h, dla_step).  slots int32 [B]; negative: idle."""
    from torch import float32 as f32, int32 as i32
    fn = "dla_step"
    sk = tuple(q.shape)
    B, H, K = sk
    V, dt, dev, n_slots = v.shape[2], q.dtype, q.get_device(), state.shape[0]
    sv = (B, H, V)
    packed = _STEP_PACK.pack(
        *_rows(fn, "q", q, sk, dt, dev), *_rows(fn, "k", k, sk, dt, dev), *_rows(fn, "v", v, sv, dt, dev),
        *_rows(fn, "o", o, sv, dt, dev), _flat(fn, "g", g, (H,), f32, dev),
        _flat(fn, "state", state, (n_slots, H, K, V), f32, dev), _flat(fn, "slots", slots, (B,), i32, dev),
        _flat(fn, "dev_status", dev_status, (1,), i32, dev), B, n_slots, H, K, V,
        K ** -0.5 if scale is None else scale, _dtype_of(q))
    _packed_call(fn, packed, stream, dev)


NORMS = {None: 0, "none": 0, "rms": 1, "l2": 2}
PAIRINGS = {"half": 0, "adjacent": 1}


def _qk_call(fn, q, k, yq, yk, dyq, dyk, dq, dk, q_weight, k_weight, dq_weight, dk_weight, cos, sin, positions, norm,
             eps, pairing, workspace, dev_status, stream, backward):
    from torch import float32 as f32, int32 as i32
    sq = tuple(q.shape)
    T, HQ, D = sq
    HK = 0 if k is None else k.shape[1]
    sk, dt, dev = (T, HK, D), q.dtype, q.get_device()
    if norm not in NORMS or pairing not in PAIRINGS:
        raise ValueError(f"{fn}: norm {norm!r} or pairing {pairing!r} is not one of {tuple(NORMS)}, "
                         f"{tuple(PAIRINGS)}")
    P = half = c = s = 0
    if (cos is None) != (sin is None):
        raise ValueError(f"{fn}: cos and sin come together")
    if cos is not None:
        P, half = cos.shape
        c, s = _flat(fn, "cos", cos, (P, half), f32, dev), _flat(fn, "sin", sin, (P, half), f32, dev)
    rq = _rows(fn, "q", q, sq, dt, dev)
    rk = _rows(fn, "k", k, sk, dt, dev) if HK else _NO_ROWS
    if backward:
        out = (*_NO_ROWS, *_NO_ROWS, *_rows(fn, "dyq", dyq, sq, dt, dev),
               *(_rows(fn, "dyk", dyk, sk, dt, dev) if HK else _NO_ROWS), *_rows(fn, "dq", dq, sq, dt, dev),
               *(_rows(fn, "dk", dk, sk, dt, dev) if HK else _NO_ROWS))
    else:
        out = (*_rows(fn, "yq", yq, sq, dt, dev), *(_rows(fn, "yk", yk, sk, dt, dev) if HK else _NO_ROWS),
               *_NO_ROWS, *_NO_ROWS, *_NO_ROWS, *_NO_ROWS)
    packed = _QK_PACK.pack(
        *rq, *rk, *out, _flat(fn, "q_weight", q_weight, (D,), dt, dev), _flat(fn, "k_weight", k_weight, (D,), dt, dev),
        _flat(fn, "dq_weight", dq_weight, (D,), f32, dev), _flat(fn, "dk_weight", dk_weight, (D,), f32, dev), c, s,
        _flat(fn, "positions", positions, (T,), i32, dev), _flat(fn, "dev_status", dev_status, (1,), i32, dev),
        *_scratch(fn, workspace, dev), T, P, HQ, HK, D, 2 * half, eps, NORMS[norm], PAIRINGS[pairing], _dtype_of(q))
    _packed_call(fn, packed, stream, dev)


def qk_norm_rope_fwd(q, k, yq, yk, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                     norm="rms", eps=1e-6, pairing="half", dev_status=None, stream=None):
    """Norm of each head's queries [T, HQ, D] and keys [T, HK, D] (k None: queries alone) and the
    rotation by the rows `positions` of cos, sin [P, R / 2], in one pass (include/gcl.h,
    qk_norm_rope)."""
    _qk_call("qk_norm_rope_fwd", q, k, yq, yk, None, None, None, None, q_weight, k_weight, None, None, cos, sin,
             positions, norm, eps, pairing, None, dev_status, stream, False)


def qk_norm_rope_bwd_workspace_bytes(q, k) -> int:
    """Workspace of qk_norm_rope_bwd with weight gradients."""
    if q.get_device() >= 0:
        _on_device("qk_norm_rope_bwd_workspace_bytes", q.get_device())
    T, HQ, D = q.shape
    a = QkArgs(t_max=T, HQ=HQ, HK=0 if k is None else k.shape[1], D=D)
    return int(lib().gcl_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(a)))


def qk_norm_rope_bwd(q, k, dyq, dyk, dq, dk, q_weight=None, k_weight=None, dq_weight=None,
                     dk_weight=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6,
                     pairing="half", workspace=None, dev_status=None, stream=None):
    """The backward of qk_norm_rope_fwd: dq, dk from dyq, dyk, and the weights' gradients fp32 [D]."""
    _qk_call("qk_norm_rope_bwd", q, k, None, None, dyq, dyk, dq, dk, q_weight, k_weight, dq_weight, dk_weight, cos, sin,
             positions, norm, eps, pairing, workspace, dev_status, stream, True)


def rope_table_build(cos, sin, base: float = 10000.0, stream=None):
    """Fills the tables cos, sin [P, R / 2] fp32 with the angles p base^(-2 i / R)."""
    from torch import float32 as f32
    fn = "rope_table_build"
    if cos.dim() != 2:
        raise ValueError(f"{fn}: cos must be [positions, R / 2]")
    shape, dev = tuple(cos.shape), cos.get_device()
    if dev < 0:
        raise ValueError(f"{fn}: cos must be a CUDA tensor (got {cos.device})")
    c, s = _flat(fn, "cos", cos, shape, f32, dev), _flat(fn, "sin", sin, shape, f32, dev)
    _on_device(fn, dev)
    _check(fn, lib().rope_table_build(c, s, shape[0], 2 * shape[1], float(base), _stream(stream)))


# ------------------------------------------------------------------ gated linear recurrence
DECAYS = {"log": 0, "sigmoid": 1, "power": 2}
MIXES = {"one": 0, "complement": 1, "root": 2}
_GLR_PACK = struct.Struct("@" + _ROWS_FMT * 8 + "PPPPPPPPPPNqiiiii0q")
_GLR_STEP_PACK = struct.Struct("@" + _ROWS_FMT * 4 + "PPPPiiiiii0q")


# What the calls below look up of torch, kept from the first call on (an import statement in the call takes 0.6 us of it).
_F32 = _I32 = _I64 = None
_DTYPE_CODES = {}


def _load_torch():
    global _F32, _I32, _I64
    import torch
    _DTYPE_CODES.update({torch.float32: GCL_F32, torch.bfloat16: GCL_BF16, torch.float16: GCL_F16})
    _I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _code_of(fn, name, dtype):
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"{fn}: {name} has dtype {dtype}, expected one of {tuple(_DTYPE_CODES)}")
    return code


def _rows2(fn, name, t, shape, dtype, device):
    """gcl_rows of a tensor [tokens, D] with contiguous D and any token stride."""
    if t.get_device() != device or device < 0 or t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor {tuple(shape)} of {dtype} on the call's device (got {tuple(t.shape)}, "
                         f"{t.dtype}, {t.device})")
    st, sd = t.stride()
    if sd != 1 or st < 0:
        raise ValueError(f"{fn}: {name} must have contiguous rows and no negative stride (strides {t.stride()})")
    # (the stride of an extent of one is free: one that fits)
    return t.data_ptr(), st if shape[0] != 1 else shape[1], shape[1]


def _kind(fn, decay, mix):
    if decay not in DECAYS or mix not in MIXES:
        raise ValueError(f"{fn}: decay {decay!r} or mix {mix!r} is not one of {tuple(DECAYS)}, {tuple(MIXES)}")
    return DECAYS[decay], MIXES[mix]


def _save_rows(T):
    return -(-T // CHUNK)


def glr_fwd_workspace_bytes(x, cu_seqlens) -> int:
    """Workspace of glr_fwd for these sizes."""
    if x.get_device() >= 0:
        _on_device("glr_fwd_workspace_bytes", x.get_device())
    a = GlrArgs(t_max=x.shape[0], n_max=cu_seqlens.shape[0] - 1, D=x.shape[1], dtype=_dtype_of(x))
    return int(lib().gcl_glr_fwd_workspace_bytes(ctypes.byref(a)))


def glr_bwd_workspace_bytes(x, cu_seqlens, h_save=None, drate=True) -> int:
    """Workspace of glr_bwd for these sizes, with the states h_save of the forward or without (None), and with
    the gradient of the rates (drate) or without."""
    if x.get_device() >= 0:
        _on_device("glr_bwd_workspace_bytes", x.get_device())
    a = GlrArgs(t_max=x.shape[0], n_max=cu_seqlens.shape[0] - 1, D=x.shape[1], dtype=_dtype_of(x),
                h_save=None if h_save is None else 16, drate=16 if drate is not None and drate is not False else None)
    return int(lib().gcl_glr_bwd_workspace_bytes(ctypes.byref(a)))


def glr_fwd(x, r, cu_seqlens, o, i=None, rate=None, h0=None, ht=None, h_save=None, decay="power", mix="root",
            dev_status=None, workspace=None, stream=None):
    """The gated linear recurrence over packed sequences (include/gcl.h, glr): o [T, D] (None: only the states) and
    ht [N, D] from x, the decay gate r, the input gate i (or None) [T, D] and h0.  x, r, i and o may have strided
    tokens.  h_save [ceil(T / 64), D] fp32 keeps the states that the backward reads."""
    if _F32 is None:
        _load_torch()
    f32, i32 = _F32, _I32
    fn = "glr_fwd"
    sx = x.shape
    T, D = sx
    N, dt, dev = cu_seqlens.shape[0] - 1, x.dtype, x.get_device()
    kd, km = _kind(fn, decay, mix)
    packed = _GLR_PACK.pack(
        *_rows2(fn, "x", x, sx, dt, dev), *_rows2(fn, "r", r, sx, dt, dev),
        *(_NO_ROWS if i is None else _rows2(fn, "i", i, sx, dt, dev)),
        *(_NO_ROWS if o is None else _rows2(fn, "o", o, sx, dt, dev)), *_NO_ROWS, *_NO_ROWS, *_NO_ROWS, *_NO_ROWS,
        0 if rate is None else _flat(fn, "rate", rate, (D,), f32, dev),
        0 if h0 is None else _flat(fn, "h0", h0, (N, D), f32, dev),
        0 if ht is None else _flat(fn, "ht", ht, (N, D), f32, dev),
        0, 0, 0, 0 if h_save is None else _flat(fn, "h_save", h_save, (_save_rows(T), D), f32, dev),
        _flat(fn, "cu_seqlens", cu_seqlens, (N + 1,), i32, dev),
        0 if dev_status is None else _flat(fn, "dev_status", dev_status, (1,), i32, dev),
        *_scratch(fn, workspace, dev), T, N, D, kd, km, _code_of(fn, "x", dt))
    _packed_call(fn, packed, stream, dev)


def glr_bwd(x, r, d_o, cu_seqlens, dx, dr, i=None, di=None, rate=None, drate=None, h0=None, dht=None, dh0=None,
            h_save=None, decay="power", mix="root", dev_status=None, workspace=None, stream=None):
    """The backward of glr_fwd: dx, dr, di (with i) of x's dtype, drate [D] and dh0 [N, D] from d_o and dht.  With the
    forward's h_save the states are not formed again."""
    if _F32 is None:
        _load_torch()
    f32, i32 = _F32, _I32
    fn = "glr_bwd"
    sx = x.shape
    T, D = sx
    N, dt, dev = cu_seqlens.shape[0] - 1, x.dtype, x.get_device()
    kd, km = _kind(fn, decay, mix)
    if (i is None) != (di is None):
        raise ValueError(f"{fn}: i and di come together")
    packed = _GLR_PACK.pack(
        *_rows2(fn, "x", x, sx, dt, dev), *_rows2(fn, "r", r, sx, dt, dev),
        *(_NO_ROWS if i is None else _rows2(fn, "i", i, sx, dt, dev)), *_NO_ROWS, *_rows2(fn, "d_o", d_o, sx, dt, dev),
        *_rows2(fn, "dx", dx, sx, dt, dev), *_rows2(fn, "dr", dr, sx, dt, dev),
        *(_NO_ROWS if di is None else _rows2(fn, "di", di, sx, dt, dev)),
        0 if rate is None else _flat(fn, "rate", rate, (D,), f32, dev),
        0 if h0 is None else _flat(fn, "h0", h0, (N, D), f32, dev), 0,
        0 if dht is None else _flat(fn, "dht", dht, (N, D), f32, dev),
        0 if dh0 is None else _flat(fn, "dh0", dh0, (N, D), f32, dev),
        0 if drate is None else _flat(fn, "drate", drate, (D,), f32, dev),
        0 if h_save is None else _flat(fn, "h_save", h_save, (_save_rows(T), D), f32, dev),
        _flat(fn, "cu_seqlens", cu_seqlens, (N + 1,), i32, dev),
        0 if dev_status is None else _flat(fn, "dev_status", dev_status, (1,), i32, dev),
        *_scratch(fn, workspace, dev), T, N, D, kd, km, _code_of(fn, "x", dt))
    _packed_call(fn, packed, stream, dev)


def glr_step(x, r, state, o, i=None, rate=None, slots=None, decay="power", mix="root", dev_status=None, stream=None):
    """One token of each request: the states [n_slots, D] of the requests' slots are updated in place and
    o [B, D] is written (include/gcl.h, glr_step).  slots int32 [B]; negative: idle."""
    if _F32 is None:
        _load_torch()
    f32, i32 = _F32, _I32
    fn = "glr_step"
    sx = x.shape
    B, D = sx
    dt, dev, n_slots = x.dtype, x.get_device(), state.shape[0]
    kd, km = _kind(fn, decay, mix)
    packed = _GLR_STEP_PACK.pack(
        *_rows2(fn, "x", x, sx, dt, dev), *_rows2(fn, "r", r, sx, dt, dev),
        *(_NO_ROWS if i is None else _rows2(fn, "i", i, sx, dt, dev)), *_rows2(fn, "o", o, sx, dt, dev),
        0 if rate is None else _flat(fn, "rate", rate, (D,), f32, dev), _flat(fn, "state", state, (n_slots, D), f32, dev),
        0 if slots is None else _flat(fn, "slots", slots, (B,), i32, dev),
        0 if dev_status is None else _flat(fn, "dev_status", dev_status, (1,), i32, dev), B, n_slots, D, kd, km,
        _code_of(fn, "x", dt))
    _packed_call(fn, packed, stream, dev)


# ------------------------------------------------------------------ norms around a block
GATE_ACTIVATIONS = {None: 0, "silu": 1, "sigmoid": 2}
_BLOCK_PACK = struct.Struct("@" + _ROWS_FMT * 10 + "PPPPPPPPNqiiifffiiiii0q")


def _rows3(fn, name, t, shape, dtype, device):
    """gcl_rows of a tensor [tokens, heads, D], or [tokens, D] where the call's rows have one head."""
    if len(shape) == 2:
        return _rows2(fn, name, t, shape, dtype, device)
    if t.get_device() != device or device < 0 or t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{fn}: {name} must be a CUDA tensor {tuple(shape)} of {dtype} on the call's device (got {tuple(t.shape)}, "
                         f"{t.dtype}, {t.device})")
    T, H, D = shape
    st, sh, sd = t.stride()
    if sd != 1 or st < 0 or sh < 0:
        raise ValueError(f"{fn}: {name} must have contiguous rows and no negative stride (strides {t.stride()})")
    if H == 1:                               # the stride of an extent of one is free: one that fits
        sh = D
    return t.data_ptr(), st if T != 1 else H * sh, sh


def _block_call(fn, y, gate, x, xo, z, dxo, dz, dy, dgate, dx, post_weight, pre_weight, dpost_weight, dpre_weight,
                post_norm, pre_norm, activation, scale, eps, dropout, rng, cu_seqlens, dev_status, workspace, stream):
    if _F32 is None:
        _load_torch()
    f32, i32, i64 = _F32, _I32, _I64
    sy = tuple(y.shape)
    T, H, D = sy if len(sy) == 3 else (sy[0], 1, sy[1])
    dt, dev = y.dtype, y.get_device()
    if post_norm not in NORMS or pre_norm not in NORMS or activation not in GATE_ACTIVATIONS:
        raise ValueError(f"{fn}: post_norm {post_norm!r}, pre_norm {pre_norm!r} or activation {activation!r} is not one of "
                         f"{tuple(NORMS)}, {tuple(GATE_ACTIVATIONS)}")
    flow = x if x is not None else xo if xo is not None else dxo            # its type is the residual stream's
    st = dt if flow is None else flow.dtype
    if st is not dt and st is not f32:
        raise ValueError(f"{fn}: x, xo and their gradients have dtype {st}, expected {dt} or {f32}")
    n = 0 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    code = _code_of(fn, "y", dt)
    no = _NO_ROWS
    packed = _BLOCK_PACK.pack(
        *_rows3(fn, "y", y, sy, dt, dev), *(no if gate is None else _rows3(fn, "gate", gate, sy, dt, dev)),
        *(no if x is None else _rows3(fn, "x", x, sy, st, dev)), *(no if xo is None else _rows3(fn, "xo", xo, sy, st, dev)),
        *(no if z is None else _rows3(fn, "z", z, sy, dt, dev)), *(no if dxo is None else _rows3(fn, "dxo", dxo, sy, st, dev)),
        *(no if dz is None else _rows3(fn, "dz", dz, sy, dt, dev)), *(no if dy is None else _rows3(fn, "dy", dy, sy, dt, dev)),
        *(no if dgate is None else _rows3(fn, "dgate", dgate, sy, dt, dev)), *(no if dx is None else _rows3(fn, "dx", dx, sy, st, dev)),
        0 if post_weight is None else _flat(fn, "post_weight", post_weight, (D,), dt, dev),
        0 if pre_weight is None else _flat(fn, "pre_weight", pre_weight, (D,), dt, dev),
        0 if dpost_weight is None else _flat(fn, "dpost_weight", dpost_weight, (D,), f32, dev),
        0 if dpre_weight is None else _flat(fn, "dpre_weight", dpre_weight, (D,), f32, dev),
        0 if rng is None else _flat(fn, "rng", rng, (2,), i64, dev),
        0 if cu_seqlens is None else _flat(fn, "cu_seqlens", cu_seqlens, (n + 1,), i32, dev),
        0 if dev_status is None else _flat(fn, "dev_status", dev_status, (1,), i32, dev),
        *_scratch(fn, workspace, dev), T, n, H, D, scale, eps, dropout, NORMS[post_norm], NORMS[pre_norm],
        GATE_ACTIVATIONS[activation], code, GCL_F32 if st is f32 else code)
    _packed_call(fn, packed, stream, dev)


def block_norm_fwd(y, xo, x=None, z=None, gate=None, post_weight=None, pre_weight=None, post_norm="rms", pre_norm="rms",
                   activation=None, scale=1.0, eps=1e-6, dropout=0.0, rng=None, cu_seqlens=None, dev_status=None, stream=None):
    """What lies between two blocks, in one pass (include/gcl.h, block_norm): xo = x + scale drop(act(gate) norm(y) w_post)
    and z = norm(xo) w_pre, for rows [T, H, D] or [T, D] with any token and head strides.  Every part but y may be left out
    (None), xo where z is given.  x and xo have y's dtype or fp32."""
    _block_call("block_norm_fwd", y, gate, x, xo, z, None, None, None, None, None, post_weight, pre_weight, None, None,
                post_norm, pre_norm, activation, scale, eps, dropout, rng, cu_seqlens, dev_status, None, stream)


def block_norm_bwd_workspace_bytes(y) -> int:
    """Workspace of block_norm_bwd with weight gradients."""
    if y.get_device() >= 0:
        _on_device("block_norm_bwd_workspace_bytes", y.get_device())
    T, H, D = y.shape if y.dim() == 3 else (y.shape[0], 1, y.shape[1])
    a = BlockArgs(t_max=T, H=H, D=D, dtype=_dtype_of(y))
    return int(lib().gcl_block_norm_bwd_workspace_bytes(ctypes.byref(a)))


def block_norm_bwd(y, dxo, dy, x=None, dx=None, dz=None, gate=None, dgate=None, post_weight=None, pre_weight=None,
                   dpost_weight=None, dpre_weight=None, post_norm="rms", pre_norm="rms", activation=None, scale=1.0, eps=1e-6,
                   dropout=0.0, rng=None, cu_seqlens=None, dev_status=None, workspace=None, stream=None):
    """The backward of block_norm_fwd: dy, dgate, dx and the weights' gradients fp32 [D] from dxo and dz (one of them may
    be None) and the forward's inputs; dropout's mask is formed again from rng."""
    if (gate is None) != (dgate is None):
        raise ValueError("block_norm_bwd: gate and dgate come together")
    _block_call("block_norm_bwd", y, gate, x, None, None, dxo, dz, dy, dgate, dx, post_weight, pre_weight, dpost_weight,
                dpre_weight, post_norm, pre_norm, activation, scale, eps, dropout, rng, cu_seqlens, dev_status, workspace, stream)
