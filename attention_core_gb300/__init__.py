"""GB300 (sm_103a) attention core under selective activation recomputation.

Thin Python binding of the C ABI in ``include/attn_core.h``: the functions
below marshal torch tensors into device pointers and the current CUDA stream
and call the library; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if ``libattn_core.so`` is missing or
cannot be loaded, the first call raises.

The attention core (QK^T, softmax, softmax dropout, attention over V) is the
part of a transformer layer that selective activation recomputation drops
after the forward pass and recomputes in the backward pass ("Reducing
Activation Recomputation in Large Transformer Models", Key takeaways, fourth
bullet).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

__all__ = [
    "AttnCoreError", "Params", "load_library", "attn_core_fwd", "attn_core_bwd_recompute",
    "attn_core_bwd_workspace_bytes", "attn_core_stored_bytes", "attn_core_strerror",
    "attn_core_bwd_recompute_noalloc",
    "fwd", "bwd_recompute", "stored_bytes", "OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED",
    "ERR_MISALIGNED", "ERR_WORKSPACE_TOO_SMALL", "ERR_CUDA", "ERR_DEVICE_TIMEOUT",
    "FLAG_TEST_WAIT_TIMEOUT", "FLAG_REDRAW_MASK", "SUPPORTED_HEAD_DIMS",
    "DalParams", "attn_core_dropout_add_ln_fwd", "attn_core_dropout_add_ln_bwd",
    "attn_core_dropout_add_ln_bwd_workspace_bytes", "dropout_add_ln_fwd", "dropout_add_ln_bwd",
    "attn_core_gelu_fwd", "attn_core_gelu_bwd", "gelu_fwd", "gelu_bwd",
    "attn_core_fwd_varlen", "attn_core_bwd_varlen", "attn_core_bwd_varlen_workspace_bytes",
    "fwd_varlen", "bwd_varlen",
    "ERR_DEVICE_TABLE", "RopeTable", "rope_table", "attn_core_rope_fwd", "attn_core_rope_bwd", "rope_fwd",
    "rope_bwd", "PAGE_SIZES", "PagedBatch", "attn_core_paged_append", "attn_core_paged_fwd",
    "attn_core_paged_workspace_bytes", "paged_append", "paged_fwd", "attn_core_page_copy", "page_copy",
    "attn_core_paged_prefix_fwd", "attn_core_paged_prefix_workspace_bytes", "paged_prefix_fwd",
    "attn_core_paged_weights", "attn_core_paged_weights_workspace_bytes", "paged_weights",
    "attn_core_paged_evict", "attn_core_paged_evict_workspace_bytes", "paged_evict",
]

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_MISALIGNED = 3
ERR_WORKSPACE_TOO_SMALL = 4
ERR_CUDA = 5
ERR_DEVICE_TIMEOUT = 6
ERR_DEVICE_TABLE = 7
FLAG_REDRAW_MASK = 0x1
FLAG_TEST_WAIT_TIMEOUT = 0x100
SUPPORTED_HEAD_DIMS = (64, 96, 128, 160)
PAGE_SIZES = (16, 32, 64, 128, 256)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libattn_core.so")


class AttnCoreError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {attn_core_strerror(code)} (code {code})")


class _CParams(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("s", ctypes.c_int32), ("d", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("p_drop", ctypes.c_float), ("scale", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("dev_status", ctypes.c_void_p), ("flags", ctypes.c_int32),
                ("wait_timeout_ms", ctypes.c_uint32), ("timing_events", ctypes.c_void_p),
                ("s_kv", ctypes.c_int32)]


class _CVarlenParams(ctypes.Structure):
    _fields_ = [("base", _CParams), ("n_seq", ctypes.c_int32),
                ("cu_seqlens_q", ctypes.POINTER(ctypes.c_int32)),
                ("cu_seqlens_k", ctypes.POINTER(ctypes.c_int32)),
                ("cu_seqlens_q_dev", ctypes.c_void_p), ("cu_seqlens_k_dev", ctypes.c_void_p)]


class _CDalParams(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int32), ("hidden", ctypes.c_int32), ("p_drop", ctypes.c_float),
                ("eps", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("dev_status", ctypes.c_void_p), ("wait_timeout_ms", ctypes.c_uint32)]


class _CBytes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("layer_none", "layer_selective", "layer_full", "core_scores_avoided",
                 "core_kept", "core_recompute_state")]


class _CRopeConfig(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("d", "rot_dim", "interleaved", "scaling")] +
                [(n, ctypes.c_double) for n in ("base", "factor", "original_len", "low_freq", "high_freq",
                                                "beta_fast", "beta_slow", "mscale")])


class RopeTable(ctypes.Structure):
    """Mirror of ``attn_core_rope_table``: made by :func:`rope_table`, kept by
    the caller and passed to every rotation."""
    _fields_ = [("d", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("mscale", ctypes.c_float), ("turns", ctypes.c_uint64 * 128)]


class _CRopeParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("b", "s", "h_q", "h_kv")] +
                [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "yq_stride", "yk_stride")] +
                [("pos0", ctypes.c_int32), ("positions", ctypes.c_void_p)])


class _CPagedParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_seq", "n_tokens", "h_q", "h_kv", "d", "page_size", "n_pages",
                                               "max_pages", "causal")] +
                [("scale", ctypes.c_float)] +
                [(n, ctypes.c_void_p) for n in ("cu_seqlens_q", "kv_lens", "page_table", "dev_status")] +
                [("flags", ctypes.c_int32), ("wait_timeout_ms", ctypes.c_uint32)])


@dataclass
class Params:
    """Mirror of ``attn_core_params`` (see include/attn_core.h)."""
    b: int
    h_q: int
    h_kv: int
    s: int
    d: int
    causal: bool = True
    p_drop: float = 0.0
    scale: float = 0.0
    seed: int = 0
    offset: int = 0
    dev_status: int = 0          # device address of an int32, or 0
    flags: int = 0
    wait_timeout_ms: int = 0
    timing_events: int = 0       # address of a void*[2 * n_kernels] array, or 0
    s_kv: int = 0                # keys per KV head; 0 means s

    @property
    def keys(self) -> int:
        return self.s_kv or self.s

    def to_c(self) -> _CParams:
        return _CParams(self.b, self.h_q, self.h_kv, self.s, self.d, int(self.causal),
                        float(self.p_drop), float(self.scale), int(self.seed) & (2**64 - 1),
                        int(self.offset) & (2**64 - 1), self.dev_status or None, int(self.flags),
                        int(self.wait_timeout_ms), self.timing_events or None, int(self.s_kv))


@dataclass
class DalParams:
    """Mirror of ``attn_core_dal_params`` (dropout + residual add + layer norm)."""
    n_rows: int
    hidden: int
    p_drop: float = 0.0
    eps: float = 1e-5
    seed: int = 0
    offset: int = 0
    dev_status: int = 0          # device address of an int32, or 0
    wait_timeout_ms: int = 0

    def to_c(self) -> _CDalParams:
        return _CDalParams(int(self.n_rows), int(self.hidden), float(self.p_drop), float(self.eps),
                           int(self.seed) & (2**64 - 1), int(self.offset) & (2**64 - 1),
                           self.dev_status or None, int(self.wait_timeout_ms))


_lib = None
# The short calls' entry points once more, with plain addresses and integers for
# arguments: converting structures costs a few microseconds of the host's time.
_FAST: dict = {}


def load_library(path: str = LIB_PATH):
    """Load libattn_core.so (raises if it is absent: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"attention-core library not built ({path} missing); run "
            "`python -m attention_core_gb300.build` or __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp = ctypes.c_void_p
    P = ctypes.POINTER(_CParams)
    lib.attn_core_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp]
    lib.attn_core_fwd.restype = ctypes.c_int
    lib.attn_core_bwd_workspace_bytes.argtypes = [P]
    lib.attn_core_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_core_bwd_recompute.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.attn_core_bwd_recompute.restype = ctypes.c_int
    lib.attn_core_bwd_recompute_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.attn_core_bwd_recompute_noalloc.restype = ctypes.c_int
    lib.attn_core_stored_bytes.argtypes = [P, ctypes.POINTER(_CBytes)]
    lib.attn_core_stored_bytes.restype = ctypes.c_int
    lib.attn_core_strerror.argtypes = [ctypes.c_int]
    lib.attn_core_strerror.restype = ctypes.c_char_p
    DP = ctypes.POINTER(_CDalParams)
    lib.attn_core_dropout_add_ln_fwd.argtypes = [DP, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.attn_core_dropout_add_ln_fwd.restype = ctypes.c_int
    lib.attn_core_dropout_add_ln_bwd_workspace_bytes.argtypes = [DP]
    lib.attn_core_dropout_add_ln_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_core_dropout_add_ln_bwd.argtypes = [DP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                 ctypes.c_size_t, vp]
    lib.attn_core_dropout_add_ln_bwd.restype = ctypes.c_int
    VP = ctypes.POINTER(_CVarlenParams)
    lib.attn_core_fwd_varlen.argtypes = [VP, vp, vp, vp, vp, vp, vp]
    lib.attn_core_fwd_varlen.restype = ctypes.c_int
    lib.attn_core_bwd_varlen_workspace_bytes.argtypes = [VP]
    lib.attn_core_bwd_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_core_bwd_varlen.argtypes = [VP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.attn_core_bwd_varlen.restype = ctypes.c_int
    lib.attn_core_gelu_fwd.argtypes = [ctypes.c_int64, vp, vp, vp]
    lib.attn_core_gelu_fwd.restype = ctypes.c_int
    lib.attn_core_gelu_bwd.argtypes = [ctypes.c_int64, vp, vp, vp, vp]
    lib.attn_core_gelu_bwd.restype = ctypes.c_int
    RT, RP = ctypes.POINTER(RopeTable), ctypes.POINTER(_CRopeParams)
    lib.attn_core_rope_init.argtypes = [ctypes.POINTER(_CRopeConfig), RT]
    lib.attn_core_rope_init.restype = ctypes.c_int
    for f in (lib.attn_core_rope_fwd, lib.attn_core_rope_bwd):
        f.argtypes = [RP, RT, vp, vp, vp, vp, vp]
        f.restype = ctypes.c_int
    PP = ctypes.POINTER(_CPagedParams)
    lib.attn_core_paged_append.argtypes = [PP, RT, vp, vp, vp, ctypes.POINTER(ctypes.c_int64), vp, vp, vp, vp]
    lib.attn_core_paged_append.restype = ctypes.c_int
    lib.attn_core_paged_workspace_bytes.argtypes = [PP]
    lib.attn_core_paged_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_core_paged_fwd.argtypes = [PP, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.attn_core_paged_fwd.restype = ctypes.c_int
    lib.attn_core_paged_prefix_workspace_bytes.argtypes = [PP, ctypes.c_int32]
    lib.attn_core_paged_prefix_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_core_paged_prefix_fwd.argtypes = [PP, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.attn_core_paged_prefix_fwd.restype = ctypes.c_int
    lib.attn_core_paged_weights_workspace_bytes.argtypes = [PP]
    lib.attn_core_paged_weights_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_core_paged_weights.argtypes = [PP, vp, vp, vp, ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp]
    lib.attn_core_paged_weights.restype = ctypes.c_int
    lib.attn_core_paged_evict_workspace_bytes.argtypes = [PP]
    lib.attn_core_paged_evict_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_core_paged_evict.argtypes = [PP, vp, ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp,
                                          ctypes.c_size_t, vp]
    lib.attn_core_paged_evict.restype = ctypes.c_int
    lib.attn_core_page_copy.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp,
                                        ctypes.c_int64, vp]
    lib.attn_core_page_copy.restype = ctypes.c_int
    i64 = ctypes.c_int64
    for name, argtypes in (("attn_core_rope_fwd", [vp] * 7), ("attn_core_rope_bwd", [vp] * 7),
                           ("attn_core_paged_append", [vp] * 10),
                           ("attn_core_paged_fwd", [vp] * 7 + [ctypes.c_size_t, vp]),
                           ("attn_core_paged_prefix_fwd",
                            [vp, ctypes.c_int32] + [vp] * 8 + [ctypes.c_size_t, vp]),
                           ("attn_core_paged_weights",
                            [vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp]),
                           ("attn_core_paged_evict",
                            [vp, vp, ctypes.c_int32, ctypes.c_int32] + [vp] * 7 + [ctypes.c_size_t, vp]),
                           ("attn_core_page_copy", [vp, i64, i64, i64, i64, vp, i64, vp])):
        f = lib[name]
        f.argtypes, f.restype = argtypes, ctypes.c_int
        _FAST[name] = f
    _lib = lib
    return lib


# ------------------------------------------------------------ raw C ABI ---
# Same names and arguments as the C functions; pointers are plain integers.

def attn_core_strerror(code: int) -> str:
    return load_library().attn_core_strerror(int(code)).decode()


def attn_core_fwd(p: Params, q: int, k: int, v: int, o: int, lse: int, stream: int) -> int:
    cp = p.to_c()
    return load_library().attn_core_fwd(ctypes.byref(cp), q, k, v, o, lse, stream or None)


def attn_core_bwd_workspace_bytes(p: Params) -> int:
    cp = p.to_c()
    return int(load_library().attn_core_bwd_workspace_bytes(ctypes.byref(cp)))


def attn_core_bwd_recompute(p: Params, q: int, k: int, v: int, o: int, lse: int, dout: int,
                            dq: int, dk: int, dv: int, workspace: int, workspace_bytes: int,
                            stream: int) -> int:
    cp = p.to_c()
    return load_library().attn_core_bwd_recompute(ctypes.byref(cp), q, k, v, o, lse, dout, dq, dk,
                                                  dv, workspace, workspace_bytes, stream or None)


def attn_core_bwd_recompute_noalloc(p: Params, q: int, k: int, v: int, o: int, lse: int, dout: int,
                                    dq: int, dk: int, dv: int, stream: int) -> int:
    """Backward for callers that cannot allocate device memory: no workspace
    argument; the library's own fixed scratch array is used (see the header
    for its size limit and for why calls that overlap on the GPU race)."""
    cp = p.to_c()
    return load_library().attn_core_bwd_recompute_noalloc(ctypes.byref(cp), q, k, v, o, lse, dout, dq,
                                                          dk, dv, stream or None)


def attn_core_stored_bytes(p: Params) -> tuple[int, dict]:
    cp = p.to_c()
    out = _CBytes()
    rc = load_library().attn_core_stored_bytes(ctypes.byref(cp), ctypes.byref(out))
    return rc, {n: int(getattr(out, n)) for n, _ in _CBytes._fields_}


def attn_core_dropout_add_ln_fwd(p: DalParams, x: int, residual: int, gamma: int, beta: int, z: int,
                                 y: int, mean: int, rstd: int, stream: int) -> int:
    cp = p.to_c()
    return load_library().attn_core_dropout_add_ln_fwd(ctypes.byref(cp), x, residual, gamma, beta, z, y,
                                                       mean, rstd, stream or None)


def attn_core_dropout_add_ln_bwd_workspace_bytes(p: DalParams) -> int:
    cp = p.to_c()
    return int(load_library().attn_core_dropout_add_ln_bwd_workspace_bytes(ctypes.byref(cp)))


def attn_core_dropout_add_ln_bwd(p: DalParams, dy: int, dz_next: int, z: int, mean: int, rstd: int,
                                 gamma: int, dx: int, d_residual: int, dgamma: int, dbeta: int,
                                 workspace: int, workspace_bytes: int, stream: int) -> int:
    cp = p.to_c()
    return load_library().attn_core_dropout_add_ln_bwd(ctypes.byref(cp), dy, dz_next or None, z, mean,
                                                       rstd, gamma, dx, d_residual, dgamma, dbeta,
                                                       workspace, workspace_bytes, stream or None)


def _varlen_c(p: Params, cu_q, cu_k, cu_q_dev: int = 0, cu_k_dev: int = 0):
    """(_CVarlenParams, keep-alive arrays) for host sequence tables and the
    device addresses of their copies."""
    aq = (ctypes.c_int32 * len(cu_q))(*[int(x) for x in cu_q])
    ak = (ctypes.c_int32 * len(cu_k))(*[int(x) for x in cu_k]) if cu_k is not None else None
    vp = _CVarlenParams(p.to_c(), len(cu_q) - 1, ctypes.cast(aq, ctypes.POINTER(ctypes.c_int32)),
                        ctypes.cast(ak, ctypes.POINTER(ctypes.c_int32)) if ak is not None else None,
                        cu_q_dev or None, cu_k_dev or None)
    return vp, (aq, ak)


def attn_core_fwd_varlen(p: Params, cu_q, cu_k, q: int, k: int, v: int, o: int, lse: int, stream: int, *,
                         cu_q_dev: int = 0, cu_k_dev: int = 0) -> int:
    """p supplies h_q, h_kv, d, causal, p_drop, scale, seed, offset, dev_status,
    flags and wait_timeout_ms; cu_q / cu_k are host sequence tables and
    cu_q_dev / cu_k_dev the device addresses of their copies."""
    vp, keep = _varlen_c(p, cu_q, cu_k, cu_q_dev, cu_k_dev)
    return load_library().attn_core_fwd_varlen(ctypes.byref(vp), q, k, v, o, lse, stream or None)


def attn_core_bwd_varlen_workspace_bytes(p: Params, cu_q, cu_k, *, cu_q_dev: int = 0, cu_k_dev: int = 0) -> int:
    vp, keep = _varlen_c(p, cu_q, cu_k, cu_q_dev, cu_k_dev)
    return int(load_library().attn_core_bwd_varlen_workspace_bytes(ctypes.byref(vp)))


def attn_core_bwd_varlen(p: Params, cu_q, cu_k, q: int, k: int, v: int, o: int, lse: int, dout: int, dq: int,
                         dk: int, dv: int, workspace: int, workspace_bytes: int, stream: int, *,
                         cu_q_dev: int = 0, cu_k_dev: int = 0) -> int:
    vp, keep = _varlen_c(p, cu_q, cu_k, cu_q_dev, cu_k_dev)
    return load_library().attn_core_bwd_varlen(ctypes.byref(vp), q, k, v, o, lse, dout, dq, dk, dv, workspace,
                                               workspace_bytes, stream or None)


def _device_tables(cq, ck, device):
    """Device copies of the host sequence tables (kept alive by the caller until
    the kernels that read them are queued: the caching allocator reuses the
    memory only in stream order)."""
    import torch
    tq = torch.tensor(cq, dtype=torch.int32, device=device)
    tk = torch.tensor(ck, dtype=torch.int32, device=device) if ck is not None else None
    return tq, tk, tq.data_ptr(), (tk.data_ptr() if tk is not None else 0)


def attn_core_gelu_fwd(n: int, x: int, y: int, stream: int) -> int:
    return load_library().attn_core_gelu_fwd(int(n), x, y, stream or None)


def attn_core_gelu_bwd(n: int, x: int, dy: int, dx: int, stream: int) -> int:
    return load_library().attn_core_gelu_bwd(int(n), x, dy, dx, stream or None)


# --------------------------------------------------- torch conveniences ---

def _check(t, name, dtype, shape):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream() -> int:
    import torch
    return torch.cuda.current_stream().cuda_stream


class _Host:
    """What a short call asks of torch, looked up once: on a Grace host the public
    ways cost several microseconds of a call's ten.

    device()  the current device
    stream(d) the current stream's handle, without the Stream object around it
    empty(size, strides, dtype)  an output on the current device: torch's compiled
              code allocates through an entry of its own that skips the dispatcher
              (two outputs and a launch cost 6.4 us with it, 10.6 with torch.empty)
    """

    def __init__(self):
        import torch
        c = torch._C
        self.bf16, self.f32, self.i32 = torch.bfloat16, torch.float32, torch.int32
        self.device = getattr(c, "_cuda_getDevice", None) or torch.cuda.current_device
        self.stream = getattr(c, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
        self.empty = getattr(getattr(getattr(c, "_dynamo", None), "guards", None), "_empty_strided_cuda", None) or (
            lambda size, strides, dtype: torch.empty_strided(size, strides, dtype=dtype, device="cuda"))


_HOST: list = []


def _host() -> _Host:
    if not _HOST:
        _HOST.append(_Host())
    return _HOST[0]


def _params_from(q, k, causal, p_drop, seed, offset, scale, **kw) -> Params:
    b, h_q, s, d = q.shape
    return Params(b=b, h_q=h_q, h_kv=k.shape[1], s=s, d=d, causal=causal, p_drop=p_drop,
                  scale=scale, seed=seed, offset=offset, s_kv=k.shape[2], **kw)


def fwd(q, k, v, *, causal: bool = True, p_drop: float = 0.0, seed: int = 0, offset: int = 0,
        scale: float = 0.0, out=None, lse=None, **kw):
    """Forward of the attention core.  Returns (O bf16 [b,h_q,s,d], LSE fp32 [b,h_q,s]).

    K and V may have a different sequence length from Q (s_kv keys,
    cross-attention) when ``causal`` is False."""
    import torch
    p = _params_from(q, k, causal, p_drop, seed, offset, scale, **kw)
    _check(q, "q", torch.bfloat16, (p.b, p.h_q, p.s, p.d))
    _check(k, "k", torch.bfloat16, (p.b, p.h_kv, p.keys, p.d))
    _check(v, "v", torch.bfloat16, (p.b, p.h_kv, p.keys, p.d))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((p.b, p.h_q, p.s), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, (p.b, p.h_q, p.s, p.d))
    _check(lse, "lse", torch.float32, (p.b, p.h_q, p.s))
    rc = attn_core_fwd(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                       _stream())
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_fwd")
    return out, lse


def bwd_recompute(q, k, v, o, lse, dout, *, causal: bool = True, p_drop: float = 0.0, seed: int = 0,
                  offset: int = 0, scale: float = 0.0, dq=None, dk=None, dv=None, workspace=None,
                  **kw):
    """Recompute-backward.  Returns (dQ, dK, dV), bf16, shaped like Q, K, V."""
    import torch
    p = _params_from(q, k, causal, p_drop, seed, offset, scale, **kw)
    _check(q, "q", torch.bfloat16, (p.b, p.h_q, p.s, p.d))
    _check(k, "k", torch.bfloat16, (p.b, p.h_kv, p.keys, p.d))
    _check(v, "v", torch.bfloat16, (p.b, p.h_kv, p.keys, p.d))
    _check(o, "o", torch.bfloat16, (p.b, p.h_q, p.s, p.d))
    _check(dout, "dout", torch.bfloat16, (p.b, p.h_q, p.s, p.d))
    _check(lse, "lse", torch.float32, (p.b, p.h_q, p.s))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(dq, "dq", torch.bfloat16, (p.b, p.h_q, p.s, p.d))
    _check(dk, "dk", torch.bfloat16, (p.b, p.h_kv, p.keys, p.d))
    _check(dv, "dv", torch.bfloat16, (p.b, p.h_kv, p.keys, p.d))
    ws_bytes = attn_core_bwd_workspace_bytes(p)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    rc = attn_core_bwd_recompute(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                 lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                 dv.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream())
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_bwd_recompute")
    return dq, dk, dv


def stored_bytes(b: int, h_q: int, h_kv: int, s: int, d: int, s_kv: int = 0) -> dict:
    """Activation-byte accounting of one layer shard (see attn_core_bytes)."""
    rc, out = attn_core_stored_bytes(Params(b=b, h_q=h_q, h_kv=h_kv, s=s, d=d, s_kv=s_kv,
                                            causal=not s_kv or s_kv == s))
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_stored_bytes")
    return out


def dropout_add_ln_fwd(x, residual, gamma, beta, *, p_drop: float = 0.0, seed: int = 0, offset: int = 0,
                       eps: float = 1e-5, **kw):
    """z = residual + dropout(x), y = LayerNorm(z).  Returns (z, y, mean, rstd)."""
    import torch
    n, h = x.shape
    p = DalParams(n_rows=n, hidden=h, p_drop=p_drop, eps=eps, seed=seed, offset=offset, **kw)
    _check(x, "x", torch.bfloat16, (n, h))
    _check(residual, "residual", torch.bfloat16, (n, h))
    _check(gamma, "gamma", torch.float32, (h,))
    _check(beta, "beta", torch.float32, (h,))
    z, y = torch.empty_like(x), torch.empty_like(x)
    mean = torch.empty(n, dtype=torch.float32, device=x.device)
    rstd = torch.empty(n, dtype=torch.float32, device=x.device)
    rc = attn_core_dropout_add_ln_fwd(p, x.data_ptr(), residual.data_ptr(), gamma.data_ptr(),
                                      beta.data_ptr(), z.data_ptr(), y.data_ptr(), mean.data_ptr(),
                                      rstd.data_ptr(), _stream())
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_dropout_add_ln_fwd")
    return z, y, mean, rstd


def dropout_add_ln_bwd(dy, z, mean, rstd, gamma, *, dz_next=None, p_drop: float = 0.0, seed: int = 0,
                       offset: int = 0, eps: float = 1e-5, workspace=None, **kw):
    """Gradients of dropout_add_ln_fwd.  Returns (dx, d_residual, dgamma, dbeta)."""
    import torch
    n, h = dy.shape
    p = DalParams(n_rows=n, hidden=h, p_drop=p_drop, eps=eps, seed=seed, offset=offset, **kw)
    _check(dy, "dy", torch.bfloat16, (n, h))
    _check(z, "z", torch.bfloat16, (n, h))
    _check(mean, "mean", torch.float32, (n,))
    _check(rstd, "rstd", torch.float32, (n,))
    _check(gamma, "gamma", torch.float32, (h,))
    if dz_next is not None:
        _check(dz_next, "dz_next", torch.bfloat16, (n, h))
    dx, dres = torch.empty_like(dy), torch.empty_like(dy)
    dgamma = torch.empty(h, dtype=torch.float32, device=dy.device)
    dbeta = torch.empty(h, dtype=torch.float32, device=dy.device)
    ws_bytes = attn_core_dropout_add_ln_bwd_workspace_bytes(p)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dy.device)
    rc = attn_core_dropout_add_ln_bwd(p, dy.data_ptr(), dz_next.data_ptr() if dz_next is not None else 0,
                                      z.data_ptr(), mean.data_ptr(), rstd.data_ptr(), gamma.data_ptr(),
                                      dx.data_ptr(), dres.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(),
                                      workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                      _stream())
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_dropout_add_ln_bwd")
    return dx, dres, dgamma, dbeta


def gelu_fwd(x, out=None):
    """GeLU (tanh form) of a contiguous bf16 CUDA tensor (numel a multiple of 8)."""
    import torch
    _check(x, "x", torch.bfloat16, tuple(x.shape))
    out = torch.empty_like(x) if out is None else out
    rc = attn_core_gelu_fwd(x.numel(), x.data_ptr(), out.data_ptr(), _stream())
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_gelu_fwd")
    return out


def gelu_bwd(x, dy, out=None):
    """dy * GeLU'(x) for contiguous bf16 CUDA tensors of one shape."""
    import torch
    _check(x, "x", torch.bfloat16, tuple(x.shape))
    _check(dy, "dy", torch.bfloat16, tuple(x.shape))
    out = torch.empty_like(x) if out is None else out
    rc = attn_core_gelu_bwd(x.numel(), x.data_ptr(), dy.data_ptr(), out.data_ptr(), _stream())
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_gelu_bwd")
    return out


def _varlen_params(q, k, causal, p_drop, seed, offset, scale, **kw) -> Params:
    _, h_q, d = q.shape
    return Params(b=1, h_q=h_q, h_kv=k.shape[1], s=1, d=d, causal=causal, p_drop=p_drop, scale=scale,
                  seed=seed, offset=offset, **kw)


def fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k=None, *, causal: bool = True, p_drop: float = 0.0,
               seed: int = 0, offset: int = 0, scale: float = 0.0, **kw):
    """Forward over a packed batch: q [total_q, h_q, d], k/v [total_k, h_kv, d];
    cu_seqlens_* host sequence tables (lists or CPU tensors; their device
    copies are made here).  The batch is one launch per kernel.  Returns (O,
    LSE [h_q, total_q])."""
    import torch
    p = _varlen_params(q, k, causal, p_drop, seed, offset, scale, **kw)
    cq = [int(x) for x in cu_seqlens_q]
    ck = [int(x) for x in cu_seqlens_k] if cu_seqlens_k is not None else None
    _check(q, "q", torch.bfloat16, (cq[-1], p.h_q, p.d))
    _check(k, "k", torch.bfloat16, ((ck or cq)[-1], p.h_kv, p.d))
    _check(v, "v", torch.bfloat16, ((ck or cq)[-1], p.h_kv, p.d))
    o = torch.empty_like(q)
    lse = torch.empty((p.h_q, cq[-1]), dtype=torch.float32, device=q.device)
    tq, tk, dq_ptr, dk_ptr = _device_tables(cq, ck, q.device)
    rc = attn_core_fwd_varlen(p, cq, ck, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              lse.data_ptr(), _stream(), cu_q_dev=dq_ptr, cu_k_dev=dk_ptr)
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_fwd_varlen")
    return o, lse


def bwd_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k=None, *, causal: bool = True,
               p_drop: float = 0.0, seed: int = 0, offset: int = 0, scale: float = 0.0, **kw):
    """Recompute-backward over a packed batch.  Returns (dQ, dK, dV)."""
    import torch
    p = _varlen_params(q, k, causal, p_drop, seed, offset, scale, **kw)
    cq = [int(x) for x in cu_seqlens_q]
    ck = [int(x) for x in cu_seqlens_k] if cu_seqlens_k is not None else None
    _check(o, "o", torch.bfloat16, tuple(q.shape))
    _check(dout, "dout", torch.bfloat16, tuple(q.shape))
    _check(lse, "lse", torch.float32, (p.h_q, cq[-1]))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    tq, tk, dq_ptr, dk_ptr = _device_tables(cq, ck, q.device)
    ws_bytes = attn_core_bwd_varlen_workspace_bytes(p, cq, ck, cu_q_dev=dq_ptr, cu_k_dev=dk_ptr)
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
    rc = attn_core_bwd_varlen(p, cq, ck, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                              ws.data_ptr(), ws.numel(), _stream(), cu_q_dev=dq_ptr, cu_k_dev=dk_ptr)
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_bwd_varlen")
    return dq, dk, dv


# ------------------------------------- rotary positions, the paged cache ---

ROPE_SCALINGS = {"none": 0, "linear": 1, "bands": 2, "yarn": 3}


def rope_table(d: int, *, rot_dim: int = 0, base: float = 10000.0, interleaved: bool = False,
               scaling: str = "none", factor: float = 1.0, original_len: float = 0.0, low_freq: float = 0.0,
               high_freq: float = 0.0, beta_fast: float = 0.0, beta_slow: float = 0.0,
               mscale: float = 0.0) -> RopeTable:
    """The frequencies of rotary positions over the first ``rot_dim`` values of
    each head (all, up to 256, by default); ``scaling`` is "none", "linear",
    "bands" or "yarn" (formulas: include/attn_core.h)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {tuple(ROPE_SCALINGS)}, got {scaling!r}")
    c = _CRopeConfig(_bits32("d", d), _bits32("rot_dim", rot_dim), int(bool(interleaved)), ROPE_SCALINGS[scaling], float(base), float(factor),
                     float(original_len), float(low_freq), float(high_freq), float(beta_fast), float(beta_slow),
                     float(mscale))
    t = RopeTable()
    rc = load_library().attn_core_rope_init(ctypes.byref(c), ctypes.byref(t))
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_rope_init")
    return t


def attn_core_rope_fwd(p: _CRopeParams, t: RopeTable, q: int, k: int, yq: int, yk: int, stream: int) -> int:
    return load_library().attn_core_rope_fwd(p, t, q or None, k or None, yq or None, yk or None, stream or None)


def attn_core_rope_bwd(p: _CRopeParams, t: RopeTable, dyq: int, dyk: int, dq: int, dk: int, stream: int) -> int:
    return load_library().attn_core_rope_bwd(p, t, dyq or None, dyk or None, dq or None, dk or None, stream or None)


def attn_core_paged_append(p: _CPagedParams, t, q: int, k: int, v: int, strides, q_out: int, k_pages: int,
                           v_pages: int, stream: int) -> int:
    """strides: three host integers (q, k, v), or None for packed tensors."""
    st = (ctypes.c_int64 * 3)(*strides) if strides is not None else None
    return load_library().attn_core_paged_append(p, t, q or None, k, v, st, q_out or None, k_pages, v_pages,
                                                 stream or None)


def attn_core_paged_workspace_bytes(p: _CPagedParams) -> int:
    return int(load_library().attn_core_paged_workspace_bytes(p))


def attn_core_paged_fwd(p: _CPagedParams, q: int, k_pages: int, v_pages: int, o: int, lse: int, workspace: int,
                        workspace_bytes: int, stream: int) -> int:
    return load_library().attn_core_paged_fwd(p, q, k_pages, v_pages, o, lse, workspace, workspace_bytes,
                                              stream or None)


def attn_core_paged_prefix_workspace_bytes(p: _CPagedParams, n_groups: int) -> int:
    return int(load_library().attn_core_paged_prefix_workspace_bytes(p, n_groups))


def attn_core_paged_prefix_fwd(p: _CPagedParams, n_groups: int, group_starts: int, prefix_pages: int, q: int,
                               k_pages: int, v_pages: int, o: int, lse: int, workspace: int, workspace_bytes: int,
                               stream: int) -> int:
    return load_library().attn_core_paged_prefix_fwd(p, n_groups, group_starts, prefix_pages, q, k_pages, v_pages, o,
                                                     lse, workspace, workspace_bytes, stream or None)


def attn_core_paged_weights_workspace_bytes(p: _CPagedParams) -> int:
    return int(load_library().attn_core_paged_weights_workspace_bytes(p))


def attn_core_paged_weights(p: _CPagedParams, q: int, k_pages: int, lse: int, decay: float, weights: int,
                            weights_out: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    return load_library().attn_core_paged_weights(p, q, k_pages, lse, decay, weights, weights_out, workspace,
                                                  workspace_bytes, stream or None)


def attn_core_paged_evict_workspace_bytes(p: _CPagedParams) -> int:
    return int(load_library().attn_core_paged_evict_workspace_bytes(p))


def attn_core_paged_evict(p: _CPagedParams, keep: int, first: int, recent: int, out_table: int, k_pages: int,
                          v_pages: int, weights: int, weights_out: int, kept: int, workspace: int,
                          workspace_bytes: int, stream: int) -> int:
    return load_library().attn_core_paged_evict(p, keep, first, recent, out_table or None, k_pages, v_pages, weights,
                                                weights_out, kept, workspace, workspace_bytes, stream or None)


def attn_core_page_copy(pages: int, n_planes: int, plane_stride: int, n_pages: int, page_bytes: int, pairs: int,
                        n_pairs: int, stream: int) -> int:
    """pairs: address of host int32 [n_pairs, 2]."""
    return load_library().attn_core_page_copy(pages, n_planes, plane_stride, n_pages, page_bytes, pairs or None,
                                              n_pairs, stream or None)


def _bits32(name: str, value, low: int = -2**31, high: int = 2**31 - 1) -> int:
    """A value for a 32-bit field, which ctypes would cut without a word."""
    value = int(value)
    if not low <= value <= high:
        raise ValueError(f"{name} does not fit 32 bits: {value}")
    return value


def _layout(shape) -> tuple:
    """(sizes, strides) of a contiguous tensor."""
    out, n = [], 1
    for d in reversed(shape):
        out.append(n)
        n *= max(int(d), 1)
    return tuple(int(d) for d in shape), tuple(reversed(out))


def _need(t, name, dtype, shape, device: int) -> None:
    """A contiguous tensor of this type and shape on the current device, where
    the library launches; _check says what else it is."""
    try:
        good = t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()
    except AttributeError:
        good = False
    if not good:
        _check(t, name, dtype, shape)
        _on_device(device, t)


def _on_device(device: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != device:      # -1 off the GPU
            raise ValueError(f"tensors must be on the current device (cuda:{device}), got {t.device}")


def _rope_view(x, name, d):
    """(b, heads, s, strides) of [b, h, s, d] or packed [tokens, h, d]; only d
    has to be contiguous.  A dimension of one element has no stride."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor")
    if x.dim() not in (3, 4) or x.shape[-1] != d:
        raise ValueError(f"{name} must be [b, h, s, {d}] or [tokens, h, {d}], got {tuple(x.shape)}")
    if x.stride(-1) != 1 and d > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if x.dim() == 4:
        (b, h, s, _), (tb, th, ts, _) = x.shape, x.stride()
    else:
        (s, h, _), (ts, th, _) = x.shape, x.stride()
        b, tb = 1, 0
    return b, h, s, (tb if b > 1 else 0, th if h > 1 else 0, ts if s > 1 else 0)


# The argument structure of a rotation follows from its tensors' shapes and
# strides alone: made once for each and copied (building it costs more than the
# launch).
_ROPE_PARAMS: dict = {}


def _rope_params(q, k, out_q, out_k, d):
    p = _CRopeParams()
    lead = None
    for x, y, name in ((q, out_q, "q"), (k, out_k, "k")):
        if x is None:
            continue
        b, h, s, st = _rope_view(x, name, d)
        if lead not in (None, (b, s, x.dim())):
            raise ValueError(f"q and k must have the same batch and tokens, got {tuple(q.shape)}, {tuple(k.shape)}")
        lead = (b, s, x.dim())
        if y is None:           # allocated like x, contiguous
            yst = (h * s * d, s * d, d) if x.dim() == 4 else (0, d, h * d)
        elif y.shape != x.shape:
            raise ValueError(f"out_{name} must have shape {tuple(x.shape)}, got {tuple(y.shape)}")
        else:
            yst = _rope_view(y, "out_" + name, d)[3]
        setattr(p, "h_" + ("q" if name == "q" else "kv"), _bits32(name + "'s heads", h))
        getattr(p, name + "_stride")[:] = st
        getattr(p, "y" + name + "_stride")[:] = yst
    if lead is None:
        raise ValueError("q or k must be given")
    p.b, p.s = _bits32("batch", lead[0]), _bits32("tokens", lead[1])
    return p


def _rope(what, q, k, table, positions, pos0, out_q, out_k):
    pos0 = _bits32("pos0", pos0) if pos0 else 0
    if (q is None and out_q is not None) or (k is None and out_k is not None):
        raise ValueError("out_q without q" if q is None and out_q is not None else "out_k without k")
    host = _host()
    dev = host.device()
    key = (table.d,
           None if q is None else (q.shape, q.stride(), q.dtype, q.get_device()),
           None if k is None else (k.shape, k.stride(), k.dtype, k.get_device()),
           None if out_q is None else (out_q.shape, out_q.stride(), out_q.dtype, out_q.get_device()),
           None if out_k is None else (out_k.shape, out_k.stride(), out_k.dtype, out_k.get_device()), dev)
    known = _ROPE_PARAMS.get(key)
    if known is None:
        _on_device(dev, q, k, out_q, out_k)
        known = (_rope_params(q, k, out_q, out_k, table.d),
                 *(None if x is None else _layout(x.shape) for x in (q, k)))
        if len(_ROPE_PARAMS) >= 256:
            _ROPE_PARAMS.clear()
        _ROPE_PARAMS[key] = known
    params, q_layout, k_layout = known
    p = _CRopeParams.from_buffer_copy(params)
    if positions is None:
        p.pos0 = pos0
    else:
        if positions.dtype != host.i32 or not positions.is_contiguous() or positions.numel() != p.b * p.s:
            raise ValueError(f"positions must be a contiguous int32 CUDA tensor of {p.b * p.s} values")
        if positions.get_device() != dev:
            _on_device(dev, positions)
        p.positions = positions.data_ptr()
    xq = xk = yq = yk = 0
    if q is not None:
        if out_q is None:
            out_q = host.empty(*q_layout, host.bf16)
        xq, yq = q.data_ptr(), out_q.data_ptr()
    if k is not None:
        if out_k is None:
            out_k = host.empty(*k_layout, host.bf16)
        xk, yk = k.data_ptr(), out_k.data_ptr()
    rc = _FAST[what](ctypes.addressof(p), ctypes.addressof(table), xq, xk, yq, yk, host.stream(dev)) if p.s else OK
    if rc != OK:
        raise AttnCoreError(rc, what)
    return out_q, out_k


def rope_fwd(q, k, table: RopeTable, *, positions=None, pos0: int = 0, out_q=None, out_k=None):
    """Rotary positions on q and k (either may be None): bf16 [b, h, s, d] or
    packed [tokens, h, d] of any strides with d contiguous.  ``positions``:
    int32, one per (batch element, token); by default pos0 + token.  ``out_q`` /
    ``out_k`` may be the inputs themselves.  Returns (q, k) rotated."""
    return _rope("attn_core_rope_fwd", q, k, table, positions, pos0, out_q, out_k)


def rope_bwd(dq, dk, table: RopeTable, *, positions=None, pos0: int = 0, out_q=None, out_k=None):
    """Gradients of rope_fwd's inputs from those of its outputs."""
    return _rope("attn_core_rope_bwd", dq, dk, table, positions, pos0, out_q, out_k)


class PagedBatch:
    """A batch of sequences whose keys and values live in pages, as
    paged_append and paged_fwd take it (layout: include/attn_core.h).

    ``cu_seqlens_q`` [n_seq + 1], ``kv_lens`` [n_seq] and ``page_table``
    [n_seq, max_pages] are int32 CUDA tensors, read by the kernels when they
    run: a step's new lengths and pages are copied into them, and a captured
    graph follows.  The batch owns the attention's workspace; calls that may
    overlap on the GPU need a batch (or a ``workspace``) each.  It may be dropped
    right after a call, on whichever stream that was made; a captured graph needs
    the batch for as long as it is replayed.

    ``group_starts`` [n_groups + 1] and ``prefix_pages`` [n_groups], two more such
    tables, make it a batch for paged_prefix_fwd: the sequences group_starts[g] ..
    group_starts[g + 1] - 1 name the same pages in their first prefix_pages[g]
    columns (PagePool.groups finds them).  A smaller count costs speed; one that
    reaches into columns that differ gives wrong results, unnoticed, so the counts
    follow the page table (a fork's copied page, PagePool.shrink), also where a
    captured graph is replayed."""

    def __init__(self, cu_seqlens_q, kv_lens, page_table, *, n_tokens: int, h_q: int, h_kv: int, d: int,
                 page_size: int, n_pages: int, causal: bool = True, scale: float = 0.0, dev_status: int = 0,
                 flags: int = 0, wait_timeout_ms: int = 0, workspace=None, group_starts=None, prefix_pages=None):
        import torch
        if page_table.dim() != 2:
            raise ValueError(f"page_table must be [n_seq, max_pages], got {tuple(page_table.shape)}")
        n_seq, max_pages = page_table.shape
        sizes = [_bits32(name, v) for name, v in
                 (("n_seq", n_seq), ("n_tokens", n_tokens), ("h_q", h_q), ("h_kv", h_kv), ("d", d),
                  ("page_size", page_size), ("n_pages", n_pages), ("max_pages", max_pages))]
        flags, wait = _bits32("flags", flags), _bits32("wait_timeout_ms", wait_timeout_ms, 0, 2**32 - 1)
        _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, (n_seq + 1,))
        _check(kv_lens, "kv_lens", torch.int32, (n_seq,))
        _check(page_table, "page_table", torch.int32, (n_seq, max_pages))
        self.tables = (cu_seqlens_q, kv_lens, page_table)
        self.params = _CPagedParams(*sizes, int(bool(causal)), float(scale), cu_seqlens_q.data_ptr(),
                                    kv_lens.data_ptr(), page_table.data_ptr(), dev_status or None, flags, wait)
        need = attn_core_paged_workspace_bytes(self.params)
        if need == 0:       # the call itself says what is wrong
            raise AttnCoreError(ERR_UNSUPPORTED if page_size not in PAGE_SIZES or d not in SUPPORTED_HEAD_DIMS
                                else ERR_INVALID_ARG, "PagedBatch")
        self._groups = None     # (number of groups, their tables' addresses)
        if (group_starts is None) != (prefix_pages is None):
            raise ValueError("group_starts and prefix_pages go together")
        if group_starts is not None:
            n_groups = group_starts.numel() - 1
            _check(group_starts, "group_starts", torch.int32, (n_groups + 1,))
            _check(prefix_pages, "prefix_pages", torch.int32, (n_groups,))
            self._groups = (n_groups, group_starts.data_ptr(), prefix_pages.data_ptr())
            self.tables += (group_starts, prefix_pages)
            more = attn_core_paged_prefix_workspace_bytes(self.params, n_groups)
            if more == 0:
                raise AttnCoreError(ERR_INVALID_ARG, "PagedBatch")
            need = max(need, more)
        names = ("kv_lens", "page_table", "group_starts", "prefix_pages")
        for name, t in zip(names, self.tables[1:]):
            if t.device != cu_seqlens_q.device:
                raise ValueError(f"{name} must be on {cu_seqlens_q.device}, got {t.device}")
        self._streams = set()   # handles of the streams that calls were made on
        self.workspace = torch.empty(need, dtype=torch.uint8, device=cu_seqlens_q.device) if workspace is None \
            else workspace
        self._address = ctypes.addressof(self.params)
        self._strides = {}      # by paged_append's layouts: three token strides
        self._q_shape = torch.Size((int(n_tokens), int(h_q), int(d)))
        self._kv_shape = torch.Size((int(n_tokens), int(h_kv), int(d)))
        self._page_shape = torch.Size((int(n_pages), int(h_kv), int(page_size), int(d)))
        self._lse_shape = torch.Size((int(h_q), int(n_tokens)))
        self._weights_shape = torch.Size((int(n_seq), int(h_kv), int(max_pages) * int(page_size)))
        self._weights_layout = _layout(self._weights_shape)
        self._seq_shape, self._table_shape = torch.Size((int(n_seq),)), torch.Size((int(n_seq), int(max_pages)))
        self._evict_bytes = attn_core_paged_evict_workspace_bytes(self.params)      # 0: more than it can count
        self._q_layout, self._lse_layout = _layout(self._q_shape), _layout(self._lse_shape)

    @property
    def workspace(self):
        """The attention's device memory; another one takes its place by assignment."""
        return self._workspace

    @workspace.setter
    def workspace(self, t) -> None:
        import torch
        if not isinstance(t, torch.Tensor) or t.device != self.tables[0].device or not t.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.tables[0].device}")   # its bytes are counted
        self._workspace = t
        self._ws = (t.data_ptr(), t.numel() * t.element_size())
        self._streams.clear()

    def _used_on(self, stream: int) -> None:
        """The first call on the current stream: the allocator is told of it, so that
        it does not hand the workspace out again, or tables that only the batch
        holds, before the calls there have run (5 us, once for each stream)."""
        import torch
        current = torch.cuda.current_stream()
        for t in (self.workspace, *self.tables):
            t.record_stream(current)
        self._streams.add(stream)


def _token_stride(x, name, shape):
    """Elements from one token to the next of [tokens, heads, d] whose heads are
    contiguous (a slice of a fused projection, for one)."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.bfloat16 or x.shape != shape:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor of shape {tuple(shape)}")
    t, h, e = x.stride()
    if (e != 1 and shape[2] > 1) or (h != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must be contiguous in its heads and their values")
    return t if shape[0] > 1 else shape[1] * shape[2]


def paged_append(batch: PagedBatch, q, k, v, k_pages, v_pages, *, table: RopeTable | None = None, out_q=None):
    """Add the new tokens' k and v [n_tokens, h_kv, d] to the cache, rotated by
    ``table`` at their positions (None: as they are), and rotate q
    [n_tokens, h_q, d] (or None).  Returns q's rotation, packed."""
    host = _host()
    dev, bf16 = host.device(), host.bf16
    # what a layout needs follows from shapes, strides and types alone
    key = (None if q is None else (q.shape, q.stride(), q.dtype), k.shape, k.stride(), k.dtype, v.shape, v.stride(),
           v.dtype)
    strides = batch._strides.get(key)
    if strides is None:
        three = (0 if q is None else _token_stride(q, "q", batch._q_shape), _token_stride(k, "k", batch._kv_shape),
                 _token_stride(v, "v", batch._kv_shape))
        if len(batch._strides) >= 64:
            batch._strides.clear()
        batch._strides[key] = strides = (ctypes.c_int64 * 3)(*three)
    _need(k_pages, "k_pages", bf16, batch._page_shape, dev)
    _need(v_pages, "v_pages", bf16, batch._page_shape, dev)
    xq = yq = 0
    if q is not None:
        if out_q is None:
            out_q = host.empty(*batch._q_layout, bf16)
        else:
            _need(out_q, "out_q", bf16, batch._q_shape, dev)
        xq, yq = q.data_ptr(), out_q.data_ptr()
    elif out_q is not None:
        raise ValueError("out_q without q")
    if k.get_device() != dev or v.get_device() != dev or (q is not None and q.get_device() != dev) \
            or batch._workspace.get_device() != dev:
        _on_device(dev, q, k, v, batch._workspace)
    if batch.params.n_tokens:
        stream = host.stream(dev)
        if stream not in batch._streams:
            batch._used_on(stream)
        rc = _FAST["attn_core_paged_append"](batch._address, 0 if table is None else ctypes.addressof(table), xq,
                                             k.data_ptr(), v.data_ptr(), ctypes.addressof(strides), yq,
                                             k_pages.data_ptr(), v_pages.data_ptr(), stream)
        if rc != OK:
            raise AttnCoreError(rc, "attn_core_paged_append")
    return out_q


def paged_fwd(batch: PagedBatch, q, k_pages, v_pages, *, out=None, lse=None):
    """Attention of the batch's new tokens q [n_tokens, h_q, d] over the cache
    (which already holds their keys and values).  Returns (O like q, LSE fp32
    [h_q, n_tokens])."""
    dev, out, lse = _attend_args(batch, q, k_pages, v_pages, out, lse)
    if batch.params.n_tokens:
        ws, ws_bytes = batch._ws
        stream = _host().stream(dev)
        if stream not in batch._streams:
            batch._used_on(stream)
        rc = _FAST["attn_core_paged_fwd"](batch._address, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                          out.data_ptr(), lse.data_ptr(), ws, ws_bytes, stream)
        if rc != OK:
            raise AttnCoreError(rc, "attn_core_paged_fwd")
    return out, lse


def _attend_args(batch: PagedBatch, q, k_pages, v_pages, out, lse):
    """The device, and O and LSE of a call of the attention over the cache."""
    host = _host()
    dev, bf16 = host.device(), host.bf16
    _need(q, "q", bf16, batch._q_shape, dev)
    _need(k_pages, "k_pages", bf16, batch._page_shape, dev)
    _need(v_pages, "v_pages", bf16, batch._page_shape, dev)
    if out is None:
        out = host.empty(*batch._q_layout, bf16)
    else:
        _need(out, "out", bf16, batch._q_shape, dev)
    if lse is None:
        lse = host.empty(*batch._lse_layout, host.f32)
    else:
        _need(lse, "lse", host.f32, batch._lse_shape, dev)
    if batch._workspace.get_device() != dev:
        _on_device(dev, batch._workspace)
    return dev, out, lse


def paged_prefix_fwd(batch: PagedBatch, q, k_pages, v_pages, *, out=None, lse=None):
    """paged_fwd of a batch with groups of sequences that share their first
    pages: the shared keys are visited once for each group.  Returns (O, LSE)."""
    if batch._groups is None:
        raise ValueError("the batch has no groups (group_starts, prefix_pages)")
    dev, out, lse = _attend_args(batch, q, k_pages, v_pages, out, lse)
    if batch.params.n_tokens:
        ws, ws_bytes = batch._ws
        stream = _host().stream(dev)
        if stream not in batch._streams:
            batch._used_on(stream)
        rc = _FAST["attn_core_paged_prefix_fwd"](batch._address, *batch._groups, q.data_ptr(), k_pages.data_ptr(),
                                                 v_pages.data_ptr(), out.data_ptr(), lse.data_ptr(), ws, ws_bytes,
                                                 stream)
        if rc != OK:
            raise AttnCoreError(rc, "attn_core_paged_prefix_fwd")
    return out, lse


def paged_weights(batch: PagedBatch, q, lse, k_pages, weights, *, decay: float = 1.0, out=None):
    """Add what the batch's new tokens pay to each key of the cache (their
    attention weights, by ``lse`` as paged_fwd returned it) to ``weights`` fp32
    [n_seq, h_kv, max_pages * page_size], whose earlier values fade by ``decay``;
    the new tokens' own keys start at 0.  In place, or into ``out``, which is
    returned; sequences without new tokens are left as they were there."""
    host = _host()
    dev = host.device()
    _need(q, "q", host.bf16, batch._q_shape, dev)
    _need(k_pages, "k_pages", host.bf16, batch._page_shape, dev)
    _need(lse, "lse", host.f32, batch._lse_shape, dev)
    _need(weights, "weights", host.f32, batch._weights_shape, dev)
    if out is None:
        out = weights
    else:
        _need(out, "out", host.f32, batch._weights_shape, dev)
    if batch._workspace.get_device() != dev:
        _on_device(dev, batch._workspace)
    if batch.params.n_tokens:
        ws, ws_bytes = batch._ws
        stream = host.stream(dev)
        if stream not in batch._streams:
            batch._used_on(stream)
        rc = _FAST["attn_core_paged_weights"](batch._address, q.data_ptr(), k_pages.data_ptr(), lse.data_ptr(),
                                              float(decay), weights.data_ptr(), out.data_ptr(), ws, ws_bytes, stream)
        if rc != OK:
            raise AttnCoreError(rc, "attn_core_paged_weights")
    return out


def paged_evict(batch: PagedBatch, weights, keep, k_pages, v_pages, *, first: int = 0, recent: int = 0,
                out_table=None, out_weights=None, kept=None):
    """Keep ``keep[i]`` keys of sequence i (int32 CUDA tensor [n_seq]), each KV head
    its own: the ``recent`` last, the ``first`` first, and of the others those with
    the largest ``weights``.  They move to the front in their order, K and V within
    the sequence's pages or to those of ``out_table`` [n_seq, max_pages]
    (PagePool.shrink), the weights in place or into ``out_weights``.  Returns
    ``kept`` int32 [n_seq, h_kv, max_pages * page_size]: the key that each was."""
    host = _host()
    dev = host.device()
    _need(weights, "weights", host.f32, batch._weights_shape, dev)
    _need(keep, "keep", host.i32, batch._seq_shape, dev)
    _need(k_pages, "k_pages", host.bf16, batch._page_shape, dev)
    _need(v_pages, "v_pages", host.bf16, batch._page_shape, dev)
    if out_table is not None:
        _need(out_table, "out_table", host.i32, batch._table_shape, dev)
    if out_weights is None:
        out_weights = weights
    else:
        _need(out_weights, "out_weights", host.f32, batch._weights_shape, dev)
    if kept is None:
        kept = host.empty(*batch._weights_layout, host.i32)
    else:
        _need(kept, "kept", host.i32, batch._weights_shape, dev)
    first, recent = _bits32("first", first), _bits32("recent", recent)
    if batch._workspace.get_device() != dev:
        _on_device(dev, batch._workspace)
    ws, ws_bytes = batch._ws
    if ws_bytes < batch._evict_bytes:       # of this call's own: very many or very long sequences
        own = host.empty((batch._evict_bytes // 4,), (1,), host.i32)
        ws, ws_bytes = own.data_ptr(), batch._evict_bytes
    stream = host.stream(dev)
    if stream not in batch._streams:
        batch._used_on(stream)
    rc = _FAST["attn_core_paged_evict"](batch._address, keep.data_ptr(), first, recent,
                                        0 if out_table is None else out_table.data_ptr(), k_pages.data_ptr(),
                                        v_pages.data_ptr(), weights.data_ptr(), out_weights.data_ptr(),
                                        kept.data_ptr(), ws, ws_bytes, stream)
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_paged_evict")
    return kept


def page_copy(pages, pairs) -> None:
    """Copy pages of a cache, pairs[i] = (from, to), in every plane of ``pages``
    [planes, n_pages, h_kv, page_size, d] (or one plane, four-dimensional).
    ``pairs``: a host list or int32 array; no target may be named twice or be
    another copy's source."""
    import numpy as np
    import torch
    if not isinstance(pages, torch.Tensor) or not pages.is_cuda or pages.dim() not in (4, 5) \
            or not pages.is_contiguous():
        raise ValueError("pages must be a contiguous CUDA tensor [planes, n_pages, h_kv, page_size, d]")
    if isinstance(pairs, torch.Tensor):
        if pairs.is_cuda:
            raise ValueError("pairs must be in host memory")
        pairs = pairs.numpy()
    arr = pairs
    if not (isinstance(arr, np.ndarray) and arr.dtype == np.int32 and arr.ndim == 2 and arr.shape[1] == 2
            and arr.flags.c_contiguous):
        wide = np.asarray(pairs)
        if wide.size and wide.dtype.kind not in "iu":
            raise ValueError("pairs must be integers")
        if wide.size and (wide.ndim != 2 or wide.shape[1] != 2):
            raise ValueError(f"pairs must be [n, 2], got {wide.shape}")
        arr = np.ascontiguousarray(wide, dtype=np.int32)
        if not np.array_equal(arr, wide):
            raise ValueError("pairs must fit 32 bits")
    host = _host()
    dev = host.device()
    _on_device(dev, pages)
    shape = pages.shape
    planes, n_pages = (shape[0] if len(shape) == 5 else 1), shape[-4]
    if pages.numel() == 0:
        if arr.size:
            raise ValueError("no pages to copy")
        return
    page_bytes = shape[-3] * shape[-2] * shape[-1] * pages.element_size()
    load_library()
    rc = _FAST["attn_core_page_copy"](pages.data_ptr(), planes, n_pages * page_bytes, n_pages, page_bytes,
                                      arr.ctypes.data, len(arr) if arr.size else 0, host.stream(dev))
    if rc != OK:
        raise AttnCoreError(rc, "attn_core_page_copy")
