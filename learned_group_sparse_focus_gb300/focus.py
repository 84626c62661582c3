"""Python binding of libfocus.so (the Focus C ABI declared in include/focus.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch provides device memory and streams.  If the compiled
library is missing, importing this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libfocus.so")

F32, BF16 = 0, 1
TILE_M = 128
TILE_N = 128
CACHE_PAGE = 64           # slots of a cache page
CACHE_MAX_QUERY = 64      # new tokens a sequence in one focus_cache_attention_fwd

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace too small",
          4: "CUDA error", 5: "device wait timed out", 6: "group id outside [0, K)",
          7: "cache page, length or position out of range"}


class FocusError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({status})")
        self.status = status


class Params(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("B", "H", "H_kv", "n", "d", "D", "d_g", "K", "A", "w")] + \
               [("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class Item(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("b", "a", "g", "row0", "rows", "keys", "key0", "pad")]


class Index(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("rank", ctypes.c_void_p), ("farlen_tok", ctypes.c_void_p),
                ("farlen_slot", ctypes.c_void_p), ("items", ctypes.c_void_p),
                ("order", ctypes.c_void_p), ("n_items", ctypes.c_void_p),
                ("max_items", ctypes.c_int32), ("w_eff", ctypes.c_int32)]


class IndexTopk(ctypes.Structure):
    _fields_ = [("entry", Index), ("pair", Index), ("pair_gid", ctypes.c_void_p),
                ("far_tok", ctypes.c_void_p), ("k", ctypes.c_int32), ("split", ctypes.c_int32),
                ("farlen_sub", ctypes.c_void_p)]


class CacheStruct(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("k", "v", "k_scale", "v_scale", "pos", "gid", "mass", "table",
                                               "len", "next")] + \
               [("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libfocus.so not built ({LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, P, C = ctypes.c_void_p, ctypes.POINTER(Params), ctypes.POINTER(CacheStruct)
    sig = {
        "focus_abi_version": ([], ctypes.c_int32),
        "focus_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "focus_workspace_bytes": ([P], ctypes.c_size_t),
        "focus_workspace_init": ([vp, vp], ctypes.c_int),
        "focus_assign": ([P, vp, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "focus_build_index": ([P, vp, ctypes.POINTER(Index), vp, ctypes.c_size_t, vp], ctypes.c_int),
        "focus_attention_fwd": ([P, vp, vp, vp, ctypes.POINTER(Index), vp, vp, vp, ctypes.c_size_t, vp],
                                ctypes.c_int),
        "focus_attention_fwd_timed": ([P, vp, vp, vp, ctypes.POINTER(Index), vp, vp, vp, ctypes.c_size_t,
                                       vp, ctypes.POINTER(ctypes.c_void_p)], ctypes.c_int),
        "focus_dense_causal_fwd": ([P, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "focus_test_attention_wait_limit": ([P, vp, vp, vp, vp, vp, ctypes.c_size_t, ctypes.c_uint64, vp],
                                            ctypes.c_int),
        "focus_sinkhorn_workspace_bytes": ([P], ctypes.c_size_t),
        "focus_assign_scores": ([P, vp, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "focus_sinkhorn_fwd": ([P, ctypes.c_int32, ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp],
                               ctypes.c_int),
        "focus_backward_workspace_bytes": ([P], ctypes.c_size_t),
        "focus_attention_bwd": ([P, vp, vp, vp, vp, vp, vp, ctypes.POINTER(Index), vp, vp, vp, vp,
                                 ctypes.c_size_t, vp], ctypes.c_int),
        "focus_attention_two_call_fwd": ([P, vp, vp, vp, ctypes.POINTER(Index), vp, vp, vp, ctypes.c_size_t,
                                          vp], ctypes.c_int),
        "focus_layer_fwd_host": ([P] + [vp] * 7 + [vp] * 8 + [vp, ctypes.c_size_t, vp], ctypes.c_int),
        "focus_check_errors": ([vp, vp], ctypes.c_int),
        "focus_build_index_static": ([P, vp, ctypes.POINTER(Index), vp, vp], ctypes.c_int),
        "focus_workspace_bytes_topk": ([P, ctypes.c_int32], ctypes.c_size_t),
        "focus_assign_topk": ([P, ctypes.c_int32, vp, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "focus_build_index_topk": ([P, ctypes.c_int32, vp, ctypes.POINTER(IndexTopk), vp, ctypes.c_size_t,
                                    vp], ctypes.c_int),
        "focus_attention_topk_fwd": ([P, vp, vp, vp, ctypes.POINTER(IndexTopk), vp, vp, vp, ctypes.c_size_t,
                                      vp], ctypes.c_int),
        "focus_attention_topk_fwd_timed": ([P, vp, vp, vp, ctypes.POINTER(IndexTopk), vp, vp, vp,
                                            ctypes.c_size_t, vp, ctypes.POINTER(ctypes.c_void_p)],
                                           ctypes.c_int),
        "focus_cache_workspace_bytes": ([P, C], ctypes.c_size_t),
        "focus_cache_append": ([P, vp, vp, vp, vp, C, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "focus_cache_attention_fwd": ([P, vp, vp, vp, C, vp, vp, ctypes.c_int32, vp, ctypes.c_size_t, vp],
                                      ctypes.c_int),
        "focus_cache_evict": ([P, ctypes.c_int32, ctypes.c_int32, C, C, vp, ctypes.c_size_t, vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()

EXPORTED = ("focus_abi_version", "focus_status_string", "focus_workspace_bytes",
            "focus_workspace_init", "focus_assign", "focus_build_index", "focus_attention_fwd",
            "focus_attention_fwd_timed", "focus_dense_causal_fwd", "focus_layer_fwd_host", "focus_check_errors",
            "focus_build_index_static", "focus_workspace_bytes_topk", "focus_assign_topk",
            "focus_build_index_topk", "focus_attention_topk_fwd", "focus_attention_topk_fwd_timed",
            "focus_attention_two_call_fwd", "focus_sinkhorn_workspace_bytes", "focus_assign_scores",
            "focus_sinkhorn_fwd", "focus_backward_workspace_bytes", "focus_attention_bwd",
            "focus_test_attention_wait_limit", "focus_cache_workspace_bytes", "focus_cache_append",
            "focus_cache_attention_fwd", "focus_cache_evict")


def lib():
    return _lib


def make_params(B, H, H_kv, n, d, D, d_g, K, A, w, scale=None, dtype=BF16) -> Params:
    if scale is None:
        scale = 1.0 / (d ** 0.5)
    if isinstance(dtype, str):
        dtype = BF16 if dtype == "bf16" else F32
    return Params(B, H, H_kv, n, d, D, d_g, K, A, w, float(scale), int(dtype))


def params_from_workload(wl, **override) -> Params:
    f = dict(B=wl.B, H=wl.H, H_kv=wl.H_kv, n=wl.n, d=wl.d, D=wl.D, d_g=wl.d_g, K=wl.K, A=wl.A,
             w=wl.w, scale=wl.scale, dtype=wl.dtype)
    f.update(override)
    return make_params(**f)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return t.data_ptr()
    return int(t)


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(fn: str, st: int):
    if st != 0:
        raise FocusError(fn, st)


def focus_workspace_bytes(p: Params) -> int:
    return int(_lib.focus_workspace_bytes(ctypes.byref(p)))


def alloc_workspace(p: Params, device="cuda", stream=None) -> torch.Tensor:
    """Caller-owned workspace (a uint8 device tensor), error word cleared."""
    nbytes = focus_workspace_bytes(p)
    if nbytes == 0:
        raise FocusError("focus_workspace_bytes", 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    focus_workspace_init(ws, stream)
    return ws


def focus_workspace_init(ws, stream=None):
    _check("focus_workspace_init", _lib.focus_workspace_init(_ptr(ws), _stream(stream)))


def focus_assign(p: Params, h, W, C, gid, ws, stream=None):
    _check("focus_assign", _lib.focus_assign(ctypes.byref(p), _ptr(h), _ptr(W), _ptr(C), _ptr(gid),
                                             _ptr(ws), ws.numel(), _stream(stream)))


def focus_build_index(p: Params, gid, ws, stream=None) -> Index:
    idx = Index()
    _check("focus_build_index", _lib.focus_build_index(ctypes.byref(p), _ptr(gid), ctypes.byref(idx),
                                                       _ptr(ws), ws.numel(), _stream(stream)))
    return idx


def focus_attention_fwd(p: Params, Q, K, V, idx: Index, O, lse, ws, stream=None):
    _check("focus_attention_fwd",
           _lib.focus_attention_fwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), ctypes.byref(idx),
                                    _ptr(O), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def focus_attention_fwd_timed(p: Params, Q, K, V, idx: Index, O, lse, ws, events, stream=None):
    """events: four recorded-once torch.cuda.Event objects (see include/focus.h)."""
    arr = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
    _check("focus_attention_fwd_timed",
           _lib.focus_attention_fwd_timed(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), ctypes.byref(idx),
                                          _ptr(O), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream), arr))


def focus_attention_two_call_fwd(p: Params, Q, K, V, idx: Index, O, lse, ws, stream=None):
    """The two-call comparator (group call, window call, separate combine)."""
    _check("focus_attention_two_call_fwd",
           _lib.focus_attention_two_call_fwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), ctypes.byref(idx),
                                             _ptr(O), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def focus_dense_causal_fwd(p: Params, Q, K, V, O, lse, ws, stream=None):
    _check("focus_dense_causal_fwd",
           _lib.focus_dense_causal_fwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse),
                                       _ptr(ws), ws.numel(), _stream(stream)))


def focus_test_attention_wait_limit(p: Params, Q, K, V, O, ws, wait_ns: int, stream=None):
    """Test hook: the dense kernel with its first Q tile withheld and every
    device wait limited to wait_ns; the device error word then holds the
    timeout bit (read it with focus_check_errors)."""
    _check("focus_test_attention_wait_limit",
           _lib.focus_test_attention_wait_limit(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(ws),
                                                ws.numel(), int(wait_ns), _stream(stream)))


def focus_layer_fwd_host(p: Params, host: dict, dev: dict, ws, stream=None):
    """host: pinned CPU tensors h, W, C, Q, K, V, O; dev: device tensors of the same
    names plus gid.  Enqueues H2D copies, the three steps and the D2H copy of O."""
    _check("focus_layer_fwd_host", _lib.focus_layer_fwd_host(
        ctypes.byref(p), *[_ptr(host[k]) for k in ("h", "W", "C", "Q", "K", "V", "O")],
        *[_ptr(dev[k]) for k in ("h", "W", "C", "Q", "K", "V", "O", "gid")],
        _ptr(ws), ws.numel(), _stream(stream)))


def focus_check_errors(ws, stream=None) -> int:
    """Synchronise the stream; return (and clear) the device error status."""
    return int(_lib.focus_check_errors(_ptr(ws), _stream(stream)))


def index_buffers(p: Params, device="cuda") -> dict:
    """Caller-owned output buffers for focus_build_index_static, sized as the
    index arrays of focus_build_index, plus a zeroed 256-byte error word."""
    P, n, K = p.B * p.A, p.n, p.K
    m = P * ((n + TILE_M - 1) // TILE_M + min(K, n))
    z = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)
    return dict(counts=z(p.B, p.A, K), offsets=z(p.B, p.A, K + 1), perm=z(p.B, p.A, n),
                rank=z(p.B, p.A, n), farlen_tok=z(p.B, p.A, n), farlen_slot=z(p.B, p.A, n),
                items=z(m, 8), order=z(m), n_items=z(1),
                err=torch.zeros(64, dtype=torch.int32, device=device))


def focus_build_index_static(p: Params, gid, bufs: dict, stream=None) -> Index:
    """focus_build_index into the caller-owned buffers of index_buffers(); the
    sort's scratch is the library's fixed device array (no workspace)."""
    idx = Index()
    for name in ("counts", "offsets", "perm", "rank", "farlen_tok", "farlen_slot", "items", "order",
                 "n_items"):
        setattr(idx, name, _ptr(bufs[name]))
    idx.max_items = bufs["order"].numel()
    _check("focus_build_index_static",
           _lib.focus_build_index_static(ctypes.byref(p), _ptr(gid), ctypes.byref(idx), _ptr(bufs["err"]),
                                         _stream(stream)))
    return idx


# ------------------------------------------------------- top-k membership ---

def focus_workspace_bytes_topk(p: Params, k: int) -> int:
    return int(_lib.focus_workspace_bytes_topk(ctypes.byref(p), int(k)))


def alloc_workspace_topk(p: Params, k: int, device="cuda", stream=None) -> torch.Tensor:
    """Caller-owned workspace for the top-k calls, error word cleared."""
    nbytes = focus_workspace_bytes_topk(p, k)
    if nbytes == 0:
        raise FocusError("focus_workspace_bytes_topk", 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    focus_workspace_init(ws, stream)
    return ws


def focus_assign_topk(p: Params, k: int, h, W, C, gid, ws, stream=None):
    """gid: [B, A, n, k] int32 device tensor (best first)."""
    _check("focus_assign_topk", _lib.focus_assign_topk(ctypes.byref(p), int(k), _ptr(h), _ptr(W), _ptr(C),
                                                       _ptr(gid), _ptr(ws), ws.numel(), _stream(stream)))


def focus_build_index_topk(p: Params, k: int, gid, ws, stream=None) -> IndexTopk:
    idx = IndexTopk()
    _check("focus_build_index_topk",
           _lib.focus_build_index_topk(ctypes.byref(p), int(k), _ptr(gid), ctypes.byref(idx), _ptr(ws),
                                       ws.numel(), _stream(stream)))
    return idx


def focus_attention_topk_fwd(p: Params, Q, K, V, idx: IndexTopk, O, lse, ws, stream=None):
    _check("focus_attention_topk_fwd",
           _lib.focus_attention_topk_fwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), ctypes.byref(idx),
                                         _ptr(O), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def focus_attention_topk_fwd_timed(p: Params, Q, K, V, idx: IndexTopk, O, lse, ws, events, stream=None):
    """events: five torch.cuda.Event objects (see include/focus.h)."""
    arr = (ctypes.c_void_p * 5)(*[e.cuda_event for e in events])
    _check("focus_attention_topk_fwd_timed",
           _lib.focus_attention_topk_fwd_timed(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), ctypes.byref(idx),
                                               _ptr(O), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream),
                                               arr))


def run_layer_topk(p: Params, k: int, h, W, C, Q, K, V, ws, stream=None, want_lse=False):
    """assign (top-k) -> index -> attention; returns (O, gid, idx, lse)."""
    dev = Q.device
    gid = torch.empty((p.B, p.A, p.n, k), dtype=torch.int32, device=dev)
    focus_assign_topk(p, k, h, W, C, gid, ws, stream)
    idx = focus_build_index_topk(p, k, gid, ws, stream)
    O = torch.empty_like(Q)
    lse = torch.empty((p.B, p.H, p.n), dtype=torch.float32, device=dev) if want_lse else None
    focus_attention_topk_fwd(p, Q, K, V, idx, O, lse, ws, stream)
    return O, gid, idx, lse


# ---------------------------------------------------------------- backward ---

def alloc_workspace_backward(p: Params, device="cuda", stream=None) -> torch.Tensor:
    nbytes = int(_lib.focus_backward_workspace_bytes(ctypes.byref(p)))
    if nbytes == 0:
        raise FocusError("focus_backward_workspace_bytes", 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    focus_workspace_init(ws, stream)
    return ws


def focus_attention_bwd(p: Params, Q, K, V, O, dO, lse, idx: Index, dQ, dK, dV, ws, stream=None):
    """Gradients over the kept pairs; lse from the forward call, idx from
    focus_build_index (forward workspace), ws a backward workspace."""
    _check("focus_attention_bwd",
           _lib.focus_attention_bwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse),
                                    ctypes.byref(idx), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(ws), ws.numel(),
                                    _stream(stream)))


# ------------------------------------------------ Sinkhorn soft assignment ---

def alloc_workspace_sinkhorn(p: Params, device="cuda", stream=None) -> torch.Tensor:
    nbytes = int(_lib.focus_sinkhorn_workspace_bytes(ctypes.byref(p)))
    if nbytes == 0:
        raise FocusError("focus_sinkhorn_workspace_bytes", 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    focus_workspace_init(ws, stream)
    return ws


def focus_assign_scores(p: Params, h, W, C, S, ws, stream=None):
    """S: [B, A, n, K] fp32 device tensor."""
    _check("focus_assign_scores", _lib.focus_assign_scores(ctypes.byref(p), _ptr(h), _ptr(W), _ptr(C), _ptr(S),
                                                           _ptr(ws), ws.numel(), _stream(stream)))


def focus_sinkhorn_fwd(p: Params, iters: int, tau: float, S, G, ws, stream=None):
    """G (may be S): [B, A, n, K] fp32 soft assignment after `iters` rounds."""
    _check("focus_sinkhorn_fwd", _lib.focus_sinkhorn_fwd(ctypes.byref(p), int(iters), float(tau), _ptr(S),
                                                         _ptr(G), _ptr(ws), ws.numel(), _stream(stream)))


# --------------------------------------------------------- key/value cache ---

def _expect(name: str, t, shape, dtype, device):
    """Address of a tensor argument of the cache calls, its shape, dtype, device
    and layout checked."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} on {device}, got {tuple(t.shape)} {t.dtype} "
                     f"on {t.device}, strides {t.stride()}")


@dataclass(frozen=True, eq=False)
class Cache:
    """A paged 8-bit key/value cache: the caller's device tensors, laid out as
    focus_cache_t in include/focus.h.  Several caches may share the pool
    tensors (k ... mass) and differ in table, len and next."""
    k: torch.Tensor          # [n_pages, H_kv, 64, d] uint8, e4m3 codes
    v: torch.Tensor          # [n_pages, H_kv, 64, d] uint8, e4m3 codes
    k_scale: torch.Tensor    # [n_pages, H_kv] fp32, powers of two
    v_scale: torch.Tensor    # [n_pages, H_kv] fp32, powers of two
    pos: torch.Tensor        # [n_pages, H_kv, 64] int32
    gid: torch.Tensor        # [n_pages, H_kv, 64] int16
    mass: torch.Tensor | None  # [n_pages, H_kv, 64] fp32
    table: torch.Tensor      # [B, max_pages] int32
    len: torch.Tensor        # [B, H_kv] int32
    next: torch.Tensor       # [B] int32

    def __post_init__(self):
        if self.k.dim() != 4 or self.table.dim() != 2:
            raise ValueError("k must be [n_pages, H_kv, 64, d] and table [B, max_pages]")
        pages, H_kv, _, d = self.k.shape
        B, max_pages = self.table.shape
        dev, page = self.k.device, (pages, H_kv, CACHE_PAGE)
        c = CacheStruct(n_pages=pages, max_pages=max_pages)
        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        for name, shape, dtype in (("k", page + (d,), u8), ("v", page + (d,), u8), ("k_scale", page[:2], f32),
                                   ("v_scale", page[:2], f32), ("pos", page, i32), ("gid", page, torch.int16),
                                   ("mass", page, f32), ("table", (B, max_pages), i32), ("len", (B, H_kv), i32),
                                   ("next", (B,), i32)):
            t = getattr(self, name)
            if name == "mass" and t is None:
                continue
            setattr(c, name, _expect(name, t, shape, dtype, dev))
        object.__setattr__(self, "struct", c)
        object.__setattr__(self, "ref", ctypes.byref(c))
        object.__setattr__(self, "device", dev)
        object.__setattr__(self, "dims", (B, H_kv, d))


def alloc_cache(p: Params, max_tokens: int, mass: bool = False, device="cuda") -> Cache:
    """An empty cache with room for max_tokens slots a sequence, pages in order."""
    if max_tokens < 1:
        raise ValueError("max_tokens must be at least 1")
    pages = -(-int(max_tokens) // CACHE_PAGE)
    n, shape = p.B * pages, (p.B * pages, p.H_kv, CACHE_PAGE)

    def zeros(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=device)

    return Cache(k=zeros(shape + (p.d,), torch.uint8), v=zeros(shape + (p.d,), torch.uint8),
                 k_scale=zeros(shape[:2], torch.float32), v_scale=zeros(shape[:2], torch.float32),
                 pos=zeros(shape, torch.int32), gid=zeros(shape, torch.int16),
                 mass=zeros(shape, torch.float32) if mass else None,
                 table=torch.arange(n, dtype=torch.int32, device=device).view(p.B, pages),
                 len=zeros((p.B, p.H_kv), torch.int32), next=zeros((p.B,), torch.int32))


def focus_cache_workspace_bytes(p: Params, cache: Cache) -> int:
    return int(_lib.focus_cache_workspace_bytes(ctypes.byref(p), ctypes.byref(cache.struct)))


def alloc_workspace_cache(p: Params, cache: Cache, stream=None) -> torch.Tensor:
    """Caller-owned workspace for the cache calls on this cache, error word
    cleared."""
    nbytes = focus_cache_workspace_bytes(p, cache)
    if nbytes == 0:
        raise FocusError("focus_cache_workspace_bytes", 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
    with torch.cuda.device(cache.device):
        focus_workspace_init(ws, stream)
    return ws


def _raw_stream(index: int) -> int:
    """Current stream of a device (torch.cuda.current_stream builds an object, at
    a third of the cost of a whole call)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _cache_call(fn: str, p: Params, cache: Cache, ws, stream, *args):
    """Runs a cache call on the cache's device (args: the C arguments between p
    and ws)."""
    dev = cache.device
    if cache.dims != (p.B, p.H_kv, p.d):
        raise ValueError(f"the cache holds (B, H_kv, d) = {cache.dims}, the call asks for {(p.B, p.H_kv, p.d)}")
    if dev.type != "cuda":
        raise ValueError(f"the cache must be on a CUDA device, not {dev}")
    if ws.device != dev or (stream is not None and stream.device != dev):
        raise ValueError(f"workspace and stream must be on the cache's device {dev}")
    call = getattr(_lib, fn)
    raw = _raw_stream(dev.index) if stream is None else stream.cuda_stream
    if dev.index == torch.cuda.current_device():
        st = call(p, *args, _ptr(ws), ws.numel(), raw)
    else:
        with torch.cuda.device(dev):
            st = call(p, *args, _ptr(ws), ws.numel(), raw)
    if st != 0:
        raise FocusError(fn, st)


def _float_type(p: Params):
    return torch.bfloat16 if p.dtype == BF16 else torch.float32


def focus_cache_append(p: Params, K, V, gid, cache: Cache, ws, n_new=None, len_out=None, next_out=None, stream=None):
    """Appends K, V [B, H_kv, n, d] and gid [B, A, n]; n_new [B] int32: valid
    tokens a sequence (None: all n).  The counts are updated in place, or written
    to len_out [B, H_kv] and next_out [B]."""
    dev, B, H_kv, n, ft, i32 = cache.device, p.B, p.H_kv, p.n, _float_type(p), torch.int32
    rows = (B, H_kv, n, p.d)
    _cache_call("focus_cache_append", p, cache, ws, stream,
                _expect("K", K, rows, ft, dev), _expect("V", V, rows, ft, dev),
                _expect("gid", gid, (B, p.A, n), i32, dev),
                None if n_new is None else _expect("n_new", n_new, (B,), i32, dev), cache.ref,
                cache.struct.len if len_out is None else _expect("len_out", len_out, (B, H_kv), i32, dev),
                cache.struct.next if next_out is None else _expect("next_out", next_out, (B,), i32, dev))


def focus_cache_attention_fwd(p: Params, Q, gid, cache: Cache, O, lse, ws, n_new=None, accumulate=False,
                              stream=None):
    """Attention of the newest tokens Q [B, H, n, d] (the last n_new[b] appended
    ones) over the cache into O and lse ([B, H, n] fp32 or None); accumulate adds
    the weights each slot received to cache.mass."""
    dev, B, H, n, ft, i32 = cache.device, p.B, p.H, p.n, _float_type(p), torch.int32
    rows = (B, H, n, p.d)
    _cache_call("focus_cache_attention_fwd", p, cache, ws, stream,
                _expect("Q", Q, rows, ft, dev), _expect("gid", gid, (B, p.A, n), i32, dev),
                None if n_new is None else _expect("n_new", n_new, (B,), i32, dev), cache.ref,
                _expect("O", O, rows, ft, dev),
                None if lse is None else _expect("lse", lse, (B, H, n), torch.float32, dev), 1 if accumulate else 0)


def focus_cache_evict(p: Params, budget: int, recent: int, src: Cache, dst: Cache, ws, stream=None):
    """Copies the at most `budget` slots a head that stay (the last `recent`
    positions, then the most mass) from src's pages into dst's."""
    if dst.device != src.device or dst.dims != src.dims:
        raise ValueError("src and dst must be on one device and agree in B, H_kv and d")
    _cache_call("focus_cache_evict", p, src, ws, stream, int(budget), int(recent), src.ref, dst.ref)


def run_decode_step(p: Params, h, W, C, Q, K, V, cache: Cache, ws, ws_cache, n_new=None, want_lse=False,
                    accumulate=False, stream=None):
    """assign -> append -> attention for p.n new tokens a sequence; returns (O,
    gid, lse).  ws: a workspace of alloc_workspace(p); ws_cache: one of
    alloc_workspace_cache(p, cache).  Rows behind n_new[b] of O are 0."""
    dev = cache.device
    with torch.cuda.device(dev), torch.cuda.stream(stream):      # the fills below run on the call's stream
        gid = torch.empty((p.B, p.A, p.n), dtype=torch.int32, device=dev)
        O = torch.empty_like(Q) if n_new is None else torch.zeros_like(Q)
        lse = None
        if want_lse:
            lse = torch.full((p.B, p.H, p.n), float("-inf"), dtype=torch.float32, device=dev)
        focus_assign(p, h, W, C, gid, ws, stream)
        focus_cache_append(p, K, V, gid, cache, ws_cache, n_new=n_new, stream=stream)
        focus_cache_attention_fwd(p, Q, gid, cache, O, lse, ws_cache, n_new=n_new, accumulate=accumulate,
                                  stream=stream)
    return O, gid, lse


# ------------------------------------------------------------ index views ---

def index_views(p: Params, idx: Index, ws: torch.Tensor, n: int | None = None,
                K: int | None = None) -> dict:
    """Torch views (no copy) of the index arrays living inside the workspace.
    n: sorted items per (b, a) (p.n; n * k for a top-k entry index); K: groups
    (p.K; K (K - 1) / 2 for a top-2 pair index)."""
    base = ws.data_ptr()
    P = p.B * p.A
    n = p.n if n is None else n
    K = p.K if K is None else K

    def view(ptr, count, dtype=torch.int32, shape=None):
        off = ptr - base
        t = ws[off:off + count * 4].view(dtype)
        return t.view(*shape) if shape else t

    out = dict(counts=view(idx.counts, P * K, shape=(p.B, p.A, K)),
               offsets=view(idx.offsets, P * (K + 1), shape=(p.B, p.A, K + 1)),
               perm=view(idx.perm, P * n, shape=(p.B, p.A, n)),
               rank=view(idx.rank, P * n, shape=(p.B, p.A, n)),
               farlen_tok=view(idx.farlen_tok, P * n, shape=(p.B, p.A, n)),
               farlen_slot=view(idx.farlen_slot, P * n, shape=(p.B, p.A, n)),
               n_items=view(idx.n_items, 1))
    m = idx.max_items
    out["items"] = view(idx.items, m * 8, shape=(m, 8))
    out["order"] = view(idx.order, m)
    return out


def run_layer(p: Params, h, W, C, Q, K, V, ws, stream=None, want_lse=False):
    """assign -> index -> attention on device tensors; returns (O, gid, idx, lse)."""
    dev = Q.device
    gid = torch.empty((p.B, p.A, p.n), dtype=torch.int32, device=dev)
    focus_assign(p, h, W, C, gid, ws, stream)
    idx = focus_build_index(p, gid, ws, stream)
    O = torch.empty_like(Q)
    lse = torch.empty((p.B, p.H, p.n), dtype=torch.float32, device=dev) if want_lse else None
    focus_attention_fwd(p, Q, K, V, idx, O, lse, ws, stream)
    return O, gid, idx, lse
