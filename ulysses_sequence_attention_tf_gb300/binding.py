"""Thin ctypes binding of ``libtf_ulysses.so`` (the C ABI in include/tf_ulysses.h).

Argument marshalling only: torch supplies device memory, streams and the
tensors' data pointers/strides; every step of the relayout runs in the
library's CUDA kernels.  There is no fallback: if the library is missing or a
call fails, a ``TfUlyssesError`` is raised.

Names follow the C ABI: ``scatter_qkv`` / ``scatter_qkv_into`` / ``gather_out``
/ ``rope_table`` / ``cache_clear`` ...
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# the in-tree build, or another build of the same library named by TF_ULYSSES_LIBRARY
LIB_PATH = os.environ.get("TF_ULYSSES_LIBRARY") or os.path.join(_PKG, "libtf_ulysses.so")

TF_OK, TF_ERR_INVALID, TF_ERR_DIVISIBILITY, TF_ERR_ALIGNMENT = 0, 1, 2, 3
TF_ERR_UNSUPPORTED, TF_ERR_OOM, TF_ERR_CUDA, TF_ERR_BUSY = 4, 5, 6, 7
STATUS_NAMES = {0: "TF_OK", 1: "TF_ERR_INVALID", 2: "TF_ERR_DIVISIBILITY", 3: "TF_ERR_ALIGNMENT",
                4: "TF_ERR_UNSUPPORTED", 5: "TF_ERR_OOM", 6: "TF_ERR_CUDA", 7: "TF_ERR_BUSY"}
TF_MODE_SCATTER, TF_MODE_SCATTER_NORM_ROPE, TF_MODE_GATHER = 0, 1, 2
TF_MODE_FLAG_FUSED_LAYOUT, TF_MODE_FLAG_ROPE_NEOX = 0x100, 0x200
MAX_SHARDS = 8
CACHE_CAPACITY = 12

_DTYPE_CODE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.int32: 2,
               torch.uint8: 3, torch.int8: 3}
for _name in ("float8_e4m3fn", "float8_e5m2"):
    if hasattr(torch, _name):
        _DTYPE_CODE[getattr(torch, _name)] = 3


class TfUlyssesError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64), ("h", ctypes.c_int64)]


class NormRope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("theta", ctypes.c_float), ("cos_sin", ctypes.c_void_p)]


class Targets(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p * MAX_SHARDS), ("k", ctypes.c_void_p * MAX_SHARDS),
                ("v", ctypes.c_void_p * MAX_SHARDS), ("done", ctypes.c_void_p)]


class Attention(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("P", "B", "Sq", "Sk", "H", "Hkv", "D", "dtype")] + \
               [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("causal", ctypes.c_int)] + \
               [(n, ctypes.c_void_p) for n in ("slopes", "prefix", "q_docs", "k_docs")]


class KvCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
               [(n, ctypes.c_int) for n in ("num_pages", "Hkv", "page_size", "D", "N", "max_pages")] + \
               [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("starts", ctypes.c_void_p)]


class KvAttention(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("P", "T", "H", "dtype", "max_tokens", "max_len")] + \
               [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("causal", ctypes.c_int), ("slopes", ctypes.c_void_p)]


class KvPlan(NamedTuple):
    """What ``kv_plan`` gives: int32 ``lens [N]``, ``starts [N + 1]``, ``positions [rows]``, ``slots [rows]``, ``span [2]``."""
    lens: torch.Tensor
    starts: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    span: torch.Tensor


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("N", "max_pages", "page_size", "num_pages", "T")] + \
               [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64)] + \
               [(n, ctypes.c_void_p) for n in ("lens", "new_tokens", "free_pages", "free_span", "lens_out", "starts", "positions",
                                               "slots", "span_out")]


class Rotary(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("P", "B", "T", "H", "Hk", "D", "rotary_dim", "dtype", "rope", "inverse")] + \
               [("magnitude", ctypes.c_float), ("frequencies", ctypes.POINTER(ctypes.c_double)), ("positions", ctypes.c_void_p),
                ("first", ctypes.c_int)]


class Linear(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("P", "B", "S", "H", "D", "dtype")] + \
               [("scale", ctypes.c_float), ("decay", ctypes.c_void_p)]


class LinearPool(ctypes.Structure):
    _fields_ = [("states", ctypes.c_void_p), ("num_slots", ctypes.c_int), ("N", ctypes.c_int), ("slots", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("max_tokens", ctypes.c_int)]


class PagedCache(NamedTuple):
    """A paged key-value cache: e4m3 codes ``[pages, Hkv, page_size, D]`` and their fp32 scales ``[pages, Hkv]``."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


ALLOC_FN = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p)
FREE_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p)

_lock = threading.Lock()
_lib = None


def _declare(lib):
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    PP = ctypes.POINTER(ctypes.c_void_p)
    lib.tf_ulysses_scatter_qkv.argtypes = [ctypes.c_char_p, PP, PP, PP, ctypes.POINTER(Strides),
                                           i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(NormRope),
                                           vp, ctypes.POINTER(Targets)]
    lib.tf_ulysses_scatter_qkv_into.argtypes = [PP, PP, PP, ctypes.POINTER(Strides), i32, i32, i32, i32, i32,
                                                i32, i32, ctypes.POINTER(NormRope), PP, PP, PP, vp]
    lib.tf_ulysses_scatter_qkv_noalloc.argtypes = lib.tf_ulysses_scatter_qkv_into.argtypes
    lib.tf_ulysses_scatter_qkv_heads_into.argtypes = [PP, PP, PP, ctypes.POINTER(Strides), i32, i32, i32, i32, i32,
                                                      i32, i32, ctypes.POINTER(NormRope), i32, i32, PP, PP, PP, vp]
    lib.tf_ulysses_exchange_chunks.argtypes = [PP, PP, i32, ctypes.c_size_t, vp]
    lib.tf_ulysses_project_qkv_into.argtypes = [PP, i64, vp, i64, i32, i32, i32, i32, i32, i32, i32, i32,
                                                ctypes.POINTER(NormRope), PP, PP, PP, vp]
    lib.tf_ulysses_gather_out.argtypes = [ctypes.c_char_p, PP, ctypes.POINTER(Strides), i32, i32, i32, i32, i32,
                                          i32, PP, ctypes.POINTER(Strides), vp, ctypes.POINTER(Targets)]
    lib.tf_ulysses_rope_table.argtypes = [ctypes.c_float, i32, i32, vp, ctypes.POINTER(ctypes.c_void_p)]
    AP, SP, size_t = ctypes.POINTER(Attention), ctypes.POINTER(Strides), ctypes.c_size_t
    lib.tf_ulysses_attention.argtypes = [AP, PP, PP, PP, SP, PP, SP, PP, vp, size_t, vp]
    lib.tf_ulysses_attention_backward.argtypes = [AP, PP, PP, PP, PP, PP, PP, SP, PP, PP, PP, SP, vp, size_t, vp]
    lib.tf_ulysses_attention_workspace.argtypes = [AP, i32, ctypes.POINTER(size_t)]
    CP, KP = ctypes.POINTER(KvCache), ctypes.POINTER(KvAttention)
    lib.tf_ulysses_kv_append.argtypes = [CP, i32, i32, i32, i32, PP, PP, PP, SP, PP, SP, ctypes.POINTER(NormRope), i32,
                                         i32, vp]
    lib.tf_ulysses_kv_attend.argtypes = [CP, KP, PP, SP, PP, SP, PP, vp, size_t, vp]
    lib.tf_ulysses_kv_attend_workspace.argtypes = [CP, KP, ctypes.POINTER(size_t)]
    lib.tf_ulysses_kv_plan.argtypes = [ctypes.POINTER(Plan), vp]
    lib.tf_ulysses_rope.argtypes = [ctypes.POINTER(Rotary), PP, PP, SP, PP, PP, SP, vp]
    f64 = ctypes.c_double
    lib.tf_ulysses_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, ctypes.POINTER(f64)]
    LP, OP = ctypes.POINTER(Linear), ctypes.POINTER(LinearPool)
    lib.tf_ulysses_linear_attention.argtypes = [LP, PP, PP, PP, SP, vp, PP, SP, vp, vp, size_t, vp]
    lib.tf_ulysses_linear_attention_backward.argtypes = [LP, PP, PP, PP, PP, SP, vp, vp, PP, PP, PP, SP, vp, vp, size_t, vp]
    lib.tf_ulysses_linear_attention_workspace.argtypes = [LP, i32, ctypes.POINTER(size_t)]
    lib.tf_ulysses_linear_attend.argtypes = [LP, OP, PP, PP, PP, SP, PP, SP, vp, size_t, vp]
    lib.tf_ulysses_linear_attend_workspace.argtypes = [LP, OP, ctypes.POINTER(size_t)]
    for name in ("tf_ulysses_kv_plan", "tf_ulysses_rope", "tf_ulysses_rope_frequencies", "tf_ulysses_linear_attention",
                 "tf_ulysses_linear_attention_backward", "tf_ulysses_linear_attention_workspace", "tf_ulysses_linear_attend",
                 "tf_ulysses_linear_attend_workspace", "tf_ulysses_kv_append", "tf_ulysses_kv_attend", "tf_ulysses_kv_attend_workspace",
                 "tf_ulysses_attention", "tf_ulysses_attention_backward", "tf_ulysses_attention_workspace",
                 "tf_ulysses_scatter_qkv_heads_into", "tf_ulysses_exchange_chunks", "tf_ulysses_project_qkv_into",
                 "tf_ulysses_scatter_qkv", "tf_ulysses_scatter_qkv_into", "tf_ulysses_scatter_qkv_noalloc",
                 "tf_ulysses_gather_out",
                 "tf_ulysses_rope_table", "tf_ulysses_cache_clear"):
        getattr(lib, name).restype = i32
    lib.tf_ulysses_cache_clear.argtypes = []
    lib.tf_ulysses_cache_entries.argtypes = []
    lib.tf_ulysses_cache_entries.restype = i32
    lib.tf_ulysses_set_allocator.argtypes = [ALLOC_FN, FREE_FN, vp]
    lib.tf_ulysses_set_allocator.restype = None
    lib.tf_ulysses_device_status.argtypes = [i32, ctypes.POINTER(ctypes.c_uint)]
    lib.tf_ulysses_device_status.restype = i32
    lib.tf_ulysses_last_error.argtypes = []
    lib.tf_ulysses_last_error.restype = ctypes.c_char_p
    lib.tf_ulysses_launch_count.argtypes = []
    lib.tf_ulysses_launch_count.restype = ctypes.c_uint64
    lib.tf_ulysses_selftest_wait.argtypes = [ctypes.c_ulonglong, vp]
    lib.tf_ulysses_selftest_wait.restype = i32
    lib.tf_ulysses_set_slots.argtypes = [ctypes.c_char_p, i32]
    lib.tf_ulysses_set_slots.restype = i32
    lib.tf_ulysses_alloc_count.argtypes = []
    lib.tf_ulysses_alloc_count.restype = ctypes.c_uint64
    lib.tf_ulysses_abi_version.argtypes = []
    lib.tf_ulysses_abi_version.restype = i32
    return lib


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise TfUlyssesError(TF_ERR_INVALID, f"{LIB_PATH} is not built (run __graft_entry__.build())")
                _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def _check(status: int):
    if status != TF_OK:
        raise TfUlyssesError(status, lib().tf_ulysses_last_error().decode(errors="replace"))


# ---------------------------------------------------------------- marshalling
def _ptr_array(ts):
    if ts is None:
        return None
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def _strides_of(ts, ndim_names="[B, tokens, heads, D]"):
    s = ts[0].stride()
    if ts[0].dim() != 4:
        raise ValueError(f"expected 4-d views {ndim_names}")
    if ts[0].shape[-1] > 1 and s[3] != 1:
        raise ValueError("the D dimension must have stride 1")
    for t in ts[1:]:
        if t.stride() != s or t.shape != ts[0].shape or t.dtype != ts[0].dtype:
            raise ValueError("all shards of a tensor must share shape, dtype and strides")
    return Strides(s[0], s[1], s[2])


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


class _DeviceBuffer:
    """Zero-copy view of library-owned device memory for torch.as_tensor."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr, "data": (ptr, False),
                                         "version": 2, "strides": None}


# Flat tensors over library-owned memory, by (address, elements, dtype, device).
# Cached targets come back at the same addresses call after call, so their views
# are cut from a cached flat tensor instead of being built from the array
# interface each time; a view owns no memory, so an entry whose memory was freed
# and reused still views exactly that address range.
_WRAP_CACHE = {}
_WRAP_CACHE_MAX = 4096


def _wrap(ptr, shape, dtype, device):
    if not ptr or 0 in shape:
        return torch.empty(shape, dtype=dtype, device=device)
    numel = 1
    for n in shape:
        numel *= n
    key = (ptr, numel, dtype, device)
    flat = _WRAP_CACHE.get(key)
    if flat is None:
        esize = torch.empty((), dtype=dtype).element_size()
        typestr = {1: "|u1", 2: "<i2", 4: "<i4", 8: "<i8"}[esize]
        with torch.cuda.device(device):
            flat = torch.as_tensor(_DeviceBuffer(ptr, (numel,), typestr), device=device).view(dtype)
        if len(_WRAP_CACHE) >= _WRAP_CACHE_MAX:
            _WRAP_CACHE.clear()
        _WRAP_CACHE[key] = flat
    return flat.view(shape)


def _dtype_code(dtype):
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}")
    return _DTYPE_CODE[dtype]


def _norm_rope(q_weight, k_weight, eps, theta, cos_sin):
    nr = NormRope()
    nr.q_weight = q_weight.data_ptr() if q_weight is not None else None
    nr.k_weight = k_weight.data_ptr() if k_weight is not None else None
    nr.eps = float(eps)
    nr.theta = float(theta)
    nr.cos_sin = cos_sin.data_ptr() if cos_sin is not None else None
    return nr


def _scatter_args(q, k, v):
    P = len(q)
    if not 1 <= P <= MAX_SHARDS:
        raise ValueError(f"P={P} outside [1, {MAX_SHARDS}]")
    B, Sl, H, D = q[0].shape
    strides = (Strides * 3)()
    for i, ts in enumerate((q, k, v)):
        if ts is None:
            continue
        if len(ts) != P or ts[0].shape != q[0].shape or ts[0].dtype != q[0].dtype:
            raise ValueError("q, k and v must have P shards of the same shape and dtype")
        strides[i] = _strides_of(ts)
    return P, B, Sl, H, D, strides


def _mode(norm_rope, rope, layout):
    if rope not in ("interleaved", "neox"):
        raise ValueError(f"rope must be 'interleaved' or 'neox', not {rope!r}")
    if layout not in ("bshd", "fused"):
        raise ValueError(f"layout must be 'bshd' or 'fused', not {layout!r}")
    mode = TF_MODE_SCATTER_NORM_ROPE if norm_rope else TF_MODE_SCATTER
    if rope == "neox":
        mode |= TF_MODE_FLAG_ROPE_NEOX  # the library rejects it without norm_rope
    if layout == "fused":
        mode |= TF_MODE_FLAG_FUSED_LAYOUT
    return mode


def _check_targets(outs, layout):
    for o in outs:
        if o is not None and any(not t.is_contiguous() for t in o):
            raise ValueError("targets must be contiguous " +
                             ("[B, S, H/P, 3*D] payloads" if layout == "fused" else "[B, S, H/P, D]"))


# ---------------------------------------------------------------- public API
def scatter_qkv(tag, q, k=None, v=None, *, norm_rope=False, q_weight=None, k_weight=None, eps=1e-6,
                theta=10000.0, cos_sin=None, rope="interleaved", layout="bshd", stream=None):
    """Sequence->head scatter of P shards ``[B, S_local, H, D]`` of Q (and K, V)
    into cached final-layout targets, in one launch.

    Returns ``(q_targets, k_targets, v_targets, done_event_handle)``: lists of P
    ``[B, P*S_local, H/P, D]`` tensors viewing library-owned memory (valid until the
    next call with the same key, eviction or ``cache_clear``), ``None`` for absent
    tensors.  With ``norm_rope=True``, Q and K get RMSNorm (eps, q_weight/k_weight)
    and RoPE at global positions (theta, or an fp32 ``cos_sin`` table
    ``[>= S, D/2, 2]``), pairs (2i, 2i+1) for ``rope="interleaved"`` or (i, i + D/2)
    for ``rope="neox"``; V is copied bit for bit.  ``layout="fused"`` (q, k, v
    all required) writes one ``[B, S, H/P, 3*D]`` payload per head group and returns
    Q, K and V as views into it (``fused_payloads`` recovers the payloads).
    """
    P, B, Sl, H, D, strides = _scatter_args(q, k, v)
    mode = _mode(norm_rope, rope, layout)
    nr = _norm_rope(q_weight, k_weight, eps, theta, cos_sin) if norm_rope else None
    out = Targets()
    _check(lib().tf_ulysses_scatter_qkv(
        tag.encode() if isinstance(tag, str) else tag, _ptr_array(q), _ptr_array(k), _ptr_array(v), strides,
        P, B, Sl, H, D, _dtype_code(q[0].dtype), mode, ctypes.byref(nr) if nr is not None else None,
        _stream_handle(stream), ctypes.byref(out)))
    S, Hl = P * Sl, H // P
    dev = q[0].device
    if layout == "fused":
        pay = [_wrap(out.q[g], (B, S, Hl, 3 * D), q[0].dtype, dev) for g in range(P)]
        return ([t[..., :D] for t in pay], [t[..., D:2 * D] for t in pay], [t[..., 2 * D:] for t in pay],
                out.done)
    res = []
    for arr, ts in ((out.q, q), (out.k, k), (out.v, v)):
        res.append(None if ts is None else [_wrap(arr[g], (B, S, Hl, D), q[0].dtype, dev) for g in range(P)])
    return res[0], res[1], res[2], out.done


def fused_payloads(q_targets):
    """The ``[B, S, H/P, 3*D]`` payloads behind the Q views returned by
    ``scatter_qkv(..., layout="fused")``."""
    res = []
    for t in q_targets:
        B, S, Hl, D = t.shape
        if t.stride() != (S * Hl * 3 * D, Hl * 3 * D, 3 * D, 1):
            raise ValueError("not a Q view of a fused-layout payload")
        res.append(t.as_strided((B, S, Hl, 3 * D), (S * Hl * 3 * D, Hl * 3 * D, 3 * D, 1)))
    return res


def scatter_qkv_into(q, k, v, q_out, k_out=None, v_out=None, *, norm_rope=False, q_weight=None, k_weight=None,
                     eps=1e-6, theta=10000.0, cos_sin=None, rope="interleaved", layout="bshd", stream=None):
    """Same scatter into caller-owned contiguous targets ``[B, P*S_local, H/P, D]``;
    with ``layout="fused"``, ``q_out`` holds the P payloads ``[B, P*S_local, H/P, 3*D]``
    and ``k_out``, ``v_out`` stay None."""
    P, B, Sl, H, D, strides = _scatter_args(q, k, v)
    _check_targets((q_out, k_out, v_out), layout)
    mode = _mode(norm_rope, rope, layout)
    nr = _norm_rope(q_weight, k_weight, eps, theta, cos_sin) if norm_rope else None
    _check(lib().tf_ulysses_scatter_qkv_into(
        _ptr_array(q), _ptr_array(k), _ptr_array(v), strides, P, B, Sl, H, D, _dtype_code(q[0].dtype), mode,
        ctypes.byref(nr) if nr is not None else None, _ptr_array(q_out), _ptr_array(k_out), _ptr_array(v_out),
        _stream_handle(stream)))
    return q_out, k_out, v_out


def scatter_qkv_noalloc(q, k, v, q_out, k_out=None, v_out=None, *, norm_rope=False, q_weight=None, k_weight=None,
                        eps=1e-6, theta=10000.0, cos_sin=None, rope="interleaved", layout="bshd", stream=None):
    """``scatter_qkv_into`` for callers that cannot allocate device memory: the
    library allocates nothing; a needed cos/sin table lives in the library's
    fixed 16 MiB device scratch (P*S_local*D <= 4 Mi floats), rebuilt only when
    it does not already hold this (theta, rows, D).  A rebuild whose work
    overlaps on the GPU with another call's scatter races with it."""
    P, B, Sl, H, D, strides = _scatter_args(q, k, v)
    _check_targets((q_out, k_out, v_out), layout)
    mode = _mode(norm_rope, rope, layout)
    nr = _norm_rope(q_weight, k_weight, eps, theta, cos_sin) if norm_rope else None
    _check(lib().tf_ulysses_scatter_qkv_noalloc(
        _ptr_array(q), _ptr_array(k), _ptr_array(v), strides, P, B, Sl, H, D, _dtype_code(q[0].dtype), mode,
        ctypes.byref(nr) if nr is not None else None, _ptr_array(q_out), _ptr_array(k_out), _ptr_array(v_out),
        _stream_handle(stream)))
    return q_out, k_out, v_out


def scatter_qkv_heads_into(q, k, v, q_out, k_out=None, v_out=None, *, h0, h1, norm_rope=False, q_weight=None,
                           k_weight=None, eps=1e-6, theta=10000.0, cos_sin=None, rope="interleaved", layout="bshd",
                           stream=None):
    """``scatter_qkv_into`` restricted to heads [h0, h1) of every head band: those
    heads of the caller's targets are written, every other element is kept."""
    P, B, Sl, H, D, strides = _scatter_args(q, k, v)
    _check_targets((q_out, k_out, v_out), layout)
    mode = _mode(norm_rope, rope, layout)
    nr = _norm_rope(q_weight, k_weight, eps, theta, cos_sin) if norm_rope else None
    _check(lib().tf_ulysses_scatter_qkv_heads_into(
        _ptr_array(q), _ptr_array(k), _ptr_array(v), strides, P, B, Sl, H, D, _dtype_code(q[0].dtype), mode,
        ctypes.byref(nr) if nr is not None else None, int(h0), int(h1), _ptr_array(q_out), _ptr_array(k_out),
        _ptr_array(v_out), _stream_handle(stream)))
    return q_out, k_out, v_out


def project_qkv_into(x, w_qkv, H, q_out, k_out=None, v_out=None, *, norm_rope=False, q_weight=None, k_weight=None,
                     eps=1e-6, theta=10000.0, cos_sin=None, rope="interleaved", layout="bshd", stream=None):
    """QKV projection fused with the scatter: ``x`` is P shards ``[B, S_local,
    hidden]`` (bf16, unit stride along hidden, rows of one shard equally spaced),
    ``w_qkv`` the ``[3*H*D, hidden]`` weight (nn.Linear layout, D = 128).  Q, K, V
    head rows land in the targets as ``scatter_qkv_into`` writes them, after the
    RMSNorm + RoPE on Q/K when ``norm_rope``."""
    P = len(x)
    B, Sl, hidden = x[0].shape
    for t in x:
        if t.shape != x[0].shape or t.stride() != x[0].stride() or t.dtype != x[0].dtype:
            raise ValueError("all x shards must share shape, strides and dtype")
    if x[0].stride(2) != 1 or (B > 1 and x[0].stride(0) != Sl * x[0].stride(1)):
        raise ValueError("x rows must be equally spaced with unit stride along hidden")
    if w_qkv.stride(1) != 1:
        raise ValueError("w_qkv needs unit stride along hidden")
    D = w_qkv.shape[0] // (3 * H)
    _check_targets((q_out, k_out, v_out), layout)
    mode = _mode(norm_rope, rope, layout)
    nr = _norm_rope(q_weight, k_weight, eps, theta, cos_sin) if norm_rope else None
    _check(lib().tf_ulysses_project_qkv_into(
        _ptr_array(x), x[0].stride(1) if Sl > 1 or B > 1 else hidden, ctypes.c_void_p(w_qkv.data_ptr()),
        w_qkv.stride(0), P, B, Sl, hidden, H, D, _dtype_code(x[0].dtype), mode,
        ctypes.byref(nr) if nr is not None else None, _ptr_array(q_out), _ptr_array(k_out), _ptr_array(v_out),
        _stream_handle(stream)))
    return q_out, k_out, v_out


def exchange_chunks(src, dst=None, *, stream=None):
    """All-to-all over destination-major payloads: P tensors ``src[r]`` of P equal
    chunks (chunk g goes to rank g) -> ``dst[g]`` holding chunk g of every rank in
    rank order.  Tensors must be contiguous with P*chunk bytes, chunk a multiple
    of 16 bytes; ``dst`` defaults to new tensors shaped like ``src``."""
    P = len(src)
    if any(not t.is_contiguous() or t.shape != src[0].shape or t.dtype != src[0].dtype for t in src):
        raise ValueError("src must be P contiguous tensors of one shape and dtype")
    nbytes = src[0].numel() * src[0].element_size()
    if nbytes % P:
        raise ValueError("a payload must split into P equal chunks")
    if dst is None:
        dst = [torch.empty_like(t) for t in src]
    if any(not t.is_contiguous() or t.numel() * t.element_size() != nbytes for t in dst):
        raise ValueError("dst must be P contiguous tensors of the payload size")
    _check(lib().tf_ulysses_exchange_chunks(_ptr_array(src), _ptr_array(dst), P, nbytes // P, _stream_handle(stream)))
    return dst


def gather_out(tag, attn, out=None, *, stream=None):
    """Head->sequence gather of P head-group outputs ``[B, S, H/P, D]`` into P shard
    outputs ``[B, S/P, H, D]`` -- cached library buffers, or ``out`` (P caller tensors,
    any strides with unit D stride).  Returns ``(outputs, done_event_handle)``."""
    P = len(attn)
    B, S, Hl, D = attn[0].shape
    if S % P:
        raise ValueError(f"S={S} is not divisible by P={P}")
    Sl, H = S // P, Hl * P
    a_str = _strides_of(attn)
    o_str = _strides_of(out) if out is not None else None
    res = Targets()
    _check(lib().tf_ulysses_gather_out(
        tag.encode() if isinstance(tag, str) else tag, _ptr_array(attn), ctypes.byref(a_str), P, B, Sl, H, D,
        _dtype_code(attn[0].dtype), _ptr_array(out), ctypes.byref(o_str) if o_str is not None else None,
        _stream_handle(stream), ctypes.byref(res)))
    if out is not None:
        return list(out), res.done
    return [_wrap(res.q[r], (B, Sl, H, D), attn[0].dtype, attn[0].device) for r in range(P)], res.done


# ---------------------------------------------------------------- attention and key-value cache
# These calls are short on the GPU: their checks and marshalling are in csrc/torch_calls.cpp.  Results of a call of the rotation,
# linear attention and the plan that are made there share one allocation up to 1 MiB altogether: one that is kept keeps the others'
# memory, and torch.save writes all of it.  clone() what is kept for long, or give the result.
_calls = None


def _torch_calls():
    """The module that marshals these calls, bound to the library's entry points; raises if it has not been built."""
    global _calls
    if _calls is None:
        L = lib()
        try:
            from . import _torch_calls as module
        except ImportError as e:
            raise TfUlyssesError(TF_ERR_INVALID, f"_torch_calls is not built (run __graft_entry__.build()): {e}") from e
        names = ("attention", "attention_backward", "attention_workspace", "kv_append", "kv_attend", "kv_attend_workspace",
                 "kv_plan", "rope", "rope_frequencies", "linear_attention", "linear_attention_backward",
                 "linear_attention_workspace", "linear_attend", "linear_attend_workspace")
        module.bind(_check, *[ctypes.cast(getattr(L, "tf_ulysses_" + n), ctypes.c_void_p).value for n in names])
        _calls = module
    return _calls


def _on_stream(stream):
    """The stream of a call as a context in which torch allocates for it, so that memory which the call's kernels use
    returns to the allocator in that stream's order."""
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _run(name, stream, before, after):
    """``name`` of the module with the device and the stream of the call between its arguments."""
    call = getattr(_calls or _torch_calls(), name)
    if stream is None:
        return _on_device(call, before, after)
    with _on_stream(stream):  # whose device is current in here
        return _on_device(call, before, after)


def _on_device(call, before, after):
    device = torch._C._cuda_getDevice()
    return call(*before, device, torch._C._cuda_getCurrentRawStream(device), *after)


def attention(q, k, v, out=None, lse=None, *, scale=None, softcap=0.0, slopes=None, causal=False, prefix=None,
              q_docs=None, k_docs=None, stream=None):
    """Attention over P head groups: ``q`` P views ``[B, Sq, H/P, D]``, ``k`` and ``v`` P views
    ``[B, Sk, Hkv/P, D]`` (bf16 or fp16, D 64 or 128; H/Hkv query heads share a key head).

    Scores are ``scale * q.k`` (default 1/sqrt(D)), capped to ``softcap * tanh(x / softcap)``
    where softcap > 0, plus ``-slopes[h] * |i + Sk - Sq - j|`` (``slopes``: fp32 ``[H]``).
    ``causal``: key j is visible up to position i + Sk - Sq, and below ``prefix[b]`` (int32
    ``[B]``) always.  ``q_docs`` / ``k_docs`` (int32 ``[B, Sq]``, ``[B, Sk]``): only equal
    document numbers see one another; negative ones are padding.  Returns ``(out, lse)``:
    P tensors ``[B, Sq, H/P, D]`` and fp32 ``[B, H/P, Sq]``, 0 and -inf for rows that see
    nothing; both are made here unless given.  The call is not recorded by autograd, also where a tensor requires a
    gradient: ``attention_backward`` gives the gradients.
    """
    return _run("attention", stream, (q, k, v, scale, softcap, slopes, causal, prefix, q_docs, k_docs), (out, lse))


def attention_backward(dout, q, k, v, out, lse, dq=None, dk=None, dv=None, *, scale=None, softcap=0.0, slopes=None,
                       causal=False, prefix=None, q_docs=None, k_docs=None, stream=None):
    """Gradients ``(dq, dk, dv)`` of ``attention`` for the gradient ``dout`` of its output, from
    the same inputs and options and its results ``out`` and ``lse`` (not those of more keys): lists of P tensors
    shaped like q, k and v, made here unless given.  Shared key heads get the sum over
    their query heads.  The same inputs give the same bits.  Not recorded by autograd."""
    return _run("attention_backward", stream, (q, k, v, scale, softcap, slopes, causal, prefix, q_docs, k_docs),
                (dout, out, lse, dq, dk, dv))


_ROPE = {None: 0, "interleaved": 1, "neox": 2}


def kv_cache(num_pages, Hkv, page_size, D, *, device="cuda"):
    """A paged cache of ``num_pages`` pages of ``page_size`` (16, 32, 64 or 128) tokens for ``Hkv`` key heads
    (over all head groups) of D 64 or 128.  Pages need no clearing: the first append to a page sets it up."""
    codes = lambda: torch.zeros((num_pages, Hkv, page_size, D), dtype=torch.float8_e4m3fn, device=device)  # noqa: E731
    scales = lambda: torch.ones((num_pages, Hkv), dtype=torch.float32, device=device)  # noqa: E731
    return PagedCache(codes(), codes(), scales(), scales())


def kv_append(cache, page_table, lens, starts, k, v, q=None, q_out=None, *, q_weight=None, k_weight=None, eps=1e-6,
              theta=10000.0, cos_sin=None, rope="interleaved", stream=None):
    """Append new rows to a paged cache (``kv_cache``): ``k`` and ``v`` are P row views ``[T, Hkv/P, D]`` whose rows
    ``[starts[n], starts[n + 1])`` are the newest tokens of sequence n, of length ``lens[n]`` with them, in the pages
    of row n of ``page_table`` (int32 ``[N, max_pages]``; ``lens`` int32 ``[N]``, ``starts`` int32 ``[N + 1]``).

    K is normalised (``k_weight`` given) and rotated at its token's position (``rope`` "interleaved", "neox" or None;
    the table ``cos_sin`` fp32 ``[rows, D/2, 2]`` or the resident one of theta) before it is stored; the queries
    ``q`` ``[T, H/P, D]`` of the same tokens likewise into ``q_out`` (made here unless given; ``q`` itself is fine).
    Returns ``q_out``, or None without q.
    """
    if rope not in _ROPE:
        raise ValueError(f"rope must be 'interleaved', 'neox' or None, not {rope!r}")
    return _run("kv_append", stream, (*cache, page_table, lens, starts),
                (k, v, q, q_out, q_weight, k_weight, eps, theta, cos_sin, _ROPE[rope]))


def kv_attend(cache, page_table, lens, starts, q, out=None, lse=None, *, max_tokens=None, max_len=None, scale=None,
              softcap=0.0, slopes=None, causal=True, stream=None):
    """Attention of each sequence's newest tokens over its cached keys and values (their own appended before):
    ``q`` P row views ``[T, H/P, D]``, rows as in ``kv_append``.  Score options are those of ``attention``, positions
    those in the sequence; ``causal=False`` lets a token see all ``lens[n]`` keys.  ``max_tokens`` and ``max_len`` bound
    the new tokens and the length of one sequence (default: T and the table's width); tight ones spare work.
    Returns ``(out, lse)``: P tensors ``[T, H/P, D]`` and fp32 ``[H/P, T]``, made here unless given (rows of no sequence
    are then undefined; given tensors keep them).
    """
    return _run("kv_attend", stream, (*cache, page_table, lens, starts),
                (q, out, lse, max_tokens, max_len, scale, softcap, slopes, causal))


def kv_plan(page_table, lens, new, free, span, *, page_size, rows, lens_out=None, starts=None, positions=None, slots=None,
            span_out=None, stream=None):
    """What a step's requests need of a paged cache, built on the device from their lengths: ``lens`` (int32 ``[N]``)
    tokens so far and ``new`` (int32 ``[N]``) tokens that each one gets now, or a negative number where it has ended.

    ``free`` (int32 ``[num_pages]``) is a ring of free page numbers, ``span`` (int32 ``[2]``) its head and how many are
    free.  New pages go into ``page_table`` (int32 ``[N, max_pages]``), those of ended requests back into ``free``; both are
    written in place, ``lens`` and ``span`` are not.  Returns ``KvPlan(lens, starts, positions, slots, span)``: the new
    lengths, the first row of each request among ``rows`` (the ``lens`` and ``starts`` of ``kv_append``), each row's position
    (that of ``rope``) and its slot ``page * page_size + position % page_size``, 0 and -1 behind the last, and the ring's new
    span.  They are made here unless given.  Requests are served in order: where pages or rows run out, the first one
    that does not fit and all behind it get nothing, which their ``starts`` tell.  The results made here share one allocation.
    """
    return KvPlan(*_run("kv_plan", stream, (page_table, lens, new, free, span),
                        (page_size, rows, lens_out, starts, positions, slots, span_out)))


_ROPE_SCALE = {None: 0, "linear": 1, "base": 2, "parts": 3}


def rope_frequencies(rotary_dim, theta=10000.0, *, scaling=None, factor=1.0, original=4096, low=1.0, high=32.0):
    """Frequencies ``[rotary_dim / 2]`` (float64 on the CPU) for ``rope``: ``theta^(-2i / rotary_dim)``, for contexts longer
    than the trained one divided by ``factor`` ("linear"), with a larger base ("base"), or divided for the
    pairs only that turn less than ``low`` times in ``original`` tokens, kept above ``high``, in between by parts ("parts",
    which goes with a magnitude of ``0.1 * log(factor) + 1`` as a rule)."""
    if scaling not in _ROPE_SCALE:
        raise ValueError(f"scaling must be 'linear', 'base', 'parts' or None, not {scaling!r}")
    if not -2 ** 31 <= rotary_dim < 2 ** 31:
        raise ValueError(f"rotary_dim={rotary_dim} is out of range")
    out = (ctypes.c_double * 128)()
    _check(lib().tf_ulysses_rope_frequencies(int(rotary_dim), float(theta), _ROPE_SCALE[scaling], float(factor), float(original),
                                             float(low), float(high), out))
    return torch.tensor(out[:rotary_dim // 2], dtype=torch.float64)


def rope(q, k=None, q_out=None, k_out=None, *, positions=None, first=0, frequencies=None, rotary_dim=None, theta=10000.0,
         magnitude=1.0, rope="interleaved", inverse=False, stream=None):
    """Rotary positions of P head groups: ``q`` and ``k`` P views ``[B, tokens, heads/P, D]`` or rows ``[T, heads/P, D]``
    (bf16 or fp16, D a multiple of 8 up to 256), at ``positions`` (int32 ``[B, tokens]`` or ``[T]``) or ``first + token``.

    Pairs (2i, 2i+1) ("interleaved") or (i, i + R/2) ("neox") of the first R elements of a head turn by
    ``position * frequencies[i]`` (``rope_frequencies``, float64 ``[R / 2]`` on the CPU; default: those of ``theta`` and
    ``rotary_dim``, which is D unless given) and are multiplied by ``magnitude``; the other elements are copied.
    ``inverse=True`` turns the other way: the gradient of the inputs from that of the outputs.  Returns
    ``(q_out, k_out)``, lists of P tensors made here unless given (``q`` and ``k`` themselves are fine); k_out is None
    without k.  The call is not recorded by autograd, also where a tensor requires a gradient.
    """
    if rope not in ("interleaved", "neox"):
        raise ValueError(f"rope must be 'interleaved' or 'neox', not {rope!r}")
    return _run("rope", stream, (q, k), (q_out, k_out, positions, first, frequencies, rotary_dim, theta, magnitude, _ROPE[rope],
                                         inverse))


def linear_attention(q, k, v, out=None, *, decay, scale=None, state=None, final_state=False, stream=None):
    """Attention without a softmax over P head groups, ``q``, ``k`` and ``v`` P views ``[B, S, H/P, D]`` (bf16 or fp16, D 64
    or 128): with ``S_t = exp(-decay[h]) S_(t-1) + k_t^T v_t`` the output is ``scale * q_t S_t`` (default 1/sqrt(D)).

    ``decay``: fp32 ``[H]``, >= 0.  ``state``: fp32 ``[B, H, D, D]``, what the sequence starts from (default: zeros);
    ``final_state=True`` (or a tensor, ``state`` itself too) asks for the one behind the last token.  Returns
    ``(out, final_state)``, the latter None unless asked for; made here, small ones (up to 1 MiB altogether) share an
    allocation, so ``clone()`` a state that is kept for long or saved, or give its tensor.  Not recorded by autograd:
    ``linear_attention_backward`` gives the gradients.
    """
    return _run("linear_attention", stream, (q, k, v, decay, scale, state), (out, final_state))


def linear_attention_backward(dout, q, k, v, dq=None, dk=None, dv=None, *, decay, scale=None, state=None, dstate=None,
                              dstate_out=None, stream=None):
    """Gradients ``(dq, dk, dv, dstate_out)`` of ``linear_attention`` for the gradients ``dout`` of its output and ``dstate`` of
    its final state (fp32 ``[B, H, D, D]`` or None), from the same inputs: lists of P tensors shaped like q, k and v, and
    the gradient of ``state`` (None without state, unless a tensor or True is given).  Small ones made here (up to 1 MiB
    altogether) share an allocation.  Not recorded by autograd.  There is no gradient of the decay."""
    return _run("linear_attention_backward", stream, (q, k, v, decay, scale, state), (dout, dstate, dq, dk, dv, dstate_out))


def linear_attend(states, slots, starts, q, k, v, out=None, *, decay, scale=None, max_tokens=None, stream=None):
    """Linear attention of each sequence's newest tokens through its state, which moves on: rows ``[starts[n],
    starts[n + 1])`` (int32 ``[N + 1]``) of the P row views ``q``, ``k``, ``v`` ``[T, H/P, D]`` belong to sequence n, whose
    state is ``states[slots[n]]`` (fp32 ``[slots, H, D, D]``, updated in place; ``slots`` int32 ``[N]``, different for
    sequences with new rows).  Prompts, chunks and single tokens alike; ``max_tokens`` bounds the rows of one sequence
    (default: T), and a tight one spares work.  Returns ``out``, P tensors ``[T, H/P, D]`` made here unless given (rows
    of no sequence are then undefined; given tensors keep them)."""
    return _run("linear_attend", stream, (q, k, v, decay, scale, states, slots, starts), (out, max_tokens))


def rope_table(theta, S, D, *, stream=None, device=None):
    """The library's resident fp32 cos/sin table ``[S, D/2, 2]`` (a view)."""
    ptr = ctypes.c_void_p()
    _check(lib().tf_ulysses_rope_table(float(theta), int(S), int(D), _stream_handle(stream), ctypes.byref(ptr)))
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    return _wrap(ptr.value, (S, D // 2, 2), torch.float32, dev)


def cache_clear():
    _check(lib().tf_ulysses_cache_clear())


def device_status(clear: bool = False) -> int:
    """The staged kernels' device status word (0 = every in-kernel wait completed)."""
    v = ctypes.c_uint()
    _check(lib().tf_ulysses_device_status(1 if clear else 0, ctypes.byref(v)))
    return int(v.value)


def selftest_wait(cycles: int, *, stream=None):
    """Launch the bounded-wait self-test (a wait nothing satisfies, given up after
    ``cycles`` clock cycles); ``device_status()`` then has bit 1 set."""
    _check(lib().tf_ulysses_selftest_wait(int(cycles), _stream_handle(stream)))


def set_slots(tag, num_slots: int):
    """Rotating target sets for cache entries of ``tag`` created from now on."""
    _check(lib().tf_ulysses_set_slots(tag.encode() if isinstance(tag, str) else tag, int(num_slots)))


def alloc_count() -> int:
    """Device allocations the library has made in this process."""
    return int(lib().tf_ulysses_alloc_count())


def cache_entries() -> int:
    return lib().tf_ulysses_cache_entries()


def launch_count() -> int:
    return int(lib().tf_ulysses_launch_count())


def abi_version() -> int:
    return lib().tf_ulysses_abi_version()


# torch-backed allocator: cached targets and tables come from torch's caching allocator
_alloc_refs = None


def _torch_alloc(nbytes, stream, ctx):
    try:
        return torch.cuda.caching_allocator_alloc(int(nbytes), stream=int(stream or 0))
    except Exception:  # noqa: BLE001 -- the library reports TF_ERR_OOM
        return None


def _torch_free(ptr, nbytes, stream, ctx):
    torch.cuda.caching_allocator_delete(ptr)


def use_torch_allocator(enable: bool = True):
    """Route the library's device allocations through torch's caching allocator
    (default: cudaMallocAsync on the calling stream)."""
    global _alloc_refs
    if enable:
        _alloc_refs = (ALLOC_FN(_torch_alloc), FREE_FN(_torch_free))
        lib().tf_ulysses_set_allocator(_alloc_refs[0], _alloc_refs[1], None)
    else:
        lib().tf_ulysses_set_allocator(ALLOC_FN(), FREE_FN(), None)
        _alloc_refs = None
