"""Python binding of the paged-cache operators (include/locks_cache.h).

Like ``locks``: argument marshalling only, on torch's current CUDA stream of the
tensors' device unless a stream is given, no fallback. Tensors of bf16 bits may be
``torch.bfloat16`` or, as elsewhere in this package, ``torch.int16``. Around a decode
step::

    rope = make_rope(128, [500000.0 ** (-i / 64) for i in range(64)])
    # the step's tokens: head norms, rotation, K/V into the cache, q in fp32
    locks_append_tokens(dims, rope, q_proj, k_proj, v_proj, positions, cache_index,
                        page_table, q, k_cache, v_cache)
    locks_decode_step(dims, q, ..., scores=scores)      # or locks_prefix_attention
    locks_accumulate_mass(dims, scores, seq_pages, mass, mass, mass_ws, decay=0.98)
    locks_evict_pages(dims, mass, page_table, seq_pages, keep_pages, mass, page_table,
                      seq_pages, evicted, n_evicted, sink_pages=1, recent_pages=4)

Every tensor of a call must be on one CUDA device; where that is not the current
one, the call is made on it.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import locks as _locks
from .locks import LocksError, _check, locks_dims_t

LOCKS_BF16, LOCKS_FP16, LOCKS_FP32 = 0, 1, 2
LOCKS_MAX_AXES = 4
_TYPES = {torch.bfloat16: LOCKS_BF16, torch.int16: LOCKS_BF16, torch.float16: LOCKS_FP16, torch.float32: LOCKS_FP32}
_BF16 = (torch.bfloat16, torch.int16)
_QUERY = (torch.float32,) + _BF16


class locks_rope_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("scale", ctypes.c_float), ("inv_freq", ctypes.c_double * 64), ("axis", ctypes.c_int32 * 64)]


_lib: Optional[ctypes.CDLL] = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = _locks.load_library()
        P, S, I32, I64, F32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        D, R = ctypes.POINTER(locks_dims_t), ctypes.POINTER(locks_rope_t)
        sig = {
            "locks_append_tokens": [D, R, P, P, P, I32, I64, I64, I64, I32, P, P, P, P, P, P, F32, P, I32, P, P, P, S,
                                    P],
            "locks_prefix_workspace_size": [D, I32, ctypes.POINTER(S)],
            "locks_prefix_attention": [D, P, I32, P, P, P, P, P, I32, I32, P, P, P, P, P, S, P],
            "locks_mass_workspace_size": [D, ctypes.POINTER(S)],
            "locks_accumulate_mass": [D, P, P, P, P, P, F32, P, S, P],
            "locks_evict_pages": [D, P, P, P, I32, I32, I32, I32, P, P, P, P, I32, P, P, S, P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _lib = lib
    return _lib


# ----------------------------------------------------------------- arguments
# These run before every launch, and for a decode step's small calls they are most of the
# call's time: one chained test per tensor, and its reason found only when it fails.

def _refuse(name: str, t: torch.Tensor, device: int, dtypes, shape) -> None:
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call is on device {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has type {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError("LOCKS buffers must be contiguous")


def _arg(name: str, t: Optional[torch.Tensor], device: int, dtypes, shape) -> Optional[int]:
    """The address of a contiguous tensor of the given kind and shape (None: null)."""
    if t is None:
        return None
    if t.get_device() != device or t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, device, dtypes, shape)
    return t.data_ptr()


def _ws(t: Optional[torch.Tensor], device: int):
    if t is None:
        return None, 0
    if t.get_device() != device or not t.is_contiguous():
        _refuse("workspace", t, device, (t.dtype,), t.shape)
    return t.data_ptr(), t.nbytes


def _rows(name: str, t: torch.Tensor, device: int, dtype, tokens: int, heads: int):
    """(address, elements from token to token) of [tokens][heads][128] rows; only the token
    axis may be strided."""
    if t.get_device() != device or t.dtype != dtype or t.shape != (tokens, heads, 128):
        _refuse(name, t, device, (dtype,), (tokens, heads, 128))
    step, head, one = t.stride()
    if one != 1 or (head != 128 and heads > 1):
        raise ValueError(f"{name}: the heads of a token must lie beside each other")
    return t.data_ptr(), step if tokens > 1 else 0


def _call(name: str, device: int, stream, *args) -> None:
    if device < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    fn = getattr(_lib or _library(), name)
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == device:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != 0:
        raise LocksError(name, status)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)   # the same without a Stream object


_I32 = (torch.int32,)
_F32 = (torch.float32,)


# -------------------------------------------------------------- entry points

def make_rope(rot_dim: int, inv_freq: Sequence[float], interleaved: bool = False, axis: Optional[Sequence[int]] = None,
              num_axes: Optional[int] = None, scale: float = 1.0) -> locks_rope_t:
    """inv_freq: rot_dim / 2 angles per position, in radians; axis: the row of positions that
    turns each pair (all 0 unless given); num_axes: rows of positions (the largest axis + 1)."""
    n = rot_dim // 2
    if len(inv_freq) != n or (axis is not None and len(axis) != n) or not 0 <= n <= 64:
        raise ValueError(f"rot_dim {rot_dim} takes {n} inverse frequencies and axes")
    axis = [0] * n if axis is None else [int(a) for a in axis]
    r = locks_rope_t(rot_dim, int(interleaved), max(axis, default=0) + 1 if num_axes is None else num_axes, scale)
    r.inv_freq[:n] = [float(f) for f in inv_freq]
    r.axis[:n] = axis
    return r


def locks_append_tokens(dims: locks_dims_t, rope: Optional[locks_rope_t], q: Optional[torch.Tensor], k: torch.Tensor,
                        v: torch.Tensor, positions: Optional[torch.Tensor], cache_index: torch.Tensor,
                        page_table: torch.Tensor, q_out: Optional[torch.Tensor], k_cache: torch.Tensor,
                        v_cache: torch.Tensor, token_seq: Optional[torch.Tensor] = None,
                        q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                        eps: float = 1e-6, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """q, k, v: [tokens][heads][128], bf16, fp16 or fp32, the token axis strided as it likes (slices
    of one projection's output). positions int32 [axes][tokens] (or [tokens] for one axis)."""
    dev, n, hq, hkv = k.get_device(), k.shape[0], dims.num_q_heads, dims.num_kv_heads
    in_type = _TYPES.get(k.dtype)
    if in_type is None:
        raise TypeError(f"k has type {k.dtype}")
    kp, ks = _rows("k", k, dev, k.dtype, n, hkv)
    vp, vs = _rows("v", v, dev, k.dtype, n, hkv)
    qp, qs, qtype = None, 0, LOCKS_FP32
    if q is not None:
        qp, qs = _rows("q", q, dev, k.dtype, n, hq)
    if q_out is not None:
        qtype = LOCKS_FP32 if q_out.dtype == torch.float32 else LOCKS_BF16
    if positions is not None and rope is not None:
        pos = _arg("positions", positions, dev, _I32,
                   (n,) if positions.dim() == 1 and rope.num_axes == 1 else (rope.num_axes, n))
    else:
        pos = None
    cache = (dims.num_phys_pages, hkv, 16, 128)
    ws, nws = _ws(workspace, dev)
    _call("locks_append_tokens", dev, stream, ctypes.byref(dims), ctypes.byref(rope) if rope is not None else None,
          qp, kp, vp, in_type, qs, ks, vs, n, pos, _arg("token_seq", token_seq, dev, _I32, (n,)),
          _arg("cache_index", cache_index, dev, _I32, (n,)),
          _arg("page_table", page_table, dev, _I32, (dims.batch, dims.max_pages_per_seq)),
          _arg("q_weight", q_weight, dev, _F32, (128,)), _arg("k_weight", k_weight, dev, _F32, (128,)), eps,
          _arg("q_out", q_out, dev, _QUERY, (n, hq, 128)), qtype,
          _arg("k_cache", k_cache, dev, _BF16, cache), _arg("v_cache", v_cache, dev, _BF16, cache), ws, nws)


def locks_prefix_workspace_size(dims: locks_dims_t, num_groups: int) -> int:
    out = ctypes.c_size_t(0)
    _check("locks_prefix_workspace_size",
           _library().locks_prefix_workspace_size(ctypes.byref(dims), num_groups, ctypes.byref(out)))
    return out.value


def alloc_prefix_workspace(dims: locks_dims_t, num_groups: int, device="cuda") -> torch.Tensor:
    """A workspace of locks_prefix_workspace_size bytes with a clear status word."""
    ws = torch.empty(locks_prefix_workspace_size(dims, num_groups), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def locks_prefix_attention(dims: locks_dims_t, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           prefix_table: Optional[torch.Tensor], prefix_tokens: Optional[torch.Tensor],
                           group_start: Optional[torch.Tensor], page_table: Optional[torch.Tensor],
                           seq_tokens: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                           lse: Optional[torch.Tensor] = None, stream=None) -> None:
    """prefix_table None: no prefixes. page_table may be None when dims.max_pages_per_seq is 0."""
    dev, b, hq = q.get_device(), dims.batch, dims.num_q_heads
    cache = (dims.num_phys_pages, dims.num_kv_heads, 16, 128)
    groups, pages = (0, 0) if prefix_table is None else prefix_table.shape
    ws, nws = _ws(workspace, dev)
    _call("locks_prefix_attention", dev, stream, ctypes.byref(dims),
          _arg("q", q, dev, _QUERY, (b, hq, 128)),
          LOCKS_FP32 if q.dtype == torch.float32 else LOCKS_BF16, _arg("k_cache", k_cache, dev, _BF16, cache),
          _arg("v_cache", v_cache, dev, _BF16, cache),
          _arg("prefix_table", prefix_table, dev, _I32, (groups, pages)),
          _arg("prefix_tokens", prefix_tokens if groups else None, dev, _I32, (groups,)),
          _arg("group_start", group_start if groups else None, dev, _I32, (groups + 1,)), groups, pages,
          _arg("page_table", page_table, dev, _I32, (b, dims.max_pages_per_seq)),
          _arg("seq_tokens", seq_tokens, dev, _I32, (b,)), _arg("out", out, dev, _BF16, (b, hq, 128)),
          _arg("lse", lse, dev, _F32, (b, hq)), ws, nws)


def locks_mass_workspace_size(dims: locks_dims_t) -> int:
    out = ctypes.c_size_t(0)
    _check("locks_mass_workspace_size", _library().locks_mass_workspace_size(ctypes.byref(dims), ctypes.byref(out)))
    return out.value


def alloc_mass_workspace(dims: locks_dims_t, device="cuda") -> torch.Tensor:
    """A workspace of locks_mass_workspace_size bytes with a clear status word."""
    ws = torch.empty(locks_mass_workspace_size(dims), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def locks_accumulate_mass(dims: locks_dims_t, scores: torch.Tensor, seq_pages: torch.Tensor, mass: torch.Tensor,
                          mass_out: torch.Tensor, workspace: torch.Tensor, decay: float = 1.0,
                          lse_partials: Optional[torch.Tensor] = None, stream=None) -> None:
    """mass_out may be mass. lse_partials: those locks_score_pages wrote beside these scores."""
    dev, b, p = scores.get_device(), dims.batch, dims.max_pages_per_seq
    ws, nws = _ws(workspace, dev)
    partials = None
    if lse_partials is not None:
        partials = _arg("lse_partials", lse_partials, dev, _F32, _locks.lse_partials_shape(dims))
    _call("locks_accumulate_mass", dev, stream, ctypes.byref(dims),
          _arg("scores", scores, dev, _F32, (b, dims.num_q_heads, p)), partials,
          _arg("seq_pages", seq_pages, dev, _I32, (b,)), _arg("mass", mass, dev, _F32, (b, p)),
          _arg("mass_out", mass_out, dev, _F32, (b, p)), decay, ws, nws)


def locks_evict_pages(dims: locks_dims_t, mass: torch.Tensor, page_table: torch.Tensor, seq_pages: torch.Tensor,
                      keep_pages: int, mass_out: torch.Tensor, page_table_out: torch.Tensor,
                      seq_pages_out: torch.Tensor, evicted: torch.Tensor, n_evicted: torch.Tensor,
                      sink_pages: int = 0, recent_pages: int = 0, extra_pages: int = 0,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The outputs mass_out, page_table_out and seq_pages_out may be the inputs. evicted: int32
    [batch][at least max(1, max_pages_per_seq - keep_pages)]."""
    dev, b, p = mass.get_device(), dims.batch, dims.max_pages_per_seq
    ws, nws = _ws(workspace, dev)
    cap = evicted.shape[-1]
    _call("locks_evict_pages", dev, stream, ctypes.byref(dims), _arg("mass", mass, dev, _F32, (b, p)),
          _arg("page_table", page_table, dev, _I32, (b, p)), _arg("seq_pages", seq_pages, dev, _I32, (b,)),
          keep_pages, sink_pages, recent_pages, extra_pages, _arg("mass_out", mass_out, dev, _F32, (b, p)),
          _arg("page_table_out", page_table_out, dev, _I32, (b, p)),
          _arg("seq_pages_out", seq_pages_out, dev, _I32, (b,)), _arg("evicted", evicted, dev, _I32, (b, cap)), cap,
          _arg("n_evicted", n_evicted, dev, _I32, (b,)), ws, nws)
