"""Python binding of the paged-cache operators (include/locks_cache.h).

Like ``locks``: argument marshalling only, on torch's current CUDA stream of the
tensors' device unless a stream is given, no fallback. Tensors of bf16 bits may be
``torch.bfloat16`` or, as elsewhere in this package, ``torch.int16``. Around a decode
step::

    rope = make_rope(128, [500000.0 ** (-i / 64) for i in range(64)])
    # the step's tokens: head norms, rotation, K/V into the cache, q in fp32
    locks_append_tokens(dims, rope, q_proj, k_proj, v_proj, positions, cache_index,
                        page_table, q, k_cache, v_cache)
    locks_decode_step(dims, q, ..., scores=scores)
    locks_accumulate_mass(dims, scores, seq_pages, mass, mass, mass_ws, decay=0.98)
    locks_evict_pages(dims, mass, page_table, seq_pages, keep_pages, mass, page_table,
                      seq_pages, evicted, n_evicted, sink_pages=1, recent_pages=4)

``locks_prefix_attention`` attends in the step's place where a batch shares prompts. It goes
over every token and writes no page scores: mass then needs ``locks_score_pages`` or
``locks_exact_scores`` beside it.

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
class locks_rope_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("scale", ctypes.c_float), ("inv_freq", ctypes.c_double * 64), ("axis", ctypes.c_int32 * 64)]


_lib: Optional[ctypes.CDLL] = None
_native = None


def load_library() -> ctypes.CDLL:
    """The library with this module's signatures; _marshal bound to its entry points."""
    global _lib, _native
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
        try:
            from . import _marshal
        except ImportError as e:
            raise RuntimeError("the _marshal extension is not built (run __graft_entry__.build())") from e
        _marshal.bind(*(ctypes.cast(getattr(lib, n), P).value for n in (
            "locks_append_tokens", "locks_prefix_attention", "locks_accumulate_mass", "locks_evict_pages")))
        _native = _marshal
        _lib = lib
    return _lib


# The tensors' checks and addresses are _marshal's (csrc/marshal.cpp): of a decode step's small
# calls, reading them through Python was most of the time.

def _place(device: int, stream):
    """The stream's handle, and whether the device has to be made current first."""
    if _native is None:
        load_library()
    if device < 0:                       # host tensors: refused by the call, after what else may be wrong
        return 0, False
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    return stream, _current_device() != device


def _call(entry: str, name: str, device: int, stream, *args) -> None:
    stream, elsewhere = _place(device, stream)
    if elsewhere:
        with torch.cuda.device(device):
            status = getattr(_native, entry)(device, stream, *args)
    else:
        status = getattr(_native, entry)(device, stream, *args)
    if status != 0:
        raise LocksError(name, status)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the same without a Stream object, and without the check that CUDA is up (a CUDA tensor is)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


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
    _call("append", "locks_append_tokens", k.get_device(), stream, ctypes.addressof(dims),
          0 if rope is None else ctypes.addressof(rope), q, k, v, positions, cache_index, page_table, q_out, k_cache,
          v_cache, token_seq, q_weight, k_weight, eps, workspace)


def locks_prefix_workspace_size(dims: locks_dims_t, num_groups: int) -> int:
    out = ctypes.c_size_t(0)
    _check("locks_prefix_workspace_size",
           load_library().locks_prefix_workspace_size(ctypes.byref(dims), num_groups, ctypes.byref(out)))
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
    _call("prefix", "locks_prefix_attention", q.get_device(), stream, ctypes.addressof(dims), q, k_cache, v_cache,
          prefix_table, prefix_tokens, group_start, page_table, seq_tokens, out, workspace, lse)


def locks_mass_workspace_size(dims: locks_dims_t) -> int:
    out = ctypes.c_size_t(0)
    _check("locks_mass_workspace_size", load_library().locks_mass_workspace_size(ctypes.byref(dims), ctypes.byref(out)))
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
    _call("mass", "locks_accumulate_mass", scores.get_device(), stream, ctypes.addressof(dims), scores, seq_pages, mass,
          mass_out, workspace, decay, lse_partials,
          0 if lse_partials is None else _locks.lse_partials_shape(dims)[0])


def locks_evict_pages(dims: locks_dims_t, mass: torch.Tensor, page_table: torch.Tensor, seq_pages: torch.Tensor,
                      keep_pages: int, mass_out: torch.Tensor, page_table_out: torch.Tensor,
                      seq_pages_out: torch.Tensor, evicted: torch.Tensor, n_evicted: torch.Tensor,
                      sink_pages: int = 0, recent_pages: int = 0, extra_pages: int = 0,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The outputs mass_out, page_table_out and seq_pages_out may be the inputs. evicted: int32
    [batch][at least max(1, max_pages_per_seq - keep_pages)]."""
    _call("evict", "locks_evict_pages", mass.get_device(), stream, ctypes.addressof(dims), mass, page_table, seq_pages,
          keep_pages, mass_out, page_table_out, seq_pages_out, evicted, n_evicted, sink_pages, recent_pages,
          extra_pages, workspace)
