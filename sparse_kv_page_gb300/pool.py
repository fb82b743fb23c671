"""Python binding of the packed cache and its page pool (include/locks_pool.h).

Like ``cache``: argument marshalling only, on torch's current CUDA stream of the tensors'
device unless a stream is given, no fallback. A cache in 4 bits around the decode step::

    # bf16 pages that filled become packed pages; their summaries go by the packed page: arrays of
    # num_packed pages and then the bf16 pool's, `tail` being the latter (Summaries(mu[num_packed:], ...))
    locks_build_summaries(dims, k_cache, filled, n, tail)
    locks_copy_pages(make_planes([mu, basis, coef, scales]), filled + num_packed, packed_ids)
    locks_pack_pages(dims, k_cache, v_cache, filled, packed_ids, n, packed)
    locks_select_pages(...)                       # scores as ever, tables of packed pages
    locks_packed_attention(dims, q, packed, page_table, seq_pages, out, ws, selected=selected,
                           n_selected=n_selected, k_cache=k_cache, v_cache=v_cache,
                           recent_table=recent_table, recent_tokens=recent_tokens)

and the pool's life, whose state is the pages' reference counts alone::

    planes = make_planes([k_cache, v_cache, ...])          # of all layers
    locks_take_pages(dims, page_table, seq_tokens, new_tokens, refs, seq_tokens, refs, ws)
    locks_fork_sequences(dims, page_table, seq_tokens, parents, refs, table_out, tokens_out,
                         refs, copy_src, copy_dst, n_copies, ws)
    locks_copy_pages(planes, copy_src, copy_dst, n_copies)
    locks_free_pages(refs, evicted, n_evicted, refs)
    locks_compact_pages(dims, page_table, seq_tokens, refs, page_table, refs, move_src,
                        move_dst, n_moves, new_page, ws)
    locks_copy_pages(planes, move_src, move_dst, n_moves)

Every tensor of a call must be on one CUDA device; where that is not the current one, the
call is made on it.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import cache as _cache
from .cache import _call
from .locks import _check, locks_dims_t

LOCKS_PACKED_BYTES = 2432
LOCKS_MAX_PLANES = 128


class locks_planes_t(ctypes.Structure):
    _fields_ = [("num_planes", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("base", ctypes.c_void_p * LOCKS_MAX_PLANES), ("page_bytes", ctypes.c_int64 * LOCKS_MAX_PLANES)]


_lib: Optional[ctypes.CDLL] = None


def load_library() -> ctypes.CDLL:
    """The library with this module's signatures; _marshal bound to its entry points."""
    global _lib
    if _lib is None:
        lib = _cache.load_library()
        P, S, I32, D = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.POINTER(locks_dims_t)
        sig = {
            "locks_pack_pages": [D, P, P, P, P, I32, P, I32, P, S, P],
            "locks_unpack_pages": [D, P, I32, P, P, I32, P, P, P, S, P],
            "locks_packed_workspace_size": [D, ctypes.POINTER(S)],
            "locks_packed_attention": [D, P, I32, P, I32, P, P, P, P, I32, P, P, P, I32, P, P, P, P, S, P],
            "locks_copy_pages": [ctypes.POINTER(locks_planes_t), P, P, I32, P, P, S, P],
            "locks_pool_workspace_size": [D, ctypes.POINTER(S)],
            "locks_fork_sequences": [D] + [P] * 11 + [S, P],
            "locks_take_pages": [D] + [P] * 8 + [S, P],
            "locks_free_pages": [P, I32, P, I32, P, I32, P, P, S, P],
            "locks_compact_pages": [D] + [P] * 7 + [I32] + [P] * 3 + [S, P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _cache._native.bind_pool(*(ctypes.cast(getattr(lib, n), P).value for n in (
            "locks_pack_pages", "locks_unpack_pages", "locks_packed_attention", "locks_copy_pages",
            "locks_fork_sequences", "locks_take_pages", "locks_free_pages", "locks_compact_pages")))
        _lib = lib
    return _lib


def _enter(*args) -> None:
    if _lib is None:
        load_library()
    _call(*args)


def _size(name: str, dims: locks_dims_t) -> int:
    out = ctypes.c_size_t(0)
    _check(name, getattr(load_library(), name)(ctypes.byref(dims), ctypes.byref(out)))
    return out.value


def _alloc(bytes_: int, device) -> torch.Tensor:
    ws = torch.empty(bytes_, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


# -------------------------------------------------------------- entry points

def locks_pack_pages(dims: locks_dims_t, k_cache: torch.Tensor, v_cache: torch.Tensor, src_pages: torch.Tensor,
                     dst_pages: Optional[torch.Tensor], n_pages: int, packed: torch.Tensor,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """packed: uint8 [packed pages][kv heads][LOCKS_PACKED_BYTES]. dst_pages None: src_pages."""
    _enter("pack", "locks_pack_pages", k_cache.get_device(), stream, ctypes.addressof(dims), k_cache, v_cache,
           src_pages, dst_pages, n_pages, packed, workspace)


def locks_unpack_pages(dims: locks_dims_t, packed: torch.Tensor, src_pages: torch.Tensor,
                       dst_pages: Optional[torch.Tensor], n_pages: int, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """src_pages are packed pages, dst_pages (None: the same ids) pages of the bf16 pool."""
    _enter("unpack", "locks_unpack_pages", k_cache.get_device(), stream, ctypes.addressof(dims), k_cache, v_cache,
           src_pages, dst_pages, n_pages, packed, workspace)


def locks_packed_workspace_size(dims: locks_dims_t) -> int:
    return _size("locks_packed_workspace_size", dims)


def alloc_packed_workspace(dims: locks_dims_t, device="cuda") -> torch.Tensor:
    """A workspace of locks_packed_workspace_size bytes with a clear status word."""
    return _alloc(locks_packed_workspace_size(dims), device)


def locks_packed_attention(dims: locks_dims_t, q: torch.Tensor, packed: Optional[torch.Tensor],
                           page_table: Optional[torch.Tensor], seq_pages: Optional[torch.Tensor], out: torch.Tensor,
                           workspace: torch.Tensor, selected: Optional[torch.Tensor] = None,
                           n_selected: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
                           v_cache: Optional[torch.Tensor] = None, recent_table: Optional[torch.Tensor] = None,
                           recent_tokens: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """selected None: every page; recent_table None: no recent tokens. packed and page_table may be
    None when dims.max_pages_per_seq is 0, seq_pages when selected is given."""
    _enter("attend", "locks_packed_attention", q.get_device(), stream, ctypes.addressof(dims), q, packed, page_table,
           seq_pages, selected, n_selected, k_cache, v_cache, recent_table, recent_tokens, out, lse, workspace)


def make_planes(arrays: Sequence[torch.Tensor]) -> locks_planes_t:
    """The arrays that locks_copy_pages copies pages of: contiguous CUDA tensors [pages][...] of any
    type, a multiple of 8 bytes a page. They are kept alive with what is returned."""
    arrays = list(arrays)
    if len(arrays) > LOCKS_MAX_PLANES:
        raise ValueError(f"{len(arrays)} arrays, more than {LOCKS_MAX_PLANES}")
    planes = locks_planes_t(len(arrays), arrays[0].shape[0] if arrays and arrays[0].dim() else 0)
    planes.device = arrays[0].get_device() if arrays else -1
    planes.arrays = arrays
    for i, x in enumerate(arrays):
        if x.dim() < 1 or x.shape[0] != planes.num_pages:
            raise ValueError(f"array {i} is not [{planes.num_pages}][...]")
        if not x.is_contiguous():
            raise ValueError("LOCKS buffers must be contiguous")
        if not x.is_cuda or x.get_device() != planes.device:
            raise ValueError(f"array {i} is no CUDA tensor of the first one's device")
        page = x.nbytes // max(1, planes.num_pages)
        if page % 8 or x.data_ptr() % 8:
            raise ValueError(f"a page of array {i} is no multiple of 8 bytes, or not 8-byte aligned")
        planes.base[i] = x.data_ptr()
        planes.page_bytes[i] = page
    return planes


def locks_copy_pages(planes: locks_planes_t, src_pages: torch.Tensor, dst_pages: torch.Tensor,
                     n_pairs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """n_pairs: int32 [1], read on the device; None: all of the lists."""
    device = src_pages.get_device()
    if planes.num_planes and planes.device != device:
        raise ValueError(f"src_pages is on device {device}, the arrays are on device {planes.device}")
    _enter("copy", "locks_copy_pages", device, stream, ctypes.addressof(planes), src_pages, dst_pages, n_pairs,
           workspace)


def locks_pool_workspace_size(dims: locks_dims_t) -> int:
    return _size("locks_pool_workspace_size", dims)


def alloc_pool_workspace(dims: locks_dims_t, device="cuda") -> torch.Tensor:
    """A workspace of locks_pool_workspace_size bytes with a clear status word."""
    return _alloc(locks_pool_workspace_size(dims), device)


def locks_fork_sequences(dims: locks_dims_t, page_table: torch.Tensor, seq_tokens: torch.Tensor,
                         parents: torch.Tensor, refs: torch.Tensor, page_table_out: torch.Tensor,
                         seq_tokens_out: torch.Tensor, refs_out: torch.Tensor, copy_src: torch.Tensor,
                         copy_dst: torch.Tensor, n_copies: torch.Tensor, workspace: torch.Tensor,
                         stream=None) -> None:
    """refs_out may be refs; the tables may not be one another. locks_copy_pages(planes, copy_src,
    copy_dst, n_copies) then copies what the new last pages begin with."""
    _enter("fork", "locks_fork_sequences", page_table.get_device(), stream, ctypes.addressof(dims), page_table,
           seq_tokens, parents, refs, page_table_out, seq_tokens_out, refs_out, copy_src, copy_dst, n_copies,
           workspace)


def locks_take_pages(dims: locks_dims_t, page_table: torch.Tensor, seq_tokens: torch.Tensor,
                     new_tokens: torch.Tensor, refs: torch.Tensor, seq_tokens_out: torch.Tensor,
                     refs_out: torch.Tensor, workspace: torch.Tensor, n_free: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """page_table is written in place; seq_tokens_out and refs_out may be the inputs."""
    _enter("take", "locks_take_pages", page_table.get_device(), stream, ctypes.addressof(dims), page_table,
           seq_tokens, new_tokens, refs, seq_tokens_out, refs_out, n_free, workspace)


def locks_free_pages(refs: torch.Tensor, pages: torch.Tensor, counts: torch.Tensor, refs_out: torch.Tensor,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """pages: int32 [rows][pages] with counts [rows] (a page table, or evicted and n_evicted of
    locks_evict_pages). refs_out may be refs."""
    _enter("free", "locks_free_pages", refs.get_device(), stream, refs, pages, counts, refs_out, workspace)


def locks_compact_pages(dims: locks_dims_t, page_table: torch.Tensor, seq_tokens: torch.Tensor, refs: torch.Tensor,
                        page_table_out: torch.Tensor, refs_out: torch.Tensor, move_src: torch.Tensor,
                        move_dst: torch.Tensor, n_moves: torch.Tensor, new_page: torch.Tensor,
                        workspace: torch.Tensor, stream=None) -> None:
    """page_table_out and refs_out may be the inputs. locks_copy_pages(planes, move_src, move_dst,
    n_moves) then moves the pages; other tables go by new_page."""
    _enter("compact", "locks_compact_pages", page_table.get_device(), stream, ctypes.addressof(dims), page_table,
           seq_tokens, refs, page_table_out, refs_out, move_src, move_dst, n_moves, new_page, workspace)
