"""Sequences and pages of caches: ``cache_fork`` and ``cache_compact``.

Argument checks and marshalling only; the work runs in the HIP kernels of
``libfp8bq.so`` on the current stream.  Both take the caches of all layers,
``KvCache`` or ``LatentCache``, that one block table serves.
"""

import ctypes
import struct

from . import _check, load_library
from .kv import _run

MAX_COMPACT_PAGES = 1 << 20

_PAGES = struct.Struct("=Qqii")   # fp8bq_pages


def _pages(caches):
    """The packed ``fp8bq_pages``, what keeps its list alive, and a cache."""
    caches = list(caches) if isinstance(caches, (list, tuple)) else [caches]
    if not caches:
        raise ValueError("caches must hold at least one cache")
    first = caches[0]
    try:
        for c in caches:
            if c.num_pages != first.num_pages or c.page_size != first.page_size or c._index != first._index:
                raise ValueError("the caches must agree in num_pages, page_size and device")
        buffers = b"".join([c._buffers for c in caches])
    except AttributeError:
        raise TypeError("caches must be KvCache or LatentCache objects") from None
    keep = ctypes.c_char_p(buffers)
    at = ctypes.cast(keep, ctypes.c_void_p).value
    return _PAGES.pack(at, first.num_pages, len(buffers) // 16, first.page_size), keep, first


def _ints(x, n, index, what):
    import torch

    if x.dtype is not torch.int32:
        raise TypeError(f"{what} must be int32")
    if x.dim() != 1 or (n is not None and x.shape[0] != n) or not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous [{'n' if n is None else n}]")
    if x.get_device() != index:
        raise ValueError(f"{what} must be on the caches' device")
    return x.data_ptr()


def _table(x, shape, index, what):
    """(pointer, row stride) of an int32 table."""
    import torch

    if x.dtype is not torch.int32:
        raise TypeError(f"{what} must be int32")
    if x.dim() != 2 or (shape is not None and tuple(x.shape) != shape):
        raise ValueError(f"{what} must be [sequences, pages]" if shape is None else
                         f"{what} has shape {tuple(x.shape)}, expected {shape}")
    n, width = x.shape
    if (width > 1 and x.stride(1) != 1) or (n > 1 and x.stride(0) < width):
        raise ValueError(f"{what}'s rows must be contiguous")
    if x.get_device() != index:
        raise ValueError(f"{what} must be on the caches' device")
    return x.data_ptr(), x.stride(0) if n > 1 else width


def cache_fork(caches, block_table, seq_lens, parents, children, pages):
    """Let sequences go on from the tokens of others (``fp8bq_cache_fork``): n
    samples of one prompt, beams.

    ``caches`` are the ``KvCache`` or ``LatentCache`` of each layer (or a single
    one), ``block_table`` (int32 [sequences, pages]) and ``seq_lens`` (int32
    [sequences]) theirs.  Sequence ``children[i]`` becomes a copy of
    ``parents[i]``: its length, and its row of the table, whose whole pages both
    share from now on.  Where the parent's last page is partly filled, that page
    is copied, in all caches, to ``pages[i]``, the child's own.  The last three are
    int32 [forks] on the GPU.

    A child is named once and is nobody's parent, and ``pages`` are in no other
    use; otherwise what these rows and pages hold is unspecified.  Forks whose
    parent or child is no sequence are left out.  The table and the lengths are
    changed in place.
    """
    packed, keep, cache = _pages(caches)
    index = cache._index
    tp, ts = _table(block_table, None, index, "block_table")
    n, width = block_table.shape
    lp = _ints(seq_lens, n, index, "seq_lens")
    ap = _ints(parents, None, index, "parents")
    forks = parents.shape[0]
    bp, pp = _ints(children, forks, index, "children"), _ints(pages, forks, index, "pages")
    if forks == 0 or n == 0:
        return
    status = _run(cache, load_library().fp8bq_cache_fork, packed, tp, ts, n, width, lp, ap, bp, pp, forks)
    if status:
        _check("fp8bq_cache_fork", status)
    del keep


def cache_compact_workspace_bytes(caches):
    """Bytes of ``cache_compact``'s workspace for these caches."""
    first = caches[0] if isinstance(caches, (list, tuple)) else caches
    return int(load_library().fp8bq_cache_compact_workspace_bytes(first.num_pages))


def cache_compact(caches, block_table, seq_lens, *, table_out=None, used=None, workspace=None):
    """Move the pages in use to the front of the caches
    (``fp8bq_cache_compact``), so that the pages behind them are free: for new
    sequences, or for the trainer to take their memory.

    Arguments as in ``cache_fork``.  In use is what the table names within the
    lengths; a sequence is freed by setting its length to 0.  With ``used`` pages
    in use, those numbered ``used`` and more move, in order, to the free ones
    before them, in all caches; pages that sequences share stay shared.

    Returns ``(table, used)``: the table with the pages' new numbers, -1 behind each
    length and for entries that were no page, in ``table_out`` (which may be
    ``block_table``) or a new tensor, and an int32 [1] tensor with the number of
    pages in use.  ``workspace`` is a uint8 GPU tensor of
    ``cache_compact_workspace_bytes`` that no overlapping call uses; by default
    each call takes one from torch's allocator.
    """
    import torch

    packed, keep, cache = _pages(caches)
    index = cache._index
    if cache.num_pages > MAX_COMPACT_PAGES:
        raise ValueError(f"at most {MAX_COMPACT_PAGES} pages, got {cache.num_pages}")
    tp, ts = _table(block_table, None, index, "block_table")
    n, width = block_table.shape
    lp = _ints(seq_lens, n, index, "seq_lens")
    if table_out is None:
        table_out = torch.empty((n, width), dtype=torch.int32, device=cache.device)
    op, os_ = _table(table_out, (n, width), index, "table_out")
    if used is None:
        used = torch.empty((1,), dtype=torch.int32, device=cache.device)
    up = _ints(used, 1, index, "used")
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(lib.fp8bq_cache_compact_workspace_bytes(cache.num_pages), dtype=torch.uint8,
                                device=cache.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the caches' device")
    status = _run(cache, lib.fp8bq_cache_compact, packed, tp, ts, n, width, lp, op, os_, up, workspace.data_ptr(),
                  workspace.numel() * workspace.element_size())
    if status:
        _check("fp8bq_cache_compact", status)
    del keep
    return table_out, used
