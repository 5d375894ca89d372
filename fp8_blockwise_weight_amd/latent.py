"""The cache of shared latents: ``LatentCache``, ``latent_append``,
``latent_attention``, and ``latent_prompt_attention`` before it.

Argument checks and marshalling only; the work runs in the HIP kernels of
``libfp8bq.so`` on the current stream.  A token's latent is a block of its own,
as ``quantize(x, (1, latent_dim))`` would make it, with a power of two for a
descale (include/fp8bq.h has the arithmetic).
"""

import struct

from . import _check, load_library
from .kv import _BATCH, _BUFFER, MAX_ROWS, PAGE_SIZES, _batch, _rows, _run, _writable

LATENT_DIMS = (256, 512)
ROPE_DIM = 64
MAX_HEADS = 1024

_CACHE = struct.Struct("=QQQqii")             # fp8bq_latent_cache
_TOKENS = struct.Struct("=QQQQQQQ9qii")       # fp8bq_latent_tokens
_QUERY = struct.Struct("=QQQQ7qif")           # fp8bq_latent_query
_PROMPT = struct.Struct("=QQQQQQQQ11qiiif")   # fp8bq_latent_prompt


class LatentCache:
    """The buffers of a paged cache of latents, checked once; other buffers are
    another ``LatentCache`` (the attributes are read-only).

    ``c`` is float8_e4m3fn [pages, page_size, latent_dim], ``r`` bfloat16
    [pages, page_size, 64] and ``scale`` float32 [pages, page_size], powers of
    two, all contiguous on one GPU.  ``LatentCache.empty`` allocates them.
    Dequantize with ``dequantize(cache.c.view(-1, latent_dim),
    cache.scale.view(-1, 1), (1, latent_dim))``.
    """

    __slots__ = ("c", "r", "scale", "num_pages", "page_size", "latent_dim", "device", "_index", "_packed", "_buffers")

    def __init__(self, c, r, scale):
        import torch

        for t, what, dims, dtype in ((c, "c", 3, torch.float8_e4m3fn), (r, "r", 3, torch.bfloat16),
                                     (scale, "scale", 2, torch.float32)):
            if not isinstance(t, torch.Tensor) or t.dim() != dims:
                raise TypeError(f"{what} must be a {dims}-D tensor")
            if t.dtype != dtype:
                raise TypeError(f"{what} must be {str(dtype).split('.')[1]}, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous")
        pages, size, dim = c.shape
        if size not in PAGE_SIZES:
            raise ValueError(f"page_size must be one of {PAGE_SIZES}, got {size}")
        if dim not in LATENT_DIMS:
            raise ValueError(f"latent_dim must be one of {LATENT_DIMS}, got {dim}")
        if pages < 1:
            raise ValueError("a cache holds at least one page")
        if tuple(r.shape) != (pages, size, ROPE_DIM):
            raise ValueError(f"r has shape {tuple(r.shape)}, expected {(pages, size, ROPE_DIM)}")
        if tuple(scale.shape) != (pages, size):
            raise ValueError(f"scale has shape {tuple(scale.shape)}, expected {(pages, size)}")
        if c.data_ptr() % 16 or r.data_ptr() % 16:
            raise ValueError("c and r must be 16-byte aligned")
        for t in (c, r, scale):
            if not t.is_cuda:
                raise TypeError("the cache must be on a GPU (there is no CPU implementation)")
            if t.device != c.device:
                raise ValueError("the cache's buffers must be on one device")
        packed = _CACHE.pack(c.data_ptr(), r.data_ptr(), scale.data_ptr(), pages, size, dim)
        buffers = b"".join(_BUFFER.pack(t.data_ptr(), t.numel() // pages * t.element_size()) for t in (c, r, scale))
        for name, value in zip(self.__slots__, (c, r, scale, pages, size, dim, c.device, c.get_device(), packed,
                                                buffers)):
            object.__setattr__(self, name, value)

    # Calls go by the addresses taken above, as those of a KvCache do.
    def __setattr__(self, name, value):
        raise AttributeError(f"LatentCache.{name} is read-only")

    def __delattr__(self, name):
        raise AttributeError(f"LatentCache.{name} is read-only")

    def __reduce__(self):
        return LatentCache, (self.c, self.r, self.scale)

    @classmethod
    def empty(cls, num_pages, latent_dim=512, page_size=64, device="cuda"):
        """A cache of ``num_pages`` zeroed pages."""
        import torch

        if page_size not in PAGE_SIZES:
            raise ValueError(f"page_size must be one of {PAGE_SIZES}, got {page_size}")
        return cls(torch.zeros((num_pages, page_size, latent_dim), dtype=torch.float8_e4m3fn, device=device),
                   torch.zeros((num_pages, page_size, ROPE_DIM), dtype=torch.bfloat16, device=device),
                   torch.ones((num_pages, page_size), dtype=torch.float32, device=device))


def _flat_rows(x, tokens, dim, index, what):
    """(pointer, token stride) of BF16 rows [tokens, dim]."""
    import torch

    if x.dtype is not torch.bfloat16 or x.dim() != 2:
        raise TypeError(f"{what} must be a 2-D torch.bfloat16 tensor")
    if x.shape[0] != tokens or x.shape[1] != dim:
        raise ValueError(f"{what} has shape {tuple(x.shape)}, expected {(tokens, dim)}")
    if x.get_device() != index:
        raise ValueError(f"{what} must be on the same device as the rest")
    st, sd = x.stride()
    ptr = x.data_ptr()
    if tokens <= 1:
        st = 0
    if sd != 1 or ptr & 15 or st & 7 or st < 0:
        raise ValueError(f"{what}'s rows must be contiguous and 16-byte aligned")
    return ptr, st


def _heads(q, tokens):
    heads = q.shape[1]
    if not 1 <= heads <= MAX_HEADS:
        raise ValueError(f"q's heads must be 1 to {MAX_HEADS}, got {heads}")
    if tokens * heads > MAX_ROWS:
        raise ValueError(f"at most {MAX_ROWS} rows (tokens x heads) per call")
    return heads


def latent_append(cache, c, r, block_table, seq_lens, query_start=None, *, q=None, q_out=None, r_out=None,
                  cos=None, sin=None, interleaved=False):
    """Store new latents and their rotated keys in ``cache``
    (``fp8bq_latent_append``).

    ``c`` is BF16 [tokens, latent_dim], ``r`` BF16 [tokens, 64], the key's rotary
    channels; both may be views of one projection's output.  ``block_table``,
    ``seq_lens`` and ``query_start`` are as in ``kv_append``.  ``cos`` and ``sin``
    (float32 [positions, 32]) rotate ``r`` and ``q``, in halves or, with
    ``interleaved``, adjacent pairs; without them nothing is rotated.  Tokens at
    positions beyond their rows are left out.

    Returns the rotated queries where ``q`` (BF16 [tokens, heads, 64], often a
    view of the last channels of each head) is given, in ``q_out`` (which may be
    ``q``) or a new tensor, else None.  ``r_out`` (BF16 [tokens, 64]; may be
    ``r``) takes the rotated keys too, which ``latent_prompt_attention`` wants.
    Rows of no sequence and of tokens that are left out are not written.
    """
    import torch

    tokens = c.shape[0]
    index, dim = cache._index, cache.latent_dim
    batch, n = _batch(cache, tokens, block_table, seq_lens, query_start)
    cp, ct = _flat_rows(c, tokens, dim, index, "c")
    rp, rt = _flat_rows(r, tokens, ROPE_DIM, index, "r")
    positions = cos_p = sin_p = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin belong together")
    if cos is not None:
        if cos.dtype is not torch.float32 or sin.dtype is not torch.float32:
            raise TypeError("cos and sin must be float32")
        if cos.dim() != 2 or cos.shape != sin.shape or cos.shape[1] != ROPE_DIM // 2 or not cos.is_contiguous() \
                or not sin.is_contiguous():
            raise ValueError(f"cos and sin must be contiguous [positions, {ROPE_DIM // 2}]")
        positions, cos_p, sin_p = cos.shape[0], cos.data_ptr(), sin.data_ptr()
        if cos.get_device() != index or sin.get_device() != index or (cos_p | sin_p) & 15:
            raise ValueError("cos and sin must be on the cache's device and 16-byte aligned")
    qp = qt = qh = op = ot = oh = heads = rop = rot = 0
    if q is not None:
        qp, qt, qh = _rows(q, tokens, None, ROPE_DIM, index, "q")
        heads = _heads(q, tokens)
        if q_out is None:
            q_out = torch.empty((tokens, heads, ROPE_DIM), dtype=torch.bfloat16, device=cache.device)
        op, ot, oh = _rows(q_out, tokens, heads, ROPE_DIM, index, "q_out")
        _writable(q_out, ot, oh, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if r_out is not None:
        rop, rot = _flat_rows(r_out, tokens, ROPE_DIM, index, "r_out")
        _writable(r_out.unsqueeze(1), rot, 0, "r_out")
    if tokens > MAX_ROWS:
        raise ValueError(f"at most {MAX_ROWS} rows (tokens x heads) per call")
    if tokens == 0 or n == 0 or (cos is not None and positions == 0):   # all are left out
        return q_out
    packed = _TOKENS.pack(cp, rp, rop, qp, op, cos_p, sin_p, ct, rt, rot, qt, qh, ot, oh, tokens, positions, heads,
                          int(bool(interleaved)))
    status = _run(cache, load_library().fp8bq_latent_append, cache._packed, batch, packed)
    if status:
        _check("fp8bq_latent_append", status)
    return q_out


def latent_attention_workspace_bytes(cache, q, block_table):
    """Bytes of ``latent_attention``'s workspace for these tensors: by their
    shapes alone."""
    n, width = block_table.shape
    batch = _BATCH.pack(0, 0, 0, width, n, width)
    return int(load_library().fp8bq_latent_attention_workspace_bytes(cache._packed, batch, q.shape[1], q.shape[0]))


def latent_attention(cache, q, q_rope, block_table, seq_lens, query_start=None, *, scale, out=None, return_lse=False,
                     lse=None, workspace=None):
    """Attention over ``cache`` in the absorbed form
    (``fp8bq_latent_attention``), one query token per sequence or, with
    ``query_start``, any number of each, the last ones of their sequence.

    ``q`` is BF16 [tokens, heads, latent_dim], the queries times their heads' key
    up-projection, ``q_rope`` BF16 [tokens, heads, 64], rotated; either may be
    strided, ``q`` the transposed output of a batched product, for one.  ``scale``
    is that of the scores: (the width of a head's expanded key) ** -0.5.  A query
    sees the tokens up to its own position; one that sees none gets zeros, one
    that sees some and holds a NaN or an infinity gets NaN.

    Returns ``out`` (BF16 [tokens, heads, latent_dim], weighted sums of latents,
    which the heads' value up-projection takes), and with ``return_lse`` also the
    logarithm of each row's sum of exponentials (float32 [tokens, heads]; ``lse``
    may supply it).  Rows of no sequence are not written.  The kernel is chosen by the
    mean number of query rows (tokens times heads) of a sequence, so that chunks and
    single tokens are served faster in calls of their own (31 tokens and a chunk of 512,
    all over 8000, 16 heads: 47 + 163 us, in one call 242).  Nothing here has a gradient.  ``workspace`` is a uint8 GPU tensor of
    ``latent_attention_workspace_bytes`` that no overlapping call uses; by default
    each call takes one from torch's allocator.
    """
    import torch

    index, dim = cache._index, cache.latent_dim
    tokens = q.shape[0]
    batch, n = _batch(cache, tokens, block_table, seq_lens, query_start)
    qp, qt, qh = _rows(q, tokens, None, dim, index, "q")
    heads = _heads(q, tokens)
    rp, rt, rh = _rows(q_rope, tokens, heads, ROPE_DIM, index, "q_rope")
    scale = float(scale)
    if scale - scale != 0.0 or abs(scale) > 2e38:
        raise ValueError(f"scale must be a finite float32, got {scale}")
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=cache.device)
        op, ot, oh = out.data_ptr(), heads * dim, dim
    else:
        op, ot, oh = _rows(out, tokens, heads, dim, index, "out")
        _writable(out, ot, oh, "out")
    lp = 0
    if lse is not None or return_lse:
        if lse is None:
            lse = torch.empty((tokens, heads), dtype=torch.float32, device=cache.device)
        elif lse.dtype is not torch.float32 or tuple(lse.shape) != (tokens, heads) \
                or not lse.is_contiguous() or lse.get_device() != index:
            raise ValueError(f"lse must be contiguous float32 {(tokens, heads)} on the cache's device")
        lp = lse.data_ptr()
    if tokens > 0 and n > 0:
        lib = load_library()
        need = lib.fp8bq_latent_attention_workspace_bytes(cache._packed, batch, heads, tokens)
        wp = size = 0
        if workspace is not None:
            if workspace.get_device() != index or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on the cache's device")
            wp, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
            wp, size = workspace.data_ptr(), need
        packed = _QUERY.pack(qp, rp, op, lp, qt, qh, rt, rh, ot, oh, tokens, heads, scale)
        status = _run(cache, lib.fp8bq_latent_attention, cache._packed, batch, packed, wp, size)
        if status:
            _check("fp8bq_latent_attention", status)
    return (out, lse) if return_lse else out


class _On:
    """What ``_run`` reads of a cache, for calls without one."""

    def __init__(self, x):
        self._index, self.device = x.get_device(), x.device


def latent_prompt_attention(q, k, k_rope, v, query_start, key_start=None, *, scale=None, out=None, return_lse=False,
                            lse=None):
    """Causal attention in the expanded form (``fp8bq_latent_prompt_attention``):
    prompts, against keys and values that the up-projections have made of the
    latents.

    ``q`` is BF16 [tokens, heads, head_dim + 64], the rotated channels last,
    ``k`` and ``v`` BF16 [keys, heads, head_dim] (64 or 128; often two views of one
    projection's output), ``k_rope`` BF16 [keys, 64], rotated, for all heads; their
    token strides are below 2^23 elements.
    Sequence b's queries are the rows ``query_start[b]`` to ``query_start[b + 1]``
    (int32 [sequences + 1]), its keys the rows ``key_start[b]`` to
    ``key_start[b + 1]``, by default the same ones; its queries are its last
    tokens.  ``scale`` defaults to (head_dim + 64) ** -0.5.

    Returns ``out`` (BF16 [tokens, heads, head_dim]), and with ``return_lse`` also
    the logarithm of each row's sum of exponentials (float32 [tokens, heads];
    ``lse`` may supply it).  A row that sees nothing gets zeros; rows of no
    sequence are not written.  Nothing here has a gradient.
    """
    import torch

    if not q.is_cuda:
        raise TypeError("q must be on a GPU (there is no CPU implementation)")
    on = _On(q)
    index = on._index
    if v.dim() != 3 or v.shape[2] not in (64, 128):
        raise ValueError(f"v must be [keys, heads, 64 or 128], got {tuple(v.shape)}")
    tokens, (keys, _, dim) = q.shape[0], v.shape
    qp, qt, qh = _rows(q, tokens, None, dim + ROPE_DIM, index, "q")
    heads = _heads(q, tokens)
    if keys * heads > MAX_ROWS:
        raise ValueError(f"at most {MAX_ROWS} rows (keys x heads) per call")
    kp, kt, kh = _rows(k, keys, heads, dim, index, "k")
    vp, vt, vh = _rows(v, keys, heads, dim, index, "v")
    rp, rt = _flat_rows(k_rope, keys, ROPE_DIM, index, "k_rope")
    n = query_start.shape[0] - 1
    for x, what in ((query_start, "query_start"), (key_start, "key_start")):
        if x is None:
            continue
        if x.dtype is not torch.int32:
            raise TypeError(f"{what} must be int32")
        if x.dim() != 1 or n < 0 or x.shape[0] != n + 1 or not x.is_contiguous():
            raise ValueError(f"{what} must be contiguous [sequences + 1]")
        if x.get_device() != index:
            raise ValueError(f"{what} must be on {on.device}")
    if key_start is None and keys != tokens:
        raise ValueError(f"without key_start every query has a key: got {tokens} queries, {keys} keys")
    scale = (dim + ROPE_DIM) ** -0.5 if scale is None else float(scale)
    if scale - scale != 0.0 or abs(scale) > 2e38:
        raise ValueError(f"scale must be a finite float32, got {scale}")
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=on.device)
        op, ot, oh = out.data_ptr(), heads * dim, dim
    else:
        op, ot, oh = _rows(out, tokens, heads, dim, index, "out")
        _writable(out, ot, oh, "out")
    lp = 0
    if lse is not None or return_lse:
        if lse is None:
            lse = torch.empty((tokens, heads), dtype=torch.float32, device=on.device)
        elif lse.dtype is not torch.float32 or tuple(lse.shape) != (tokens, heads) \
                or not lse.is_contiguous() or lse.get_device() != index:
            raise ValueError(f"lse must be contiguous float32 {(tokens, heads)} on q's device")
        lp = lse.data_ptr()
    if tokens > 0 and n > 0:
        packed = _PROMPT.pack(qp, kp, rp, vp, op, lp, query_start.data_ptr(),
                              0 if key_start is None else key_start.data_ptr(), qt, qh, kt, kh, rt, vt, vh, ot, oh,
                              tokens, keys, heads, dim, n, scale)
        status = _run(on, load_library().fp8bq_latent_prompt_attention, packed)
        if status:
            _check("fp8bq_latent_prompt_attention", status)
    return (out, lse) if return_lse else out
