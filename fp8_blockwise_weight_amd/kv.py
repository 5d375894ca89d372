"""The blockwise e4m3 key/value cache: ``KvCache``, ``kv_append``, ``kv_attention``.

Argument checks and marshalling only; the work runs in the HIP kernels of
``libfp8bq.so`` on the current stream.  A cache page of one head is a block of
tokens by channels with one fp32 descale, as ``quantize`` makes of a weight's
tiles, except that the descale is a power of two, so that a page can take in
tokens one by one (include/fp8bq.h has the arithmetic).
"""

import struct

from . import _check, load_library

PAGE_SIZES = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128, 192, 256)
MAX_ROWS = 1 << 25             # tokens x query heads of a call

_CACHE = struct.Struct("=QQQQqiiii")       # fp8bq_kv_cache
_BUFFER = struct.Struct("=Qq")             # fp8bq_page_buffer
_BATCH = struct.Struct("=QQQqii")          # fp8bq_kv_batch
_TOKENS = struct.Struct("=QQQQQQ10qiiii")  # fp8bq_kv_tokens
_QUERY = struct.Struct("=QQQ5qiifi")       # fp8bq_kv_query


class KvCache:
    """The buffers of a paged cache, checked once; other buffers are another
    ``KvCache`` (the attributes are read-only).

    ``k`` is float8_e4m3fn [pages, kv_heads, page_size, head_dim], ``v``
    float8_e4m3fn [pages, kv_heads, head_dim, page_size] (a channel's tokens
    side by side) and ``k_scale``, ``v_scale`` are float32 [pages, kv_heads],
    all contiguous on one GPU.  ``KvCache.empty`` allocates them.  Dequantize a
    page with ``dequantize(cache.k[i, h], cache.k_scale[i, h].view(1, 1),
    (page_size, head_dim))``.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "num_pages", "page_size", "kv_heads", "head_dim",
                 "device", "_index", "_packed", "_buffers")

    def __init__(self, k, v, k_scale, v_scale):
        import torch

        for t, what, dims in ((k, "k", 4), (v, "v", 4), (k_scale, "k_scale", 2), (v_scale, "v_scale", 2)):
            if not isinstance(t, torch.Tensor) or t.dim() != dims:
                raise TypeError(f"{what} must be a {dims}-D tensor")
            if t.dtype != (torch.float8_e4m3fn if dims == 4 else torch.float32):
                raise TypeError(f"{what} must be {'float8_e4m3fn' if dims == 4 else 'float32'}, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous")
        pages, heads, size, dim = k.shape
        if size not in PAGE_SIZES:
            raise ValueError(f"page_size must be one of {PAGE_SIZES}, got {size}")
        if dim not in HEAD_DIMS:
            raise ValueError(f"head_dim must be one of {HEAD_DIMS}, got {dim}")
        if pages < 1 or heads < 1:
            raise ValueError("a cache holds at least one page and one head")
        if tuple(v.shape) != (pages, heads, dim, size):
            raise ValueError(f"v has shape {tuple(v.shape)}, expected {(pages, heads, dim, size)}")
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if tuple(t.shape) != (pages, heads):
                raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(pages, heads)}")
        if k.data_ptr() % 16 or v.data_ptr() % 16:
            raise ValueError("k and v must be 16-byte aligned")
        for t in (k, v, k_scale, v_scale):
            if not t.is_cuda:
                raise TypeError("the cache must be on a GPU (there is no CPU implementation)")
            if t.device != k.device:
                raise ValueError("the cache's buffers must be on one device")
        packed = _CACHE.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                             pages, size, heads, dim, 0)
        buffers = b"".join(_BUFFER.pack(t.data_ptr(), t.numel() // pages * t.element_size())
                           for t in (k, v, k_scale, v_scale))
        for name, value in zip(self.__slots__, (k, v, k_scale, v_scale, pages, size, heads, dim, k.device,
                                                k.get_device(), packed, buffers)):
            object.__setattr__(self, name, value)

    # Calls go by the addresses taken above: another tensor put in a buffer's
    # place would change nothing that they read, and free what they do.
    def __setattr__(self, name, value):
        raise AttributeError(f"KvCache.{name} is read-only")

    def __delattr__(self, name):
        raise AttributeError(f"KvCache.{name} is read-only")

    # A copy, or one loaded from a file, takes its own buffers' addresses.
    def __reduce__(self):
        return KvCache, (self.k, self.v, self.k_scale, self.v_scale)

    @classmethod
    def empty(cls, num_pages, kv_heads, head_dim, page_size=64, device="cuda"):
        """A cache of ``num_pages`` zeroed pages."""
        import torch

        if page_size not in PAGE_SIZES:
            raise ValueError(f"page_size must be one of {PAGE_SIZES}, got {page_size}")
        f8, f32 = torch.float8_e4m3fn, torch.float32
        return cls(torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=f8, device=device),
                   torch.zeros((num_pages, kv_heads, head_dim, page_size), dtype=f8, device=device),
                   torch.ones((num_pages, kv_heads), dtype=f32, device=device),
                   torch.ones((num_pages, kv_heads), dtype=f32, device=device))


def _batch(cache, tokens, block_table, seq_lens, query_start):
    """The packed ``fp8bq_kv_batch``, and the number of sequences."""
    import torch

    i32, index = torch.int32, cache._index
    if block_table.dtype is not i32 or seq_lens.dtype is not i32:
        raise TypeError("block_table and seq_lens must be int32")
    if block_table.dim() != 2 or seq_lens.dim() != 1 or block_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("block_table must be [sequences, pages] and seq_lens [sequences]")
    if block_table.get_device() != index or seq_lens.get_device() != index:
        raise ValueError(f"block_table and seq_lens must be on {cache.device}")
    n, width = block_table.shape
    if (width > 1 and block_table.stride(1) != 1) or (n > 1 and block_table.stride(0) < width) \
            or not seq_lens.is_contiguous():
        raise ValueError("block_table's rows and seq_lens must be contiguous")
    starts = 0
    if query_start is None:
        if n != tokens:
            raise ValueError(f"without query_start every sequence has one token: got {tokens} tokens, {n} sequences")
    else:
        if query_start.dtype is not i32:
            raise TypeError("query_start must be int32")
        if query_start.dim() != 1 or query_start.shape[0] != n + 1 or not query_start.is_contiguous():
            raise ValueError("query_start must be contiguous [sequences + 1]")
        if query_start.get_device() != index:
            raise ValueError(f"query_start must be on {cache.device}")
        starts = query_start.data_ptr()
    return _BATCH.pack(block_table.data_ptr(), seq_lens.data_ptr(), starts,
                       block_table.stride(0) if n > 1 else width, n, width), n


def _rows(x, tokens, heads, dim, index, what):
    """(pointer, token stride, head stride) of BF16 rows [tokens, heads, dim]."""
    import torch

    if x.dtype is not torch.bfloat16 or x.dim() != 3:
        raise TypeError(f"{what} must be a 3-D torch.bfloat16 tensor")
    t, h, d = x.shape
    if t != tokens or d != dim or (heads is not None and h != heads):
        raise ValueError(f"{what} has shape {(t, h, d)}, expected {(tokens, heads if heads else 'heads', dim)}")
    if x.get_device() != index:
        raise ValueError(f"{what} must be on the cache's device")
    st, sh, sd = x.stride()
    ptr = x.data_ptr()
    if t <= 1:
        st = 0
    if h <= 1:
        sh = 0
    if sd != 1 or ptr & 15 or st & 7 or sh & 7 or st < 0 or sh < 0:
        raise ValueError(f"{what}'s rows must be contiguous and 16-byte aligned")
    return ptr, st, sh


def _writable(x, stride_t, stride_h, what):
    """Rows that are written may not share elements."""
    t, h, d = x.shape
    if (h > 1 and stride_h < d) or (t > 1 and stride_t < d) or \
            (t > 1 and h > 1 and stride_t < (h - 1) * stride_h + d and stride_h < (t - 1) * stride_t + d):
        raise ValueError(f"{what}'s rows must not overlap")


def _run(cache, f, *args):
    """``f(*args, stream)`` on the current stream of the cache's device.

    The stream's handle is taken from torch's own lookup: building a Stream
    object around it took 2.8 us of a 12.5 us call.
    """
    import torch

    index = cache._index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        return f(*args, stream)
    with torch.cuda.device(index):
        return f(*args, stream)


def kv_append(cache, k, v, block_table, seq_lens, query_start=None, *, q=None, q_out=None, cos=None,
              sin=None, interleaved=False):
    """Store new keys and values in ``cache``, keys rotated by their positions
    (``fp8bq_kv_append``).

    ``k`` and ``v`` are BF16 [tokens, kv_heads, head_dim]; rows may be strided
    views of one projection's output.  ``seq_lens`` (int32 [sequences]) counts
    each sequence's tokens with the new ones, ``block_table`` (int32
    [sequences, pages]) names its pages, and its new tokens are the rows
    ``query_start[b]`` to ``query_start[b + 1]`` (int32 [sequences + 1];
    without it, row b).  ``cos`` and ``sin`` (float32 [positions, rot / 2])
    rotate the first ``rot`` channels of keys and queries, in halves or, with
    ``interleaved``, adjacent pairs; without them nothing is rotated.  Tokens at
    positions beyond their rows are left out.

    Returns the rotated queries where ``q`` (BF16 [tokens, q_heads, head_dim])
    is given, in ``q_out`` (which may be ``q``) or a new tensor, else None.
    Rows of no sequence (padding before ``query_start[0]`` or from
    ``query_start[-1]`` on) and of tokens that are left out are not written:
    what ``q_out`` held stays there, and a new tensor holds anything.
    """
    import torch

    tokens = k.shape[0]
    index, heads, dim = cache._index, cache.kv_heads, cache.head_dim
    batch, n = _batch(cache, tokens, block_table, seq_lens, query_start)
    kp, kt, kh = _rows(k, tokens, heads, dim, index, "k")
    vp, vt, vh = _rows(v, tokens, heads, dim, index, "v")
    rot = positions = cp = sp = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin belong together")
    if cos is not None:
        if cos.dtype is not torch.float32 or sin.dtype is not torch.float32:
            raise TypeError("cos and sin must be float32")
        if cos.dim() != 2 or cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous [positions, rot / 2]")
        positions, half = cos.shape
        rot = 2 * half
        if rot > dim or rot % 16:
            raise ValueError(f"rotated channels must be a multiple of 16 up to {dim}, got {rot}")
        cp, sp = cos.data_ptr(), sin.data_ptr()
        if rot and (cos.get_device() != index or sin.get_device() != index or (cp | sp) & 15):
            raise ValueError("cos and sin must be on the cache's device and 16-byte aligned")
    qp = qt = qh = op = ot = oh = q_heads = 0
    if q is not None:
        qp, qt, qh = _rows(q, tokens, None, dim, index, "q")
        q_heads = q.shape[1]
        if q_heads < 1 or q_heads % heads:
            raise ValueError(f"q's heads must be a multiple of {heads}, got {q_heads}")
        if q_out is None:
            q_out = torch.empty((tokens, q_heads, dim), dtype=torch.bfloat16, device=cache.device)
        op, ot, oh = _rows(q_out, tokens, q_heads, dim, index, "q_out")
        _writable(q_out, ot, oh, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if tokens * max(q_heads, heads) > MAX_ROWS:
        raise ValueError(f"at most {MAX_ROWS} rows (tokens x heads) per call")
    if tokens == 0 or n == 0:
        return q_out
    packed = _TOKENS.pack(kp, vp, qp, op, cp, sp, kt, kh, vt, vh, qt, qh, ot, oh, tokens, positions,
                          q_heads, rot, int(bool(interleaved)), 0)
    status = _run(cache, load_library().fp8bq_kv_append, cache._packed, batch, packed)
    if status:
        _check("fp8bq_kv_append", status)
    return q_out


def kv_attention_workspace_bytes(cache, q, block_table):
    """Bytes of ``kv_attention``'s workspace for these tensors: by their shapes
    alone."""
    n, width = block_table.shape
    batch = _BATCH.pack(0, 0, 0, width, n, width)
    return int(load_library().fp8bq_kv_attention_workspace_bytes(cache._packed, batch, q.shape[1], q.shape[0]))


def kv_attention(cache, q, block_table, seq_lens, query_start=None, *, scale=None, window=0, out=None,
                 return_lse=False, lse=None, workspace=None):
    """Attention of ``q`` (BF16 [tokens, q_heads, head_dim]) over ``cache``
    (``fp8bq_kv_attention``), one query token per sequence or, with
    ``query_start``, any number of each, the last ones of their sequence.

    Arguments as in ``kv_append``.  A query sees the tokens up to its own
    position, with ``window`` no more than that many of them; one that sees
    none gets zeros, one that sees some and holds a NaN or an infinity gets NaN.
    ``scale`` defaults to head_dim ** -0.5.  Returns ``out``
    (BF16, like q), and with ``return_lse`` also the logarithm of each row's
    sum of exponentials (float32 [tokens, q_heads]; ``lse`` may supply it).
    Rows of no sequence (padding before ``query_start[0]`` or from
    ``query_start[-1]`` on) are not written: what ``out`` and ``lse`` held stays
    there, and new tensors hold anything.
    The kernel is chosen by the mean number of query tokens, so that prompts
    and single tokens are served faster in calls of their own (128 tokens over
    8192 each and a prompt of 2048: 337 + 58 us, in one call 553).  Nothing here
    has a gradient.
    ``workspace`` is a uint8 GPU tensor of ``kv_attention_workspace_bytes`` that
    no overlapping call uses; by default each call takes one from torch's
    allocator.
    """
    import torch

    index, heads, dim = cache._index, cache.kv_heads, cache.head_dim
    tokens = q.shape[0]
    batch, n = _batch(cache, tokens, block_table, seq_lens, query_start)
    qp, qt, qh = _rows(q, tokens, None, dim, index, "q")
    q_heads = q.shape[1]
    if q_heads < 1 or q_heads % heads:
        raise ValueError(f"q's heads must be a multiple of {heads}, got {q_heads}")
    if tokens * q_heads > MAX_ROWS:
        raise ValueError(f"at most {MAX_ROWS} rows (tokens x heads) per call")
    scale = dim ** -0.5 if scale is None else float(scale)
    if scale - scale != 0.0 or abs(scale) > 2e38:
        raise ValueError(f"scale must be a finite float32, got {scale}")
    if not 0 <= window <= 0x7FFFFFFF:
        raise ValueError(f"window must be 0 (none) or a positive number of tokens, got {window}")
    if out is None:
        out = torch.empty((tokens, q_heads, dim), dtype=torch.bfloat16, device=cache.device)
        op, ot, oh = out.data_ptr(), q_heads * dim, dim
    else:
        op, ot, oh = _rows(out, tokens, q_heads, dim, index, "out")
        _writable(out, ot, oh, "out")
    lp = 0
    if lse is not None or return_lse:
        if lse is None:
            lse = torch.empty((tokens, q_heads), dtype=torch.float32, device=cache.device)
        elif lse.dtype is not torch.float32 or tuple(lse.shape) != (tokens, q_heads) \
                or not lse.is_contiguous() or lse.get_device() != index:
            raise ValueError(f"lse must be contiguous float32 {(tokens, q_heads)} on the cache's device")
        lp = lse.data_ptr()
    if tokens > 0 and n > 0:
        lib = load_library()
        need = lib.fp8bq_kv_attention_workspace_bytes(cache._packed, batch, q_heads, tokens)
        wp = size = 0
        if workspace is not None:
            if workspace.get_device() != index or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on the cache's device")
            wp, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
            wp, size = workspace.data_ptr(), need
        packed = _QUERY.pack(qp, op, lp, qt, qh, ot, oh, tokens, q_heads, window, scale, 0)
        status = _run(cache, lib.fp8bq_kv_attention, cache._packed, batch, packed, wp, size)
        if status:
            _check("fp8bq_kv_attention", status)
    return (out, lse) if return_lse else out
