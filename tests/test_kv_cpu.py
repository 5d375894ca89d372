"""The key/value cache's calls without a GPU: every bad argument is refused
before a device is touched, shapes alone size the workspace, and the plain
reference that the GPU tests compare with meets the format's definition."""

import concurrent.futures
import ctypes
import functools

import numpy as np
import pytest
import torch

import fp8_blockwise_weight_amd as fq
from fp8_blockwise_weight_amd import kv
import kv_reference as ref

INVALID, WORKSPACE = fq.ERR_INVALID_ARGUMENT, fq.ERR_WORKSPACE
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fake addresses are passed only where no GPU is visible")


def on_a_thread(test):
    """For calls that pass the checks and find no GPU: the error that they leave
    is their thread's own."""
    @functools.wraps(test)
    def run(*args, **kw):
        with concurrent.futures.ThreadPoolExecutor(1) as pool:
            pool.submit(test, *args, **kw).result()
    return run


# Fake, never dereferenced addresses.
K, V, KS, VS, TB, LN, ST, A, B, C, D, CO, SI, WS = (0x10_0000_0000 * i for i in range(1, 15))


def cache(k=K, v=V, ks=KS, vs=VS, pages=100, size=64, heads=8, dim=128):
    return kv._CACHE.pack(k, v, ks, vs, pages, size, heads, dim, 0)


def batch(table=TB, lens=LN, starts=ST, stride=40, count=4, width=40):
    return kv._BATCH.pack(table, lens, starts, stride, count, width)


def tokens(k=A, v=B, q=C, q_out=D, cos=CO, sin=SI, strides=(1024, 128, 1024, 128, 4096, 128, 4096, 128), tokens=9,
           positions=4096, q_heads=32, rot=128, interleaved=0):
    return kv._TOKENS.pack(k, v, q, q_out, cos, sin, *strides, tokens, positions, q_heads, rot, interleaved, 0)


def query(q=A, out=B, lse=0, strides=(4096, 128, 4096, 128), tokens=9, q_heads=32, window=0, scale=0.1):
    return kv._QUERY.pack(q, out, lse, *strides, tokens, q_heads, window, scale, 0)


BAD_CACHES = [dict(k=0), dict(v=0), dict(ks=0), dict(vs=0), dict(k=K + 8), dict(v=V + 1), dict(ks=KS + 2),
              dict(pages=0), dict(pages=1 << 31), dict(size=8), dict(size=48), dict(size=512), dict(heads=0),
              dict(heads=-1), dict(heads=1 << 16), dict(dim=0), dict(dim=96), dict(dim=320), dict(v=K + 16),
              dict(ks=K + 64), dict(vs=KS + 4)]
BAD_BATCHES = [dict(table=0), dict(lens=0), dict(stride=39), dict(width=-1), dict(count=-1), dict(count=1 << 21),
               dict(table=TB + 2), dict(lens=LN + 1), dict(starts=ST + 2), dict(starts=0)]


@no_gpu
@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_cache(bad):
    lib = fq.load_library()
    assert lib.fp8bq_kv_append(cache(**bad), batch(), tokens(), None) == INVALID
    assert lib.fp8bq_kv_attention(cache(**bad), batch(), query(), WS, 1 << 40, None) == INVALID


@no_gpu
@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_bad_batch(bad):
    lib = fq.load_library()
    assert lib.fp8bq_kv_append(cache(), batch(**bad), tokens(), None) == INVALID
    assert lib.fp8bq_kv_attention(cache(), batch(**bad), query(), WS, 1 << 40, None) == INVALID


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(k=0), dict(v=0), dict(k=A + 8), dict(v=B + 2), dict(q_out=0), dict(q=C + 4), dict(q_out=D + 8),
    dict(strides=(1020, 128, 1024, 128, 4096, 128, 4096, 128)), dict(strides=(1024, 132, 1024, 128, 4096, 128, 4096, 128)),
    dict(strides=(1024, 128, 1024, 128, 4096, 128, -4096, 128)), dict(tokens=-1), dict(q_heads=0), dict(q_heads=12),
    dict(rot=-16), dict(rot=24), dict(rot=144), dict(cos=0), dict(sin=0), dict(cos=CO + 4), dict(positions=-1),
    dict(tokens=1 << 25), dict(k=K + 4096), dict(v=V + 4096), dict(q_out=K - 4096), dict(q_out=VS),
    dict(strides=(1 << 36, 128, 1024, 128, 4096, 128, 4096, 128)),
])
def test_bad_tokens(bad):
    assert fq.load_library().fp8bq_kv_append(cache(), batch(), tokens(**bad), None) == INVALID


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(q=0), dict(out=0), dict(q=A + 8), dict(out=B + 2), dict(lse=2), dict(strides=(4100, 128, 4096, 128)),
    dict(strides=(4096, 128, 4096, -128)), dict(tokens=-1), dict(tokens=1 << 25), dict(q_heads=0), dict(q_heads=-8),
    dict(q_heads=20), dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(scale=3e38), dict(out=K + 64), dict(out=V - 128), dict(lse=KS), dict(out=B, lse=B + 64), dict(out=WS), dict(lse=WS),
    dict(strides=(4096, 128, 4096, 1 << 36)),
])
def test_bad_query(bad):
    assert fq.load_library().fp8bq_kv_attention(cache(), batch(), query(**bad), WS, 1 << 40, None) == INVALID


@no_gpu
@pytest.mark.parametrize("token,head", [(0, 128), (4096, 0), (4096, 120), (128, 128), (2048, 128),
                                         (120, 4096), (128, 1024)])
def test_written_rows_that_overlap(token, head):
    lib = fq.load_library()
    bad = tokens(strides=(1024, 128, 1024, 128, 4096, 128, token, head))
    assert lib.fp8bq_kv_append(cache(), batch(), bad, None) == INVALID
    bad = query(strides=(4096, 128, token, head))
    assert lib.fp8bq_kv_attention(cache(), batch(), bad, WS, 1 << 40, None) == INVALID


ROWS = 9 * 4096 * 2   # bytes of nine tokens of 32 heads


@no_gpu
@pytest.mark.parametrize("at,strides,ok", [
    (A, (4096, 128), True),                # in place
    (A + ROWS, (4096, 128), True),         # behind the queries
    (A + 8192, (4096, 128), False),        # a token further on
    (A - 256, (4096, 128), False),         # a head before
    (A, (128, 9 * 128), False),            # the same memory in another order
    (A + 16, (4096, 128), False),
])
@on_a_thread
def test_outputs_over_their_queries(at, strides, ok):
    lib = fq.load_library()
    status = lib.fp8bq_kv_attention(cache(), batch(), query(out=at, strides=(4096, 128, *strides)), WS, 1 << 40, None)
    assert (status != INVALID) == ok
    status = lib.fp8bq_kv_append(cache(), batch(),
                                 tokens(k=C, v=D, q=A, q_out=at, strides=(1024, 128, 1024, 128, 4096, 128, *strides)),
                                 None)
    assert (status != INVALID) == ok


@no_gpu
@pytest.mark.parametrize("token,head,k,v,q_out,ok", [
    (6144, 128, 4096, 5120, 0, True),      # q, k and v of one projection, queries in place
    (6144, 128, 4096, 5120, 128, False),
    (6144, 128, 4088, 5120, 0, False),     # k begins within the queries
    (6144, 128, 4096, 5128, 0, False),     # v ends in the next token's queries
    (128, 3 * 9 * 128, 9 * 128, 18 * 128, 0, True),    # head by head
    (128, 3 * 9 * 128, 9 * 128 - 8, 18 * 128, 0, False),
    (128, 3 * 9 * 128, 18 * 128, 18 * 128 + 8, 0, False),
])
@on_a_thread
def test_queries_beside_keys_and_values(token, head, k, v, q_out, ok):
    args = tokens(k=A + 2 * k, v=A + 2 * v, q=A, q_out=A + 2 * q_out, strides=(token, head) * 4)
    assert (fq.load_library().fp8bq_kv_append(cache(), batch(), args, None) != INVALID) == ok


@no_gpu
def test_null_structs_and_workspace():
    lib = fq.load_library()
    assert lib.fp8bq_kv_append(None, batch(), tokens(), None) == INVALID
    assert lib.fp8bq_kv_append(cache(), None, tokens(), None) == INVALID
    assert lib.fp8bq_kv_append(cache(), batch(), None, None) == INVALID
    assert lib.fp8bq_kv_attention(None, batch(), query(), WS, 1 << 40, None) == INVALID
    assert lib.fp8bq_kv_attention(cache(), None, query(), WS, 1 << 40, None) == INVALID
    assert lib.fp8bq_kv_attention(cache(), batch(), None, WS, 1 << 40, None) == INVALID
    need = lib.fp8bq_kv_attention_workspace_bytes(cache(), batch(), 32, 9)
    assert need > 0
    assert lib.fp8bq_kv_attention(cache(), batch(), query(), None, need, None) == WORKSPACE
    assert lib.fp8bq_kv_attention(cache(), batch(), query(), WS, need - 1, None) == WORKSPACE
    assert lib.fp8bq_kv_attention(cache(), batch(), query(), WS + 8, need, None) == WORKSPACE


def test_nothing_to_do_touches_no_device():
    lib = fq.load_library()
    assert lib.fp8bq_kv_append(cache(), batch(count=0), tokens(), None) == fq.OK
    assert lib.fp8bq_kv_append(cache(), batch(), tokens(tokens=0), None) == fq.OK
    assert lib.fp8bq_kv_attention(cache(), batch(count=0), query(), None, 0, None) == fq.OK
    assert lib.fp8bq_kv_attention(cache(), batch(), query(tokens=0), None, 0, None) == fq.OK


def test_workspace_depends_on_shapes_alone():
    f = fq.load_library().fp8bq_kv_attention_workspace_bytes
    none = dict(table=0, lens=0, starts=0)
    for c, b, heads, tokens in ((dict(heads=0), {}, 32, 9), (dict(size=24), {}, 32, 9), ({}, dict(count=0), 32, 9),
                                ({}, {}, 12, 9), ({}, {}, 32, 0), ({}, {}, 32, 1 << 40), ({}, dict(width=-1), 32, 9)):
        assert f(cache(**c), batch(**none, **b), heads, tokens) == 0
    assert f(None, batch(), 32, 9) == 0 and f(cache(), None, 32, 9) == 0
    assert 0 < f(cache(k=0, v=0, ks=0, vs=0), batch(**none, width=10000, stride=10000, count=1), 32, 1) < 1 << 28
    assert f(cache(), batch(**none, width=16, count=9), 32, 9) == 0          # short tables: no splits
    assert f(cache(), batch(**none, width=17, stride=17, count=9), 32, 9) > 0


@no_gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@on_a_thread
def test_a_window_never_needs_more_workspace(dim):
    """The size is asked for without the window that a call then has."""
    lib, refused = fq.load_library(), []
    for heads, group in ((1, 1), (1, 16), (4, 8), (8, 4), (16, 3)):
        one = cache(heads=heads, dim=dim)
        for count in (1, 3, 9, 20, 35, 40, 60, 75, 130):
            for new in (1, 3, 4, 12, 18, 40, 300):
                for width in (1, 7, 12, 17, 20, 33, 500):
                    held = batch(count=count, width=width, stride=width)
                    tokens = count * new
                    need = lib.fp8bq_kv_attention_workspace_bytes(one, held, heads * group, tokens)
                    for window in (1, 100, 400, 500, 600, 900, 1000, 1900, 5000):
                        q = query(strides=(heads * group * dim, dim) * 2, tokens=tokens, q_heads=heads * group,
                                  window=window)
                        if lib.fp8bq_kv_attention(one, held, q, WS, need, None) == WORKSPACE:
                            refused.append((heads, group, count, new, width, window))
    assert not refused, (len(refused), refused[:5])


def test_struct_sizes():
    assert (kv._CACHE.size, kv._BATCH.size, kv._TOKENS.size, kv._QUERY.size) == (56, 40, 144, 80)


def test_cpu_tensors_are_refused():
    k = torch.zeros((2, 1, 16, 64), dtype=torch.float8_e4m3fn)
    v = torch.zeros((2, 1, 64, 16), dtype=torch.float8_e4m3fn)
    s = torch.ones((2, 1))
    with pytest.raises(TypeError, match="GPU"):
        fq.KvCache(k, v, s, s.clone())
    with pytest.raises(TypeError, match="float8"):
        fq.KvCache(k.float(), v, s, s)
    with pytest.raises(ValueError, match="expected"):
        fq.KvCache(k, k, s, s)
    with pytest.raises(ValueError, match="page_size"):
        fq.KvCache(k[:, :, :8].contiguous(), v, s, s)
    with pytest.raises(ValueError, match="head_dim"):
        fq.KvCache(k[..., :32].contiguous(), v, s, s)
    with pytest.raises(ValueError, match="contiguous"):
        fq.KvCache(k, v.transpose(2, 3), s, s)
    with pytest.raises(ValueError, match="k_scale"):
        fq.KvCache(k, v, s[:1], s)
    with pytest.raises(TypeError, match="4-D"):
        fq.KvCache(k[0], v, s, s)


def test_reference_codes_are_the_format():
    """Every code decodes and encodes to itself, and midpoints go to even."""
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert np.array_equal(ref.encode(ref.decode(codes)), codes)
    pos = ref.decode(np.arange(0, 127, dtype=np.uint8))
    mids = (pos[:-1] + pos[1:]) / 2
    want = np.arange(0, 126) + (np.arange(0, 126) & 1)
    assert np.array_equal(ref.encode(mids), want.astype(np.uint8))


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.0, 2.0 ** -42),
                                       (3.0e38, 2.0 ** 120), (7.0, 2.0 ** -6), (6.9, 2.0 ** -6), (7.1, 2.0 ** -5)])
def test_reference_scale(amax, want):
    s = ref.fit(amax)
    assert s == want and 448.0 * s >= amax and (amax < 1e-9 or 448.0 * s / 2 < amax)


@pytest.mark.parametrize("dim,page,heads,group,lens,new,window", [
    (64, 16, 2, 3, [40, 17], [5, 17], 0), (128, 32, 1, 2, [90, 33], [9, 1], 20),
])
def test_reference_attention_of_long_is_the_same(dim, page, heads, group, lens, new, window):
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 126, (9, heads, page, dim), generator=g).to(torch.uint8).numpy()
    turned = np.ascontiguousarray(codes[::-1].transpose(0, 1, 3, 2)) | 0x80
    scales = [(0.001 + torch.rand((9, heads), generator=g)).numpy() for _ in range(2)]
    q = torch.randn((sum(new), heads * group, dim), generator=g).to(torch.bfloat16)
    args = ([codes, turned, *scales], q, [[4, 1, 3, 0], [2, 5, 8, 7]], lens, [0, new[0], sum(new)])
    for a, b in zip(ref.attention(*args, window=window), ref.attention_of_long(*args, window=window)):
        assert torch.allclose(a, b, rtol=1e-9, atol=0)


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(q=WS), dict(q=WS - ROWS + 16), dict(q=WS + 4096), dict(lse=A), dict(lse=A + ROWS - 4), dict(lse=A - 9 * 32 * 4 + 4),
    dict(q=WS, out=WS),
])
def test_sums_and_workspace_over_the_queries(bad):
    """Rows that finish early are written while others still read their queries."""
    lib = fq.load_library()
    need = lib.fp8bq_kv_attention_workspace_bytes(cache(), batch(), 32, 9)
    assert need > 4096
    assert lib.fp8bq_kv_attention(cache(), batch(), query(**bad), WS, need, None) == INVALID


@no_gpu
@pytest.mark.parametrize("good", [dict(q=WS - ROWS), dict(lse=A + ROWS), dict(lse=A - 9 * 32 * 4)])
@on_a_thread
def test_sums_and_workspace_beside_the_queries(good):
    lib = fq.load_library()
    need = lib.fp8bq_kv_attention_workspace_bytes(cache(), batch(), 32, 9)
    assert lib.fp8bq_kv_attention(cache(), batch(), query(**good), WS, need, None) not in (INVALID, WORKSPACE)


LENGTHS, TABLE = 4 * 4, 4 * 4 * 40   # bytes of the batch's arrays (the offsets are one longer than the lengths)


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(table=B), dict(table=B - TABLE + 4), dict(lens=B + ROWS - 4), dict(lens=B - LENGTHS + 4), dict(starts=B - LENGTHS),
    dict(table=SI), dict(lens=SI + 64), dict(starts=SI + 9 * 32 * 4 - 4), dict(table=WS), dict(lens=WS + 400), dict(starts=WS),
])
def test_attention_over_the_arrays_it_reads(bad):
    lib = fq.load_library()
    need = lib.fp8bq_kv_attention_workspace_bytes(cache(), batch(), 32, 9)
    assert lib.fp8bq_kv_attention(cache(), batch(**bad), query(lse=SI), WS, need, None) == INVALID


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(table=D), dict(lens=D + ROWS - 4), dict(starts=D - LENGTHS), dict(table=K + 4096), dict(lens=V + 64),
    dict(starts=KS), dict(table=VS - TABLE + 4), dict(lens=K - 4), dict(starts=VS + 100 * 8 * 4 - 4),
])
def test_append_over_the_arrays_it_reads(bad):
    assert fq.load_library().fp8bq_kv_append(cache(), batch(**bad), tokens(), None) == INVALID


@no_gpu
@pytest.mark.parametrize("good", [
    dict(table=B - TABLE), dict(lens=B + ROWS), dict(starts=D - LENGTHS - 4), dict(lens=KS - LENGTHS), dict(starts=VS + 100 * 8 * 4),
    dict(table=K + 100 * 8 * 64 * 128), dict(table=0, width=0),
])
@on_a_thread
def test_arrays_beside_what_is_written(good):
    lib = fq.load_library()
    assert lib.fp8bq_kv_append(cache(), batch(**good), tokens(), None) != INVALID
    need = lib.fp8bq_kv_attention_workspace_bytes(cache(), batch(), 32, 9)
    assert lib.fp8bq_kv_attention(cache(), batch(**good), query(lse=SI), WS, need, None) not in (INVALID, WORKSPACE)


TURNS = 4096 * 64 * 4   # bytes of 4096 rows of cos or sin


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(q=K + 4096), dict(q=V - 128), dict(q=KS), dict(q=VS - ROWS + 16),
    dict(cos=K), dict(sin=V + 4096), dict(cos=KS - TURNS + 16), dict(sin=VS + 16), dict(cos=D), dict(sin=D + ROWS - 16),
    dict(cos=D - TURNS + 16), dict(cos=D - 64, positions=1 << 62), dict(q=CO, q_out=CO),
])
def test_append_over_its_inputs(bad):
    assert fq.load_library().fp8bq_kv_append(cache(), batch(), tokens(**bad), None) == INVALID


@no_gpu
@pytest.mark.parametrize("good", [
    dict(q=K - ROWS), dict(q=KS + 100 * 8 * 4), dict(cos=K - TURNS), dict(sin=D + ROWS), dict(cos=D - TURNS),
    dict(cos=K, sin=V, rot=0), dict(cos=K, sin=D, positions=0), dict(q=0, q_out=0, cos=D), dict(cos=K - TURNS // 2, rot=64),
])
@on_a_thread
def test_append_beside_its_inputs(good):
    assert fq.load_library().fp8bq_kv_append(cache(), batch(), tokens(**good), None) != INVALID


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "num_pages", "page_size", "kv_heads", "head_dim", "device"])
def test_a_cache_keeps_its_buffers(name):
    """Calls go by the addresses that the constructor took."""
    held = object.__new__(fq.KvCache)
    object.__setattr__(held, name, 1)
    with pytest.raises(AttributeError, match="read-only"):
        setattr(held, name, 2)
    with pytest.raises(AttributeError, match="read-only"):
        delattr(held, name)
    assert getattr(held, name) == 1


def test_a_copied_cache_is_made_anew():
    """From its buffers alone: no address goes along."""
    held = object.__new__(fq.KvCache)
    for i, name in enumerate(fq.KvCache.__slots__):
        object.__setattr__(held, name, i)
    for protocol in (2, 4):
        assert held.__reduce_ex__(protocol) == (fq.KvCache, (0, 1, 2, 3))
