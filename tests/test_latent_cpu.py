"""The latent cache's and the pages' calls without a GPU: every bad argument is
refused before a device is touched, shapes alone size the workspaces, and the
struct layouts are the header's."""

import ctypes
import os
import subprocess
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import fp8_blockwise_weight_amd as fq
import latent_reference as ref
from fp8_blockwise_weight_amd import kv, latent, pages
from test_kv_cpu import BAD_BATCHES, batch, no_gpu, on_a_thread

INVALID, WORKSPACE = fq.ERR_INVALID_ARGUMENT, fq.ERR_WORKSPACE
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Fake, never dereferenced addresses, beside those of test_kv_cpu's batch.
C, R, SC, X, XR, RO, Q, QO, CO, SI, OUT, LSE, WS = (0x10_0000_0000 * i for i in range(20, 33))


def cache(c=C, r=R, scale=SC, pages=100, size=64, dim=512):
    return latent._CACHE.pack(c, r, scale, pages, size, dim)


def tokens(c=X, r=XR, r_out=RO, q=Q, q_out=QO, cos=CO, sin=SI, strides=(576, 576, 64, 3200, 192, 1024, 64), tokens=9,
           positions=4096, heads=16, interleaved=0):
    return latent._TOKENS.pack(c, r, r_out, q, q_out, cos, sin, *strides, tokens, positions, heads, interleaved)


def query(q=Q, r=QO, out=OUT, lse=0, strides=(512, 4608, 3200, 192, 8192, 512), tokens=9, heads=16, scale=0.1):
    return latent._QUERY.pack(q, r, out, lse, *strides, tokens, heads, scale)


def prompt(q=Q, k=X, r=XR, v=X + 256, out=OUT, lse=0, q_at=CO, k_at=SI,
           strides=(3200, 192, 4096, 256, 64, 4096, 256, 2048, 128), tokens=9, keys=20, heads=16, dim=128, count=2, scale=0.1):
    return latent._PROMPT.pack(q, k, r, v, out, lse, q_at, k_at, *strides, tokens, keys, heads, dim, count, scale)


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(c=0), dict(r=0), dict(scale=0), dict(c=C + 8), dict(r=R + 2), dict(scale=SC + 2), dict(pages=0),
    dict(pages=1 << 31), dict(size=8), dict(size=48), dict(dim=0), dict(dim=128), dict(dim=576), dict(r=C + 64),
    dict(scale=R + 4)])
def test_bad_cache(bad):
    lib = fq.load_library()
    assert lib.fp8bq_latent_append(cache(**bad), batch(), tokens(), None) == INVALID
    assert lib.fp8bq_latent_attention(cache(**bad), batch(), query(), WS, 1 << 40, None) == INVALID


@no_gpu
@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_bad_batch(bad):
    lib = fq.load_library()
    assert lib.fp8bq_latent_append(cache(), batch(**bad), tokens(), None) == INVALID
    assert lib.fp8bq_latent_attention(cache(), batch(**bad), query(), WS, 1 << 40, None) == INVALID


def strides(base, **at):
    return tuple(at.get(f"s{i}", x) for i, x in enumerate(base))


T = (576, 576, 64, 3200, 192, 1024, 64)


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(c=0), dict(r=0), dict(c=X + 8), dict(r=XR + 2), dict(r_out=RO + 8), dict(q=Q + 4), dict(q_out=0),
    dict(q_out=QO + 8), dict(strides=strides(T, s0=580)), dict(strides=strides(T, s1=4)), dict(strides=strides(T, s2=56)),
    dict(strides=strides(T, s2=0)), dict(strides=strides(T, s3=1 << 36)), dict(strides=strides(T, s5=-1024)),
    dict(strides=strides(T, s6=56)), dict(strides=strides(T, s5=960)), dict(tokens=-1), dict(heads=0), dict(heads=1025),
    dict(tokens=1 << 25), dict(cos=0), dict(sin=0), dict(cos=CO + 4), dict(positions=-1),
    # what is written lies apart from what is read, and from itself
    dict(c=C + 1024), dict(r=SC), dict(q=R - 64), dict(q_out=C), dict(r_out=R + 128), dict(q_out=X), dict(r_out=X),
    dict(q_out=Q + 64), dict(r_out=XR + 64), dict(q_out=RO), dict(q_out=CO), dict(r_out=SI + 512), dict(cos=C),
    dict(sin=SC), dict(c=RO),
])
def test_bad_tokens(bad):
    assert fq.load_library().fp8bq_latent_append(cache(), batch(), tokens(**bad), None) == INVALID


@no_gpu
@on_a_thread
def test_tokens_that_pass(what=None):
    """In place, without queries, without rotation, outputs as slices of one
    tensor: these get as far as looking for a device."""
    lib = fq.load_library()
    for good in (dict(), dict(r_out=0), dict(q=0, q_out=0), dict(cos=0, sin=0), dict(r_out=XR, strides=strides(T, s2=576)),
                 dict(q_out=Q, strides=strides(T, s5=3200, s6=192)), dict(positions=0), dict(tokens=9, heads=1024,
                 strides=strides(T, s3=192 * 1024, s5=65536)),
                 dict(c=X, r=X + 1024, r_out=X + 1024, strides=strides(T, s2=576))):
        assert lib.fp8bq_latent_append(cache(), batch(), tokens(**good), None) == fq.ERR_HIP, good


A = (512, 4608, 3200, 192, 8192, 512)


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(q=0), dict(r=0), dict(out=0), dict(q=Q + 8), dict(r=QO + 2), dict(out=OUT + 8), dict(lse=LSE + 2),
    dict(strides=strides(A, s0=508)), dict(strides=strides(A, s3=1 << 36)), dict(strides=strides(A, s4=8190)),
    dict(strides=strides(A, s5=504)), dict(strides=strides(A, s4=0)), dict(tokens=-1), dict(tokens=1 << 25),
    dict(heads=0), dict(heads=1025), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=3e38),
    dict(out=C), dict(lse=R), dict(out=Q), dict(out=QO), dict(lse=Q), dict(lse=OUT + 64), dict(out=WS), dict(lse=WS + 4096),
    dict(q=WS), dict(r=WS + 64)])
def test_bad_query(bad):
    assert fq.load_library().fp8bq_latent_attention(cache(), batch(), query(**bad), WS, 1 << 40, None) == INVALID


@no_gpu
def test_workspace():
    lib = fq.load_library()
    b = batch(count=4, width=40)
    for heads in (1, 16, 40, 128, 1024):
        need = lib.fp8bq_latent_attention_workspace_bytes(cache(), b, heads, 9)
        assert need > 0
        for ws, size in ((0, need), (WS, need - 1), (WS + 8, need)):
            bad = query(heads=heads, strides=(512, 4608, 192 * heads, 192, 512 * heads, 512))
            assert lib.fp8bq_latent_attention(cache(), b, bad, ws, size, None) == WORKSPACE
        # addresses and pages say nothing
        assert need == lib.fp8bq_latent_attention_workspace_bytes(cache(0, 0, 0, pages=7), batch(0, 0, 0), heads, 9)
    for bad in ((None, b, 16, 9), (cache(), None, 16, 9), (cache(size=5), b, 16, 9), (cache(dim=64), b, 16, 9),
                (cache(), b, 0, 9), (cache(), b, 16, 0), (cache(), b, 2000, 9)):
        assert lib.fp8bq_latent_attention_workspace_bytes(*bad) == 0
    assert lib.fp8bq_latent_attention(cache(), batch(count=0, starts=0), query(tokens=0), None, 0, None) == fq.OK


@no_gpu
def test_workspace_of_small_calls():
    """Room for no more partial sums than a call can make: two for each key tile, and
    four tiles more, of each row tile, in whole eights; and never more than the
    largest calls take."""
    lib = fq.load_library()
    for dim in (256, 512):
        for heads, rows in ((16, 32), (40, 64), (128, 128), (300, 256)):
            for count, width in ((1, 5), (1, 13), (1, 100), (4, 6), (30, 9), (1, 100000), (200, 300)):
                need = lib.fp8bq_latent_attention_workspace_bytes(cache(dim=dim), batch(count=count, width=width), heads, count)
                units = (count * heads // rows + count) * (width + 4)
                shares = min(-(-units // 8) * 8, 256 * 64 // rows)
                assert need == 2 * shares * rows * (4 * dim + 8) + 8 * count * heads, (dim, heads, count, width)


P = (3200, 192, 4096, 256, 64, 4096, 256, 2048, 128)


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k=0), dict(r=0), dict(v=0), dict(out=0), dict(q_at=0), dict(q=Q + 8), dict(k=X + 2), dict(r=XR + 4),
    dict(v=X + 248), dict(out=OUT + 8), dict(lse=LSE + 1), dict(q_at=CO + 2), dict(k_at=SI + 1), dict(k_at=0),
    dict(strides=strides(P, s0=3198)), dict(strides=strides(P, s2=-8)), dict(strides=strides(P, s4=1 << 36)),
    dict(strides=strides(P, s2=1 << 23)), dict(strides=strides(P, s4=1 << 23)), dict(strides=strides(P, s5=1 << 23)),
    dict(strides=strides(P, s7=0)), dict(strides=strides(P, s8=120)), dict(tokens=-1), dict(keys=-1), dict(count=-1),
    dict(count=1 << 21), dict(heads=0), dict(heads=1025), dict(dim=96), dict(dim=192), dict(tokens=1 << 25),
    dict(keys=1 << 25), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=Q), dict(out=X), dict(out=X + 4096),
    dict(out=XR), dict(lse=Q), dict(lse=X), dict(lse=OUT), dict(out=CO), dict(lse=SI)])
def test_bad_prompt(bad):
    assert fq.load_library().fp8bq_latent_prompt_attention(prompt(**bad), None) == INVALID


# ---------------------------------------------------------------- pages

BUFFERS = [(C, 64 * 512), (R, 64 * 128), (SC, 256), (X, 20)]


def pool(buffers=BUFFERS, num_pages=100, count=None, size=64):
    raw = b"".join(kv._BUFFER.pack(*x) for x in buffers)
    keep = ctypes.create_string_buffer(raw, max(len(raw), 1))
    packed = pages._PAGES.pack(ctypes.addressof(keep), num_pages, len(buffers) if count is None else count, size)
    return packed, keep


TB, LN, PA, CH, FR, TO, US = (0x10_0000_0000 * i for i in range(40, 47))


def fork(p, table=TB, stride=40, count=8, width=40, lens=LN, parents=PA, children=CH, fresh=FR, forks=3):
    packed, keep = p
    return fq.load_library().fp8bq_cache_fork(packed, table, stride, count, width, lens, parents, children, fresh, forks,
                                              None)


def compact(p, table=TB, stride=40, count=8, width=40, lens=LN, out=TO, out_stride=40, used=US, ws=WS, size=1 << 30):
    packed, keep = p
    return fq.load_library().fp8bq_cache_compact(packed, table, stride, count, width, lens, out, out_stride, used, ws,
                                                 size, None)


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(buffers=[]), dict(num_pages=0), dict(num_pages=1 << 31), dict(size=0), dict(size=24), dict(count=-1),
    dict(count=4097), dict(buffers=[(0, 64)]), dict(buffers=[(C + 2, 64)]), dict(buffers=[(C, 0)]), dict(buffers=[(C, 6)]),
    dict(buffers=[(C, 1 << 31)]), dict(buffers=[(C, 64), (C + 6396, 64)]), dict(buffers=BUFFERS + [(C + 64, 64)])])
def test_bad_pages(bad):
    assert fork(pool(**bad)) == INVALID
    assert compact(pool(**bad)) == INVALID


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(table=0), dict(table=TB + 1), dict(stride=39), dict(stride=1 << 36), dict(count=-1), dict(count=(1 << 20) + 1),
    dict(width=-1), dict(lens=0), dict(lens=LN + 2), dict(parents=0), dict(children=0), dict(fresh=0), dict(fresh=FR + 3),
    dict(forks=-1), dict(forks=(1 << 20) + 1), dict(table=C), dict(lens=R + 64), dict(parents=SC), dict(fresh=X),
    dict(lens=TB + 64), dict(children=TB), dict(parents=LN), dict(fresh=LN + 4)])
def test_bad_fork(bad):
    assert fork(pool(), **bad) == INVALID


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(table=0), dict(out=0), dict(stride=39), dict(out_stride=39), dict(count=-1), dict(width=-1), dict(lens=0),
    dict(used=0), dict(used=US + 2), dict(out=TO + 2), dict(table=C), dict(out=R), dict(used=SC), dict(ws=X), dict(lens=X),
    dict(out=TB + 4), dict(out=TB, out_stride=48), dict(used=TB), dict(used=LN), dict(out=LN), dict(ws=TO), dict(used=WS + 64),
    dict(ws=TB), dict(used=TO)])
def test_bad_compact(bad):
    assert compact(pool(), **bad) == INVALID


@no_gpu
def test_compact_workspace():
    lib = fq.load_library()
    need = lib.fp8bq_cache_compact_workspace_bytes(100)
    assert need >= 1200
    for ws, size in ((0, need), (WS, need - 1), (WS + 8, need)):
        assert compact(pool(), ws=ws, size=size) == WORKSPACE
    assert lib.fp8bq_cache_compact_workspace_bytes(0) == 0 == lib.fp8bq_cache_compact_workspace_bytes((1 << 20) + 1)
    assert compact(pool(buffers=[(C, 4)], num_pages=(1 << 20) + 1)) == INVALID
    assert fork(pool(), forks=0) == fq.OK and fork(pool(), count=0) == fq.OK


@no_gpu
@on_a_thread
def test_pages_that_pass():
    assert fork(pool()) == fq.ERR_HIP
    assert fork(pool(), width=0, table=0, stride=0) == fq.ERR_HIP
    assert compact(pool()) == fq.ERR_HIP
    assert compact(pool(), out=TB) == fq.ERR_HIP
    assert compact(pool(), count=0, table=0, out=0, lens=0) == fq.ERR_HIP


# -------------------------------------------------------------- layouts

LAYOUT = r"""
#include <stdio.h>
#include "fp8bq.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu\n", sizeof(fp8bq_latent_cache), sizeof(fp8bq_latent_tokens),
         sizeof(fp8bq_latent_query), sizeof(fp8bq_latent_prompt), sizeof(fp8bq_page_buffer), sizeof(fp8bq_pages));
  fp8bq_latent_tokens t = {0};
  fp8bq_latent_query q = {0};
  fp8bq_latent_prompt p = {0};
  printf("%zu %zu %zu %zu\n", (size_t)((char*)&t.c_token_stride - (char*)&t), (size_t)((char*)&t.q_heads - (char*)&t),
         (size_t)((char*)&q.scale - (char*)&q), (size_t)((char*)&p.scale - (char*)&p));
  return 0;
}
"""


def test_struct_layouts(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(LAYOUT)
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes, offsets = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    assert [int(x) for x in sizes.split()] == [latent._CACHE.size, latent._TOKENS.size, latent._QUERY.size,
                                               latent._PROMPT.size, kv._BUFFER.size, pages._PAGES.size]
    assert [int(x) for x in offsets.split()] == [56, latent._TOKENS.size - 8, latent._QUERY.size - 4,
                                                 latent._PROMPT.size - 4]


# ------------------------------------------------------- the Python side

def test_no_cpu_implementation():
    c = torch.zeros((2, 16, 256), dtype=torch.float8_e4m3fn)
    r, s = torch.zeros((2, 16, 64), dtype=torch.bfloat16), torch.ones((2, 16))
    with pytest.raises(TypeError, match="GPU"):
        fq.LatentCache(c, r, s)
    for bad, error in (((c.float(), r, s), TypeError), ((c, r.float(), s), TypeError), ((c, r, s.double()), TypeError),
                       ((c[0], r, s), TypeError), ((c[:, ::2], r, s), ValueError), ((c, r[:1], s), ValueError),
                       ((c, r, s[:, :8].contiguous()), ValueError), ((c[:, :8].contiguous(), r, s), ValueError),
                       ((c[..., :128].contiguous(), r, s), ValueError)):
        with pytest.raises(error):
            fq.LatentCache(*bad)
    with pytest.raises(ValueError):
        fq.LatentCache.empty(2, 256, 24, device="cpu")
    z = torch.zeros((3, 1, 192), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="GPU"):
        fq.latent_prompt_attention(z, z[..., :128], z[:, 0, :64], z[..., :128], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="KvCache or LatentCache"):
        fq.cache_fork([c], None, None, None, None, None)
    with pytest.raises(ValueError):
        fq.cache_compact([], None, None)


def test_append_without_positions_is_checked():
    """Zero rows of cos and sin leave all tokens out, and let nothing pass that is
    refused otherwise."""
    cache = SimpleNamespace(_index=-1, latent_dim=256, device=torch.device("cpu"))     # of tensors on the CPU
    bf = torch.bfloat16
    c, r, q = torch.zeros((3, 256), dtype=bf), torch.zeros((3, 64), dtype=bf), torch.zeros((3, 2, 192), dtype=bf)[..., 128:]
    args = (cache, c, r, torch.zeros((3, 1), dtype=torch.int32), torch.ones(3, dtype=torch.int32))
    turn = dict(cos=torch.zeros((0, 32)), sin=torch.zeros((0, 32)))
    assert fq.latent_append(*args, **turn) is None
    out = fq.latent_append(*args, q=q, **turn)
    assert out.shape == q.shape and out.dtype is bf and out.is_contiguous()
    assert fq.latent_append(*args, q=q, q_out=out, r_out=r, **turn) is out
    for bad, error in ((dict(q=q.float()), TypeError), (dict(q=q[:2]), ValueError), (dict(q=q[..., :32]), ValueError),
                       (dict(q_out=out), ValueError), (dict(q=q, q_out=out[:, :1]), ValueError),
                       (dict(q=q, q_out=out.float()), TypeError), (dict(q=q, q_out=out[:1].expand(3, 2, 64)), ValueError),
                       (dict(r_out=r.float()), TypeError), (dict(r_out=r[:2]), ValueError),
                       (dict(r_out=r[:1].expand(3, 64)), ValueError)):
        with pytest.raises(error):
            fq.latent_append(*args, **bad, **turn)


# ------------------------------------------------------------- the oracle

def test_reference_of_forks_and_compaction():
    """Worked by hand: pages of 16, page p holding p."""
    x = np.arange(10, dtype=np.int64)[:, None].copy()
    table, lens = np.array([[7, 2, 9], [4, -1, -1], [7, 5, -1]], dtype=np.int32), np.array([33, 0, 20])
    t, l, y = table.copy(), lens.copy(), x.copy()
    ref.fork([y], t, l, [0], [1], [8], 16)
    assert t.tolist() == [[7, 2, 9], [7, 2, 8], [7, 5, -1]] and l.tolist() == [33, 33, 20] and y[8, 0] == 9
    out, used = ref.compact([y], t, l, 16)
    # in use: 2 5 7 8 9; five pages: holes 0 1 3 4, movers 5 7 8 9
    assert used == 5 and out.tolist() == [[1, 2, 4], [1, 2, 3], [1, 0, -1]]
    assert y[:5, 0].tolist() == [5, 7, 2, 9, 9]


def test_reference_of_attention():
    """One key, then two alike: outputs are the key's latent, sums count."""
    L = 256
    c = np.zeros((1, 16, L), dtype=np.uint8)
    c[0, :2, 0] = 0x38                                      # 1.0
    cache = [c, torch.zeros((1, 16, 64), dtype=torch.bfloat16), np.full((1, 16), 0.5, dtype=np.float32)]
    q, r = torch.ones((2, 1, L), dtype=torch.bfloat16), torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    out, lse, _, _ = ref.absorbed(cache, q, r, [[0]], [2], [0, 2], 2.0)
    assert out[:, 0, 0].tolist() == [0.5, 0.5] and np.allclose(lse[:, 0], [1.0, 1.0 + np.log(2)])
    k, v = torch.ones((2, 1, 64), dtype=torch.bfloat16), torch.full((2, 1, 64), 3.0, dtype=torch.bfloat16)
    q = torch.ones((2, 1, 128), dtype=torch.bfloat16)
    out, lse, _, _ = ref.expanded(q, k, torch.zeros((2, 64), dtype=torch.bfloat16), v, [0, 2], [0, 2], 0.25)
    assert out[:, 0, 0].tolist() == [3.0, 3.0] and np.allclose(lse[:, 0], [16.0, 16.0 + np.log(2)])
