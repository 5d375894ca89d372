"""The latent cache on the GPU against the plain definitions of
latent_reference.py: stored bytes, scales and rotated rows equal, attention in
both forms within the error that its documented roundings allow."""

import concurrent.futures
import copy
import math

import numpy as np
import pytest
import torch

import latent_reference as ref
from kv_reference import decode
from test_kv_gpu import i32, rotation, starts_of, tables

pytestmark = pytest.mark.gpu

DEV = "cuda"


def random_cache(fq, g, pages, size, dim, spread=0.5):
    """Latents as appends leave them, all slots filled."""
    x = torch.randn((pages, size, dim), generator=g) * torch.exp(spread * torch.randn((pages, size, 1), generator=g))
    s = torch.from_numpy(np.vectorize(ref.fit)(x.abs().amax(2).numpy()).astype(np.float32))
    codes = torch.from_numpy(ref.encode((x.double() / s[..., None].double()).numpy()))
    r = torch.randn((pages, size, 64), generator=g).to(torch.bfloat16)
    return fq.LatentCache(codes.to(DEV).view(torch.float8_e4m3fn), r.to(DEV), s.to(DEV))


def host(cache):
    return [cache.c.view(torch.uint8).cpu().numpy().copy(), cache.r.cpu().clone(), cache.scale.cpu().numpy().copy()]


def same_cache(cache, want):
    got = host(cache)
    assert np.array_equal(got[0], want[0]), np.argwhere(got[0] != want[0])[:4].tolist()
    assert torch.equal(got[1].view(torch.int16), want[1].view(torch.int16))
    assert np.array_equal(got[2], want[2])


def close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.equal(got.isnan(), want.isnan()), what
    off = (got - want).abs() - tol
    off = torch.where((got == want) | want.isnan(), torch.full_like(off, -1), off)      # infinities too
    assert float(off.max()) <= 0, (what, float(off.max()), np.argwhere(off.numpy() > 0)[:4].tolist())


# ---------------------------------------------------------------- append

APPEND = [
    # latent, page, heads, interleaved, turned, lens, new
    (512, 64, 16, False, True, [1, 64, 65, 200, 7], None),
    (256, 16, 3, True, True, [16, 17, 33, 1], None),
    (512, 32, 0, False, True, [31, 32, 33], None),
    (512, 256, 128, True, True, [300, 256, 5], None),
    (256, 128, 5, False, False, [129, 128], None),
    (512, 64, 25, False, True, [64, 65, 200, 7, 130], [64, 1, 150, 7, 2]),
    (256, 16, 24, True, True, [100, 16, 33, 9, 50], [100, 3, 17, 0, 33]),
    (512, 16, 40, True, True, [40], [39]),
]


@pytest.mark.parametrize("dim,page,heads,interleaved,turned,lens,new", APPEND)
def test_append_equals_the_definition(gpu_lib, dim, page, heads, interleaved, turned, lens, new):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + page + heads)
    one = new is None
    starts = starts_of([1] * len(lens) if one else new)
    T, width = starts[-1], max(-(-x // page) for x in lens)
    pages = len(lens) * width + 2
    table = tables(g, [-(-x // page) for x in lens], width, pages)
    cache = random_cache(fq, g, pages, page, dim)
    want = host(cache)
    # latents and keys side by side, queries behind other channels
    x = (torch.randn((T, dim + 64), generator=g) * torch.exp(2 * torch.randn((T, 1), generator=g))).to(torch.bfloat16)
    x[T // 2, :dim] = 0
    qs = torch.randn((T, max(heads, 1), 192), generator=g).to(torch.bfloat16)
    cos, sin = rotation(max(lens), 64) if turned else (None, None)
    q_want, r_want = torch.zeros((T, max(heads, 1), 64), dtype=torch.bfloat16), torch.zeros((T, 64), dtype=torch.bfloat16)
    ref.append(want, x[:, :dim], x[:, dim:], table, lens, starts, qs[:, :, 128:] if heads else None, q_want, r_want,
               cos, sin, interleaved)
    d, dq = x.to(DEV), qs.to(DEV)
    turn = dict(cos=torch.from_numpy(cos).to(DEV), sin=torch.from_numpy(sin).to(DEV)) if turned else {}
    r_out = torch.zeros((T, 64), dtype=torch.bfloat16, device=DEV)
    args = (cache, d[:, :dim], d[:, dim:], i32(table), i32(lens), None if one else i32(starts))
    got = fq.latent_append(*args, q=dq[:, :, 128:] if heads else None, r_out=r_out, interleaved=interleaved, **turn)
    torch.cuda.synchronize()
    same_cache(cache, want)
    assert torch.equal(r_out.cpu().view(torch.int16), r_want.view(torch.int16))
    assert (got is None) == (heads == 0)
    if heads:
        assert torch.equal(got.cpu().view(torch.int16), q_want.view(torch.int16))
    assert torch.equal(d.cpu().view(torch.int16), x.view(torch.int16))
    # in place, and the same again
    again = fq.latent_append(*args, q=dq[:, :, 128:] if heads else None, q_out=dq[:, :, 128:] if heads else None,
                             r_out=d[:, dim:], interleaved=interleaved, **turn)
    torch.cuda.synchronize()
    same_cache(cache, want)
    assert torch.equal(d[:, dim:].cpu().view(torch.int16), r_want.view(torch.int16))
    assert torch.equal(d[:, :dim].cpu().view(torch.int16), x[:, :dim].view(torch.int16))
    if heads:
        assert torch.equal(again.cpu().view(torch.int16), q_want.view(torch.int16))
        assert torch.equal(dq[:, :, :128].cpu().view(torch.int16), qs[:, :, :128].view(torch.int16))


def test_append_leaves_out_what_has_no_place(gpu_lib):
    """Pages that are none, tables that are too short, negative positions,
    positions without a row of cos, rows of no sequence, offsets that are none."""
    fq, g = gpu_lib, torch.Generator().manual_seed(3)
    dim, page, pages = 256, 16, 6
    lens, starts = [20, 40, 3, 70, 33], [2, 8, 12, 17, 20, 22]
    table = [[0, 9], [-1, 3], [1, 1], [5, 2], [4, 1 << 30]]
    cache = random_cache(fq, g, pages, page, dim)
    want = host(cache)
    T = 26
    c, r = (torch.randn((T, n), generator=g).to(torch.bfloat16) for n in (dim, 64))
    q = torch.randn((T, 2, 64), generator=g).to(torch.bfloat16)
    cos, sin = rotation(69, 64)
    q_out, r_out = torch.full((T, 2, 64), 7.0, dtype=torch.bfloat16), torch.full((T, 64), 7.0, dtype=torch.bfloat16)
    dq, dr = q_out.to(DEV), r_out.to(DEV)
    ref.append(want, c, r, table, lens, starts, q, q_out, r_out, cos, sin)
    fq.latent_append(cache, c.to(DEV), r.to(DEV), i32(table), i32(lens), i32(starts), q=q.to(DEV), q_out=dq, r_out=dr,
                     cos=torch.from_numpy(cos).to(DEV), sin=torch.from_numpy(sin).to(DEV))
    torch.cuda.synchronize()
    same_cache(cache, want)
    assert torch.equal(dq.cpu().view(torch.int16), q_out.view(torch.int16))
    assert torch.equal(dr.cpu().view(torch.int16), r_out.view(torch.int16))
    # offsets out of range are clamped: nothing outside the buffers is written
    for bad in ([0, 5, 3, 9, 1 << 30, 2], [-7, -3, 4, 1 << 30, 5, 6]):
        fq.latent_append(cache, c.to(DEV), r.to(DEV), i32(table), i32(lens), i32(bad), q=q.to(DEV), q_out=dq, r_out=dr)
    torch.cuda.synchronize()


def test_append_of_extreme_values(gpu_lib):
    fq = gpu_lib
    x = torch.zeros((6, 256))
    x[0, 3], x[1, 5], x[2, :] = 3.38e38, 1e-30, 448.0
    x[3, 7], x[4, 9], x[5, 1] = 449.0, 2.0 ** -126, -1e-10
    x = x.to(torch.bfloat16)
    cache = fq.LatentCache.empty(1, 256, 16)
    want = host(cache)
    r = torch.zeros((6, 64), dtype=torch.bfloat16)
    ref.append(want, x, r, [[0]], [6], [0, 6])
    fq.latent_append(cache, x.to(DEV), r.to(DEV), i32([[0]]), i32([6]), i32([0, 6]))
    torch.cuda.synchronize()
    same_cache(cache, want)


# -------------------------------------------------------------- absorbed

ABSORBED = [
    # latent, page, heads, lens, new
    (512, 64, 16, [1, 64, 65, 200, 7, 0], None),
    (256, 16, 5, [16, 17, 33, 1, 300], None),
    (512, 16, 1, [130, 2], None),
    (512, 32, 32, [31, 90], None),
    (512, 128, 33, [129, 300], None),
    (256, 64, 64, [100, 5, 260], None),
    (512, 256, 65, [257, 10], None),
    (256, 256, 128, [64, 200, 0], None),
    (512, 64, 128, [190, 1], None),
    (512, 64, 12, [64, 65, 200, 7, 130], [3, 1, 5, 7, 2]),
    (256, 16, 20, [100, 16, 33, 9, 50], [4, 3, 2, 0, 4]),
    (512, 64, 40, [150, 90], [5, 3]),
    (256, 32, 16, [70, 33], [70, 33]),
    (512, 64, 7, [77], [77]),
    (512, 64, 16, [3, 10], [5, 12]),          # the first queries lie before the sequence
]


def absorbed_inputs(g, T, heads, dim, spread=0.0):
    q = torch.randn((heads, T, dim), generator=g) * torch.exp(spread * torch.randn((heads, T, 1), generator=g))
    return q.to(torch.bfloat16).transpose(0, 1), torch.randn((T, heads, 192), generator=g).to(torch.bfloat16)[..., 128:]


def check_absorbed(got, lse, want, what=""):
    out, l, tol, tol_lse = want
    close(got, out, tol, ("out", what))
    if lse is not None:
        close(lse, l, tol_lse, ("lse", what))
    # and over all: the elementwise bound is the worst case, roundings at random come to less than half
    # a step of BF16 for the weights and as much for the output
    live = torch.isfinite(out).all(-1)
    e = (got.double().cpu() - out)[live].norm() / out[live].norm().clamp_min(1e-30)
    assert float(e) < 2 ** -8, (what, float(e))


@pytest.mark.parametrize("dim,page,heads,lens,new", ABSORBED)
def test_absorbed_attention(gpu_lib, dim, page, heads, lens, new):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + page + heads + len(lens))
    one = new is None
    starts = starts_of([1] * len(lens) if one else new)
    T, width = starts[-1], max(-(-x // page) for x in lens)
    pages = len(lens) * width + 2
    table = tables(g, [-(-x // page) for x in lens], width, pages)
    cache = random_cache(fq, g, pages, page, dim)
    q, qr = absorbed_inputs(g, T, heads, dim)
    scale = 0.06
    want = ref.absorbed(host(cache), q, qr, table, lens, starts, scale)
    args = (cache, q.to(DEV), qr.to(DEV), i32(table), i32(lens), None if one else i32(starts))
    got, lse = fq.latent_attention(*args, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    check_absorbed(got, lse, want)
    assert torch.equal(got, fq.latent_attention(*args, scale=scale))           # the same again
    # a table with more columns than are used: other shapes, other splits
    wide = torch.full((len(lens), width + 40), -1, dtype=torch.int32, device=DEV)
    wide[:, :width] = i32(table)
    got, lse = fq.latent_attention(cache, args[1], args[2], wide, *args[4:], scale=scale, return_lse=True)
    check_absorbed(got, lse, want, "wide")
    want = ref.absorbed(host(cache), q, qr, table, lens, starts, -scale)
    got, lse = fq.latent_attention(*args, scale=-scale, return_lse=True)
    check_absorbed(got, lse, want, "negative scale")


@pytest.mark.parametrize("heads", [16, 40, 128])
def test_absorbed_over_long_sequences(gpu_lib, heads):
    """Keys split over many workgroups, ragged; heads picked for the comparison."""
    fq, g = gpu_lib, torch.Generator().manual_seed(heads)
    lens = [3001, 1, 0, 1500, 64, 777]
    table = tables(g, [-(-x // 64) for x in lens], 47, 100)
    cache = random_cache(fq, g, 100, 64, 512)
    q, qr = absorbed_inputs(g, len(lens), heads, 512)
    some = [0, 3, heads - 1]
    want = ref.absorbed(host(cache), q, qr, table, lens, range(len(lens) + 1), 0.06, some)
    got, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), i32(table), i32(lens), scale=0.06, return_lse=True)
    check_absorbed(got[:, some], lse[:, some], want)
    # queries of zero see every key alike: the sum of exponentials counts the keys
    zero, zr = torch.zeros_like(q).to(DEV), torch.zeros_like(qr).to(DEV)
    _, lse = fq.latent_attention(cache, zero, zr, i32(table), i32(lens), scale=0.06, return_lse=True)
    count = torch.exp(lse.double().cpu()).round()
    assert torch.equal(count, torch.tensor(lens, dtype=torch.float64)[:, None].expand(-1, heads))


def test_absorbed_of_sharp_rows(gpu_lib):
    """One key far above the others, whose weights are still summed rightly: the
    terms of a weight are taken relative to its 32 neighbours."""
    fq, g = gpu_lib, torch.Generator().manual_seed(5)
    n, heads, dim = 2000, 16, 512
    table = [list(range(32))]
    cache = random_cache(fq, g, 32, 64, dim, spread=0.0)
    q, qr = absorbed_inputs(g, 1, heads, dim)
    k = decode(host(cache)[0][0, 5]) * host(cache)[2][0, 5]
    q = q + torch.from_numpy(k).to(torch.bfloat16)[None, None] * 0.6      # key 5 gets some hundred more
    want = ref.absorbed(host(cache), q, qr, table, [n], [0, 1], 0.04)
    got, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), i32(table), i32([n]), scale=0.04, return_lse=True)
    check_absorbed(got, lse, want)


@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_absorbed_of_mixed_magnitudes(gpu_lib, spread):
    """Scales of tokens and of queries over many powers of two."""
    fq, g = gpu_lib, torch.Generator().manual_seed(9)
    table = tables(g, [5, 3], 5, 9)
    cache = random_cache(fq, g, 9, 64, 256, spread=spread)
    q, qr = absorbed_inputs(g, 2, 24, 256, spread=spread)
    scale = 0.05 * math.exp(-2 * spread)
    want = ref.absorbed(host(cache), q, qr, table, [300, 170], [0, 1, 2], scale)
    got, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), i32(table), i32([300, 170]), scale=scale, return_lse=True)
    out, l, tol, tol_lse = want
    close(got, out, tol, "out")
    close(lse, l, tol_lse, "lse")


@pytest.mark.parametrize("heads", [5, 40])
@pytest.mark.parametrize("power", [-60, 60])
def test_absorbed_at_the_ends_of_the_scales(gpu_lib, heads, power):
    """Powers of two of the scales pass through: scores stay, outputs move by them.
    A weight times its scale has no meaning below 2^-121, at 2^-60 so a weight (of at
    most 1) below 2^-61: codes are at most 448, so an output moves by at most n 448
    2^-61, and then may round the other way, a step of BF16 being 2^-7 at most."""
    fq, g = gpu_lib, torch.Generator().manual_seed(heads)
    cache = random_cache(fq, g, 8, 64, 512)
    one = torch.ones_like(cache.scale)
    q, qr = absorbed_inputs(g, 2, heads, 512)
    args = (q.to(DEV), torch.zeros_like(qr).to(DEV), i32([[0, 1, 2, 3, 4], [7, 6, 5, -1, -1]]), i32([290, 129]))
    want, lse = fq.latent_attention(fq.LatentCache(cache.c, cache.r, one), *args, scale=2.0 ** -9, return_lse=True)
    moved = fq.LatentCache(cache.c, cache.r, one * 2.0 ** power)
    got, same = fq.latent_attention(moved, *args, scale=2.0 ** (-9 - power), return_lse=True)
    lost = torch.tensor([290, 129], dtype=torch.float64)[:, None, None] * 448 * 2.0 ** (-121 - power)
    want, got = want.double().cpu(), got * 2.0 ** -power
    assert bool(want.isfinite().all())
    close(got, want, lost + (2.0 ** -7 * want.abs() if power < 0 else 0.0), "out")
    close(same, lse.double().cpu(), 1e-6 * lse.abs().double().cpu() + 1e-5, "lse")


@pytest.mark.parametrize("heads,new", [(16, [1, 1, 1, 1]), (50, [1, 1, 1, 1]), (128, [1, 1, 1, 1]), (40, [3, 1, 4, 2])])
@pytest.mark.parametrize("spare", [0, 3])        # columns of the table: without shares, and with
def test_absorbed_with_bad_pages_and_numbers(gpu_lib, heads, new, spare):
    """Pages that are none are not seen; what lies behind a sequence, NaN and
    infinite scales among it, has no effect; rows that are not numbers stay so
    and leave the others alone; rows of no sequence are left as they were."""
    fq, g = gpu_lib, torch.Generator().manual_seed(11)
    lens = [150, 70, 20, 0]
    starts = [2 + s for s in starts_of(new)]
    T = starts[-1] + 3
    table = [row + [5] * spare for row in ([0, 99, 2], [3, -1, -1], [1 << 30, 1, 1], [4, 4, 4])]
    cache = random_cache(fq, g, 6, 64, 512)
    hostc = host(cache)
    q, qr = (x.contiguous() for x in absorbed_inputs(g, T, heads, 512))
    q[starts[0], 1, 5], q[starts[1], 0, 7], qr[starts[0], 2, 3] = math.nan, math.inf, -math.inf
    want = ref.absorbed(hostc, torch.nan_to_num(q, 0, 0, 0), torch.nan_to_num(qr, 0, 0, 0), table, lens, starts, 0.06)
    for x, y in ((want[0], want[2]), (want[1], want[3])):
        for row, h in ((starts[0], 1), (starts[0], 2), (starts[1], 0)):
            x[row, h], y[row, h] = math.nan, 0.0
    # beyond the sequences: codes, keys and scales that are not numbers
    c = cache.c.view(torch.uint8)
    for pg, slot in ((2, 150 - 128), (3, 64), (1, 0)):
        c[pg, slot:] = 0x7F
        cache.r[pg, slot:] = math.nan
        cache.scale[pg, slot:] = math.inf if pg == 2 else math.nan
    c[4], c[5] = 0xFF, 0x7F
    out = torch.full((T, heads, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, heads), 3.0, device=DEV)
    fq.latent_attention(cache, q.to(DEV), qr.to(DEV), i32(table), i32(lens), i32(starts), scale=0.06, out=out, lse=lse)
    rows = slice(starts[0], starts[-1])
    check_absorbed(out[rows], lse[rows], [x[rows] for x in want])
    for x in (out, lse):
        assert bool((x[:starts[0]] == 3).all()) and bool((x[starts[-1]:] == 3).all())


def test_absorbed_splits_of_one_call(gpu_lib):
    """A part of a row with NaN scores, split over workgroups, stays NaN."""
    fq, g = gpu_lib, torch.Generator().manual_seed(2)
    cache = random_cache(fq, g, 40, 64, 256)
    q, qr = (x.contiguous() for x in absorbed_inputs(g, 1, 20, 256))
    q[0, 3, 100] = math.nan
    out, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), i32([list(range(40))]), i32([2500]), scale=0.1,
                                   return_lse=True)
    bad = torch.zeros(20, dtype=torch.bool)
    bad[3] = True
    assert torch.equal(out[0].isnan().all(-1).cpu(), bad) and torch.equal(out[0].isnan().any(-1).cpu(), bad)
    assert torch.equal(lse[0].isnan().cpu(), bad)


@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("width", [4, 9])       # without shares, and with
def test_absorbed_strides_and_buffers(gpu_lib, heads, width):
    fq, g = gpu_lib, torch.Generator().manual_seed(heads)
    lens, starts, table = [200, 90], [0, 2, 3], [[0, 1, 2, 3] + [-1] * (width - 4), [4, 5, 6, 7] + [-1] * (width - 4)]
    cache = random_cache(fq, g, 8, 64, 512)
    q, qr = absorbed_inputs(g, 3, heads, 512)
    want = ref.absorbed(host(cache), q, qr, table, lens, starts, 0.06)
    args = (i32(table), i32(lens), i32(starts))
    big = torch.full((3, heads, 520), 5.0, dtype=torch.bfloat16, device=DEV)
    head_major = torch.empty((heads, 3, 512), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    need = fq.latent_attention_workspace_bytes(cache, q, args[0])
    assert (need > 0) == (width > 4)
    work = torch.full((need + 16,), 255, dtype=torch.uint8, device=DEV)
    for out in (big[..., :512], head_major):
        got = fq.latent_attention(cache, q.to(DEV), qr.contiguous().to(DEV), *args, scale=0.06, out=out, workspace=work)
        assert got is out
        check_absorbed(out, None, want)
    assert bool((big[..., 512:] == 5).all())
    with pytest.raises(fq.Fp8bqError):
        if need == 0:
            raise fq.Fp8bqError("no workspace", fq.ERR_WORKSPACE, 0)
        fq.latent_attention(cache, q.to(DEV), qr.to(DEV), *args, scale=0.06, workspace=work[:need - 1])


@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("width", [4, 9, 40])
def test_absorbed_workspace(gpu_lib, heads, width):
    """One byte less than it takes is refused, nothing beyond it is written, and
    where it takes none an empty one does."""
    fq, g = gpu_lib, torch.Generator().manual_seed(heads + width)
    cache = random_cache(fq, g, 8, 64, 512)
    q, qr = (x.to(DEV) for x in absorbed_inputs(g, 3, heads, 512))
    table = i32([[0, 1, 2, 3] + [-1] * (width - 4), [4, 5, 6, 7] + [-1] * (width - 4)])
    args = (cache, q, qr, table, i32([200, 90]), i32([0, 2, 3]))
    want = fq.latent_attention(*args, scale=0.06)
    need = fq.latent_attention_workspace_bytes(cache, q, table)
    work = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    got = fq.latent_attention(*args, scale=0.06, workspace=work[:need])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((work[need:] == 255).all())
    if width <= 4:
        assert need == 0
        return
    out = torch.full((3, heads, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    for short in (work[:need - 1], work[:0]):
        with pytest.raises(fq.Fp8bqError) as error:
            fq.latent_attention(*args, scale=0.06, workspace=short, out=out)
        assert error.value.status == fq.ERR_WORKSPACE
    torch.cuda.synchronize()
    assert bool((out == 7).all())


def test_far_pages(gpu_lib):
    """Codes beyond 2^32 bytes from the cache's start."""
    fq, g = gpu_lib, torch.Generator().manual_seed(1)
    pages = (1 << 32) // (256 * 512) + 3
    cache = fq.LatentCache.empty(pages, 512, 256)
    small = random_cache(fq, g, 2, 256, 512)
    far = [pages - 1, pages - 2]
    c = torch.randn((300, 512), generator=g).to(torch.bfloat16).to(DEV)
    r = torch.randn((300, 64), generator=g).to(torch.bfloat16).to(DEV)
    q, qr = absorbed_inputs(g, 1, 16, 512)
    outs = []
    for to, row in ((cache, far), (small, [1, 0])):
        fq.latent_append(to, c, r, i32([row]), i32([300]), i32([0, 300]))
        outs.append(fq.latent_attention(to, q.to(DEV), qr.to(DEV), i32([row]), i32([300]), scale=0.06))
    assert torch.equal(outs[0], outs[1])


# -------------------------------------------------------------- expanded

EXPANDED = [
    # head_dim, heads, new, keys (None: the same)
    (128, 2, [1, 64, 65, 200, 7], None),
    (64, 3, [130, 1, 129, 0, 31], None),
    (128, 1, [300], None),
    (64, 16, [5, 257], None),
    (128, 3, [1, 1, 1], [300, 64, 1]),
    (64, 2, [70, 5, 128], [200, 5, 640]),
    (128, 2, [130, 3], [131, 700]),
    (128, 1, [10, 5, 4], [4, 0, 4]),          # the first queries see nothing
    (64, 24, [300] * 9, None),                # many row tiles: one set of waves each
    (128, 33, [130, 7, 260, 0, 1, 64], [130, 400, 300, 9, 0, 65]),
]


@pytest.mark.parametrize("dim,heads,new,keys", EXPANDED)
def test_expanded_attention(gpu_lib, dim, heads, new, keys):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + heads + len(new))
    q_at, k_at = starts_of(new), starts_of(keys or new)
    T, K = q_at[-1], k_at[-1]
    q = torch.randn((T, heads, dim + 64), generator=g).to(torch.bfloat16)
    kv = torch.randn((K, heads, 2 * dim), generator=g).to(torch.bfloat16)
    kr = torch.randn((K, 64), generator=g).to(torch.bfloat16)
    want = ref.expanded(q, kv[..., :dim], kr, kv[..., dim:], q_at, k_at)
    d = kv.to(DEV)
    args = (q.to(DEV), d[..., :dim], kr.to(DEV), d[..., dim:], i32(q_at), None if keys is None else i32(k_at))
    got, lse = fq.latent_prompt_attention(*args, return_lse=True)
    check_absorbed(got, lse, want)
    assert torch.equal(got, fq.latent_prompt_attention(*args))
    # other strides, a negative scale
    out = torch.empty((heads, T, dim + 8), dtype=torch.bfloat16, device=DEV).transpose(0, 1)[..., :dim]
    q3 = torch.zeros((T, 3, heads, dim + 64), dtype=torch.bfloat16, device=DEV)
    q3[:, 1] = q.to(DEV)
    fq.latent_prompt_attention(q3[:, 1], args[1].contiguous(), args[2], args[3].transpose(0, 1).contiguous().transpose(0, 1),
                               *args[4:], scale=-0.1, out=out)
    check_absorbed(out, None, ref.expanded(q, kv[..., :dim], kr, kv[..., dim:], q_at, k_at, -0.1))


def test_expanded_rows_and_offsets(gpu_lib):
    """Rows of no sequence stay; rows that are not numbers too; what lies behind
    a sequence's keys has no effect; offsets that are none reach nothing."""
    fq, g = gpu_lib, torch.Generator().manual_seed(4)
    dim, heads, T, K = 64, 2, 200, 400
    q_at, k_at = [3, 80, 80, 190], [0, 100, 110, 300]
    q = torch.randn((T, heads, dim + 64), generator=g).to(torch.bfloat16)
    k, v = (torch.randn((K, heads, dim), generator=g).to(torch.bfloat16) for _ in range(2))
    kr = torch.randn((K, 64), generator=g).to(torch.bfloat16)
    q[10, 1, 100], q[90, 0, 2] = math.nan, math.inf
    want = ref.expanded(torch.nan_to_num(q, 0, 0, 0), k, kr, v, q_at, k_at)
    for x, y in ((want[0], want[2]), (want[1], want[3])):
        for row, h in ((10, 1), (90, 0)):
            x[row, h], y[row, h] = math.nan, 0.0
    for x in (k, kr, v):
        x[100:110], x[300:] = math.nan, math.inf
    out = torch.full((T, heads, dim), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, heads), 3.0, device=DEV)
    args = [x.to(DEV) for x in (q, k, kr, v)]
    fq.latent_prompt_attention(*args, i32(q_at), i32(k_at), out=out, lse=lse)
    close(out[3:190], want[0][3:190], want[2][3:190], "out")
    close(lse[3:190], want[1][3:190], want[3][3:190], "lse")
    for x in (out, lse):
        assert bool((x[:3] == 3).all()) and bool((x[190:] == 3).all())
    for bad in ([0, 150, 90, 1 << 30], [-5, 10, 5, 2], [1 << 30, 0, -1, 200]):
        fq.latent_prompt_attention(*args, i32(bad), i32(k_at))
        fq.latent_prompt_attention(*args, i32(q_at), i32(bad))
    torch.cuda.synchronize()


def test_expanded_counts_keys(gpu_lib):
    fq = gpu_lib
    T, keys = 700, 1500
    q = torch.zeros((T, 4, 192), dtype=torch.bfloat16, device=DEV)
    k = torch.ones((keys, 4, 128), dtype=torch.bfloat16, device=DEV)
    kr = torch.ones((keys, 64), dtype=torch.bfloat16, device=DEV)
    out, lse = fq.latent_prompt_attention(q, k, kr, k, i32([0, T]), i32([0, keys]), return_lse=True)
    count = torch.exp(lse.double().cpu()).round()
    assert torch.equal(count, (keys - T + 1 + torch.arange(T, dtype=torch.float64))[:, None].expand(-1, 4))
    assert bool((out == 1).all())


# ------------------------------------------------------------ together

def test_a_rollout(gpu_lib):
    """A prompt in the expanded form, stored; then single tokens in the absorbed
    form, whose outputs agree with the expanded form over the whole sequence, up
    to the rounding of stored latents to e4m3."""
    fq, g = gpu_lib, torch.Generator().manual_seed(6)
    H, L, D, page, prompt, more = 8, 512, 128, 64, 150, 5
    n = prompt + more
    c = torch.randn((n, L), generator=g).to(torch.bfloat16).to(DEV)
    r = torch.randn((n, 64), generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn((n, H, D + 64), generator=g).to(torch.bfloat16).to(DEV)
    uk, uv = (torch.randn((H, L, D), generator=g).to(DEV) * L ** -0.5 for _ in range(2))
    cos, sin = (torch.from_numpy(x).to(DEV) for x in rotation(n, 64))
    cache = fq.LatentCache.empty(4, L, page)
    table = i32([[2, 0, 3]])

    def expand(x, up):
        return torch.matmul(x.float(), up).to(torch.bfloat16).transpose(0, 1).contiguous()

    # the whole sequence in the expanded form, from the stored latents
    whole = fq.LatentCache.empty(4, L, page)
    qr = q.clone()
    rr = torch.empty_like(r)
    fq.latent_append(whole, c, r, table, i32([n]), i32([0, n]), q=q[..., D:], q_out=qr[..., D:], r_out=rr, cos=cos, sin=sin)
    rows = table[0].long()
    stored = fq.dequantize(whole.c[rows].view(-1, L), whole.scale[rows].view(-1, 1), (1, L))[:n].to(torch.bfloat16)
    full = fq.latent_prompt_attention(qr, expand(stored, uk), rr, expand(stored, uv), i32([0, n]))
    # step by step
    fq.latent_append(cache, c[:prompt], r[:prompt], table, i32([prompt]), i32([0, prompt]), cos=cos, sin=sin)
    for t in range(prompt, n):
        qt = fq.latent_append(cache, c[t:t + 1], r[t:t + 1], table, i32([t + 1]), q=q[t:t + 1, :, D:], cos=cos, sin=sin)
        absorbed = torch.matmul(q[t, :, None, :D].float(), uk.transpose(1, 2).contiguous())[:, 0].to(torch.bfloat16)
        got = fq.latent_attention(cache, absorbed[None], qt, table, i32([t + 1]), scale=(D + 64) ** -0.5)
        y = torch.matmul(got[0, :, None].float(), uv)[:, 0]
        # roundings to BF16 on either side (queries, keys, weights, sums), each of 2^-8 at most
        assert float((y - full[t].float()).norm() / full[t].float().norm()) < 6 * 2 ** -8
    torch.cuda.synchronize()
    assert torch.equal(cache.c.view(torch.uint8)[rows].view(-1, L)[:n], whole.c.view(torch.uint8)[rows].view(-1, L)[:n])


@pytest.mark.parametrize("heads", [16, 40, 128])
def test_graphs_follow_the_lengths(gpu_lib, heads):
    """A captured step, replayed while sequences grow, with eager work between."""
    fq, g = gpu_lib, torch.Generator().manual_seed(8)
    B, L = 3, 512
    cache = random_cache(fq, g, 30, 64, L)
    table = i32([list(range(10)), list(range(10, 20)), list(range(20, 30))])
    lens = i32([1, 100, 500])
    c, r = (torch.randn((B, n), generator=g).to(torch.bfloat16).to(DEV) for n in (L, 64))
    q, qr = (x.contiguous().to(DEV) for x in absorbed_inputs(g, B, heads, L))
    cos, sin = (torch.from_numpy(x).to(DEV) for x in rotation(700, 64))

    def step(to):
        turned = fq.latent_append(to, c, r, table, lens, q=qr, cos=cos, sin=sin)
        return fq.latent_attention(to, q, turned, table, lens, scale=0.06)

    step(cache)
    mirror = fq.LatentCache(cache.c.clone(), cache.r.clone(), cache.scale.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    for _ in range(4):
        lens += 37
        c.copy_(torch.randn((B, L), generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(mirror))
        assert torch.equal(cache.c.view(torch.uint8), mirror.c.view(torch.uint8))


@pytest.mark.parametrize("dim,heads", [(128, 4), (64, 4), (128, 40), (64, 40)])   # two sets of waves, and one
def test_expanded_graphs_follow_the_offsets(gpu_lib, dim, heads):
    """A captured call, replayed over other offsets, queries and keys, with eager
    work between."""
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + heads)
    T, K = 700, 900
    q = torch.randn((T, heads, dim + 64), generator=g).to(torch.bfloat16).to(DEV)
    kv = torch.randn((K, heads, 2 * dim), generator=g).to(torch.bfloat16).to(DEV)
    kr = torch.randn((K, 64), generator=g).to(torch.bfloat16).to(DEV)
    q_at, k_at = i32([0, 300, 300, 700]), i32([0, 400, 400, 900])
    out, lse = torch.empty((T, heads, dim), dtype=torch.bfloat16, device=DEV), torch.empty((T, heads), device=DEV)

    def call(**to):
        return fq.latent_prompt_attention(q, kv[..., :dim], kr, kv[..., dim:], q_at, k_at, return_lse=True, **to)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, lse=lse)
    for queries, keys in (([0, 300, 300, 700], [0, 400, 400, 900]), ([0, 1, 699, 700], [0, 1, 850, 900]),
                          ([5, 5, 200, 600], [0, 0, 10, 700]), ([0, 0, 0, 700], [0, 0, 0, 900])):
        q_at.copy_(i32(queries))
        k_at.copy_(i32(keys))
        kv.copy_(torch.randn((K, heads, 2 * dim), generator=g).to(torch.bfloat16))
        for x in (out, lse):
            x.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = call()
        rows = slice(queries[0], queries[-1])
        assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], want_lse[rows])
        for x in (out, lse):
            assert bool((x[:queries[0]] == 3).all()) and bool((x[queries[-1]:] == 3).all())


def test_streams_and_threads(gpu_lib):
    fq, g = gpu_lib, torch.Generator().manual_seed(10)
    cache = random_cache(fq, g, 20, 64, 512)
    table, lens = i32([list(range(10)), list(range(10, 20))]), i32([600, 333])
    q, qr = (x.contiguous().to(DEV) for x in absorbed_inputs(g, 2, 32, 512))
    want = fq.latent_attention(cache, q, qr, table, lens, scale=0.06)
    x = torch.randn((300, 6, 192), generator=g).to(torch.bfloat16).to(DEV)
    kv = torch.randn((300, 6, 256), generator=g).to(torch.bfloat16).to(DEV)
    kr, at = torch.randn((300, 64), generator=g).to(torch.bfloat16).to(DEV), i32([0, 100, 300])
    wide = fq.latent_prompt_attention(x, kv[..., :128], kr, kv[..., 128:], at)
    torch.cuda.synchronize()

    def work(_):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                a = fq.latent_attention(cache, q, qr, table, lens, scale=0.06)
                b = fq.latent_prompt_attention(x, kv[..., :128], kr, kv[..., 128:], at)
            torch.cuda.current_stream().synchronize()
            return torch.equal(a, want) and torch.equal(b, wide)

    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(4)))


def test_copies_of_a_cache(gpu_lib):
    fq, g = gpu_lib, torch.Generator().manual_seed(1)
    a = random_cache(fq, g, 2, 16, 256)
    for b in (copy.copy(a), copy.deepcopy(a)):
        assert b._packed == fq.LatentCache(b.c, b.r, b.scale)._packed
    with pytest.raises(AttributeError):
        a.c = a.c.clone()
    with pytest.raises(AttributeError):
        del a.scale
