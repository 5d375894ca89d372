"""The key/value cache on the GPU against the plain definitions of
kv_reference.py: stored bytes, scales and rotated queries equal, attention
within the error that its documented roundings allow."""

import concurrent.futures
import copy
import io
import math

import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def host(cache):
    """The reference's form of a cache: numpy bytes and scales."""
    return [cache.k.view(torch.uint8).cpu().numpy().copy(), cache.v.view(torch.uint8).cpu().numpy().copy(),
            cache.k_scale.cpu().numpy().copy(), cache.v_scale.cpu().numpy().copy()]


def same_cache(cache, want):
    for name, got, exp in zip(("k", "v", "k_scale", "v_scale"), host(cache), want):
        off = np.argwhere(got.view(np.uint8) != exp.view(np.uint8))
        assert len(off) == 0, (name, len(off), off[:4].tolist())


def random_cache(fq, g, pages, heads, size, dim, pow2=True):
    """Finite codes everywhere, mixed scales."""
    def codes(*shape):
        c = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
        c[(c & 0x7F) == 0x7F] = 0x38
        return c.to(DEV).view(torch.float8_e4m3fn)

    def scales():
        s = torch.exp2(torch.randint(-9, -5, (pages, heads), generator=g).float())
        return (s if pow2 else s * (1 + 0.9 * torch.rand((pages, heads), generator=g))).to(DEV)

    return fq.KvCache(codes(pages, heads, size, dim), codes(pages, heads, dim, size), scales(), scales())


def tables(g, counts, width, pages):
    order = torch.randperm(pages, generator=g).tolist()
    rows, at = [], 0
    for c in counts:
        rows.append(order[at:at + c] + [-1] * (width - c))
        at += c
    return rows


def rotation(positions, rot):
    half = rot // 2
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(half) / max(1, half))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def starts_of(new):
    return [0] + list(np.cumsum(new))


# ---------------------------------------------------------------- append

APPEND = [
    # dim, page, heads, group, rot, interleaved, lens, new
    (128, 64, 2, 4, 128, False, [1, 64, 65, 200, 7], None),
    (64, 16, 3, 1, 32, True, [16, 17, 33, 1], None),
    (192, 32, 1, 5, 192, False, [31, 32, 33], None),
    (256, 256, 2, 2, 64, True, [300, 256, 5], None),
    (128, 128, 1, 1, 0, False, [129, 128], None),
    (128, 64, 2, 4, 128, False, [64, 65, 200, 7, 130], [64, 1, 150, 7, 2]),
    (64, 16, 5, 3, 32, True, [100, 16, 33, 9, 50], [100, 3, 17, 0, 33]),
    (192, 32, 2, 1, 96, False, [70, 1, 64], [70, 1, 32]),
    (256, 256, 1, 2, 256, False, [513, 256], [300, 256]),
    (256, 16, 1, 1, 16, True, [40], [39]),
    (128, 128, 4, 8, 128, True, [255, 1], [250, 1]),
]


def append_inputs(g, T, heads, group, dim, spread=1.0):
    qkv = torch.randn((T, heads * (group + 2) * dim), generator=g)
    qkv = (qkv * torch.exp(spread * torch.randn((T, 1), generator=g))).to(torch.bfloat16)
    at = heads * group * dim
    q = qkv[:, :at].view(T, heads * group, dim)
    k = qkv[:, at:at + heads * dim].view(T, heads, dim)
    v = qkv[:, at + heads * dim:].view(T, heads, dim)
    return qkv, q, k, v


@pytest.mark.parametrize("dim,page,heads,group,rot,interleaved,lens,new", APPEND)
def test_append_equals_the_definition(gpu_lib, dim, page, heads, group, rot, interleaved, lens, new):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + page + len(lens))
    one = new is None
    n = [1] * len(lens) if one else new
    starts = starts_of(n)
    width = max(-(-x // page) for x in lens)
    table = tables(g, [-(-x // page) for x in lens], width, len(lens) * width + 2)
    cache = random_cache(fq, g, len(lens) * width + 2, heads, page, dim)
    want = host(cache)
    qkv, q, k, v = append_inputs(g, starts[-1], heads, group, dim)
    cos, sin = rotation(max(lens), rot)
    q_want = torch.zeros_like(q)
    ref.append(want, k, v, table, lens, starts, q, q_want, cos, sin, interleaved)
    d = qkv.to(DEV)
    T, at = starts[-1], heads * group * dim
    dq = d[:, :at].view(T, heads * group, dim)
    dk = d[:, at:at + heads * dim].view(T, heads, dim)
    dv = d[:, at + heads * dim:].view(T, heads, dim)
    got = fq.kv_append(cache, dk, dv, i32(table), i32(lens), None if one else i32(starts), q=dq,
                       cos=torch.from_numpy(cos).to(DEV) if rot else None,
                       sin=torch.from_numpy(sin).to(DEV) if rot else None, interleaved=interleaved)
    torch.cuda.synchronize()
    same_cache(cache, want)
    assert torch.equal(got.cpu().view(torch.int16), q_want.view(torch.int16))
    assert torch.equal(d.cpu().view(torch.int16), qkv.view(torch.int16))
    # the queries in place, within the projection's output, and the same again
    out = fq.kv_append(cache, dk, dv, i32(table), i32(lens), None if one else i32(starts), q=dq, q_out=dq,
                       cos=torch.from_numpy(cos).to(DEV) if rot else None,
                       sin=torch.from_numpy(sin).to(DEV) if rot else None, interleaved=interleaved)
    torch.cuda.synchronize()
    assert out is dq
    assert torch.equal(dq.cpu().view(torch.int16), q_want.view(torch.int16))
    assert torch.equal(d[:, at:].cpu().view(torch.int16), qkv[:, at:].view(torch.int16))
    same_cache(cache, want)


@pytest.mark.parametrize("dim,page,step", [(128, 64, 1), (64, 16, 1), (192, 128, 1), (128, 64, 5), (256, 32, 7)])
def test_page_grows_token_by_token(gpu_lib, dim, page, step):
    """Magnitudes that double again and again: the earlier codes of the page
    follow the scale at each call, through the subnormal codes to zero."""
    fq, g = gpu_lib, torch.Generator().manual_seed(7)
    heads, total = 2, page + page // 2
    width = -(-total // page)
    table = [list(range(width))]
    cache = random_cache(fq, g, width, heads, page, dim)
    want = host(cache)
    k = (torch.randn((total, heads, dim), generator=g) * torch.exp2(torch.arange(total) / 3.0)[:, None, None]).to(torch.bfloat16)
    v = (torch.randn((total, heads, dim), generator=g) * torch.exp2(torch.arange(total) / 2.0 - 9)[:, None, None]).to(torch.bfloat16)
    for at in range(0, total, step):
        n = min(step, total - at)
        kk, vv = k[at:at + n], v[at:at + n]
        ref.append(want, kk, vv, table, [at + n], [0, n])
        assert fq.kv_append(cache, kk.to(DEV), vv.to(DEV), i32(table), i32([at + n]),
                            None if step == 1 else i32([0, n])) is None
    torch.cuda.synchronize()
    same_cache(cache, want)
    # a page decodes as the package's dequantize decodes any block
    x = fq.dequantize(cache.k[0, 1], cache.k_scale[0, 1].view(1, 1), (page, dim))
    assert np.array_equal(x.cpu().numpy(), (ref.decode(want[0][0, 1]) * want[2][0, 1]).astype(np.float32))


def test_power_of_two_growth_rounds_once(gpu_lib):
    """Codes of a page filled token by token equal those of the whole page
    stored at once wherever they are normal numbers at every step."""
    fq, g = gpu_lib, torch.Generator().manual_seed(11)
    S, D = 64, 128
    x = ((1 + torch.rand((S, 1, D), generator=g)) * torch.exp2(torch.arange(S) / 16.0)[:, None, None]).to(torch.bfloat16).to(DEV)
    one, all_ = (fq.KvCache.empty(1, 1, D, S, device=DEV) for _ in range(2))
    table = i32([[0]])
    fq.kv_append(all_, x, x, table, i32([S]), i32([0, S]))
    for t in range(S):
        fq.kv_append(one, x[t:t + 1], x[t:t + 1], table, i32([t + 1]))
    torch.cuda.synchronize()
    same_cache(one, host(all_))


@pytest.mark.parametrize("new", [None, 1, 3])
@pytest.mark.parametrize("loud", [True, False])
def test_append_to_pages_whose_scale_is_no_power_of_two(gpu_lib, new, loud):
    """Pages that something else has filled: the scale stays where the new
    tokens fit, and gives way to a power of two where they do not."""
    fq, g = gpu_lib, torch.Generator().manual_seed(11)
    heads, size, dim, held, n = 3, 64, 128, 21, new or 1
    cache = random_cache(fq, g, 1, heads, size, dim, pow2=False)
    want = host(cache)
    k, v = (torch.randn((n, heads, dim), generator=g).to(torch.bfloat16) * (64.0 if loud else 0.0625) for _ in range(2))
    one = np.float32(1)
    for x, codes, scale, turned in ((k, want[0], want[2], False), (v, want[1], want[3], True)):
        for h in range(heads):
            at = codes[0, h].T if turned else codes[0, h]
            x32, was = x[:, h].float().numpy(), scale[0, h]
            s = np.float32(max(ref.fit(np.abs(x32).max()), was))
            assert (s > was) == loud
            if loud:
                at[:held] = ref.encode((ref.decode(at[:held]).astype(np.float32) * (was * (one / s))).astype(np.float64))
            at[held:held + n] = ref.encode((x32 * (one / s)).astype(np.float64))
            scale[0, h] = s
    fq.kv_append(cache, k.to(DEV), v.to(DEV), i32([[0]]), i32([held + n]), None if new is None else i32([0, n]))
    same_cache(cache, want)


@pytest.mark.parametrize("single", [True, False])
def test_append_leaves_out_what_has_no_place(gpu_lib, single):
    """Pages that are none, positions beyond the table, beyond the rotation's
    rows or below zero, sequences of no tokens, rows of no sequence: nothing of
    theirs is stored, everything else is."""
    fq, g = gpu_lib, torch.Generator().manual_seed(3)
    D, S, heads, group, pages, width = 64, 16, 2, 2, 12, 3
    cache = random_cache(fq, g, pages, heads, S, D)
    want = host(cache)
    table = [[0, 1, -1], [2, 99, 3], [4, -2147483648, 2147483647], [5, 6, 7], [8, 12, 9], [10, 11, 3]]   # 3: read by two, stored by one
    lens = [33, 20, 40, 100, 0, 48]
    new = [1] * 6 if single else [20, 9, 40, 60, 3, 17]
    starts = starts_of(new)
    if not single:
        starts = [s + 2 for s in starts]            # two rows before the first sequence, three behind the last
    T = starts[-1] + (0 if single else 3)
    _, q, k, v = append_inputs(g, T, heads, group, D)
    cos, sin = rotation(46, 64)
    marker = torch.full((T, heads * group, D), 7.0, dtype=torch.bfloat16)
    q_want = marker.clone()
    ref.append(want, k, v, table, lens, starts, q, q_want, cos, sin)
    got = marker.to(DEV)
    fq.kv_append(cache, k.to(DEV), v.to(DEV), i32(table), i32(lens), None if single else i32(starts), q=q.to(DEV),
                 q_out=got, cos=torch.from_numpy(cos).to(DEV), sin=torch.from_numpy(sin).to(DEV))
    torch.cuda.synchronize()
    same_cache(cache, want)
    assert torch.equal(got.cpu().view(torch.int16), q_want.view(torch.int16))


@pytest.mark.parametrize("single", [True, False])
def test_positions_that_attention_does_not_see_are_not_stored(gpu_lib, single):
    """The last positions below 2^31 - 1024 are stored, those from there on are
    not, though the table has pages for them; their queries are rotated all the
    same (here by nothing)."""
    fq, g = gpu_lib, torch.Generator().manual_seed(23)
    S, D, limit = 256, 64, (1 << 31) - 1024
    lens = [limit, limit + 1, (1 << 31) - 1] if single else [limit + 2, limit + 300, (1 << 31) - 1]
    new = [1, 1, 1] if single else [4, 301, 9]
    starts = starts_of(new)
    cache = random_cache(fq, g, 12, 1, S, D)
    want = host(cache)
    table = torch.full((3, 1 << 23), -1, dtype=torch.int32, device=DEV)
    for b in range(3):
        table[b, -5:-1] = i32([4 * b, 4 * b + 1, 4 * b + 2, 4 * b + 3])
    table[2, -1] = 11
    near = [[-1] * 3 + [4 * b] for b in range(3)]    # the same slots of short sequences
    _, q, k, v = append_inputs(g, starts[-1], 1, 2, D)
    keep = [(b, r) for b in range(3) for r in range(new[b]) if lens[b] - new[b] + r < limit]
    if keep:
        kept = [starts[b] + r for b, r in keep]
        counts = [sum(1 for x, _ in keep if x == b) for b in range(3)]
        ref.append(want, k[kept], v[kept], near, [4 * S if c else 0 for c in counts], starts_of(counts))
    got = fq.kv_append(cache, k.to(DEV), v.to(DEV), table, i32(lens), None if single else i32(starts), q=q.to(DEV))
    torch.cuda.synchronize()
    same_cache(cache, want)
    assert torch.equal(got.cpu().view(torch.int16), q.contiguous().view(torch.int16))


# -------------------------------------------------------------- attention

def check_attention(fq, cache, q, table, lens, starts, one, **kw):
    """Against the definition with a table just as wide as the sequences and
    with room for long ones (keys then split over workgroups), each twice."""
    out, lse, tol, tol_lse = ref.attention(host(cache), q, table, lens, starts, **kw)
    rows = [r for b in range(len(lens)) for r in range(starts[b], starts[b + 1])]
    empty = torch.isinf(lse[rows])
    dq, st = q.to(DEV), None if one else i32(starts)
    for room in (0, 20 * 64 // cache.page_size):
        wide = i32([list(r) + [-1] * room for r in table])
        got, got_lse = fq.kv_attention(cache, dq, wide, i32(lens), st, return_lse=True, **kw)
        again = fq.kv_attention(cache, dq, wide, i32(lens), st, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), again.view(torch.int16))
        got, got_lse = got.cpu().double(), got_lse.cpu().double()
        off = (got[rows] - out[rows]).abs()
        assert not torch.isnan(off).any()
        assert (off <= tol[rows]).all(), (room, float((off / tol[rows]).max()))
        assert torch.equal(empty, torch.isinf(got_lse[rows])) and (got_lse[rows][empty] < 0).all()
        off = (got_lse[rows] - lse[rows])[~empty].abs()
        assert (off <= tol_lse[rows][~empty]).all(), room
    return got


ATTENTION = [
    # dim, page, heads, group, lens, new, window
    (128, 64, 2, 4, [1, 64, 65, 300, 2], None, 0),
    (64, 16, 3, 1, [1, 16, 17, 63, 129], None, 0),
    (192, 32, 1, 5, [31, 257], None, 0),
    (256, 256, 2, 2, [1, 255, 513], None, 0),
    (128, 128, 1, 16, [129, 1000], None, 0),
    (64, 64, 1, 37, [200, 3], None, 0),                 # more query heads than a tile's rows
    (128, 16, 2, 3, [700, 5], None, 100),
    (64, 16, 2, 1, [500, 64, 65], None, 1),
    (128, 64, 2, 4, [300, 70, 9, 64], [5, 3, 9, 1], 0),
    (64, 32, 1, 7, [129, 33, 10], [29, 33, 0], 0),
    (192, 16, 2, 2, [90, 200], [17, 40], 33),
    (256, 128, 1, 1, [300], [70], 0),
    (128, 64, 1, 8, [200, 131], [150, 131], 0),         # prompts
    (128, 64, 2, 2, [330], [257], 64),
    (64, 64, 1, 1, [400], [400], 0),
    # 33 to 64 query rows a sequence: tiles of two waves
    (128, 64, 2, 8, [200, 71, 130], [5, 6, 4], 0),
    (128, 16, 1, 5, [333], [9], 50),
    (64, 256, 2, 3, [300, 17], [13, 12], 0),
    (64, 32, 1, 50, [65], [1], 0),
    # tiles of four waves at every kind of page and width
    (128, 16, 1, 4, [190], [90], 0),
    (128, 256, 1, 4, [390], [65], 0),
    (64, 16, 2, 2, [130, 64], [70, 64], 20),
    (192, 128, 1, 3, [260], [50], 0),
    (256, 32, 1, 2, [170], [77], 0),
    (256, 64, 1, 1, [129], [129], 0),
    # few keys: two row tiles of 64 and a rest; many sequences of 17 to 32 rows
    (128, 64, 1, 9, [170, 20], [20, 16], 0),
    (128, 32, 3, 3, [40 + b for b in range(90)], [7] * 90, 0),
    # 33 to 64 rows of wide heads, few and many row tiles
    (256, 64, 2, 8, [200, 71, 130], [5, 6, 4], 0),
    (192, 16, 3, 6, [20 + b for b in range(40)], [8] * 40, 30),
]


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("dim,page,heads,group,lens,new,window", ATTENTION)
def test_attention_within_its_roundings(gpu_lib, dim, page, heads, group, lens, new, window, pow2):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + page + sum(lens))
    one = new is None
    starts = starts_of([1] * len(lens) if one else new)
    width = max(-(-x // page) for x in lens)
    pages = len(lens) * width + 1
    cache = random_cache(fq, g, pages, heads, page, dim, pow2)
    table = tables(g, [-(-x // page) for x in lens], width, pages)
    q = torch.randn((starts[-1], heads * group, dim), generator=g).to(torch.bfloat16)
    check_attention(fq, cache, q, table, lens, starts, one, window=window)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 3.0])
@pytest.mark.parametrize("new", [None, [3, 2], [9, 8], [40, 31]])
def test_attention_with_other_scales(gpu_lib, scale, new):
    """Negative, zero, tiny and large factors of the scores in every kernel."""
    fq, g = gpu_lib, torch.Generator().manual_seed(21)
    lens, starts = [150, 77], starts_of(new or [1, 1])
    cache = random_cache(fq, g, 7, 1, 32, 64)
    q = (0.1 * torch.randn((starts[-1], 5, 64), generator=g)).to(torch.bfloat16)
    check_attention(fq, cache, q, [[0, 1, 2, 3, 4], [5, 6, 0, -1, -1]], lens, starts, new is None, scale=scale)


def test_attention_without_splits_over_many_row_tiles(gpu_lib):
    """Enough row tiles to fill the chip: keys are not split, and no workspace
    is taken; the first sequences share their pages."""
    fq, g = gpu_lib, torch.Generator().manual_seed(22)
    n, heads, group, new = 64, 8, 8, 9
    lens = [9 + (11 * b) % 80 for b in range(n)]
    cache = random_cache(fq, g, 2 * n, heads, 64, 64)
    table = [[2 * b, 2 * b + 1] for b in range(n)]
    table[1] = table[0]
    starts = starts_of([new] * n)
    q = torch.randn((n * new, heads * group, 64), generator=g).to(torch.bfloat16)
    assert fq.kv_attention_workspace_bytes(cache, q.to(DEV), i32(table)) == 0
    check_attention(fq, cache, q, table, lens, starts, False)


@pytest.mark.parametrize("window", [60, 900, 1500, 3000])
@pytest.mark.parametrize("new", [1, 6, 30, 140])
def test_attention_under_windows_in_long_tables(gpu_lib, new, window):
    """Whether keys are split goes by what the window leaves to see."""
    fq, g = gpu_lib, torch.Generator().manual_seed(window + new)
    lens = [3000, 40, 2500]
    news = [new, min(new, 40), 2]
    counts = [-(-x // 64) for x in lens]
    cache = random_cache(fq, g, sum(counts) + 1, 1, 64, 64)
    table = tables(g, counts, max(counts), cache.num_pages)
    starts = starts_of(news)
    q = torch.randn((starts[-1], 2, 64), generator=g).to(torch.bfloat16)
    check_attention(fq, cache, q, table, lens, starts, False, window=window)


@pytest.mark.parametrize("length", [5000, 20001])
def test_attention_split_over_a_long_sequence(gpu_lib, length):
    fq, g = gpu_lib, torch.Generator().manual_seed(5)
    cache = random_cache(fq, g, -(-length // 64) + 1, 1, 64, 128)
    table = tables(g, [-(-length // 64)], -(-length // 64), cache.num_pages)
    q = torch.randn((1, 8, 128), generator=g).to(torch.bfloat16)
    check_attention(fq, cache, q, table, [length], [0, 1], True)
    q = torch.randn((3, 8, 128), generator=g).to(torch.bfloat16)
    check_attention(fq, cache, q, table, [length], [0, 3], False, scale=0.05)


def test_attention_of_many_sequences(gpu_lib):
    """More than 64 sequences, two rounds of the planning scan, mixed lengths
    and some without tokens."""
    fq, g = gpu_lib, torch.Generator().manual_seed(6)
    n = 150
    lens = [(37 * b) % 210 for b in range(n)]
    counts = [-(-x // 16) for x in lens]
    cache = random_cache(fq, g, sum(counts) + 1, 1, 16, 64)
    table = tables(g, counts, max(counts), cache.num_pages)
    q = torch.randn((n, 2, 64), generator=g).to(torch.bfloat16)
    got = check_attention(fq, cache, q, table, lens, list(range(n + 1)), True)
    assert (got[[b for b in range(n) if lens[b] == 0]] == 0).all()
    new = [min(lens[b], b % 5) for b in range(n)]
    starts = starts_of(new)
    q = torch.randn((starts[-1], 2, 64), generator=g).to(torch.bfloat16)
    check_attention(fq, cache, q, table, lens, starts, False)


@pytest.mark.parametrize("new", [1, 5, 12, 40])
def test_attention_with_few_sequences_awake(gpu_lib, new):
    """Long runs of sequences without query tokens, which hold some all the
    same, before, between and behind the others."""
    fq, g = gpu_lib, torch.Generator().manual_seed(new)
    n, awake = 300, {70: 700, 71: 333, 139: 90, 267: 1200}
    lens = [awake.get(b, 16 * (b % 3)) for b in range(n)]
    counts = [-(-x // 16) for x in lens]
    cache = random_cache(fq, g, sum(counts) + 1, 1, 16, 128)
    table = tables(g, counts, max(counts), cache.num_pages)
    starts = starts_of([new if b in awake else 0 for b in range(n)])
    q = torch.randn((starts[-1], 3, 128), generator=g).to(torch.bfloat16)
    check_attention(fq, cache, q, table, lens, starts, False)


@pytest.mark.parametrize("one", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_what_no_query_sees_has_no_effect(gpu_lib, one, dim):
    """NaN codes and NaN scales in slots behind the sequence, in pages of
    nobody, below the window, and page numbers that are none: the tokens that
    are there count, nothing else does; a row that sees nothing is zero."""
    fq, g = gpu_lib, torch.Generator().manual_seed(8)
    S = 16
    cache = random_cache(fq, g, 24, 2, S, dim)
    table = [[0, 1, 2, 3, 4, 5], [6, -1, 7, 99, 8, 9], [10, 11, 2147483647, -5, 12, 13], [-1] * 6, [14, 15, 16, 17, 18, 19]]
    lens, window = [37, 96, 61, 50, 200], 70
    new = [1] * 5 if one else [3, 20, 1, 2, 120]
    starts = starts_of(new)
    kb, vb = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    used = {(p, j) for b in range(5) for j, p in enumerate(table[b]) if 0 <= p < 24}
    clean = set()
    for b in range(5):
        lo = max(0, lens[b] - new[b] + 1 - window)
        for j, p in enumerate(table[b]):
            if not 0 <= p < 24:
                continue
            for s in range(S):
                if lo <= j * S + s < lens[b]:
                    clean.add((p, s))
    for p in range(24):
        for s in range(S):
            if (p, s) not in clean:
                kb[p, :, s] = 0x7F
                vb[p, :, :, s] = 0xFF
        if not any((p, s) in clean for s in range(S)):
            cache.k_scale[p] = float("nan")
            cache.v_scale[p] = float("inf")
    assert used
    q = torch.randn((starts[-1], 6, dim), generator=g).to(torch.bfloat16)
    got = check_attention(fq, cache, q, table, lens, starts, one, window=window)
    assert (got[starts[3]:starts[4]] == 0).all()


def test_more_query_tokens_than_the_sequence_holds(gpu_lib):
    """Rows before a sequence's first token see nothing; rows of no sequence
    keep what they hold, in every output."""
    fq, g = gpu_lib, torch.Generator().manual_seed(9)
    cache = random_cache(fq, g, 6, 1, 16, 64)
    lens, starts, table = [3, 20], [2, 9, 12], [[0, 1], [2, 3]]
    q = torch.randn((15, 4, 64), generator=g).to(torch.bfloat16)
    want, lse, tol, _ = ref.attention(host(cache), q, table, lens, starts)
    out = torch.full((15, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((15, 4), 9.0, device=DEV)
    fq.kv_attention(cache, q.to(DEV), i32(table), i32(lens), i32(starts), out=out, lse=ls)
    torch.cuda.synchronize()
    assert (out[:2] == 5).all() and (out[12:] == 5).all() and (ls[:2] == 9).all() and (ls[12:] == 9).all()
    assert (out[2:6] == 0).all() and torch.isinf(ls[2:6]).all()
    assert ((out.cpu().double() - want).abs()[2:12] <= tol[2:12]).all()


def test_starts_that_are_no_offsets_stay_in_bounds(gpu_lib):
    """query_start is clamped: negative, decreasing and far values reach no
    memory outside the buffers (their rows are unspecified)."""
    fq, g = gpu_lib, torch.Generator().manual_seed(10)
    pad = 4
    cache = random_cache(fq, g, 8, 2, 16, 64)
    before = host(cache)
    buf = torch.full((pad + 9 + pad, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    q = torch.randn((9, 4, 64), generator=g).to(torch.bfloat16).to(DEV)
    kv = q[:, :2].contiguous()
    table = i32([[0, 1], [2, 3], [4, 5]])
    for starts in ([-5, 3, 2, 1 << 30], [9, 0, 9, 0], [1 << 30, -1, 1 << 30, 4], [4, 4, 4, 4]):
        for lens in ([20, 30, 7], [-3, 1 << 30, 0]):
            fq.kv_attention(cache, q, table, i32(lens), i32(starts), out=buf[pad:pad + 9])
            fq.kv_append(cache, kv, kv, table, i32(lens), i32(starts), q=q, q_out=buf[pad:pad + 9])
    torch.cuda.synchronize()
    assert (buf[:pad] == 3).all() and (buf[pad + 9:] == 3).all()
    after = host(cache)
    for a, b in zip(before, after):
        assert np.array_equal(a[6:].view(np.uint8), b[6:].view(np.uint8))


def test_strided_rows_and_in_place_output(gpu_lib):
    fq, g = gpu_lib, torch.Generator().manual_seed(12)
    cache = random_cache(fq, g, 10, 2, 32, 128)
    lens, starts, table = [70, 40], [0, 6, 8], [[0, 1, 2], [3, 4, 5]]
    q = torch.randn((8, 8, 128), generator=g).to(torch.bfloat16)
    want = fq.kv_attention(cache, q.to(DEV), i32(table), i32(lens), i32(starts))
    wide = torch.zeros((8, 12, 136), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10, 8:] = q.to(DEV)
    view = wide[:, 2:10, 8:]
    heads_first = q.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    big = torch.full((2, 5), -7, dtype=torch.int32, device=DEV)
    big[:, :3] = i32(table)
    got = fq.kv_attention(cache, view, big[:, :3], i32(lens), i32(starts))
    got2 = fq.kv_attention(cache, heads_first, i32(table), i32(lens), i32(starts), out=torch.empty_like(heads_first))
    assert torch.equal(got, want) and torch.equal(got2, want)
    back = fq.kv_attention(cache, view, i32(table), i32(lens), i32(starts), out=view)
    torch.cuda.synchronize()
    assert torch.equal(back, want)
    wide[:, 2:10, 8:] = 0
    assert (wide == 0).all()


def test_offsets_beyond_32_bits(gpu_lib):
    """Blocks that lie more than 2^32 bytes into the cache."""
    fq, g = gpu_lib, torch.Generator().manual_seed(13)
    heads, S, D = 8, 256, 256
    pages = (1 << 32) // (heads * S * D) + 4
    cache = fq.KvCache(*(torch.empty(s, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
                         for s in ((pages, heads, S, D), (pages, heads, D, S))),
                       torch.ones((pages, heads), device=DEV), torch.ones((pages, heads), device=DEV))
    small = fq.KvCache.empty(4, heads, D, S, device=DEV)
    lens, starts = [300, 258], [0, 300, 303]
    k, v = (torch.randn((303, heads, D), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn((303, heads, D), generator=g).to(torch.bfloat16).to(DEV)
    far = [[pages - 1, pages - 3], [pages - 2, pages - 4]]
    near = [[3, 1], [2, 0]]
    for b in (0, 1):
        small.k[near[b][0]].zero_()
        cache.k[far[b][0]].zero_()
        cache.v[far[b][0]].zero_()
        cache.k[far[b][1]].zero_()
        cache.v[far[b][1]].zero_()
    outs = []
    for c, table in ((cache, far), (small, near)):
        fq.kv_append(c, k, v, i32(table), i32(lens), i32(starts))
        fq.kv_append(c, k[:2], v[:2], i32(table), i32([301, 259]))
        outs.append(fq.kv_attention(c, q, i32(table), i32(lens), i32(starts)))
        outs.append(fq.kv_attention(c, q[:2], i32(table), i32([301, 259])))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    for b in (0, 1):
        for x, y in zip(far[b], near[b]):
            assert torch.equal(cache.k[x].view(torch.uint8), small.k[y].view(torch.uint8))
            assert torch.equal(cache.v[x].view(torch.uint8), small.v[y].view(torch.uint8))


# ------------------------------------------------------------ run together

def test_prompt_steps_and_drafts_together(gpu_lib):
    """As a rollout runs them: prompts enter the cache, then single tokens,
    then drafted tokens of which some are taken back; every attention is that
    of the tokens stored so far, in 64 bits."""
    fq, g = gpu_lib, torch.Generator().manual_seed(14)
    dim, page, heads, group = 128, 32, 2, 4
    B, width = 3, 5
    cache = fq.KvCache.empty(B * width + 1, heads, dim, page, device=DEV)
    want = host(cache)
    table = tables(g, [width] * B, width, B * width + 1)
    cos, sin = rotation(160, 128)
    dcos, dsin = torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV)
    lens = [0] * B
    for new, taken in (([70, 5, 33], None), ([1] * 3, None), ([1] * 3, None), ([4, 1, 6], [2, 1, 0]), ([1] * 3, None),
                       ([0, 3, 8], None)):
        starts = starts_of(new)
        lens = [a + b for a, b in zip(lens, new)]
        one = new == [1] * B
        _, q, k, v = append_inputs(g, starts[-1], heads, group, dim, 0.3)
        q_want = torch.zeros_like(q)
        ref.append(want, k, v, table, lens, starts, q, q_want, cos, sin)
        ds = None if one else i32(starts)
        turned = fq.kv_append(cache, k.to(DEV), v.to(DEV), i32(table), i32(lens), ds, q=q.to(DEV), cos=dcos, sin=dsin)
        assert torch.equal(turned.cpu().view(torch.int16), q_want.view(torch.int16))
        got = fq.kv_attention(cache, turned, i32(table), i32(lens), ds)
        out, _, tol, _ = ref.attention(want, q_want, table, lens, starts)
        torch.cuda.synchronize()
        same_cache(cache, want)
        assert ((got.cpu().double() - out).abs() <= tol).all()
        if taken is not None:
            lens = [n - a + t for n, a, t in zip(lens, new, taken)]


def test_captured_step_follows_the_lengths(gpu_lib):
    """One graph of a decoding step (append, then attention), replayed while
    the sequences grow across pages, equals the eager calls each time; two
    graphs on streams of their own do not disturb each other."""
    fq, g = gpu_lib, torch.Generator().manual_seed(15)
    dim, page, heads, group, B, width = 128, 16, 2, 4, 5, 8
    cos, sin = (torch.from_numpy(x).to(DEV) for x in rotation(width * page, 128))
    table = i32([r + [-1] * 80 for r in tables(g, [width] * B, width, B * width)])   # room: keys are split
    sets = []
    for i in range(2):
        cache, eager = (fq.KvCache.empty(B * width, heads, dim, page, device=DEV) for _ in range(2))
        lens = i32([1 + 7 * i, 15, 16, 30, 2])
        qkv = torch.zeros((B, heads * (group + 2), dim), dtype=torch.bfloat16, device=DEV)
        q, k, v = qkv[:, :heads * group], qkv[:, heads * group:heads * (group + 1)], qkv[:, heads * (group + 1):]
        turned = torch.empty((B, heads * group, dim), dtype=torch.bfloat16, device=DEV)
        out = torch.empty_like(turned)
        ws = torch.empty(max(16, fq.kv_attention_workspace_bytes(cache, turned, table)), dtype=torch.uint8, device=DEV)
        stream = torch.cuda.Stream()

        def step(c, o):
            fq.kv_append(c, k, v, table, lens, q=q, q_out=turned, cos=cos, sin=sin)
            fq.kv_attention(c, turned, table, lens, out=o, workspace=ws)

        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            step(cache, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(cache, out)
        for c in (cache, eager):
            c.k.view(torch.uint8).zero_()
            c.v.view(torch.uint8).zero_()
        sets.append((graph, stream, cache, eager, lens, qkv, out, q, k, v))
    torch.cuda.synchronize()
    for _ in range(12):
        for graph, stream, cache, eager, lens, qkv, out, *_ in sets:
            qkv.copy_(torch.randn(qkv.shape, generator=g).to(torch.bfloat16))
        torch.cuda.synchronize()
        for graph, stream, *_ in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, cache, eager, lens, qkv, out, q, k, v in sets:
            t = fq.kv_append(eager, k, v, table, lens, q=q, cos=cos, sin=sin)
            want = fq.kv_attention(eager, t, table, lens)
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
            same_cache(cache, host(eager))
            lens += 3
        torch.cuda.synchronize()


def test_graphs_that_share_a_workspace_in_turn(gpu_lib):
    """Nothing is kept in the workspace from one call for the next: two graphs
    of different shapes replayed in turn over one, with other bytes in it
    before each; and a graph whose call takes its own."""
    fq, g = gpu_lib, torch.Generator().manual_seed(17)
    cache = random_cache(fq, g, 60, 2, 64, 128)
    table = i32([list(range(30)), list(range(30, 60))])
    lens = i32([1900, 1500])
    calls = []
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    for heads, new, own in ((8, None, False), (4, [6, 3], False), (16, [90, 33], False), (8, None, True)):
        starts = None if new is None else i32(starts_of(new))
        q = torch.randn((2 if new is None else sum(new), heads, 128), generator=g).to(torch.bfloat16).to(DEV)
        out = torch.zeros_like(q)
        need = fq.kv_attention_workspace_bytes(cache, q, table)
        assert 0 < need <= ws.numel()

        def call(q=q, starts=starts, out=out, own=own):
            fq.kv_attention(cache, q, table, lens, starts, out=out, workspace=None if own else ws)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        calls.append((graph, q, starts, out))
    for i in range(4):
        lens.copy_(i32([1900 - 301 * i, 1500 - 377 * i]))
        for graph, q, starts, out in calls:
            ws.fill_(255 if i % 2 else 0x3C)
            out.zero_()
            graph.replay()
            want = fq.kv_attention(cache, q, table, lens, starts)
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_side_stream(gpu_lib):
    """Work goes to the current stream, in order with the caller's other work."""
    fq, g = gpu_lib, torch.Generator().manual_seed(16)
    cache = random_cache(fq, g, 40, 4, 64, 128)
    table, lens = i32([list(range(20)), list(range(20, 40))]), i32([1270, 1100])
    q = torch.randn((2, 16, 128), generator=g).to(torch.bfloat16).to(DEV)
    want = fq.kv_attention(cache, q, table, lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = torch.zeros_like(q)
        for _ in range(20):
            x.copy_(q * 0.5)
            x.add_(x)
            got = fq.kv_attention(cache, x, table, lens)
    s.synchronize()
    assert torch.equal(got, want)


# ----------------------------------------------------------------- refusals

def test_refusals(gpu_lib):
    fq = gpu_lib
    cache = fq.KvCache.empty(4, 2, 64, 16, device=DEV)
    table, lens, starts = i32([[0, 1]]), i32([5]), i32([0, 3])
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device=DEV)
    cos = torch.zeros((8, 32), device=DEV)
    ap = lambda k=x, v=x, tb=table, ln=lens, st=starts, **kw: fq.kv_append(cache, k, v, tb, ln, st, **kw)  # noqa: E731
    at = lambda q=q, tb=table, ln=lens, st=starts, **kw: fq.kv_attention(cache, q, tb, ln, st, **kw)       # noqa: E731
    ap()
    at()
    for call in (lambda: ap(k=x.float()), lambda: at(q=q.half()), lambda: ap(tb=table.long()), lambda: at(ln=lens.long()),
                 lambda: at(st=starts.long()), lambda: ap(cos=cos.half(), sin=cos.half())):
        with pytest.raises(TypeError):
            call()
    odd = torch.zeros((3, 2, 68), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: ap(k=x[:2]), lambda: ap(v=x[:, :1]), lambda: ap(st=None), lambda: at(st=None),
                 lambda: ap(k=odd[:, :, 4:]), lambda: ap(k=x.transpose(1, 2).contiguous().transpose(1, 2)),
                 lambda: at(q=q[:, :3]), lambda: at(q=q[:, :, :32]), lambda: at(window=-1), lambda: at(window=1 << 31),
                 lambda: at(scale=float("nan")), lambda: at(scale=1e39), lambda: ap(cos=cos), lambda: ap(sin=cos),
                 lambda: ap(cos=cos[:, :4].contiguous(), sin=cos[:, :4].contiguous()), lambda: ap(cos=cos, sin=cos[:4]),
                 lambda: ap(cos=torch.zeros((8, 40), device=DEV), sin=torch.zeros((8, 40), device=DEV)),
                 lambda: ap(q_out=q), lambda: ap(q=q[:, :3]), lambda: ap(q=q, q_out=q[:2]),
                 lambda: ap(q=q, q_out=q[:1].expand(3, 4, 64)), lambda: at(out=q[:, :1].expand(3, 4, 64)),
                 lambda: at(tb=table[0]), lambda: at(tb=i32([[0], [1]])), lambda: at(tb=i32([[0, 1], [2, 3]]).t()[:1]),
                 lambda: at(st=i32([0, 1, 3])), lambda: ap(k=x.cpu()), lambda: at(tb=table.cpu()), lambda: at(st=starts.cpu()),
                 lambda: at(lse=torch.zeros((3, 3), device=DEV)), lambda: at(workspace=torch.zeros(64, dtype=torch.uint8)),
                 lambda: fq.KvCache.empty(1, 1, 64, 24, device=DEV), lambda: fq.KvCache.empty(0, 1, 64, 16, device=DEV)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(fq.Fp8bqError, match="workspace"):
        at(tb=i32([[0, 1] + [-1] * 80]), workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    empty = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    assert at(q=empty, st=i32([0, 0])).shape == (0, 4, 64)
    assert ap(k=empty[:, :2], v=empty[:, :2], st=i32([0, 0])) is None
    none = torch.zeros((0, 2), dtype=torch.int32, device=DEV)
    assert at(q=empty, tb=none, ln=i32([]), st=None).shape == (0, 4, 64)
    assert (at(q=q, tb=torch.zeros((1, 0), dtype=torch.int32, device=DEV)) == 0).all()
    torch.cuda.synchronize()
    assert math.isfinite(float(at().float().sum()))


FORMS = [
    # dim, page, heads, group, new: every kernel, its rows split over workgroups and not
    (64, 16, 2, 3, None), (128, 64, 2, 4, None), (256, 128, 1, 2, None),
    (64, 64, 1, 5, [6, 4, 4, 1]), (128, 32, 2, 4, [6, 5, 6, 1]), (256, 64, 1, 8, [6, 5, 5, 1]),
    (64, 32, 1, 8, [6, 5, 7, 1]), (128, 64, 2, 8, [5, 6, 4, 1]),
    (64, 64, 2, 4, [40, 33, 50, 1]), (128, 16, 1, 4, [50, 40, 33, 1]), (256, 64, 1, 2, [70, 90, 50, 1]),
]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("dim,page,heads,group,new", FORMS)
def test_query_rows_that_are_no_numbers(gpu_lib, dim, page, heads, group, new, split):
    """A row of queries with a NaN or an infinity is NaN, and so is its sum, if
    it sees a token: not the zeros of a row that sees none.  Its neighbours are
    as without it.  Keys are positive in channel 0, so that an infinity of
    either sign there makes all of its row's scores infinite alike."""
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + page)
    lens = [1300, 700, 130, 1] if split else [250, 130, 70, 1]
    n = [1] * 4 if new is None else new
    starts = starts_of(n)
    counts = [-(-x // page) for x in lens]
    cache = random_cache(fq, g, sum(counts) + 1, heads, page, dim)
    first = cache.k.view(torch.uint8)[..., 0]
    first &= 0x7F
    first[first == 0] = 0x38
    room = 1300 // page if split else 0
    table = i32([r + [-1] * room for r in tables(g, counts, max(counts), cache.num_pages)])
    q = torch.randn((starts[-1], heads * group, dim), generator=g).to(torch.bfloat16).to(DEV)
    st = None if new is None else i32(starts)
    assert (fq.kv_attention_workspace_bytes(cache, q, table) > 0) == split
    want, want_lse = fq.kv_attention(cache, q, table, i32(lens), st, return_lse=True)
    marks = [(0, 0, 3, math.nan), (0, heads * group - 1, 0, math.inf), (1, 0, 0, -math.inf), (1, heads, 0, math.inf),
             (2, 1, dim - 1, math.nan), (3, 0, 0, -math.inf), (3, heads * group - 1, 5, math.nan)]
    bad = torch.zeros((starts[-1], heads * group), dtype=torch.bool)
    x = q.clone()
    for b, h, c, value in marks:
        for row in {starts[b], starts[b + 1] - 1}:
            x[row, h, c] = value
            bad[row, h] = True
    bad = bad.to(DEV)
    got, lse = fq.kv_attention(cache, x, table, i32(lens), st, return_lse=True)
    torch.cuda.synchronize()
    assert torch.isnan(got[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(got[~bad].view(torch.int16), want[~bad].view(torch.int16))
    assert torch.equal(lse[~bad], want_lse[~bad])
    # rows that see nothing are zero whatever they hold
    x[:] = math.nan
    got, lse = fq.kv_attention(cache, x, table, i32([0, lens[1], -5, 1]), st, return_lse=True)
    torch.cuda.synchronize()
    none = torch.zeros(starts[-1], dtype=torch.bool)
    none[:starts[1]] = none[starts[2]:starts[3]] = True
    assert (got[none.to(DEV)] == 0).all() and (lse[none.to(DEV)] == -math.inf).all()
    assert torch.isnan(got[~none.to(DEV)]).all() and torch.isnan(lse[~none.to(DEV)]).all()


# ------------------------------------------------- shares of many key tiles

LONG = [6000, 2000, 4500, 3301]
SHARES = [
    # dim, page, heads, group, lens, new: totals of key tiles that make a share,
    # or a chunk, of 8 to 60 tiles in each kernel, and prompts and single tokens in one call
    (64, 16, 32, 1, LONG, None), (128, 64, 32, 2, LONG, None), (256, 128, 32, 1, LONG, None),
    (64, 64, 32, 1, LONG, [24, 20, 29, 17]), (128, 64, 16, 1, LONG, [24, 31, 9, 28]), (256, 32, 16, 1, LONG, [44, 50, 9, 60]),
    (64, 32, 32, 1, LONG, [48, 64, 33, 40]), (128, 64, 32, 1, LONG, [48, 64, 33, 40]),
    (64, 64, 32, 1, LONG, [100, 128, 70, 129]), (128, 16, 32, 1, LONG, [100, 128, 70, 129]), (192, 64, 16, 1, LONG, [70, 1, 130, 66]),
    (128, 64, 1, 8, [20001, 17], None), (128, 64, 2, 4, [20001], [400]), (128, 64, 2, 2, [1500, 900], [1500, 700]),
    (256, 64, 1, 2, [1200], [1200]),
    # a prompt among single tokens, by groups that choose each kernel
    (128, 64, 2, 1, [700] + [40 + 31 * b for b in range(70)], [700] + [1] * 70),
    (128, 64, 2, 2, [40 + 31 * b for b in range(70)] + [900], [1] * 70 + [700]),
    (64, 16, 1, 4, [40 + 31 * b for b in range(35)] + [900] + [2000 - 31 * b for b in range(35)], [1] * 35 + [700] + [1] * 35),
    (128, 32, 1, 8, [1300] + [40 + 31 * b for b in range(70)], [700] + [1] * 70),
]


@pytest.mark.parametrize("window", [0, 1111])
@pytest.mark.parametrize("dim,page,heads,group,lens,new", SHARES)
def test_every_key_counts_once(gpu_lib, dim, page, heads, group, lens, new, window):
    """Queries of zero weigh all keys they see alike.  The sum of weights is
    then their number, a sum of ones that fp32 holds exactly.  Its logarithm, up
    to 9.91, errs by the hardware's log2 (an ulp below 16: 2^-20, times ln 2), the
    product's rounding (2^-21) and that of ln 2 (9.91 * 2^-25): 1.5e-6, below
    2^-19; one key too many or too few among 20001 changes it by 5e-5.  Channel
    t % dim of a value is 1 in key tile t and 0 elsewhere, so that the output has
    each tile's share, rounded once to BF16 (the weights are 1 exactly)."""
    fq, g = gpu_lib, torch.Generator().manual_seed(31)
    one = new is None
    n = [1] * len(lens) if one else new
    starts = starts_of(n)
    counts = [-(-x // page) for x in lens]
    pages = sum(counts) + 1
    cache = random_cache(fq, g, pages, heads, page, dim)
    cache.v_scale.fill_(1.0)
    table = tables(g, counts, max(counts), pages)
    codes = torch.zeros((pages, dim, page), dtype=torch.uint8)
    for b, x in enumerate(lens):
        pos = torch.arange(x)
        rows = torch.tensor(table[b][:counts[b]])
        codes[rows[pos // page], (pos // 64) % dim, pos % page] = 0x38      # 1
    cache.v.view(torch.uint8).copy_(codes.to(DEV)[:, None].expand(pages, heads, dim, page))
    q = torch.zeros((starts[-1], heads * group, dim), dtype=torch.bfloat16, device=DEV)
    got, lse = fq.kv_attention(cache, q, i32(table), i32(lens), None if one else i32(starts), window=window, return_lse=True)
    torch.cuda.synchronize()
    got, lse = got.cpu().double(), lse.cpu().double()
    for b, x in enumerate(lens):
        pos = torch.arange(x - n[b], x)[:, None]
        key = torch.arange(x)[None, :]
        seen = (key <= pos) & ((key > pos - window) if window else (key >= 0))
        share = torch.zeros((n[b], dim), dtype=torch.float64).index_add_(1, (key[0] // 64) % dim, seen.double())
        share /= seen.sum(1, keepdim=True)
        mine = slice(starts[b], starts[b + 1])
        assert ((lse[mine] - seen.sum(1, keepdim=True).double().log()).abs() <= 2.0 ** -19).all(), b
        assert ((got[mine] - share[:, None]).abs() <= 1.001 * 2.0 ** -8 * share[:, None]).all(), b


@pytest.mark.parametrize("dim,page,heads,group,lens,new", SHARES)
def test_attention_over_many_key_tiles(gpu_lib, dim, page, heads, group, lens, new):
    """Random keys and values against 64 bits at the same sizes."""
    fq, g = gpu_lib, torch.Generator().manual_seed(32)
    one = new is None
    starts = starts_of([1] * len(lens) if one else new)
    counts = [-(-x // page) for x in lens]
    cache = random_cache(fq, g, sum(counts) + 1, heads, page, dim, False)
    table = tables(g, counts, max(counts), cache.num_pages)
    q = torch.randn((starts[-1], heads * group, dim), generator=g).to(torch.bfloat16)
    out, lse, tol, tol_lse = ref.attention_of_long(host(cache), q, table, lens, starts)
    got, got_lse = fq.kv_attention(cache, q.to(DEV), i32(table), i32(lens), None if one else i32(starts), return_lse=True)
    torch.cuda.synchronize()
    off = (got.cpu().double() - out).abs()
    assert (off <= tol).all(), float((off / tol).max())
    off = (got_lse.cpu().double() - lse).abs()
    assert (off <= tol_lse).all(), float((off / tol_lse).max())


def test_threads_at_once(gpu_lib):
    """Threads with a cache and a stream each append and attend at the same
    time, and get what each gets alone."""
    fq = gpu_lib
    cos, sin = (torch.from_numpy(x).to(DEV) for x in rotation(64, 128))

    def work(i, stream):
        g = torch.Generator().manual_seed(40 + i)
        with torch.cuda.stream(stream):
            cache = fq.KvCache.empty(24, 2, 128, 16, device=DEV)
            table = i32([r + [-1] * 80 for r in tables(g, [4] * 3, 4, 24)])
            outs = []
            for lens, new in (([20, 9, 1], [20, 9, 1]), ([21, 10, 2], None), ([30, 11, 9], [9, 1, 7]), ([31, 12, 10], None)) * 5:
                starts = None if new is None else i32(starts_of(new))
                T = 3 if new is None else sum(new)
                qkv = torch.randn((T, 12 + 2 * i, 128), generator=g).to(torch.bfloat16).to(DEV)
                q = fq.kv_append(cache, qkv[:, :2], qkv[:, 2:4], table, i32(lens), starts, q=qkv[:, 4:], cos=cos, sin=sin)
                outs.append(fq.kv_attention(cache, q, table, i32(lens), starts))
        stream.synchronize()
        return [o.cpu() for o in outs], host(cache)

    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    want = [work(i, streams[i]) for i in range(4)]
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        got = [f.result() for f in [pool.submit(work, i, streams[i]) for i in range(4)]]
    for (a, ca), (b, cb) in zip(want, got):
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))
        assert all(np.array_equal(x.view(np.uint8), y.view(np.uint8)) for x, y in zip(ca, cb))


def test_a_cache_keeps_its_buffers(gpu_lib):
    fq, g = gpu_lib, torch.Generator().manual_seed(18)
    cache, other = (random_cache(fq, g, 4, 2, 16, 64) for _ in range(2))
    k, packed = cache.k, cache._packed
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError, match="read-only"):
            setattr(cache, name, getattr(other, name))
    assert cache.k is k and cache._packed == packed
    assert (cache.num_pages, cache.kv_heads, cache.page_size, cache.head_dim) == (4, 2, 16, 64)
    assert cache.device == cache.k.device


def test_a_copied_cache_has_its_own_buffers(gpu_lib):
    """Appends to a deep copy, or to a cache that was saved and loaded, reach
    the copy; a shallow copy shares the buffers."""
    fq, g = gpu_lib, torch.Generator().manual_seed(19)
    cache = random_cache(fq, g, 4, 2, 16, 64)
    x = torch.randn((1, 2, 64), generator=g).to(torch.bfloat16).to(DEV)
    before = host(cache)
    after = host(cache)
    ref.append(after, x.cpu(), x.cpu(), [[3]], [5], [0, 1])
    saved = io.BytesIO()
    torch.save(cache, saved)
    saved.seek(0)
    for again in (copy.deepcopy(cache), torch.load(saved, weights_only=False)):
        fq.kv_append(again, x, x, i32([[3]]), i32([5]))
        torch.cuda.synchronize()
        same_cache(cache, before)
        same_cache(again, after)
    fq.kv_append(copy.copy(cache), x, x, i32([[3]]), i32([5]))
    torch.cuda.synchronize()
    same_cache(cache, after)
