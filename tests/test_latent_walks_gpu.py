"""Attention over latents where one workgroup walks many key tiles and several
row tiles: long runs of whole tiles, shares that end inside a row tile, batches
of more than 64 sequences, prompts among single tokens, and rows whose maximum
rises far while they are walked, so that sums are scaled on the way."""

import math

import pytest
import torch

import latent_reference as ref
from test_kv_gpu import i32, starts_of
from test_latent_gpu import absorbed_inputs, close, host

pytestmark = pytest.mark.gpu

DEV = "cuda"


def row_tile(tokens, heads, count):
    """Rows of a workgroup, and how many of them take the same keys side by side."""
    per_seq = -(-tokens * heads // count)
    return (32 if per_seq <= 32 else 64), (1 if per_seq <= 64 else 2 if per_seq <= 128 else 4)


def share_of(fq, cache, q, table, lens, new):
    """Key tiles of a share: the number of shares follows from the workspace
    (two places for the partial sums of a row tile each), what they hold from the
    lengths (a row tile counts for four more than its key tiles)."""
    T, heads, dim = q.shape
    rows, subs = row_tile(T, heads, len(lens))
    need = fq.latent_attention_workspace_bytes(cache, q, table)
    target, rest = divmod(need - T * heads * 8, 2 * rows * subs * (4 * dim + 8))
    assert rest == 0
    total = sum(-(-n * heads // (rows * subs)) * (max(-(-x // 64), 1) + 4) for n, x in zip(new, lens))
    return -(-total // target)


def some_cache(fq, g, pages, page, dim, low=-9, high=-5):
    """Codes as a normal distribution leaves them, scales of 2^low to 2^high."""
    c = (64 * torch.randn((pages, page, dim), generator=g)).clamp(-448, 448).to(DEV).to(torch.float8_e4m3fn)
    r = torch.randn((pages, page, 64), generator=g).to(torch.bfloat16).to(DEV)
    s = torch.exp2(torch.randint(low, high + 1, (pages, page), generator=g).float()).to(DEV)
    return fq.LatentCache(c, r, s)


def check_rows(hostc, q, qr, table, lens, starts, scale, got, lse, sequences, heads):
    """The rows of these sequences and heads against 64 bits."""
    for b in sequences:
        rows = slice(starts[b], starts[b + 1])
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        out, l, tol, tol_lse = ref.absorbed(hostc, q[rows], qr[rows], [table[b]], [lens[b]], [0, n], scale, heads)
        close(got[rows][:, heads], out, tol, ("out", b, lens[b]))
        close(lse[rows][:, heads], l, tol_lse, ("lse", b, lens[b]))


def counts(lens, new):
    """Keys that each query token sees."""
    return torch.cat([torch.arange(x - n + 1, x + 1, dtype=torch.float64).clamp_min(0) for x, n in zip(lens, new)])


# heads and new tokens that make row tiles of 32 rows, of 64, and of two and four times 64
SHAPES = [
    # latent, page, heads, sequences, longest, most new tokens, least share
    (512, 64, 16, 150, 3000, 1, 6),
    (256, 16, 5, 140, 9000, 5, 16),         # more than 64 entries of the table in a share
    (512, 64, 40, 100, 3000, 1, 8),
    (256, 16, 64, 90, 6000, 1, 16),         # the same
    (512, 16, 128, 110, 3000, 1, 20),       # the same
    (256, 64, 100, 130, 2000, 1, 16),
    (512, 128, 40, 70, 2500, 8, 24),
    (256, 32, 128, 66, 2000, 3, 16),
]


@pytest.mark.parametrize("dim,page,heads,count,longest,most,least", SHAPES)
def test_absorbed_shares_of_many_tiles(gpu_lib, dim, page, heads, count, longest, most, least):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + page + heads + count)
    lens = torch.randint(0, longest, (count,), generator=g).tolist()
    lens[1], lens[7], lens[count // 2], lens[-2], lens[-1] = 0, 1, longest, 64, 0
    new = torch.randint(0 if most > 1 else 1, most + 1, (count,), generator=g).tolist()
    new[count // 2] = most
    starts = [int(x) for x in starts_of(new)]
    width, pages = -(-longest // page), 2 * (-(-longest // page)) + 3
    # pages are read only: sequences may name the same ones
    table = [torch.randperm(pages, generator=g)[:width].tolist() for _ in range(count)]
    cache = some_cache(fq, g, pages, page, dim)
    q, qr = absorbed_inputs(g, starts[-1], heads, dim)
    t, l, at = i32(table), i32(lens), None if most == 1 else i32(starts)
    assert share_of(fq, cache, q, t, lens, new) >= least
    dq, dr = q.to(DEV), qr.to(DEV)
    got, lse = fq.latent_attention(cache, dq, dr, t, l, at, scale=0.06, return_lse=True)
    again = fq.latent_attention(cache, dq, dr, t, l, at, scale=0.06)
    # queries of zero see every key alike: the sum of exponentials counts the keys
    _, zero = fq.latent_attention(cache, torch.zeros_like(dq), torch.zeros_like(dr), t, l, at, scale=0.06, return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(got, again)
    want = counts(lens, new)[:, None].expand(-1, heads)
    assert torch.equal(torch.exp(zero.double().cpu()).round(), want)
    pick = sorted({0, heads // 3, heads - 1})
    some = [1, 7, count // 2, 64, 65, count - 1] + torch.randperm(count, generator=g)[:9].tolist()
    check_rows(host(cache), q, qr, table, lens, starts, 0.06, got, lse, some, pick)


@pytest.mark.parametrize("heads,chunk,longest", [(16, 512, 2000), (128, 130, 1500)])
def test_absorbed_chunk_among_single_tokens(gpu_lib, heads, chunk, longest):
    """The row tiles are those of the mean, so most of them are nearly empty."""
    fq, g = gpu_lib, torch.Generator().manual_seed(heads)
    lens = torch.randint(1, longest, (32,), generator=g).tolist()
    new = [1] * 32
    new[11], lens[11] = chunk, chunk + 200
    new[12] = 0
    starts = [int(x) for x in starts_of(new)]
    width = -(-longest // 64)
    table = [torch.randperm(70, generator=g)[:width].tolist() for _ in range(32)]
    cache = some_cache(fq, g, 70, 64, 512)
    q, qr = absorbed_inputs(g, starts[-1], heads, 512)
    t, l, at = i32(table), i32(lens), i32(starts)
    assert row_tile(starts[-1], heads, 32) == (64, 4) and share_of(fq, cache, q, t, lens, new) > 8
    got, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), t, l, at, scale=0.06, return_lse=True)
    zero = torch.zeros_like(q).to(DEV), torch.zeros_like(qr).to(DEV)
    _, flat = fq.latent_attention(cache, *zero, t, l, at, scale=0.06, return_lse=True)
    torch.cuda.synchronize()
    want = counts(lens, new)[:, None].expand(-1, heads)
    assert torch.equal(torch.exp(flat.double().cpu()).round(), want)
    check_rows(host(cache), q, qr, table, lens, starts, 0.06, got, lse, range(32), [heads - 2])


# Scores in steps, as powers of two: with a scale of ln 2, a key's score is its
# rotated channel 0 times the query's, to which channel 1 adds noise.  Scales go
# down as scores go up, so that what is summed before a step counts as much as
# what comes behind it.
LN2 = math.log(2.0)


def stepped(fq, g, dim, page, levels, exponents):
    """A cache of one run of pages whose halves of tiles (32 keys) have these
    scores and exponents of scales."""
    n = 32 * len(levels)
    assert n % page == 0
    cache = some_cache(fq, g, n // page, page, dim, 0, 0)
    r = torch.zeros((n, 64))
    r[:, 0] = torch.tensor(levels, dtype=torch.float32).repeat_interleave(32)
    r[:, 1] = torch.randn(n, generator=g)
    s = torch.exp2(torch.tensor(exponents, dtype=torch.float32)).repeat_interleave(32)
    return fq.LatentCache(cache.c, r.to(torch.bfloat16).view(-1, page, 64).to(DEV), s.view(-1, page).to(DEV))


def stepped_queries(g, T, heads, dim):
    """Heads that go up with the steps, down, half as steep, or not at all."""
    qr = torch.zeros((T, heads, 64))
    qr[..., 0] = torch.tensor([1.0, 0.0, -1.0, 0.5])[torch.randint(0, 4, (T, heads), generator=g)]
    qr[:, 0, 0], qr[:, -1, 0] = 1.0, 1.0
    qr[..., 1] = torch.randn((T, heads), generator=g)
    return torch.zeros((T, heads, dim), dtype=torch.bfloat16), qr.to(torch.bfloat16)


@pytest.mark.parametrize("dim", [256, 512])
@pytest.mark.parametrize("heads,new", [(16, 1), (50, 1), (128, 1), (40, 4)])
@pytest.mark.parametrize("levels", [
    [0, 0, 34, 34, 68, 68, 102, 102],        # both waves of a pair
    [0, 0, 0, 37, 0, 37, 0, 74],             # one of them, the other stays behind
    [0, 0, 37, 0, 37, 0, 74, 0],
    [0, -40, 0, 33, 36, 70, 100, 70],        # in turn, from far behind
    [-20, 0, 20, 0, 20, 52, 84, 52],         # in steps that a wave's maximum follows late
])
def test_absorbed_rising_rows(gpu_lib, dim, heads, new, levels):
    """Up to four tiles in one workgroup."""
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + heads)
    cache = stepped(fq, g, dim, 64, levels, [min(50 - x, 60) for x in levels])
    lens, starts, table = [256, 200, 131], [0, new, 2 * new, 3 * new], [[0, 1, 2, 3]] * 3
    q, qr = stepped_queries(g, 3 * new, heads, dim)
    assert fq.latent_attention_workspace_bytes(cache, q, i32(table)) == 0
    got, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), i32(table), i32(lens), None if new == 1 else i32(starts),
                                   scale=LN2, return_lse=True)
    check_rows(host(cache), q, qr, table, lens, starts, LN2, got, lse, range(3), list(range(min(heads, 20))) + [heads - 1])


@pytest.mark.parametrize("dim,heads,new,count", [(512, 16, 1, 300), (256, 16, 1, 300), (512, 50, 1, 150), (256, 64, 1, 150),
                                                 (512, 128, 1, 80), (256, 40, 5, 40)])
def test_absorbed_rising_rows_in_shares(gpu_lib, dim, heads, new, count):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + heads + count)
    tiles = 36
    steps = [0] * (2 * tiles)
    for i, (at, part) in enumerate(((3, 0), (4, 1), (9, 1), (15, 0), (16, 1), (22, 0), (23, 1), (30, 1))):
        for x in range(at, tiles):
            steps[2 * x + part] += 36 if i % 2 == 0 else 33
    # at most 102 above the first, scales within 2^51
    levels = [min(x, 102) for x in steps]
    cache = stepped(fq, g, dim, 64, levels, [51 - x for x in levels])
    lens = torch.randint(1, 64 * tiles + 1, (count,), generator=g).tolist()
    lens[0], lens[3] = 64 * tiles, 64 * tiles - 1
    starts = [new * i for i in range(count + 1)]
    table = [list(range(tiles))] * count
    q, qr = stepped_queries(g, new * count, heads, dim)
    t, l, at = i32(table), i32(lens), None if new == 1 else i32(starts)
    assert share_of(fq, cache, q, t, lens, [new] * count) >= 8
    got, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), t, l, at, scale=LN2, return_lse=True)
    hostc = host(cache)
    some = [0, 3] + torch.randperm(count, generator=g)[:12].tolist()
    check_rows(hostc, q, qr, table, lens, starts, LN2, got, lse, some, [0, 1, 2, 3, heads - 1])


@pytest.mark.parametrize("dim", [256, 512])
@pytest.mark.parametrize("heads", [16, 50, 128])
@pytest.mark.parametrize("levels", [[0, -40, 0, 31, 0, 62, 0, 62], [-40, 0, 31, 0, 62, 0, 62, 0], [0, 0, 31, 31, 31, 31, 31, 31],
                                    [0, -40, 31, 31, 62, 62, 62, 62]])
def test_absorbed_rising_rows_at_the_end_of_the_scales(gpu_lib, dim, heads, levels):
    """Sums over the largest scales stay below the largest float, however scores rise."""
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + heads)
    cache = stepped(fq, g, dim, 64, levels, [60] * len(levels))
    q, qr = stepped_queries(g, 1, heads, dim)
    qr[..., 1] = 0
    got, lse = fq.latent_attention(cache, q.to(DEV), qr.to(DEV), i32([[0, 1, 2, 3]]), i32([256]), scale=LN2, return_lse=True)
    assert bool(got.isfinite().all())
    check_rows(host(cache), q, qr, [[0, 1, 2, 3]], [256], [0, 1], LN2, got, lse, [0], list(range(heads)))


# -------------------------------------------------------------- expanded

def check_expanded(q, k, kr, v, q_at, k_at, scale, got, lse, heads):
    out, l, tol, tol_lse = ref.expanded(q[:, heads], k[:, heads], kr, v[:, heads], q_at, k_at, scale)
    close(got[:, heads], out, tol, "out")
    close(lse[:, heads], l, tol_lse, "lse")


# one set of waves for a row tile from 289 of them on, two below
LONG = [
    # head_dim, heads, new, keys
    (128, 64, [700], [1500]),
    (64, 80, [513], [2100]),
    (128, 40, [300, 1, 700, 130], [1400, 1300, 700, 2000]),
    (64, 64, [1300], None),
    (128, 8, [700], [1500]),
    (64, 5, [300, 1, 700, 130], [1400, 1300, 700, 2000]),
]


@pytest.mark.parametrize("dim,heads,new,keys", LONG)
def test_expanded_over_many_tiles(gpu_lib, dim, heads, new, keys):
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + heads)
    q_at, k_at = [int(x) for x in starts_of(new)], [int(x) for x in starts_of(keys or new)]
    q = torch.randn((q_at[-1], heads, dim + 64), generator=g).to(torch.bfloat16)
    k, v = (torch.randn((k_at[-1], heads, dim), generator=g).to(torch.bfloat16) for _ in range(2))
    kr = torch.randn((k_at[-1], 64), generator=g).to(torch.bfloat16)
    args = [x.to(DEV) for x in (q, k, kr, v)] + [i32(q_at), None if keys is None else i32(k_at)]
    got, lse = fq.latent_prompt_attention(*args, return_lse=True)
    assert torch.equal(got, fq.latent_prompt_attention(*args))
    check_expanded(q, k, kr, v, q_at, k_at, None, got, lse, [0, heads // 2, heads - 1])
    # zeros see every key alike
    args[0] = torch.zeros_like(args[0])
    _, lse = fq.latent_prompt_attention(*args, return_lse=True)
    want = counts(keys or new, new)[:, None].expand(-1, heads)
    assert torch.equal(torch.exp(lse.double().cpu()).round(), want)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [4, 64])
@pytest.mark.parametrize("step", [10, 30])
def test_expanded_rising_rows(gpu_lib, dim, heads, step):
    """Maxima that rise by 2^10 and more every few tiles, in all rows or in some,
    in either half of a tile."""
    fq, g = gpu_lib, torch.Generator().manual_seed(dim + heads + step)
    n, keys = 650, 1300
    level = torch.zeros(keys)
    for at in (70, 160, 225, 400, 470, 700):       # within tiles, in odd and even ones
        if float(level.max()) + step <= 90:
            level[at:] += step
    q = torch.zeros((n, heads, dim + 64))
    q[..., dim] = torch.tensor([1.0, 0.0, -1.0, 0.5])[torch.randint(0, 4, (n, heads), generator=g)]
    q[..., dim + 1] = torch.randn((n, heads), generator=g)
    q[..., :dim] = 0.1 * torch.randn((n, heads, dim), generator=g)
    kr = torch.zeros((keys, 64))
    kr[:, 0], kr[:, 1] = level, torch.randn(keys, generator=g)
    k = torch.randn((keys, heads, dim), generator=g)
    v = torch.randn((keys, heads, dim), generator=g) * torch.exp2(40 - level)[:, None, None]
    q, k, kr, v = (x.to(torch.bfloat16) for x in (q, k, kr, v))
    q_at, k_at = [0, n], [0, keys]
    got, lse = fq.latent_prompt_attention(q.to(DEV), k.to(DEV), kr.to(DEV), v.to(DEV), i32(q_at), i32(k_at), scale=LN2,
                                          return_lse=True)
    check_expanded(q, k, kr, v, q_at, k_at, LN2, got, lse, [0, 1, heads - 1])
