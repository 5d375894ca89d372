"""Attention over latents where one workgroup walks many key tiles, and rows'
maxima rise far on the way, so that sums are scaled."""

import math

import pytest
import torch

import latent_reference as ref
from test_kv_gpu import i32
from test_latent_gpu import close, host

pytestmark = pytest.mark.gpu

DEV = "cuda"


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
