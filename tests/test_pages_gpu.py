"""Forks and compaction of caches' pages on the GPU against the plain
definitions of latent_reference.py: every byte of every page, the tables and
the lengths equal."""

import numpy as np
import pytest
import torch

import latent_reference as ref
from test_kv_gpu import i32

pytestmark = pytest.mark.gpu

DEV = "cuda"


def caches_of(fq, g, kinds, pages, size):
    """Caches with random bytes, (kind, heads or latent, dim) each."""
    def fill(t):
        b = torch.randint(0, 256, (t.numel() * t.element_size(),), generator=g, dtype=torch.uint8)
        t.view(torch.uint8).view(-1).copy_(b.to(DEV))

    out = []
    for kind, n, dim in kinds:
        c = fq.KvCache.empty(pages, n, dim, size) if kind == "kv" else fq.LatentCache.empty(pages, n, size)
        for t in ((c.k, c.v, c.k_scale, c.v_scale) if kind == "kv" else (c.c, c.r, c.scale)):
            fill(t)
        out.append(c)
    return out


def buffers(caches):
    """numpy bytes of every buffer, [pages, bytes]."""
    return [t.view(torch.uint8).reshape(t.shape[0], -1).cpu().numpy().copy()
            for c in caches for t in ((c.k, c.v, c.k_scale, c.v_scale) if hasattr(c, "k") else (c.c, c.r, c.scale))]


def same(caches, want):
    for i, (a, b) in enumerate(zip(buffers(caches), want)):
        assert np.array_equal(a, b), (i, np.argwhere((a != b).any(1))[:4].tolist())


KINDS = [
    [("kv", 8, 128)],
    [("latent", 512, 0)] * 3,
    [("kv", 1, 64), ("latent", 256, 0), ("kv", 5, 192)],
    [("kv", 2, 256)] * 2,
]


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("size", [16, 64, 256])
def test_fork(gpu_lib, kinds, size):
    fq, g = gpu_lib, torch.Generator().manual_seed(size + len(kinds))
    pages, width = 40, 5
    lens = [3 * size, 2 * size + 1, size - 1, 0, 7, 9, 11, 4 * size + size // 2, -3, 5 * size]
    table = np.random.default_rng(size).permutation(pages)[:24].tolist()
    rows = np.full((10, width), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        if b in (0, 1, 2, 7, 8, 9):
            for j in range(min(-(-max(n, 0) // size), width)):
                rows[b, j] = table.pop() if table else 0
    rows[9, 2] = 4000                                  # no page: handed on as it is
    free = [p for p in range(pages) if p not in rows]
    parents, children = [0, 1, 1, 2, 7, 8], [3, 4, 5, 6, 10, 11]
    lens, rows = lens + [5, 6], np.vstack([rows, rows[:2]])
    caches = caches_of(fq, g, kinds, pages, size)
    want, wt, wl = buffers(caches), rows.copy(), np.array(lens)
    fresh = free[:len(parents)]
    ref.fork(want, wt, wl, parents, children, fresh, size)
    t, l = i32(rows.tolist()), i32(lens)
    fq.cache_fork(caches, t, l, i32(parents), i32(children), i32(fresh))
    same(caches, want)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(l.cpu().numpy(), wl)


def test_fork_of_what_is_none(gpu_lib):
    """Rows that are none, pages that are none, a parent whose last page is none,
    tables with spare columns."""
    fq, g = gpu_lib, torch.Generator().manual_seed(1)
    caches = caches_of(fq, g, [("latent", 256, 0)], 12, 16)
    rows = np.array([[0, 1, 2, -1], [3, 99, -1, -1], [4, 5, -1, -1]] + [[7, 7, 7, 7]] * 6, dtype=np.int32)
    lens = [40, 20, 17, 1, 1, 1, 1, 1, 1]
    parents, children = [0, 1, 2, 0, -1, 50, 0, 3], [3, 4, 5, 6, 7, 8, 60, 3]
    fresh = [8, 9, 1 << 30, -5, 10, 11, 11, 11]
    want, wt, wl = buffers(caches), rows.copy(), np.array(lens)
    ref.fork(want, wt, wl, parents, children, fresh, 16)
    big = torch.full((9, 10), 77, dtype=torch.int32, device=DEV)
    big[:, :4] = i32(rows.tolist())
    l = i32(lens)
    fq.cache_fork(caches[0], big[:, :4], l, i32(parents), i32(children), i32(fresh))
    same(caches, want)
    assert np.array_equal(big[:, :4].cpu().numpy(), wt) and np.array_equal(l.cpu().numpy(), wl)
    assert bool((big[:, 4:] == 77).all())


def random_rows(rng, count, width, size, pages, shared, ended):
    lens = rng.integers(1, width * size + 1, count)
    lens[rng.random(count) < ended] = 0
    rows = np.full((count, width), -1, dtype=np.int32)
    order = rng.permutation(pages).tolist()
    for b in range(count):
        for j in range(-(-int(lens[b]) // size)):
            if b and j < width // 2 and rng.random() < shared and rows[b - 1, j] >= 0:
                rows[b, j] = rows[b - 1, j]
            elif order:
                rows[b, j] = order.pop()
    return rows, lens


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("count,width,size,pages,ended", [
    (1, 1, 64, 1, 0.0), (5, 4, 16, 33, 0.3), (70, 3, 32, 300, 0.6), (9, 40, 16, 400, 0.5), (4, 3, 64, 64, 1.0),
])
def test_compact(gpu_lib, kinds, count, width, size, pages, ended):
    fq, g = gpu_lib, torch.Generator().manual_seed(count)
    rng = np.random.default_rng(count + pages)
    rows, lens = random_rows(rng, count, width, size, pages, 0.5, ended)
    caches = caches_of(fq, g, kinds, pages, size)
    want = buffers(caches)
    table, n = ref.compact(want, rows, lens, size)
    t, l = i32(rows.tolist()), i32(lens.tolist())
    got, used = fq.cache_compact(caches, t, l)
    same(caches, want)
    assert int(used) == n and np.array_equal(got.cpu().numpy(), table)
    assert np.array_equal(t.cpu().numpy(), rows)
    # what is compact stays as it is; in place
    again, used = fq.cache_compact(caches, got, l, table_out=got)
    same(caches, want)
    assert again is got and int(used) == n and np.array_equal(got.cpu().numpy(), table)


def test_compact_of_what_is_none(gpu_lib):
    fq, g = gpu_lib, torch.Generator().manual_seed(2)
    rows = np.array([[31, 1 << 30, 30], [-1, 29, 31], [5, 6, 7], [-2, -3, 28]], dtype=np.int32)
    lens = np.array([48, 1000, -7, 33])
    caches = caches_of(fq, g, [("kv", 3, 64)], 32, 16)
    want = buffers(caches)
    table, n = ref.compact(want, rows, lens, 16)
    big = torch.full((4, 7), 9, dtype=torch.int32, device=DEV)
    got, used = fq.cache_compact(caches, i32(rows.tolist()), i32(lens.tolist()), table_out=big[:, 2:5])
    same(caches, want)
    assert int(used) == n == 4 and np.array_equal(got.cpu().numpy(), table)
    assert bool((big[:, :2] == 9).all()) and bool((big[:, 5:] == 9).all())
    # no sequence at all
    _, used = fq.cache_compact(caches, big[:0, :3], i32([]))
    assert int(used) == 0
    same(caches, want)


def test_compact_of_many_pages(gpu_lib):
    """The largest number of pages, most of them empty, in use at both ends."""
    fq = gpu_lib
    pages = fq.pages.MAX_COMPACT_PAGES
    cache = fq.KvCache.empty(pages, 1, 64, 16)
    at = np.concatenate([np.arange(0, 3000, 3), np.arange(pages - 3500, pages, 7)])
    np.random.default_rng(0).shuffle(at)
    rows = at.reshape(10, -1).astype(np.int32)
    cache.k_scale[:, 0] = torch.arange(pages, dtype=torch.float32, device=DEV)
    got, used = fq.cache_compact(cache, i32(rows.tolist()), i32([16 * rows.shape[1]] * 10))
    n = len(at)
    assert int(used) == n
    name = got.cpu().numpy()
    assert sorted(name.ravel().tolist()) == list(range(n))
    # each page's contents have gone with its name
    assert torch.equal(cache.k_scale[got.long().view(-1), 0].cpu(), torch.from_numpy(rows.ravel()).float())
    movers = sorted(p for p in at.tolist() if p >= n)
    order = {int(a): int(b) for a, b in zip(rows.ravel(), name.ravel())}
    assert [order[p] for p in movers] == sorted(order[p] for p in movers)
    with pytest.raises(ValueError):
        fq.cache_compact(fq.KvCache.empty(pages + 1, 1, 64, 16), i32([[0]]), i32([1]))


def test_many_layers(gpu_lib):
    """More buffers than a launch's arguments hold."""
    fq, g = gpu_lib, torch.Generator().manual_seed(3)
    caches = caches_of(fq, g, [("kv", 1, 64)] * 70, 12, 16)
    rows, lens = np.array([[11, 3, -1], [-1, -1, -1], [11, 9, 10]], dtype=np.int32), np.array([30, 0, 48])
    want, wt, wl = buffers(caches), rows.copy(), lens.copy()
    ref.fork(want, wt, wl, [0], [1], [5], 16)
    t, l = i32(rows.tolist()), i32(lens.tolist())
    fq.cache_fork(caches, t, l, i32([0]), i32([1]), i32([5]))
    same(caches, want)
    table, n = ref.compact(want, wt, wl, 16)
    got, used = fq.cache_compact(caches, t, l)
    same(caches, want)
    assert int(used) == n and np.array_equal(got.cpu().numpy(), table)


@pytest.mark.parametrize("kind", ["kv", "latent"])
def test_samples_of_a_prompt(gpu_lib, kind):
    """A prompt, four samples that go their own ways, two that end, the rest moved
    to the front: attention over what is left is what it was.  Captured in a graph
    and replayed."""
    fq, g = gpu_lib, torch.Generator().manual_seed(12)
    H, D, L, size, prompt = 4, 128, 512, 16, 41
    cache = fq.KvCache.empty(40, 2, D, size) if kind == "kv" else fq.LatentCache.empty(40, L, size)
    rows = torch.full((4, 6), -1, dtype=torch.int32, device=DEV)
    rows[0, :3] = i32([39, 20, 31])
    lens = i32([prompt, 0, 0, 0])

    def x(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)

    def append(n, table, lens, starts=None):
        if kind == "kv":
            fq.kv_append(cache, x(n, 2, D), x(n, 2, D), table, lens, starts)
        else:
            fq.latent_append(cache, x(n, L), x(n, 64), table, lens, starts)

    q, qr = (x(4, H, D), None) if kind == "kv" else (x(4, H, L), x(4, H, 64))

    def attend(at, table, lens):
        if kind == "kv":
            return fq.kv_attention(cache, q[at], table, lens)
        return fq.latent_attention(cache, q[at], qr[at], table, lens, scale=0.06)

    append(prompt, rows[:1], lens[:1], i32([0, prompt]))
    before = attend([0, 0], rows[[0, 0]], lens[[0, 0]])[0]
    parents, children, fresh = i32([0, 0, 0]), i32([1, 2, 3]), i32([5, 38, 0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fq.cache_fork(cache, rows, lens, parents, children, fresh)
    graph.replay()
    assert lens.tolist() == [prompt] * 4
    assert rows[:, :2].tolist() == [[39, 20]] * 4 and rows[:, 2].tolist() == [31, 5, 38, 0]
    after = attend([0, 0, 0, 0], rows, lens)
    assert all(torch.equal(after[i], after[0]) for i in range(4))
    assert torch.equal(attend([0, 0], rows[[0, 0]], lens[[0, 0]])[0], before)
    rows[1:, 3] = i32([11, 12, 13])
    rows[0, 3] = 14
    for _ in range(9):                       # over the page's end
        lens += 1
        append(4, rows, lens)
    lens[0] = lens[2] = 0                    # two end
    was = attend([1, 3], rows[[1, 3]], lens[[1, 3]])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        table, used = fq.cache_compact(cache, rows, lens)
    graph.replay()
    torch.cuda.synchronize()
    assert int(used) == 6                    # two shared, two of each
    assert int(table.max()) == 5 and bool((table[[0, 2]] == -1).all())
    assert torch.equal(attend([1, 3], table[[1, 3]], lens[[1, 3]]), was)
    # replayed with nothing left to move but the table's old names: pages keep what they hold
    rows.copy_(table)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert int(used) == 6 and torch.equal(table, rows)
        assert torch.equal(attend([1, 3], table[[1, 3]], lens[[1, 3]]), was)
