"""Plain definitions of the latent cache's operators and of those on caches'
pages, on the CPU, written from their formulas and apart from the package: what
the GPU tests compare with.  Rotation and quantization are reproduced rounding
by rounding, so stored bytes have to be equal; attention is in 64 bits with the
error that the documented roundings allow."""

import math

import numpy as np
import torch

from kv_reference import decode, encode, fit, rotate, to_bf16

U, E = 2.0 ** -8, 2.0 ** -24      # half a step of BF16 and of fp32
KEPT = 2.0 ** -13                 # of the largest of 8 products: what may be lost of each of the others


def append(cache, c, r, table, lens, starts, q=None, q_out=None, r_out=None, cos=None, sin=None, interleaved=False):
    """``cache``: numpy uint8 c [P, S, L], torch BF16 r [P, S, 64], float32
    scale [P, S], changed in place; c, r, q and outputs torch BF16 on the CPU."""
    codes, rope, scale = cache
    pages, size, _ = codes.shape
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        for i in range(n):
            pos, row = int(lens[b]) - n + i, int(starts[b]) + i
            if pos < 0 or (cos is not None and pos >= cos.shape[0]):
                continue

            def turn(x):
                x = x.float().numpy()
                return to_bf16(x if cos is None else rotate(x, cos[pos], sin[pos], interleaved))

            if q is not None:
                q_out[row] = turn(q[row])
            key = turn(r[row][None])[0]
            if r_out is not None:
                r_out[row] = key
            pg = int(table[b][pos // size]) if pos // size < len(table[b]) else -1
            if not 0 <= pg < pages:
                continue
            x = c[row].float().numpy()
            s = fit(np.abs(x).max())
            scale[pg, pos % size] = s
            codes[pg, pos % size] = encode(x.astype(np.float64) / s)
            rope[pg, pos % size] = key


def _bound(s, ds, w, z, v, N, split):
    """Elementwise errors of softmax(s) v.  ``w`` = exp(s - max), ``z`` its sum.

    Relative to a weight, twice (numerator and denominator): the score's error
    ds, exp2 and its argument (5 + 3 |s - max|) e, sums N e each and as much for
    rescaling.  ``split``: the weights are two e4m3 terms, rounded by (2^-4)^2 of
    themselves and by 2^-22 of the largest of their 32 neighbours, and of eight
    products each of the seven others loses up to 2^-13 of the largest, and again
    for the second term, 2^-4 as large.  Else they are BF16."""
    far = torch.where(w > 0, -torch.log(w.clamp_min(1e-300)), torch.zeros_like(w)).amax(-1, keepdim=True)
    a = w @ v.abs() / z
    o = w @ v / z
    rel = 2 * (ds + (5 + 3 * far) * E + 2 * N * E)
    tol = U * o.abs() + (U * (1 + U) + rel) * a + 1e-30
    if split:
        pad = -w.shape[1] % 32
        wp = torch.nn.functional.pad(w, (0, pad))
        vp = torch.nn.functional.pad(v.abs(), (0, 0, 0, pad))
        # weights times scales, against codes: the scale is a factor of either, as a power of two
        top = wp.view(w.shape[0], -1, 32)
        for g in range(top.shape[1]):
            block = vp[32 * g:32 * g + 32]
            size = block.amax(1)                                   # of a token's values
            # w s <= w |c|max / (smallest nonzero code ...): bounded by the largest w * value / 1 code step,
            # values being at most 448 codes and at least 224 codes at their largest
            most = (top[:, g] * (size / 224.0)).amax(1, keepdim=True)
            tol = tol + 2.0 ** -22 * most * torch.where(size > 0, 448.0, 0.0).sum() / z
        for g in range(0, wp.shape[1], 8):
            prod = wp[:, g:g + 8, None] * vp[None, g:g + 8]
            tol = tol + 7 * KEPT * (1 + 2.0 ** -4) * prod.amax(1) / z
    return o, a, tol, rel, far


def _lse(m, z, rel):
    return (m + z.log())[:, 0], (rel + 8 * E * (m.abs() + z.log().abs() + 1))[:, 0]


def absorbed(cache, q, q_rope, table, lens, starts, scale, heads=None):
    """float64 out [T, H, L], lse [T, H] and the errors allowed for each; with
    ``heads``, of these heads alone."""
    codes, rope, scales = cache
    pages, size, dim = codes.shape
    T, H = q.shape[:2]
    heads = list(range(H)) if heads is None else heads
    out, lse = torch.zeros(T, len(heads), dim, dtype=torch.float64), torch.full((T, len(heads)), -math.inf,
                                                                               dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(lens)):
        n, L = int(starts[b + 1] - starts[b]), int(lens[b])
        seen = [p for p in range(max(L, 0)) if p // size < len(table[b]) and 0 <= int(table[b][p // size]) < pages]
        if not seen or n == 0:
            continue
        pg = np.array([int(table[b][p // size]) for p in seen])
        sl = np.array([p % size for p in seen])
        at = np.array(seen)
        # at their places in the sequence, zeros between, so that groups of eight and of 32 are the kernel's
        c = torch.zeros(max(L, 0), dim, dtype=torch.float64)
        r = torch.zeros(max(L, 0), 64, dtype=torch.float64)
        c[at] = torch.from_numpy(decode(codes[pg, sl]) * scales[pg, sl][:, None].astype(np.float64))
        r[at] = rope[torch.from_numpy(pg), torch.from_numpy(sl)].double()
        hidden = torch.ones(max(L, 0), dtype=torch.bool)
        hidden[at] = False
        for i in range(n):
            pos, row = L - n + i, int(starts[b]) + i
            if pos < 0:
                continue
            mask = hidden[:pos + 1]
            if bool(mask.all()):
                continue
            x, y = q[row, heads].double(), q_rope[row, heads].double()
            k, kr = c[:pos + 1], r[:pos + 1]
            s = (x @ k.T + y @ kr.T) * scale
            lost = torch.stack([(x[h].abs() * k.abs()).view(pos + 1, -1, 8).amax(2).sum(1) for h in range(len(heads))])
            every = x.abs() @ k.abs().T + y.abs() @ kr.abs().T
            # queries as two terms: all but 2^-22 of the row's largest value
            rest = 2.0 ** -22 * x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None]
            ds = abs(scale) * (7 * KEPT * (1 + 2.0 ** -4) * lost + (dim + 68) * E * every + rest) + 4 * E * s.abs()
            s, ds = s.masked_fill(mask, -math.inf), ds.masked_fill(mask, 0).amax(1, keepdim=True)
            m = s.amax(1, keepdim=True)
            w = torch.exp(s - m)
            z = w.sum(1, keepdim=True)
            o, _, t, rel, _ = _bound(s, ds, w, z, k, pos + 1, True)
            out[row], tol[row] = o, t
            lse[row], tol_lse[row] = _lse(m, z, rel)
    return out, lse, tol, tol_lse


def expanded(q, k, k_rope, v, q_at, k_at, scale=None):
    """float64 out [T, H, D], lse [T, H] and the errors allowed for each."""
    T, H, D = q.shape[0], v.shape[1], v.shape[2]
    scale = (D + 64) ** -0.5 if scale is None else scale
    out, lse = torch.zeros(T, H, D, dtype=torch.float64), torch.full((T, H), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(q_at) - 1):
        rows, keys = slice(int(q_at[b]), int(q_at[b + 1])), slice(int(k_at[b]), int(k_at[b + 1]))
        n, N = rows.stop - rows.start, keys.stop - keys.start
        if n <= 0 or N <= 0:
            continue
        hidden = torch.arange(N)[None] > (N - n + torch.arange(n))[:, None]
        some = ~hidden.all(1)
        for h in range(H):
            x = q[rows, h].double()[some]
            key = torch.cat((k[keys, h], k_rope[keys]), 1).double()
            s = x @ key.T * scale
            ds = (D + 68) * E * (x.abs() @ key.abs().T) * abs(scale) + 4 * E * s.abs()
            s, ds = s.masked_fill(hidden[some], -math.inf), ds.masked_fill(hidden[some], 0).amax(1, keepdim=True)
            m = s.amax(1, keepdim=True)
            w = torch.exp(s - m)
            z = w.sum(1, keepdim=True)
            o, _, t, rel, _ = _bound(s, ds, w, z, v[keys, h].double(), N, False)
            at = torch.arange(rows.start, rows.stop)[some]
            out[at, h], tol[at, h] = o, t
            lse[at, h], tol_lse[at, h] = _lse(m, z, rel)
    return out, lse, tol, tol_lse


def fork(buffers, table, lens, parents, children, fresh, size):
    """``buffers``: numpy arrays [P, ...]; all changed in place."""
    pages = buffers[0].shape[0]
    was, was_len = table.copy(), lens.copy()
    for a, b, to in zip(parents, children, fresh):
        if not (0 <= a < len(lens) and 0 <= b < len(lens)) or a == b:
            continue
        n = max(int(was_len[a]), 0)
        whole = min(n // size, table.shape[1])
        table[b] = -1
        table[b, :whole] = was[a, :whole]
        lens[b] = n
        if n % size and whole < table.shape[1] and 0 <= was[a, whole] < pages and 0 <= to < pages:
            table[b, whole] = to
            for x in buffers:
                x[to] = x[was[a, whole]]


def compact(buffers, table, lens, size):
    """The renamed table and the number of pages in use; buffers are changed in place."""
    pages = buffers[0].shape[0]
    live = np.zeros(table.shape, dtype=bool)
    for b in range(len(lens)):
        live[b, :min(-(-max(int(lens[b]), 0) // size), table.shape[1])] = True
    live &= (table >= 0) & (table < pages)
    used = sorted(set(table[live].tolist()))
    n = len(used)
    holes = [p for p in range(n) if p not in set(used)]
    movers = [p for p in used if p >= n]
    name = {p: p for p in used}
    for to, p in zip(holes, movers):
        name[p] = to
        for x in buffers:
            x[to] = x[p]
    out = np.full(table.shape, -1, dtype=np.int32)
    for at in np.argwhere(live):
        out[tuple(at)] = name[int(table[tuple(at)])]
    return out, n
