"""Plain definitions of the key/value cache's operators, on the CPU, written
from their formulas and apart from the package: what the GPU tests compare
with.  Rotation and quantization are reproduced rounding by rounding (each
fp32 product and sum is one numpy operation, codes by the format's
definition), so stored bytes have to be equal; attention is in 64 bits."""

import math

import numpy as np
import torch

EPS = np.float32(1e-10)


def decode(codes):
    """uint8 codes -> float64 values."""
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def encode(x):
    """float64 values within +-448 -> the nearest code, ties to even."""
    mag = np.minimum(np.abs(x), 448.0)
    e = np.maximum(np.floor(np.log2(np.maximum(mag, 2.0 ** -30))), -6).astype(np.int64)
    n = np.rint(mag / np.exp2((e - 3).astype(np.float64))).astype(np.int64)   # 0 .. 16 steps
    code = np.where(n == 16, (e + 8) * 8, np.where(n >= 8, (e + 7) * 8 + n - 8, n))
    return np.where(np.signbit(x), code + 128, code).astype(np.uint8)


def fit(amax):
    """The smallest power of two s with 448 s >= amax."""
    a = float(max(np.float32(amax), EPS))
    e = math.ceil(math.log2(a / 448.0)) - 1
    while 448.0 * 2.0 ** e < a:
        e += 1
    return 2.0 ** e


def rotate(x, cos, sin, interleaved):
    """float32 [heads, dim] rotated by one row of cos and sin (float32)."""
    half = cos.shape[0]
    y = x.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    xa, xb = x[:, a], x[:, b]
    y[:, a] = xa * cos - xb * sin
    y[:, b] = xb * cos + xa * sin
    return y


def to_bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16)


def append(cache, k, v, table, lens, starts, q=None, q_out=None, cos=None, sin=None, interleaved=False):
    """``cache``: numpy uint8 k [P, h, S, D], v [P, h, D, S], float32 scales
    [P, h], changed in place; k, v, q, q_out: torch BF16 on the CPU."""
    kc, vc, ks, vs = cache
    pages, heads, size, dim = kc.shape
    kf, vf = k.float().numpy(), v.float().numpy()
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        first = int(lens[b]) - n
        by_page = {}
        for i in range(n):
            pos, row = first + i, int(starts[b]) + i
            if pos < 0 or (cos is not None and cos.shape[1] and pos >= cos.shape[0]):
                continue
            turn = cos is not None and cos.shape[1] > 0
            if q is not None:
                x = q[row].float().numpy()
                q_out[row] = to_bf16(rotate(x, cos[pos], sin[pos], interleaved) if turn else x)
            by_page.setdefault(pos // size, []).append(
                (pos % size, rotate(kf[row], cos[pos], sin[pos], interleaved) if turn else kf[row], vf[row]))
        for j, toks in by_page.items():
            pg = int(table[b][j]) if j < len(table[b]) else -1
            if not 0 <= pg < pages:
                continue
            held = toks[0][0]
            for h in range(heads):
                for codes, scale, which in ((kc[pg, h], ks, 1), (vc[pg, h].T, vs, 2)):
                    s = fit(max(np.abs(t[which][h]).max() for t in toks))
                    if held:
                        was = float(scale[pg, h])
                        s = max(s, was)
                        if s != was:
                            codes[:held] = encode(decode(codes[:held]) * (was / s))
                    scale[pg, h] = s
                    for t in toks:
                        codes[t[0]] = encode(t[which][h].astype(np.float64) / s)


def attention(cache, q, table, lens, starts, scale=None, window=0):
    """float64 out [T, H, D], lse [T, H], and the elementwise error that the
    documented roundings allow for each.

    With unit roundoffs u = 2^-8 (BF16) and e = 2^-24 (fp32), A = sum w |v| /
    sum w and N the keys seen:
      scores: products of BF16 values are exact in fp32, sums of D terms and
        the two multiplications by scales err by (D + 4) e sum |q k| scale =: ds,
        the exponent's argument by another 2 e |s|;
      weights: exp2 and its argument (3 + 2 |s log2 e|) e more, another
        4 |log2 v_scale| e where that scale enters as a logarithm (its own
        rounding, the sum's and the product's), then u by the rounding to BF16;
      sums: N e each for numerator and denominator;
      output: u |out|.
    The rescaling of sums by exp2 at each new maximum adds at most 2 e per key
    tile, counted as N e.  Errors relative to a weight act twice (numerator
    and denominator)."""
    kc, vc, ks, vs = cache
    pages, heads, size, dim = kc.shape
    T, H = q.shape[0], q.shape[1]
    group = H // heads
    scale = dim ** -0.5 if scale is None else scale
    u, e = 2.0 ** -8, 2.0 ** -24
    out, lse = torch.zeros(T, H, dim, dtype=torch.float64), torch.full((T, H), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(lens)):
        n, L = int(starts[b + 1] - starts[b]), int(lens[b])
        seen = [p for p in range(max(L, 0)) if p // size < len(table[b]) and 0 <= int(table[b][p // size]) < pages]
        for i in range(n):
            pos, row = L - n + i, int(starts[b]) + i
            keys = [p for p in seen if p <= pos and (window == 0 or p > pos - window)]
            if not keys:
                continue
            pg = np.array([int(table[b][p // size]) for p in keys])
            sl = np.array([p % size for p in keys])
            for h in range(heads):
                k = torch.from_numpy(decode(kc[pg, h, sl])) * torch.from_numpy(ks[pg, h].astype(np.float64))[:, None]
                v = torch.from_numpy(decode(vc[pg, h][np.arange(len(pg)), :, sl])) * \
                    torch.from_numpy(vs[pg, h].astype(np.float64))[:, None]
                x = q[row, h * group:(h + 1) * group].double()
                s = x @ k.T * scale
                ds = ((dim + 4) * e * (x.abs() @ k.abs().T) * abs(scale) + 4 * e * s.abs()).amax(1, keepdim=True)
                m = s.amax(1, keepdim=True)
                w = torch.exp(s - m)
                z = w.sum(1, keepdim=True)
                o, a = w @ v / z, w @ v.abs() / z
                N = len(keys)
                lv = float(np.abs(np.log2(vs[pg, h].astype(np.float64))).max())
                rel = 2 * (ds + (5 + 3 * (m - s).amax(1, keepdim=True) + 4 * lv) * e + 2 * N * e)
                out[row, h * group:(h + 1) * group] = o
                tol[row, h * group:(h + 1) * group] = u * o.abs() + (u * (1 + u) + rel) * a + 1e-30
                lse[row, h * group:(h + 1) * group] = (m + z.log())[:, 0]
                tol_lse[row, h * group:(h + 1) * group] = (rel + 8 * e * (m.abs() + z.log() + 1))[:, 0]
    return out, lse, tol, tol_lse


def attention_of_long(cache, q, table, lens, starts, scale=None, window=0):
    """The same as ``attention``, a sequence and head at a time, for long
    sequences whose pages are all pages and that hold all of their queries."""
    kc, vc, ks, vs = cache
    heads, size, dim = kc.shape[1:]
    group = q.shape[1] // heads
    scale = dim ** -0.5 if scale is None else scale
    u, e = 2.0 ** -8, 2.0 ** -24
    out, lse = torch.zeros(q.shape, dtype=torch.float64), torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(lens)):
        n, L, rows = int(starts[b + 1] - starts[b]), int(lens[b]), slice(int(starts[b]), int(starts[b + 1]))
        pg = np.array(table[b][:-(-L // size)])
        pos, key = torch.arange(L - n, L)[:, None], torch.arange(L)
        hidden = ((key > pos) | ((key <= pos - window) if window else (key < 0)))[:, None]
        N = (~hidden).sum(2, keepdim=True).double()
        for h in range(heads):
            at = slice(h * group, (h + 1) * group)
            k = torch.from_numpy((decode(kc[pg, h]) * ks[pg, h, None, None].astype(np.float64)).reshape(-1, dim)[:L])
            v = torch.from_numpy((decode(vc[pg, h]) * vs[pg, h, None, None].astype(np.float64)).transpose(0, 2, 1)
                                 .reshape(-1, dim)[:L])
            lv = torch.from_numpy(np.abs(np.log2(vs[pg, h].astype(np.float64))).repeat(size)[:L])
            lv = lv.expand(n, 1, L).masked_fill(hidden, 0).amax(2, keepdim=True)
            x = q[rows, at].double().reshape(n * group, dim)
            s = (x @ k.T * scale).view(n, group, L)
            ds = ((dim + 4) * e * (x.abs() @ k.abs().T).view(n, group, L) * abs(scale) + 4 * e * s.abs())
            ds = ds.masked_fill(hidden, 0).amax(2, keepdim=True)
            s = s.masked_fill(hidden, -math.inf)
            m = s.amax(2, keepdim=True)
            far = (m - s).masked_fill(hidden, 0).amax(2, keepdim=True)
            w = torch.exp(s - m)
            z = w.sum(2, keepdim=True)
            w = w.view(n * group, L)
            o, a = (w @ v).view(n, group, dim) / z, (w @ v.abs()).view(n, group, dim) / z
            rel = 2 * (ds + (5 + 3 * far + 4 * lv) * e + 2 * N * e)
            out[rows, at] = o
            tol[rows, at] = u * o.abs() + (u * (1 + u) + rel) * a + 1e-30
            lse[rows, at] = (m + z.log())[..., 0]
            tol_lse[rows, at] = (rel + 8 * e * (m.abs() + z.log() + 1))[..., 0]
    return out, lse, tol, tol_lse
