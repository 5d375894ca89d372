"""The operators of the blockwise e4m3 key/value cache, as cases to measure.

A case is one call of ``kv_append`` (rotate, quantize and store new tokens in
a paged cache) or of ``kv_attention`` (attention of queries over that cache).
``run`` computes it in elementary torch operations where ``own`` is false and
through the package where it is true.

The cache, for P pages of ``page`` tokens:
  k        e4m3  [P, kv_heads, page, dim]    a token's values are contiguous
  v        e4m3  [P, kv_heads, dim, page]    a channel's tokens are contiguous
  k_scale, v_scale  fp32 [P, kv_heads]       one scale per page and head

Lengths, new tokens and page counts follow from the case alone; values, page
order and what the unused pages hold follow from the seed.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-10          # floor of a block's largest magnitude
GOLDEN = 0.6180339887498949


def listed():
    """The cases.  Heads 32/8 and 32/4 of 128 are the attention shapes beside
    the dense and the mixture-of-experts weight sets of this repository."""
    base = {"q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "rot": 128,
            "interleaved": False, "ragged": False, "window": 0}

    def case(name, op, batch, longest, new, **more):
        return {"name": name, "op": op, "batch": batch, "longest": longest, "new": new, **base, **more}

    return [
        # the next token of one sequence: nothing but latency
        case("append_one", "append", 1, 1000, 1),
        # one step of a rollout batch: 256 sequences of mixed lengths, a token each
        case("append_step_256", "append", 256, 4096, 1, ragged=True),
        # drafted tokens in small pages, adjacent-pair rotation of half the channels, odd counts
        case("append_drafts_odd", "append", 37, 777, 9, ragged=True, q_heads=15, kv_heads=5, dim=64,
             page=16, rot=32, interleaved=True),
        # prompts of mixed lengths entering an empty cache
        case("append_prompts", "append", 8, 4096, 4096, ragged=True),
        # the next token of one short and one very long sequence
        case("decode_one_short", "attention", 1, 777, 1),
        case("decode_one_long", "attention", 1, 131071, 1),
        # one step of a rollout batch with mixed response lengths
        case("decode_step_128", "attention", 128, 16384, 1, ragged=True),
        # every query head with its own key head, small pages, 64 channels
        case("decode_unshared_d64", "attention", 64, 4097, 1, ragged=True, q_heads=16, kv_heads=16,
             dim=64, page=16, rot=64),
        # a sliding window over long sequences, wide heads, pages of 128
        case("decode_window_d256", "attention", 48, 32768, 1, ragged=True, q_heads=16, kv_heads=4,
             dim=256, page=128, rot=256, window=4096),
        # up to eight drafted tokens a sequence, checked in one call
        case("verify_drafts", "attention", 32, 8192, 8, ragged=True, kv_heads=4),
        # a chunk of a long prompt over what is cached of it already
        case("chunk_over_long", "attention", 1, 32768 + 500, 500),
        # whole prompts against their own keys
        case("prompts", "attention", 2, 4096, 4096),
    ]


def draw(rng):
    """One more case of the same ranges: batches of 1 to 256 sequences of 1 to
    131072 tokens, 1 to all of them new, at most what the largest case costs."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["append", "attention", "attention"])
    dim = rng.choice([64, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16]) if kv_heads <= 8 else rng.choice([1, 2, 4])
    batch = log_int(1, 256)
    longest = log_int(1, 131072)
    kind = rng.choice(["step", "step", "drafts", "chunk"])
    new = 1 if kind == "step" else min(longest, log_int(2, 16 if kind == "drafts" else 4096))
    token = 2 * kv_heads * dim
    # no more than the largest listed case: cached bytes, rows and products
    while batch > 1 and batch * longest * token > 2.0e9:
        batch = max(1, batch // 2)
    longest = max(1, min(longest, int(1.0e9 / token)))
    new = min(new, longest)
    heads = kv_heads * group
    while new > 1 and batch * new * heads * dim > 3.0e7:
        new = max(1, new // 2)
    while new > 1 and 4.0 * batch * new * longest * heads * dim > 2.0e11:
        new = max(1, new // 2)
    rot = rng.choice([dim, dim, dim // 2, 0])
    return {"op": op, "batch": batch, "longest": longest, "new": new, "q_heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128, 256]), "rot": rot,
            "interleaved": rng.choice([False, True]), "ragged": rng.choice([False, True, True]),
            "window": rng.choice([0, 0, log_int(1, 8192)]) if op == "attention" else 0}


def _lengths(case):
    """Tokens of each sequence after the call, and how many of them are new."""
    n, longest, new = case["batch"], case["longest"], case["new"]
    if not case["ragged"]:
        return [longest] * n, [new] * n
    lens = [longest] + [1 + int((longest - 1) * ((b * GOLDEN) % 1.0)) for b in range(1, n)]
    if new == longest:
        return lens, lens
    return lens, [min(lens[b], 1 + (new - 1 + 5 * b) % new) for b in range(n)]


def _fit(amax):
    """The smallest power of two that brings ``amax`` within e4m3: 448 is
    0.875 * 2^9."""
    m, e = torch.frexp(amax.clamp_min(EPS))
    return ((e + (127 - 9) + (m > 0.875).to(e.dtype)) << 23).view(torch.float32)


def _quantize_pages(x):
    """Codes [n, heads, ., .] and scales [n, heads] of pages of values."""
    s = _fit(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, H, KV, D, page = (case[k] for k in ("batch", "q_heads", "kv_heads", "dim", "page"))
    lens, new = _lengths(case)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3                       # three pages belong to nobody
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu().tolist()
    width = max(counts)
    rows, at = [], 0
    for c in counts:
        rows.append(order[at:at + c] + [-1] * (width - c))
        at += c
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    # keys with some strong channels, values without
    strong = 1 + 3 * (torch.rand((1, KV, 1, D), generator=g, device=dev) < 0.05).float()
    k, ks, v, vs = [], [], [], []
    some = max(1, (1 << 26) // (KV * page * D))   # pages made at a time
    for p in range(0, pages, some):
        n = min(some, pages - p)
        for codes, scales, x in ((k, ks, torch.randn((n, KV, page, D), generator=g, device=dev) * strong),
                                 (v, vs, torch.randn((n, KV, D, page), generator=g, device=dev))):
            q, s = _quantize_pages(x)
            codes.append(q)
            scales.append(s)
    T = starts[-1]
    state = {
        "case": case,
        "k_cache": torch.cat(k), "v_cache": torch.cat(v),
        "k_scale": torch.cat(ks), "v_scale": torch.cat(vs),
        "table": torch.tensor(rows, dtype=torch.int32, device=dev),
        "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
        "starts": torch.tensor(starts, dtype=torch.int32, device=dev),
        "longest": max(lens), "new": max(new), "tokens": T,
    }
    # queries, keys and values lie side by side, as one projection writes them
    qkv = torch.randn((T, (H + 2 * KV) * D), generator=g, device=dev).to(torch.bfloat16)
    state["q"] = qkv[:, :H * D].view(T, H, D)
    state["k"] = qkv[:, H * D:(H + KV) * D].view(T, KV, D)
    state["v"] = qkv[:, (H + KV) * D:].view(T, KV, D)
    if case["op"] == "append":
        half = case["rot"] // 2
        turn = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / max(1, half))
        angle = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * turn
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
        state["q_out"] = torch.zeros((T, H, D), dtype=torch.bfloat16, device=dev)
    else:
        state["q"] = state["q"].contiguous()
    if own:
        import fp8_blockwise_weight_amd as fq

        state["cache"] = fq.KvCache(state["k_cache"], state["v_cache"], state["k_scale"], state["v_scale"])
    return state


# ----------------------------------------------------------------- plain form

def _rotate(x, cos, sin, interleaved):
    """[T, heads, dim] in 32 bits, the first 2 * cos.shape[1] channels rotated."""
    half = cos.shape[1]
    x = x.float()
    if half == 0:
        return x
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _positions(state):
    """Sequence and position of each new token."""
    starts, lens = state["starts"].long(), state["lens"].long()
    t = torch.arange(state["tokens"], device=starts.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    return seq, lens[seq] - starts[seq + 1] + t


def _store(codes, scale, x, where, slot, head_page, held):
    """Quantizes tokens ``x`` [T, heads, dim] into pages ``codes`` [P, heads,
    page, dim] (bytes).  ``held`` [B] tokens of page ``head_page`` [B] are
    there already: where the page's scale grows, their codes follow it."""
    amax = torch.zeros_like(scale).index_reduce_(0, where, x.abs().amax(-1), "amax")
    fit = _fit(amax)
    before = torch.where(held[:, None] > 0, scale[head_page], torch.zeros_like(scale[head_page]))
    after = torch.maximum(before, fit[head_page])
    was = codes[head_page]
    again = was.view(torch.float8_e4m3fn).float() * (before / after)[:, :, None, None]
    old = torch.arange(codes.shape[2], device=codes.device)[None, :] < held[:, None]
    codes[head_page] = torch.where(old[:, None, :, None], again.to(torch.float8_e4m3fn).view(torch.uint8), was)
    scale[where] = fit[where]
    scale[head_page] = after
    q = (x / scale[where][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    heads = torch.arange(codes.shape[1], device=codes.device)[None, :]
    codes[where[:, None], heads, slot[:, None]] = q.view(torch.uint8)


def _plain_append(state):
    case, page = state["case"], state["case"]["page"]
    seq, pos = _positions(state)
    where, slot = state["table"][seq, pos // page].long(), pos % page
    cos, sin = state["cos"][pos], state["sin"][pos]
    state["q_out"].copy_(_rotate(state["q"], cos, sin, case["interleaved"]))
    # the first page that each sequence writes, and the earlier tokens in it
    starts = state["starts"].long()
    held = (state["lens"].long() - starts.diff()) % page
    head_page = where[starts[:-1]]
    _store(state["k_cache"].view(torch.uint8), state["k_scale"],
           _rotate(state["k"], cos, sin, case["interleaved"]), where, slot, head_page, held)
    _store(state["v_cache"].view(torch.uint8).transpose(2, 3), state["v_scale"],
           state["v"].float(), where, slot, head_page, held)
    return {"k": state["k_cache"], "v": state["v_cache"], "k_scale": state["k_scale"],
            "v_scale": state["v_scale"], "q": state["q_out"]}


def _plain_attention(state):
    case = state["case"]
    B, H, KV, D, page = (case[k] for k in ("batch", "q_heads", "kv_heads", "dim", "page"))
    G, n, L = H // KV, state["new"], state["longest"]
    pages = state["table"].long().clamp_min(0)                                # [B, W]
    W = pages.shape[1]
    k = state["k_cache"][pages].float() * state["k_scale"][pages][..., None, None]
    k = k.transpose(1, 2).reshape(B, KV, W * page, D)[:, :, :L]
    lens, starts = state["lens"].long(), state["starts"].long()
    count = starts.diff()
    step = torch.arange(n, device=lens.device)
    row = (starts[:-1, None] + step[None, :]).clamp_max(state["tokens"] - 1)  # [B, n]
    live = step[None, :] < count[:, None]
    pos = lens[:, None] - count[:, None] + step[None, :]
    q = state["q"][row].float().view(B, n, KV, G, D).permute(0, 2, 3, 1, 4).reshape(B, KV, G * n, D)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) * D ** -0.5
    del k
    key = torch.arange(L, device=lens.device)
    seen = (key[None, None, :] <= pos[:, :, None]) & live[:, :, None]         # [B, n, L]
    if case["window"]:
        seen &= key[None, None, :] > pos[:, :, None] - case["window"]
    s = s.view(B, KV, G, n, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = state["v_cache"][pages].float() * state["v_scale"][pages][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, KV, W * page, D)[:, :, :L]
    o = torch.matmul(p.view(B, KV, G * n, L), v).view(B, KV, G, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, H, D)
    return o[live.view(-1).nonzero()[:, 0]].to(torch.bfloat16)


def run(state):
    case = state["case"]
    one_each = state["new"] == 1                 # a token for every sequence
    if own:
        import fp8_blockwise_weight_amd as fq

        starts = None if one_each else state["starts"]
        if case["op"] == "append":
            fq.kv_append(state["cache"], state["k"], state["v"], state["table"], state["lens"], starts,
                         q=state["q"], q_out=state["q_out"], cos=state["cos"], sin=state["sin"],
                         interleaved=case["interleaved"])
            return {"k": state["k_cache"], "v": state["v_cache"], "k_scale": state["k_scale"],
                    "v_scale": state["v_scale"], "q": state["q_out"]}
        return fq.kv_attention(state["cache"], state["q"], state["table"], state["lens"], starts,
                               window=case["window"])
    return _plain_append(state) if case["op"] == "append" else _plain_attention(state)


def work(case):
    """Bytes: codes, scales, page numbers and rows, each once.  Products: the
    scores and the weighted sum over the keys that a query sees."""
    H, KV, D, page, window = (case[k] for k in ("q_heads", "kv_heads", "dim", "page", "window"))
    lens, new = _lengths(case)
    T = sum(new)
    touched = sum(-(-n // page) - (n - m) // page for n, m in zip(lens, new))
    if case["op"] == "append":
        # bf16 in, codes out, rotated queries out, the rotation's rows, scales out
        move = T * (2 * (H + 2 * KV) * D + 2 * KV * D + 2 * H * D + 4 * case["rot"]) + 8 * touched * KV
        return {"bytes": move + 4 * touched + 8 * len(lens), "flops": 3 * T * (H + KV) * case["rot"]}
    keys = pairs = held = 0
    for n, m in zip(lens, new):
        first = max(0, n - m + 1 - window) if window else 0
        keys += n - first
        held += -(-n // page) - first // page
        if not window:
            pairs += m * (n - m) + m * (m + 1) // 2
        else:
            pairs += sum(min(window, i + 1) for i in range(n - m, n))
    return {"bytes": keys * 2 * KV * D + held * (8 * KV + 4) + 4 * T * H * D + 8 * len(lens),
            "flops": 4 * pairs * H * D}


# ------------------------------------------------- the definition, in 64 bits

def _to_e4m3(x):
    """The nearest e4m3 value (ties to even), in 64 bits."""
    e = torch.frexp(x).exponent.double().sub_(1).clamp_min_(-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step).mul_(step).clamp_(-E4M3_MAX, E4M3_MAX)


def _exact_append(s, case):
    page, half = case["page"], case["rot"] // 2
    lens, new = _lengths(case)
    k, v = s["k_cache"].double(), s["v_cache"].double().transpose(2, 3).contiguous()
    scales = [s["k_scale"].double(), s["v_scale"].double()]
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        c, z = s["cos"][n - m:n, None].double(), s["sin"][n - m:n, None].double()
        turned = []
        for x in (s["q"], s["k"]):
            x = x[at:at + m].double()
            y = x.clone()
            lo = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
            hi = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
            y[..., lo] = x[..., lo] * c - x[..., hi] * z
            y[..., hi] = x[..., lo] * z + x[..., hi] * c
            turned.append(y)
        q_out[at:at + m] = turned[0]
        row = s["table"][b].tolist()
        for cache, scale, x in zip((k, v), scales, (turned[1], s["v"][at:at + m].double())):
            for j in range((n - m) // page, -(-n // page)):
                lo, hi = max(n - m, j * page), min(n, (j + 1) * page)
                part = x[lo - (n - m):hi - (n - m)]                            # [tokens, heads, dim]
                largest = part.abs().amax((0, 2)).clamp_min(EPS)
                fit = torch.exp2(torch.ceil(torch.log2(largest / E4M3_MAX)))
                fit = torch.where(fit / 2 * E4M3_MAX >= largest, fit / 2, fit)
                fit = torch.where(fit * E4M3_MAX < largest, fit * 2, fit)
                held = lo - j * page
                if held:
                    before = scale[row[j]].clone()
                    fit = torch.maximum(fit, before)
                    cache[row[j], :, :held] = _to_e4m3(cache[row[j], :, :held] * (before / fit)[:, None, None])
                scale[row[j]] = fit
                cache[row[j], :, held:hi - j * page] = _to_e4m3(part.transpose(0, 1) / fit[:, None, None])
        at += m
    return {"k": k, "v": v.transpose(2, 3).contiguous(), "k_scale": scales[0], "v_scale": scales[1], "q": q_out}


def _exact_attention(s, case):
    H, KV, D, window = (case[k] for k in ("q_heads", "kv_heads", "dim", "window"))
    lens, new = _lengths(case)
    out, at = [], 0
    for b, (n, m) in enumerate(zip(lens, new)):
        row = s["table"][b, :-(-n // case["page"])].long()
        k = (s["k_cache"][row].double() * s["k_scale"][row][..., None, None].double()).transpose(0, 1)
        v = (s["v_cache"][row].double() * s["v_scale"][row][..., None, None].double()).permute(1, 0, 3, 2)
        k, v = k.reshape(KV, -1, D)[:, :n], v.reshape(KV, -1, D)[:, :n]
        mine = s["q"][at:at + m].double().transpose(0, 1)                      # [heads, m, dim]
        key = torch.arange(n, device=k.device)
        pos = torch.arange(n - m, n, device=k.device)[:, None]
        hidden = (key > pos) | ((key <= pos - window) if window else False)
        heads = []
        for h in range(H):
            z = (mine[h] @ k[h // (H // KV)].t()) / math.sqrt(D)
            heads.append(torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ v[h // (H // KV)])
        out.append(torch.stack(heads, 1))
        at += m
    return torch.cat(out)


def exact(case, seed):
    return (_exact_append if case["op"] == "append" else _exact_attention)(prepare(case, seed), case)
