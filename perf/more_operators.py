"""The operators of the latent cache and of the caches' pages, as cases to
measure.

A case is one call of
  latent_append            new tokens into a paged cache of shared latents
  latent_attention         attention in the absorbed form over that cache
  latent_prompt_attention  attention in the expanded form, before any cache
  cache_fork               sequences that go on from another one's tokens
  cache_compact            the pages in use moved to the front
``run`` computes it in elementary torch operations where ``own`` is false and
through the package where it is true.

The latent cache, for P pages of ``page`` tokens:
  c      e4m3  [P, page, latent]   the latent of a token, for all heads, keys and values
  r      BF16  [P, page, 64]       its rotated key channels
  scale  fp32  [P, page]           a power of two for each latent
The key/value cache, whose pages are forked and compacted too:
  k      e4m3  [P, heads, page, dim]
  v      e4m3  [P, heads, dim, page]
  k_scale, v_scale  fp32 [P, heads]

Lengths, tables and page counts follow from the case alone, values from the
seed.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-10          # floor of a latent's largest magnitude
GOLDEN = 0.6180339887498949
ROPE = 64


def listed():
    """The cases.  Latents of 512 and 256 with 64 rotated channels, heads of
    128 + 64 and 64 + 64; pages of a key/value cache of 8 heads of 128."""
    def case(name, op, **more):
        return {"name": name, "op": op, "ragged": False, **more}

    def cache(name, op, batch, longest, new, heads, **more):
        base = {"latent": 512, "page": 64, "interleaved": False, "keys_out": False}
        return case(name, op, batch=batch, longest=longest, new=new, heads=heads, **{**base, **more})

    return [
        # a step of a rollout batch, a token for each sequence, odd count, an eighth of the heads
        cache("append_step", "append", 250, 4096, 1, 16, ragged=True, interleaved=True),
        # prompts of mixed lengths, all heads, keys kept for the expanded form
        cache("append_prompts", "append", 8, 4096, 4096, 128, ragged=True, keys_out=True),
        # the next token of one sequence: latency
        cache("absorbed_one", "absorbed", 1, 777, 1, 16),
        # a step of a rollout batch with mixed lengths, an eighth of the heads: the cache's bytes count
        cache("absorbed_step_16", "absorbed", 96, 16384, 1, 16, ragged=True),
        # the same with all heads on one card: products count
        cache("absorbed_step_128", "absorbed", 60, 12000, 1, 128, ragged=True),
        # up to five drafted tokens, small latents in small pages
        cache("absorbed_drafts", "absorbed", 30, 5000, 5, 40, ragged=True, latent=256, page=16),
        # short prompts of odd lengths, small heads
        case("expanded_short", "expanded", batch=9, longest=777, new=777, heads=12, dim=64, ragged=True),
        # whole prompts against their own keys
        case("expanded_prompts", "expanded", batch=2, longest=4096, new=4096, heads=32, dim=128),
        # four samples of one prompt, latents of 27 layers: latency
        case("fork_one", "fork", kind="latent", layers=27, latent=512, page=64, groups=1, samples=4, longest=777),
        # 16 samples of each of 32 prompts, key/value pages of 8 layers
        case("fork_samples", "fork", kind="kv", layers=8, kv_heads=8, dim=128, page=64, groups=32, samples=16,
             longest=1000, ragged=True),
        # a few short sequences left of many, small pages
        case("compact_small", "compact", kind="kv", layers=4, kv_heads=5, dim=64, page=16, groups=9, samples=4,
             longest=300, ragged=True, keep=3),
        # a quarter of 256 samples still running, latents of 8 layers
        case("compact_latents", "compact", kind="latent", layers=8, latent=512, page=64, groups=16, samples=16,
             longest=2000, ragged=True, keep=4),
    ]


def draw(rng):
    """One more case of the same ranges, at most what the largest case costs."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["append", "absorbed", "absorbed", "expanded", "expanded", "fork", "compact"])
    ragged = rng.choice([False, True, True])
    if op in ("append", "absorbed"):
        latent, heads = rng.choice([256, 512, 512]), rng.choice([1, 5, 8, 16, 16, 32, 40, 64, 128])
        batch, longest = log_int(1, 256), log_int(1, 65536)
        kind = rng.choice(["step", "step", "drafts", "chunk"])
        new = 1 if kind == "step" else min(longest, log_int(2, 8 if kind == "drafts" else 2048))
        while batch > 1 and batch * longest * latent > 4.0e8:
            batch = max(1, batch // 2)
        longest = max(1, min(longest, int(2.0e8 / latent)))
        new = min(new, longest)
        while new > 1 and batch * new * heads * latent > 6.0e7:
            new = max(1, new // 2)
        while new > 1 and 4.0 * batch * new * longest * heads * latent > 1.0e11:
            new = max(1, new // 2)
        return {"op": op, "batch": batch, "longest": longest, "new": new, "heads": heads, "latent": latent,
                "page": rng.choice([16, 32, 64, 128, 256]), "ragged": ragged,
                "interleaved": rng.choice([False, True]), "keys_out": rng.choice([False, True])}
    if op == "expanded":
        dim, heads = rng.choice([64, 128, 128]), rng.choice([1, 3, 8, 12, 16, 32, 64])
        batch, longest = log_int(1, 32), log_int(1, 8192)
        new = longest if rng.random() < 0.6 else log_int(1, longest)
        while batch > 1 and batch * longest * heads * dim > 6.0e7:
            batch = max(1, batch // 2)
        while longest > 1 and batch * new * longest * heads * dim > 1.3e11:
            longest = max(1, longest // 2)
            new = min(new, longest)
        return {"op": op, "batch": batch, "longest": longest, "new": new, "heads": heads, "dim": dim,
                "ragged": ragged}
    kind = rng.choice(["kv", "latent"])
    case = {"op": op, "kind": kind, "layers": log_int(1, 27), "page": rng.choice([16, 32, 64, 128, 256]),
            "groups": log_int(1, 32), "samples": log_int(1 if op == "compact" else 2, 16),
            "longest": log_int(1, 2000), "ragged": ragged}
    case.update({"latent": rng.choice([256, 512])} if kind == "latent" else
                {"kv_heads": rng.choice([1, 2, 5, 8]), "dim": rng.choice([64, 128, 192, 256])})
    if op == "compact":
        case["keep"] = rng.choice([1, 2, 4, 8])
    while case["layers"] > 1 and case["layers"] * _page_bytes(case) * len(_pool(case)[2]) > 1.2e9:
        case["layers"] //= 2
    return case


def _spread(n, longest, ragged):
    if not ragged:
        return [longest] * n
    return [longest] + [1 + int((longest - 1) * ((b * GOLDEN) % 1.0)) for b in range(1, n)]


def _lengths(case):
    """Tokens of each sequence after the call, and how many of them are new."""
    n, longest, new = case["batch"], case["longest"], case["new"]
    lens = _spread(n, longest, case["ragged"])
    if new == longest:
        return lens, list(lens)
    if not case["ragged"]:
        return lens, [new] * n
    return lens, [min(lens[b], 1 + (new - 1 + 5 * b) % new) for b in range(n)]


def _page_bytes(case):
    if case["kind"] == "latent":
        return case["page"] * (case["latent"] + 2 * ROPE + 4)
    return case["kv_heads"] * (2 * case["page"] * case["dim"] + 8)


def _pool(case):
    """(lengths, table rows, page order) of forked or compacted sequences.

    A row for each sample of each group.  To be forked, a group's first row
    holds its prompt, the others nothing yet.  To be compacted, samples share
    the whole pages of the first half of their tokens, and one in ``keep``
    still runs, the others have length 0 and their pages in the table yet."""
    page, groups, samples = case["page"], case["groups"], case["samples"]
    lens, rows, at = [], [], 0
    if case["op"] == "fork":
        for n in _spread(groups, case["longest"], case["ragged"]):
            count = -(-n // page)
            rows.append(list(range(at, at + count)))
            at += count
            lens += [n] + [0] * (samples - 1)
            rows += [[] for _ in range(samples - 1)]
        at += groups * (samples - 1)              # the pages that forks take
    else:
        every = _spread(groups * samples, case["longest"], case["ragged"])
        for g in range(groups):
            mine = every[g * samples:(g + 1) * samples]
            shared = list(range(at, at + min(mine) // 2 // page))
            at += len(shared)
            for i, n in enumerate(mine):
                own_pages = -(-n // page) - len(shared)
                rows.append(shared + list(range(at, at + own_pages)))
                at += own_pages
                lens.append(n if (g * samples + i) % case["keep"] == 0 else 0)
    order = list(range(at + 3))                   # three pages belong to nobody
    random.Random(at).shuffle(order)
    return lens, [[order[p] for p in r] for r in rows], order


def _fit(amax):
    """The smallest power of two that brings ``amax`` within e4m3: 448 is
    0.875 * 2^9."""
    m, e = torch.frexp(amax.clamp_min(EPS))
    return ((e + (127 - 9) + (m > 0.875).to(e.dtype)) << 23).view(torch.float32)


def _latents(shape, strong, g, dev):
    """Latents as a norm leaves them: even, with some strong channels."""
    x = torch.randn(shape, generator=g, device=dev) * strong
    return x * torch.exp(0.3 * torch.randn(shape[:-1] + (1,), generator=g, device=dev))


def _latent_pages(pages, page, latent, g, dev):
    strong = 1 + 3 * (torch.rand((latent,), generator=g, device=dev) < 0.05).float()
    codes, scales = [], []
    some = max(1, (1 << 26) // (page * latent))   # pages made at a time
    for p in range(0, pages, some):
        x = _latents((min(some, pages - p), page, latent), strong, g, dev)
        s = _fit(x.abs().amax(-1))
        codes.append((x / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
        scales.append(s)
    r = torch.randn((pages, page, ROPE), generator=g, device=dev).to(torch.bfloat16)
    return {"c": torch.cat(codes), "r": r, "scale": torch.cat(scales)}


def _codes(shape, g, dev):
    """Any finite codes: for pages that are only moved."""
    x = torch.randint(0, 254, shape, generator=g, device=dev, dtype=torch.uint8)
    return torch.where(x == 127, x + 127, x).view(torch.float8_e4m3fn)


def _table(rows, width, dev):
    return torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32, device=dev)


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _prepare_cache(case, g, dev):
    H, L, page = case["heads"], case["latent"], case["page"]
    lens, new = _lengths(case)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    order = list(range(pages))
    random.Random(pages).shuffle(order)
    rows, starts = [], [0]
    for c, n in zip(counts, new):
        rows.append([order.pop() for _ in range(c)])
        starts.append(starts[-1] + n)
    T = starts[-1]
    state = {"case": case, **_latent_pages(pages, page, L, g, dev), "table": _table(rows, max(counts), dev),
             "lens": _i32(lens, dev), "starts": _i32(starts, dev), "longest": max(lens), "new": max(new),
             "tokens": T}
    # the rotary channels of the queries lie behind the others, as a projection writes them
    state["q_r"] = torch.randn((T, H, 128 + ROPE), generator=g, device=dev).to(torch.bfloat16)[:, :, 128:]
    if case["op"] == "append":
        strong = 1 + 3 * (torch.rand((L,), generator=g, device=dev) < 0.05).float()
        state["x"] = _latents((T, L), strong, g, dev).to(torch.bfloat16)
        # the rotary channels of the keys are the last ones of the projection that makes the latents
        state["x_r"] = torch.randn((T, L + ROPE), generator=g, device=dev).to(torch.bfloat16)[:, L:]
        turn = 10000.0 ** (-torch.arange(ROPE // 2, device=dev, dtype=torch.float64) / (ROPE // 2))
        angle = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * turn
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
        state["q_out"] = torch.zeros((T, H, ROPE), dtype=torch.bfloat16, device=dev)
        state["r_out"] = torch.zeros((T, ROPE), dtype=torch.bfloat16, device=dev) if case["keys_out"] else None
    else:
        # head by head, as the batched product that absorbs the up-projection writes them
        state["q_c"] = torch.randn((H, T, L), generator=g, device=dev).to(torch.bfloat16).transpose(0, 1)
        state["scale_by"] = (128 + ROPE) ** -0.5
    if own:
        import fp8_blockwise_weight_amd as fq

        state["cache"] = fq.LatentCache(state["c"], state["r"], state["scale"])
    return state


def _prepare_expanded(case, g, dev):
    H, D = case["heads"], case["dim"]
    lens, new = _lengths(case)
    q_at, k_at = [0], [0]
    for n, m in zip(lens, new):
        q_at.append(q_at[-1] + m)
        k_at.append(k_at[-1] + n)
    T, K = q_at[-1], k_at[-1]
    # keys and values of a head side by side, as the up-projection writes them
    kv = torch.randn((K, H, 2 * D), generator=g, device=dev).to(torch.bfloat16)
    return {"case": case, "q": torch.randn((T, H, D + ROPE), generator=g, device=dev).to(torch.bfloat16),
            "k": kv[:, :, :D], "v": kv[:, :, D:],
            "k_r": torch.randn((K, ROPE), generator=g, device=dev).to(torch.bfloat16),
            "q_at": _i32(q_at, dev), "k_at": None if lens == new else _i32(k_at, dev)}


def _prepare_pages(case, g, dev):
    lens, rows, order = _pool(case)
    pages, page = len(order), case["page"]
    n = case["layers"]                            # one tensor for all layers
    if case["kind"] == "latent":
        buffers = {"c": _codes((n, pages, page, case["latent"]), g, dev),
                   "r": torch.randn((n, pages, page, ROPE), generator=g, device=dev).to(torch.bfloat16),
                   "scale": torch.exp2(torch.randint(-12, -4, (n, pages, page), generator=g, device=dev).float())}
    else:
        h, d = case["kv_heads"], case["dim"]
        buffers = {"k": _codes((n, pages, h, page, d), g, dev), "v": _codes((n, pages, h, d, page), g, dev),
                   **{x: torch.exp2(torch.randint(-12, -4, (n, pages, h), generator=g, device=dev).float())
                      for x in ("k_scale", "v_scale")}}
    width = max(1, -(-case["longest"] // page))
    state = {"case": case, "buffers": buffers, "table": _table(rows, width, dev), "lens": _i32(lens, dev)}
    if case["op"] == "fork":
        s = case["samples"]
        children = [b for b in range(len(lens)) if b % s]
        state["parents"] = _i32([b - b % s for b in children], dev)
        state["children"] = _i32(children, dev)
        taken = {p for r in rows for p in r}
        state["pages"] = _i32([p for p in order if p not in taken][:len(children)], dev)
    if own:
        import fp8_blockwise_weight_amd as fq

        make = fq.LatentCache if case["kind"] == "latent" else fq.KvCache
        state["handles"] = [make(*(x[i] for x in buffers.values())) for i in range(n)]
    return state


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] in ("append", "absorbed"):
        return _prepare_cache(case, g, dev)
    return (_prepare_expanded if case["op"] == "expanded" else _prepare_pages)(case, g, dev)


# ----------------------------------------------------------------- plain form

def _rotate(x, cos, sin, interleaved):
    """[..., 64] in 32 bits, rotated."""
    x, half = x.float(), ROPE // 2
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_append(state):
    case, page = state["case"], state["case"]["page"]
    starts, lens = state["starts"].long(), state["lens"].long()
    t = torch.arange(state["tokens"], device=starts.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[seq] - starts[seq + 1] + t
    where, slot = state["table"][seq, pos // page].long(), pos % page
    cos, sin = state["cos"][pos], state["sin"][pos]
    x = state["x"].float()
    s = _fit(x.abs().amax(-1))
    q = (x / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    r = _rotate(state["x_r"], cos, sin, case["interleaved"]).to(torch.bfloat16)
    state["c"].view(torch.uint8)[where, slot] = q.view(torch.uint8)
    state["scale"][where, slot] = s
    state["r"][where, slot] = r
    state["q_out"].copy_(_rotate(state["q_r"], cos[:, None], sin[:, None], case["interleaved"]))
    if state["r_out"] is not None:
        state["r_out"].copy_(r)


def _plain_absorbed(state):
    case = state["case"]
    B, H, L, page = (case[k] for k in ("batch", "heads", "latent", "page"))
    n, N = state["new"], state["longest"]
    pages = state["table"].long().clamp_min(0)
    W = pages.shape[1]
    c = (state["c"][pages].float() * state["scale"][pages][..., None]).view(B, W * page, L)[:, :N]
    r = state["r"][pages].float().view(B, W * page, ROPE)[:, :N]
    lens, starts = state["lens"].long(), state["starts"].long()
    count = starts.diff()
    step = torch.arange(n, device=lens.device)
    row = (starts[:-1, None] + step[None, :]).clamp_max(state["tokens"] - 1)
    live = step[None, :] < count[:, None]
    pos = lens[:, None] - count[:, None] + step[None, :]
    q = torch.cat((state["q_c"][row].float(), state["q_r"][row].float()), -1).view(B, n * H, L + ROPE)
    s = torch.matmul(q, torch.cat((c, r), -1).transpose(1, 2).contiguous()) * state["scale_by"]
    key = torch.arange(N, device=lens.device)
    seen = (key[None, None, :] <= pos[:, :, None]) & live[:, :, None]
    s = s.view(B, n, H, N).masked_fill_(~seen[:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, n * H, N), c).view(B, n, H, L)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).view(B * n, H, L)
    return o[live.view(-1).nonzero()[:, 0]].to(torch.bfloat16)


def _plain_expanded(state):
    case = state["case"]
    H, D = case["heads"], case["dim"]
    lens, new = _lengths(case)
    out = torch.empty((state["q"].shape[0], H, D), dtype=torch.bfloat16, device=state["q"].device)
    q_at = k_at = 0
    for n, m in zip(lens, new):
        keys = torch.cat((state["k"][k_at:k_at + n].float(),
                          state["k_r"][k_at:k_at + n].float()[:, None].expand(n, H, ROPE)), -1)
        q = state["q"][q_at:q_at + m].float().transpose(0, 1).contiguous()
        s = torch.matmul(q, keys.permute(1, 2, 0).contiguous()) * (D + ROPE) ** -0.5
        key = torch.arange(n, device=s.device)
        s.masked_fill_(key[None, None, :] > (n - m + torch.arange(m, device=s.device))[None, :, None], -math.inf)
        p = s.sub_(s.amax(-1, keepdim=True)).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, state["v"][k_at:k_at + n].float().transpose(0, 1).contiguous()) / total
        out[q_at:q_at + m] = o.transpose(0, 1)
        q_at, k_at = q_at + m, k_at + n
    return out


def _plain_fork(state):
    table, lens, page = state["table"], state["lens"], state["case"]["page"]
    a, b = state["parents"].long(), state["children"].long()
    n, width = lens[a].long(), table.shape[1]
    column = torch.arange(width, device=table.device)
    last, part = n // page, n % page > 0
    source = table[a, last.clamp_max(width - 1)].long()
    rows = torch.where(column < last[:, None], table[a], torch.full_like(table[a], -1))
    table[b] = torch.where((column == last[:, None]) & part[:, None], state["pages"][:, None], rows)
    lens[b] = lens[a]
    to, source = state["pages"][part].long(), source[part]
    for x in state["buffers"].values():
        for y in x.view(torch.uint8) if x.element_size() == 1 else x:
            y[to] = y[source]


def _plain_compact(state):
    table, lens, page = state["table"], state["lens"].long(), state["case"]["page"]
    pages = next(iter(state["buffers"].values())).shape[1]
    live = torch.arange(table.shape[1], device=table.device) < ((lens + page - 1) // page)[:, None]
    mark = torch.zeros((pages,), dtype=torch.bool, device=table.device)
    mark[table[live].long()] = True
    used = mark.sum()
    number = torch.arange(pages, device=table.device)
    holes, movers = number[~mark & (number < used)], number[mark & (number >= used)]
    name = number.clone()
    name[movers] = holes
    for x in state["buffers"].values():
        for y in x.view(torch.uint8) if x.element_size() == 1 else x:
            y[holes] = y[movers]
    renamed = torch.where(live, name[table.clamp_min(0).long()], torch.full_like(number[:1], -1))
    return renamed.to(torch.int32), used.to(torch.int32).view(1)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import fp8_blockwise_weight_amd as fq
    if op in ("append", "absorbed"):
        starts = None if state["new"] == 1 else state["starts"]   # a token for every sequence
    if op == "append":
        if own:
            fq.latent_append(state["cache"], state["x"], state["x_r"], state["table"], state["lens"], starts,
                             q=state["q_r"], q_out=state["q_out"], r_out=state["r_out"], cos=state["cos"],
                             sin=state["sin"], interleaved=case["interleaved"])
        else:
            _plain_append(state)
        out = {name: state[name] for name in ("c", "r", "scale", "q_out")}
        return out if state["r_out"] is None else {**out, "r_out": state["r_out"]}
    if op == "absorbed":
        if not own:
            return _plain_absorbed(state)
        return fq.latent_attention(state["cache"], state["q_c"], state["q_r"], state["table"], state["lens"], starts,
                                   scale=state["scale_by"])
    if op == "expanded":
        if not own:
            return _plain_expanded(state)
        return fq.latent_prompt_attention(state["q"], state["k"], state["k_r"], state["v"], state["q_at"],
                                          state["k_at"])
    if op == "fork":
        if own:
            fq.cache_fork(state["handles"], state["table"], state["lens"], state["parents"], state["children"],
                          state["pages"])
        else:
            _plain_fork(state)
        return {**state["buffers"], "table": state["table"], "lens": state["lens"]}
    renamed, used = fq.cache_compact(state["handles"], state["table"], state["lens"]) if own else _plain_compact(state)
    return {**state["buffers"], "table": renamed, "used": used}


def work(case):
    """Bytes: what is read and written, each once.  Products: the scores and
    the weighted sum over the keys that a query sees."""
    op = case["op"]
    if op in ("fork", "compact"):
        lens, rows, order = _pool(case)
        page, size = case["page"], _page_bytes(case) * case["layers"]
        entries = sum(-(-n // page) for n in lens)
        if op == "fork":
            partly = sum(1 for n in lens if n % page)          # parents that hold a partly filled page
            s = case["samples"]
            return {"bytes": partly * s * size + 4 * (entries * s + len(lens) * 2), "flops": 0}
        live = {p for n, r in zip(lens, rows) for p in r[:-(-n // page)]}
        moved = sum(1 for p in live if p >= len(live))
        width = max(1, -(-case["longest"] // page))
        return {"bytes": 2 * moved * size + 4 * (entries + len(lens) * (width + 1)), "flops": 0}
    H = case["heads"]
    lens, new = _lengths(case)
    T = sum(new)
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
    if op == "expanded":
        D = case["dim"]
        return {"bytes": 2 * T * H * (2 * D + ROPE) + sum(lens) * 2 * (2 * H * D + ROPE) + 8 * len(lens),
                "flops": 2 * pairs * H * (2 * D + ROPE)}
    L, page = case["latent"], case["page"]
    if op == "append":
        token = 2 * (L + ROPE) + L + 2 * ROPE + 4 + 4 * ROPE * H + 4 * ROPE + (2 * ROPE if case["keys_out"] else 0)
        touched = sum(-(-n // page) - (n - m) // page for n, m in zip(lens, new))
        return {"bytes": T * token + 4 * touched + 8 * len(lens), "flops": 3 * T * (H + 1) * ROPE}
    held = sum(-(-n // page) for n in lens)
    return {"bytes": sum(lens) * (L + 2 * ROPE + 4) + 4 * held + T * H * 2 * (2 * L + ROPE) + 8 * len(lens),
            "flops": 2 * pairs * H * (2 * L + ROPE)}


# ------------------------------------------------- the definition, in 64 bits

def _to_e4m3(x):
    """The nearest e4m3 value (ties to even), in 64 bits."""
    e = torch.frexp(x).exponent.double().sub_(1).clamp_min_(-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step).mul_(step).clamp_(-E4M3_MAX, E4M3_MAX)


def _exact_append(s, case):
    page, half = case["page"], ROPE // 2
    lens, new = _lengths(case)
    lo = slice(0, ROPE, 2) if case["interleaved"] else slice(0, half)
    hi = slice(1, ROPE, 2) if case["interleaved"] else slice(half, ROPE)
    c, r, scale = s["c"].double(), s["r"].double(), s["scale"].double()
    q_out = torch.zeros(s["q_r"].shape, dtype=torch.float64, device=c.device)
    r_out = torch.zeros(s["x_r"].shape, dtype=torch.float64, device=c.device)
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        cs, sn = s["cos"][n - m:n].double(), s["sin"][n - m:n].double()
        for x, y, a, z in ((s["q_r"][at:at + m].double(), q_out[at:at + m], cs[:, None], sn[:, None]),
                           (s["x_r"][at:at + m].double(), r_out[at:at + m], cs, sn)):
            y[..., lo] = x[..., lo] * a - x[..., hi] * z
            y[..., hi] = x[..., lo] * z + x[..., hi] * a
        x = s["x"][at:at + m].double()
        largest = x.abs().amax(1).clamp_min(EPS)
        fit = torch.exp2(torch.ceil(torch.log2(largest / E4M3_MAX)))
        fit = torch.where(fit / 2 * E4M3_MAX >= largest, fit / 2, fit)
        fit = torch.where(fit * E4M3_MAX < largest, fit * 2, fit)
        pos = torch.arange(n - m, n, device=c.device)
        where, slot = s["table"][b].long()[pos // page], pos % page
        c[where, slot], scale[where, slot], r[where, slot] = _to_e4m3(x / fit[:, None]), fit, r_out[at:at + m]
        at += m
    out = {"c": c, "r": r, "scale": scale, "q_out": q_out}
    return {**out, "r_out": r_out} if case["keys_out"] else out


def _exact_rows(q, k, v, first, scale_by):
    """Attention of rows [m, .] at positions first, first + 1, ... ."""
    z = (q @ k.t()) * scale_by
    late = torch.arange(k.shape[0], device=k.device)[None, :] > first + torch.arange(q.shape[0], device=k.device)[:, None]
    return torch.softmax(z.masked_fill_(late, -math.inf), -1) @ v


def _exact_absorbed(s, case):
    lens, new = _lengths(case)
    out, at = [], 0
    for b, (n, m) in enumerate(zip(lens, new)):
        row = s["table"][b, :-(-n // case["page"])].long()
        c = (s["c"][row].double() * s["scale"][row][..., None].double()).flatten(0, 1)[:n]
        k = torch.cat((c, s["r"][row].double().flatten(0, 1)[:n]), -1)
        heads = [_exact_rows(torch.cat((s["q_c"][at:at + m, h], s["q_r"][at:at + m, h]), -1).double(), k, c, n - m,
                             s["scale_by"]) for h in range(case["heads"])]
        out.append(torch.stack(heads, 1))
        at += m
    return torch.cat(out)


def _exact_expanded(s, case):
    lens, new = _lengths(case)
    out, q_at, k_at = [], 0, 0
    for n, m in zip(lens, new):
        r = s["k_r"][k_at:k_at + n]
        heads = [_exact_rows(s["q"][q_at:q_at + m, h].double(),
                             torch.cat((s["k"][k_at:k_at + n, h], r), -1).double(),
                             s["v"][k_at:k_at + n, h].double(), n - m, (case["dim"] + ROPE) ** -0.5)
                 for h in range(case["heads"])]
        out.append(torch.stack(heads, 1))
        q_at, k_at = q_at + m, k_at + n
    return torch.cat(out)


def exact(case, seed):
    exacts = {"append": _exact_append, "absorbed": _exact_absorbed, "expanded": _exact_expanded}
    if case["op"] not in exacts:
        return None               # pages and their names are moved, not computed
    return exacts[case["op"]](prepare(case, seed), case)
