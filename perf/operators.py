"""The paged-cache operators as measured: cases, inputs, their plain forms and their values in 64 bits.

A paged KV cache keeps the tokens of all requests in pages of page_size tokens, [n_pages, page_size, n_kv, d];
row b of block_table lists the pages of request b in order.  Four operators work on it:

* plan    - page_plan: block tables, slots and positions of a step's new tokens from the requests' lengths
* append  - kv_append_paged: new keys (rotated at their positions) and values written to their slots
* decode  - decode_paged: one new query per request against its pages
* shared  - decode_shared: the same for a batch whose requests all start with the same pages (a system prompt),
            the shared part read and computed once for the whole batch
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _plan(name, B, lo, hi, new, page, short=False):
    """B requests holding lo..hi tokens, adding 1..new tokens each; short: the free pages run out on the way."""
    return {"name": name, "op": "plan", "B": B, "lo": lo, "hi": hi, "new": new, "page": page, "short": short}


def _append(name, T, pad, n_kv, d, page, base, half, dtype):
    """T new tokens in a buffer of T + pad rows (the rows behind have slot -1)."""
    return {"name": name, "op": "append", "T": T, "pad": pad, "n_kv": n_kv, "d": d, "page": page, "base": base,
            "half": half, "dtype": dtype}


def _attend(name, B, pad, prefix, lo, hi, n_h, n_kv, d, page, base, dtype):
    """B requests (pad of them empty places of a padded batch) with prefix shared tokens and lo..hi of their own."""
    return {"name": name, "op": "shared" if prefix else "decode", "B": B, "pad": pad, "prefix": prefix, "lo": lo,
            "hi": hi, "n_h": n_h, "n_kv": n_kv, "d": d, "page": page, "base": base, "dtype": dtype}


def listed():
    return [
        # a decode step of the 59-request batch: one new token each (pure latency)
        _plan("plan_step_59", 59, 4096, 8192, 1, 64),
        # a step that admits prompts: 512 requests, 1..255 new tokens each, 16-token pages
        _plan("plan_prompts_512", 512, 0, 2000, 255, 16),
        # the append of that decode step, keys rotated at their positions (latency)
        _append("append_step_59", 59, 5, 8, 128, 64, 500000.0, False, "bf16"),
        # four 8192-token prompts written to pages at once (HBM)
        _append("append_prompts_32768", 32768, 0, 8, 128, 64, 500000.0, False, "bf16"),
        # one short chat, a few hundred tokens (latency of a single request)
        _attend("decode_one_short", 1, 0, 0, 333, 333, 32, 8, 128, 16, 500000.0, "bf16"),
        # the 59-request decode batch, 4096..8192 keys each, 64-token pages (HBM)
        _attend("decode_59_requests", 59, 0, 0, 4096, 8192, 32, 8, 128, 64, 500000.0, "bf16"),
        # two long documents in 16-token pages: the key axis has to be split (HBM)
        _attend("decode_two_long", 2, 0, 0, 98001, 131071, 32, 8, 128, 16, 500000.0, "bf16"),
        # a small full-precision model with as many KV heads as heads, and an empty place in the batch
        _attend("decode_f32_mha", 8, 1, 0, 1, 1024, 12, 12, 64, 32, 0.0, "f32"),
        # eight requests behind a 4096-token system prompt, a few tokens of their own (latency)
        _attend("shared_8_short", 8, 1, 4096, 1, 100, 32, 8, 128, 64, 500000.0, "bf16"),
        # 64 requests over one 32768-token document (HBM, the prefix read once)
        _attend("shared_64_document", 64, 0, 32768, 16, 512, 32, 8, 128, 64, 500000.0, "bf16"),
        # 256 requests behind a 16384-token prompt: the prefix becomes a matrix product (tensor cores)
        _attend("shared_256_prompt", 256, 3, 16384, 1, 256, 32, 8, 128, 64, 500000.0, "bf16"),
        # full precision with a shared prompt
        _attend("shared_f32", 6, 0, 1024, 1, 200, 12, 12, 64, 32, 0.0, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8), (12, 12), (8, 1), (28, 4), (16, 8), (40, 8), (6, 2)]


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 2048)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(1024, 120000 // B)))
        hi = _log(rng, 1, 8192)
        return _strip(_plan("", B, rng.randint(0, hi), hi, new, page, rng.random() < 0.25))
    n_h, n_kv = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    base = rng.choice([0.0, 10000.0, 500000.0])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op == "append":
        top = 32768 if dtype == "bf16" else 16384
        return _strip(_append("", _log(rng, 1, max(1, min(top, top * 8 * 128 // (n_kv * d)))), rng.choice([0, 1, 37]),
                              n_kv, d, page, base, rng.random() < 0.5, dtype))
    B = _log(rng, 2, 256) if op == "shared" else _log(rng, 1, 128)
    pad = rng.randint(0, 2) if B > 3 else 0
    room = 200000 if dtype == "bf16" else 16000  # tokens of all requests together
    prefix = 0
    if op == "shared":
        prefix = page * max(1, _log(rng, 256, min(32768, (1 << 27) // (B * n_h)) if dtype == "bf16" else 2048) // page)
        hi = _log(rng, 1, max(1, min(1024, room // B)))
    else:
        hi = _log(rng, 1, max(1, room // B))
    return _strip(_attend("", B, pad, prefix, rng.randint(1, hi), hi, n_h, n_kv, d, page, base, dtype))


def _strip(case):
    return {k: v for k, v in case.items() if k != "name"}


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread (so that the work does not depend on the seed)."""
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [hi] * n


def _lengths(case):
    """Keys of each live request, the new token included."""
    return [case["prefix"] + x for x in _spread(case["lo"], case["hi"], case["B"] - case["pad"])]


def _pages_of(n, page):
    return (n + page - 1) // page


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(TYPES[case["dtype"]])

    def ints(values):
        return torch.tensor(values, dtype=torch.int32).to(DEV)

    page = case["page"]
    if case["op"] == "plan":
        B = case["B"]
        lens = torch.tensor(_spread(case["lo"], case["hi"], B))[torch.randperm(B, generator=gc)]
        new = torch.tensor(_spread(1, case["new"], B))[torch.randperm(B, generator=gc)]
        have, want = (lens + page - 1) // page, (lens + new + page - 1) // page
        held, need = int(have.sum()), int((want - have).sum())
        free = max(1, need * 2 // 3) if case["short"] else need + B
        order = torch.randperm(held + free, generator=gc).to(torch.int32)
        width = int(want.max()) + 1
        table = torch.full((B, width), -1, dtype=torch.int32)
        table[torch.arange(width)[None, :] < have[:, None]] = order[:held]
        return {"case": case, "lens": lens.to(torch.int32).to(DEV), "new": new.to(torch.int32).to(DEV),
                "table": table.to(DEV), "free": order[held:].clone().to(DEV), "n_free": ints([free]),
                "n_pages": held + free, "max_tokens": int(new.sum()) + 16}
    if case["op"] == "append":
        T, pad, n_kv, d = case["T"], case["pad"], case["n_kv"], case["d"]
        n_pages = _pages_of(T, page) + 3
        where = torch.randperm(n_pages, generator=gc)[: _pages_of(T, page)]
        slots = (where[:, None] * page + torch.arange(page)[None, :]).reshape(-1)[:T]
        start = int(torch.randint(0, 8192, (1,), generator=gc))
        return {"case": case, "k": normal(T + pad, n_kv, d), "v": normal(T + pad, n_kv, d),
                "k_pages": normal(n_pages, page, n_kv, d), "v_pages": normal(n_pages, page, n_kv, d),
                "slots": torch.cat([slots, torch.full((pad,), -1)]).to(torch.int32).to(DEV),
                "positions": torch.cat([start + torch.arange(T), torch.full((pad,), -1)]).to(torch.int32).to(DEV)}
    B, prefix, n_h, n_kv, d = case["B"], case["prefix"], case["n_h"], case["n_kv"], case["d"]
    lens = torch.tensor(_lengths(case) + [0] * case["pad"])[torch.randperm(B, generator=gc)]
    n_shared = prefix // page
    tail = torch.clamp((lens + page - 1) // page - n_shared, min=0)
    n_pages = n_shared + int(tail.sum()) + 2
    order = torch.randperm(n_pages, generator=gc).to(torch.int32)
    width = n_shared + int(tail.max())
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[:, :n_shared] = order[:n_shared]
    table[:, n_shared:][torch.arange(width - n_shared)[None, :] < tail[:, None]] = order[n_shared:n_pages - 2]
    return {"case": case, "q": normal(B, n_h, d), "k_pages": normal(n_pages, page, n_kv, d),
            "v_pages": normal(n_pages, page, n_kv, d), "table": table.to(DEV),
            "prefix_pages": order[:n_shared].clone().to(DEV), "lens": lens.to(torch.int32).to(DEV)}


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"plan": _plain_plan, "append": _plain_append, "decode": _plain_attend,
            "shared": _plain_attend}[case["op"]](case, state)


def _own(case, s):
    import transformer_causal_attention_gb300 as attn

    if case["op"] == "plan":
        seqlens, cu, slots, positions, left = attn.page_plan(
            s["lens"], s["new"], s["table"], s["free"], s["n_free"], page_size=case["page"], n_pages=s["n_pages"],
            max_tokens=s["max_tokens"])
        return {"table": s["table"], "seqlens": seqlens, "cu_new": cu, "slots": slots, "positions": positions,
                "n_left": left}
    if case["op"] == "append":
        attn.kv_append_paged(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], s["positions"],
                             rope_base=case["base"], pairing="half" if case["half"] else "adjacent")
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if case["op"] == "decode":
        out, _ = attn.decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], rope_base=case["base"])
    else:
        out, _ = attn.decode_shared(s["q"], s["k_pages"], s["v_pages"], s["prefix_pages"], s["table"], s["lens"],
                                    rope_base=case["base"])
    return {"out": out}


# ------------------------------------------------------------------------------------------ plain forms
def _plain_plan(case, s):
    page, table, N = case["page"], s["table"], s["max_tokens"]
    B, width = table.shape
    lens, new = s["lens"].long(), s["new"].long()
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    have = (lens + page - 1) // page
    want = (lens + new + page - 1) // page
    fits = (want <= width) & (cu[1:] <= N)
    need = torch.where(fits, want - have, 0)
    end = torch.cumsum(need, 0)
    n_free = s["n_free"].long()
    ok = fits & ((need == 0) | (end <= n_free))
    taken = torch.where(ok & (need > 0), end, 0).max()
    # page k of request b comes from the top of the free stack, after the pages of the requests before it
    col = torch.arange(width, device=DEV)[None, :]
    fresh = ok[:, None] & (col >= have[:, None]) & (col < want[:, None])
    place = n_free - 1 - ((end - need)[:, None] + col - have[:, None])
    pages = s["free"][torch.clamp(place, 0, s["free"].numel() - 1)]
    table.copy_(torch.where(fresh, pages, table))
    t = torch.arange(N, device=DEV)
    owner = torch.clamp(torch.searchsorted(cu, t, right=True) - 1, max=B - 1)
    live = (t < cu[B]) & ok[owner]
    at = torch.where(live, lens[owner] + t - cu[owner], 0)
    slots = torch.where(live, table[owner, at // page].long() * page + at % page, -1)
    return {"table": table, "seqlens": torch.where(ok, lens + new, lens).int(), "cu_new": cu.int(),
            "slots": slots.int(), "positions": torch.where(live, at, -1).int(), "n_left": (n_free - taken).int()}


def _angles(positions, d, base):
    """cos and sin of the rotation angles [n, d / 2] (the angle in 64 bits: positions are large)."""
    theta = base ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    a = positions.double()[:, None] * theta[None, :]
    return a.cos().float(), a.sin().float()


def _rotate(x, positions, base, half):
    """x [n, heads, d] in 32 bits, rotated at the positions [n]."""
    if base <= 0:
        return x
    c, s = (t[:, None, :] for t in _angles(positions, x.shape[-1], base))
    if half:
        x0, x1 = x[..., : x.shape[-1] // 2], x[..., x.shape[-1] // 2:]
        return torch.cat([x0 * c - x1 * s, x0 * s + x1 * c], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], -1).flatten(-2)


def _plain_append(case, s):
    k = _rotate(s["k"].float(), s["positions"], case["base"], case["half"]).to(s["k"].dtype)
    at = s["slots"].long()
    live = at >= 0
    # rows without a slot write the first row's values to the first row's slot once more
    src = torch.where(live, torch.arange(at.numel(), device=DEV), 0)
    at = at[src]
    s["k_pages"].view(-1, case["n_kv"], case["d"])[at] = k[src]
    s["v_pages"].view(-1, case["n_kv"], case["d"])[at] = s["v"][src]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(case, s):
    B, n_h, n_kv, d, page, prefix = (case[x] for x in ("B", "n_h", "n_kv", "d", "page", "prefix"))
    G = n_h // n_kv
    lens = s["lens"].long()
    q = _rotate(s["q"].float(), torch.clamp(lens - 1, min=0), case["base"], False).view(B, n_kv, G, d) / math.sqrt(d)
    tail = s["table"][:, prefix // page:].long().clamp(min=0)  # pages of each request behind the prefix
    k = s["k_pages"][tail].float().view(B, -1, n_kv, d).permute(0, 2, 3, 1)
    v = s["v_pages"][tail].float().view(B, -1, n_kv, d).permute(0, 2, 1, 3)
    score = q @ k  # [B, n_kv, G, n]
    seen = prefix + torch.arange(k.shape[-1], device=DEV)[None, :] < lens[:, None]
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    v = v * seen[:, None, :, None]
    if prefix:
        pages = s["prefix_pages"].long()
        pk = s["k_pages"][pages].float().view(prefix, n_kv, d).permute(1, 2, 0)
        pv = s["v_pages"][pages].float().view(prefix, n_kv, d).permute(1, 0, 2)
        rows = q.permute(1, 0, 2, 3).reshape(n_kv, B * G, d)
        both = (rows @ pk).view(n_kv, B, G, prefix).permute(1, 0, 2, 3)
        score = torch.cat([both, score], -1)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = p[..., prefix:] @ v
    if prefix:
        rows = p[..., :prefix].permute(1, 0, 2, 3).reshape(n_kv, B * G, prefix)
        out = out + (rows @ pv).view(n_kv, B, G, d).permute(1, 0, 2, 3)
    out = torch.where((lens > prefix)[:, None, None, None], out / total, 0.0)
    return {"out": out.reshape(B, n_h, d).to(s["q"].dtype)}


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "decode": _exact_attend,
            "shared": _exact_attend}[case["op"]](case, s)


def _exact_plan(case, s):
    """Request after request, as one would by hand."""
    page, N = case["page"], s["max_tokens"]
    table, free = s["table"].tolist(), s["free"].tolist()
    width, left = len(table[0]), int(s["n_free"][0])
    start, seqlens, cu, slots, positions = left, [], [0], [-1] * N, [-1] * N
    asked = 0
    for row, n, more in zip(table, s["lens"].tolist(), s["new"].tolist()):
        first = cu[-1]
        cu.append(first + more)
        have, want = -(-n // page), -(-(n + more) // page)
        fits = want <= width and first + more <= N
        if fits:
            asked += want - have
        if not fits or (want > have and asked > start):
            seqlens.append(n)
            continue
        for c in range(have, want):
            left -= 1
            row[c] = free[left]
        for i in range(more):
            slots[first + i] = row[(n + i) // page] * page + (n + i) % page
            positions[first + i] = n + i
        seqlens.append(n + more)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).to(DEV)

    return {"table": ints(table), "seqlens": ints(seqlens), "cu_new": ints(cu), "slots": ints(slots),
            "positions": ints(positions), "n_left": ints([left])}


def _exact_append(case, s):
    n, d = case["T"], case["d"]
    x, at = s["k"][:n].double(), s["slots"][:n].long()
    if case["base"] > 0:
        # each pair of dims as a complex number, multiplied by exp(i * position * theta)
        pair = torch.arange(d // 2, device=DEV)
        a, b = (pair, pair + d // 2) if case["half"] else (2 * pair, 2 * pair + 1)
        turn = s["positions"][:n].double()[:, None] * torch.pow(torch.tensor(case["base"], dtype=torch.float64, device=DEV),
                                                                -2.0 * pair.double() / d)[None, :]
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(turn), turn)[:, None, :]
        x = x.clone()
        x[..., a], x[..., b] = z.real, z.imag
    k, v = s["k_pages"].double().flatten(0, 1), s["v_pages"].double().flatten(0, 1)
    k[at], v[at] = x, s["v"][:n].double()
    return {"k_pages": k.view(s["k_pages"].shape), "v_pages": v.view(s["v_pages"].shape)}


def _exact_attend(case, s):
    n_h, n_kv, d, page = (case[x] for x in ("n_h", "n_kv", "d", "page"))
    q, out = s["q"].double(), torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    pair = torch.arange(d // 2, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, : _pages_of(n, page)].long()
        k = s["k_pages"][pages].flatten(0, 1)[:n].double()
        v = s["v_pages"][pages].flatten(0, 1)[:n].double()
        x = q[b]
        if case["base"] > 0:
            turn = (n - 1) * torch.pow(torch.tensor(case["base"], dtype=torch.float64, device=DEV), -2.0 * pair.double() / d)
            z = torch.complex(x[:, 0::2].contiguous(), x[:, 1::2].contiguous()) * torch.polar(torch.ones_like(turn), turn)
            x = torch.view_as_real(z).flatten(1)
        score = torch.einsum("gid,ngd->gin", x.view(n_kv, n_h // n_kv, d), k) / math.sqrt(d)
        p = torch.exp(score - torch.logsumexp(score, -1, keepdim=True))
        out[b] = torch.einsum("gin,ngd->gid", p, v).reshape(n_h, d)
    return {"out": out}


def work(case):
    page = case["page"]
    if case["op"] == "plan":
        lens, new, B = _spread(case["lo"], case["hi"], case["B"]), _spread(1, case["new"], case["B"]), case["B"]
        taken = sum(_pages_of(a + b, page) - _pages_of(a, page) for a, b in zip(lens, new))
        # lengths in, open pages' entries, lengths and offsets out; ids of new pages in and out; slot and position out
        return {"bytes": 20 * B + 8 * taken + 8 * sum(new), "flops": 10 * sum(new)}
    size = 2 if case["dtype"] == "bf16" else 4
    row = case["n_kv"] * case["d"] * size
    if case["op"] == "append":
        return {"bytes": case["T"] * (4 * row + 8), "flops": 3 * case["T"] * case["n_kv"] * case["d"]}
    lens, prefix = _lengths(case), case["prefix"]
    keys = prefix + sum(n - prefix for n in lens)
    return {"bytes": 2 * keys * row + 2 * case["B"] * case["n_h"] * case["d"] * size + 4 * _pages_of(keys, page),
            "flops": 4 * sum(lens) * case["n_h"] * case["d"]}
