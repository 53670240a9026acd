"""Steps that add several tokens per request over the paged cache, as measured: cases, inputs, plain forms, 64-bit values.

A step's new tokens are packed, request b's n_b being rows cu_new[b] .. of q; they are in the cache already, at the
last n_b of its seqlens[b] places.  Four operators:

* prefill - prefill_paged: packed prompts, or chunks of them behind what the cache holds, causal
* tree    - decode_tree: drafted tokens that form a tree, each seeing the cache in front of the drafts, its ancestors
            and itself
* plan    - draft_plan: positions and visibility bits of drafted tokens from their parents
* commit  - draft_commit: the accepted drafts move to consecutive places, and pages that fall free go back
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attend(name, op, B, lo, hi, ctx_lo, ctx_hi, pad, n_h, n_kv, d, page, base, half, dtype):
    """B requests with lo..hi new tokens each behind ctx_lo..ctx_hi cached ones; pad rows behind the last request."""
    return {"name": name, "op": op, "B": B, "lo": lo, "hi": hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "pad": pad,
            "n_h": n_h, "n_kv": n_kv, "d": d, "page": page, "base": base, "half": half, "dtype": dtype}


def _plan(name, B, lo, hi, pad):
    """B requests with lo..hi drafted tokens each."""
    return {"name": name, "op": "plan", "B": B, "lo": lo, "hi": hi, "pad": pad}


def _commit(name, B, n, ctx_lo, ctx_hi, n_kv, d, page, dtype):
    """B requests of ctx_lo..ctx_hi tokens with n drafted ones each, of which the path to some leaf is accepted."""
    return {"name": name, "op": "commit", "B": B, "n": n, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "n_kv": n_kv, "d": d,
            "page": page, "dtype": dtype}


def listed():
    return [
        # one short chat message (latency of a single prompt)
        _attend("prefill_one_short", "prefill", 1, 77, 77, 0, 0, 0, 32, 8, 128, 16, 500000.0, False, "bf16"),
        # prompts of very different lengths admitted in one step, in a padded buffer
        _attend("prefill_16_prompts", "prefill", 16, 33, 2001, 0, 0, 100, 32, 8, 128, 64, 500000.0, False, "bf16"),
        # two long documents read in chunks: 2048 new tokens behind some thirty thousand
        _attend("prefill_2_chunks", "prefill", 2, 2048, 2048, 28672, 30720, 0, 32, 8, 128, 64, 500000.0, False, "bf16"),
        # four prompts of 8192 tokens (tensor cores)
        _attend("prefill_4x8192", "prefill", 4, 8192, 8192, 0, 0, 0, 32, 8, 128, 64, 500000.0, False, "bf16"),
        # a small full-precision model with as many KV heads as heads
        _attend("prefill_f32_mha", "prefill", 8, 1, 500, 0, 100, 3, 12, 12, 64, 32, 0.0, False, "f32"),
        # one chat whose next 25 tokens are drafted (latency)
        _attend("tree_one", "tree", 1, 25, 25, 900, 900, 0, 32, 8, 128, 16, 500000.0, False, "bf16"),
        # the 59-request decode batch with 32 drafted tokens each (HBM)
        _attend("tree_59_requests", "tree", 59, 32, 32, 4096, 8192, 0, 32, 8, 128, 64, 500000.0, False, "bf16"),
        # two long documents with large trees in 16-token pages: the key axis has to be split
        _attend("tree_2_long", "tree", 2, 60, 64, 98001, 131000, 4, 32, 8, 128, 16, 500000.0, True, "bf16"),
        # the plan of the 59-request step (latency)
        _plan("plan_59", 59, 32, 32, 0),
        # large trees for many requests
        _plan("plan_512", 512, 1, 100, 64),
        # the end of the 59-request step (latency)
        _commit("commit_59", 59, 32, 500, 1000, 8, 128, 64, "bf16"),
        # the same for many requests, in small pages
        _commit("commit_512", 512, 48, 1, 300, 8, 128, 16, "bf16"),
    ]


HEADS = [(32, 8), (12, 12), (8, 1), (28, 4), (16, 8), (40, 8), (6, 2)]
MOST = 4 * 4 * 128 * 32 * (8192 * 8193 // 2)  # flop of the largest listed case


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "tree", "tree", "plan", "commit"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        hi = _log(rng, 1, 128)
        case = _plan("", _log(rng, 1, 1024), rng.randint(1, hi), hi, rng.choice([0, 0, 1, 50]))
    elif op == "commit":
        n_kv, d = rng.choice([(8, 128), (4, 64), (1, 128), (12, 64)])
        ctx = _log(rng, 1, 1000)
        case = _commit("", _log(rng, 1, 512), _log(rng, 1, 128), rng.randint(0, ctx), ctx, n_kv, d, page,
                       "f32" if rng.random() < 0.2 else "bf16")
    else:
        n_h, n_kv = rng.choice(HEADS)
        d = rng.choice([64, 128, 128])
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        most = MOST // 200 if dtype == "f32" else MOST // 2
        B = _log(rng, 1, 64)
        if op == "prefill":
            hi = _log(rng, 1, 8192)
            ctx = 0 if rng.random() < 0.5 else _log(rng, 1, 32768)
        else:
            hi = _log(rng, 1, 128)
            ctx = _log(rng, 1, 65536)
        while B > 1 and (B * hi * (ctx + hi) * 4 * n_h * d > most or B * (ctx + hi) > 400000):
            B = (B + 1) // 2
        while hi > 1 and B * hi * (ctx + hi) * 4 * n_h * d > most:
            hi = (hi + 1) // 2
        case = _attend("", op, B, rng.randint(1, hi), hi, rng.randint(0, ctx), ctx, rng.choice([0, 0, 1, 37]), n_h,
                       n_kv, d, page, rng.choice([0.0, 10000.0, 500000.0]), rng.random() < 0.5, dtype)
    return {k: v for k, v in case.items() if k != "name"}


def _spread(lo, hi, n):
    """n numbers from lo to hi, evenly spread (so that the work does not depend on the seed)."""
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)] if n > 1 else [hi] * n


def _requests(case):
    """(new tokens, tokens in front of them) of each request: the most new ones behind the fewest."""
    return list(zip(_spread(case["lo"], case["hi"], case["B"]), _spread(case["ctx_lo"], case["ctx_hi"], case["B"])[::-1]))


def _pages_of(n, page):
    return (n + page - 1) // page


def _words(case):
    """32-bit words of a visibility row."""
    return (case["hi"] + 31) // 32


def _tree(n, gc):
    """Parents of n drafted tokens: the first is the tree's root, later ones hang from one of the ten before them."""
    back = torch.randint(1, 11, (n,), generator=gc).tolist()
    return [-1] + [max(0, i - back[i]) for i in range(1, n)]


def _lineage(parents):
    """For each token its ancestors and itself, in rising order."""
    lines = []
    for i, p in enumerate(parents):
        lines.append((lines[p] if p >= 0 else []) + [i])
    return lines


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32).to(DEV)

    B = case["B"]
    if case["op"] == "plan":
        counts = [_spread(case["lo"], case["hi"], B)[i] for i in torch.randperm(B, generator=gc).tolist()]
        held = torch.randint(0, 8192, (B,), generator=gc).tolist()
        parents = [_tree(n, gc) for n in counts]
        places = [held[b] + i for b in range(B) for i in range(counts[b])]
        return {"case": case, "host": parents, "parents": ints(sum(parents, []) + [-1] * case["pad"]),
                "places": ints(places + [-1] * case["pad"]),
                "cu": ints([0] + torch.tensor(counts).cumsum(0).tolist())}
    page, n_kv, d = case["page"], case["n_kv"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(TYPES[case["dtype"]])

    if case["op"] == "commit":
        requests = [(case["n"], c) for c in _spread(case["ctx_lo"], case["ctx_hi"], B)]
    else:
        requests = _requests(case)
    requests = [requests[i] for i in torch.randperm(B, generator=gc).tolist()]
    pages = [_pages_of(n + c, page) for n, c in requests]
    n_pages, width = sum(pages) + 2, max(pages)
    order = torch.randperm(n_pages, generator=gc).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[torch.arange(width)[None, :] < torch.tensor(pages)[:, None]] = order[: n_pages - 2]
    s = {"case": case, "host": requests, "table": table.to(DEV), "lens": ints([n + c for n, c in requests]),
         "k_pages": normal(n_pages, page, n_kv, d), "v_pages": normal(n_pages, page, n_kv, d)}
    if case["op"] == "commit":
        lines = [_lineage(_tree(n, gc)) for n, _ in requests]
        leaf = torch.randint(0, case["n"], (B,), generator=gc).tolist()
        paths = [line[i] for line, i in zip(lines, leaf)]
        most = max(len(p) for p in paths)
        s.update(held=ints([c for _, c in requests]), path=ints([p + [-1] * (most - len(p)) for p in paths]),
                 n_path=ints([len(p) for p in paths]), paths=paths,
                 free=torch.cat([order[n_pages - 2:], torch.full((n_pages - 2,), -1, dtype=torch.int32)]).to(DEV),
                 n_free=ints([2]))
        return s
    cu = [0]
    for n, _ in requests:
        cu.append(cu[-1] + n)
    s.update(q=normal(cu[-1] + case["pad"], case["n_h"], d), cu=ints(cu))
    if case["op"] == "tree":
        s["parents"] = [_tree(n, gc) for n, _ in requests]
        words = [[0] * _words(case) for _ in range(cu[-1] + case["pad"])]
        positions = [-1] * (cu[-1] + case["pad"])
        for b, (n, c) in enumerate(requests):
            for i, line in enumerate(_lineage(s["parents"][b])):
                positions[cu[b] + i] = c + len(line) - 1
                for j in line:
                    words[cu[b] + i][j // 32] |= 1 << (j % 32)
        s["positions"] = ints(positions)
        s["visible"] = torch.tensor([[w - (1 << 32) if w >> 31 else w for w in row] for row in words],
                                    dtype=torch.int32).to(DEV)
    else:
        s["positions"] = ints([c + i for n, c in requests for i in range(n)] + [-1] * case["pad"])
    return s


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"prefill": _plain_attend, "tree": _plain_attend, "plan": _plain_plan, "commit": _plain_commit}[case["op"]](
        case, state)


def _own(case, s):
    import transformer_causal_attention_gb300 as attn

    if case["op"] == "plan":
        positions, visible = attn.draft_plan(s["places"], s["cu"], s["parents"], words=_words(case))
        return {"positions": positions, "visible": visible}
    if case["op"] == "commit":
        seqlens, n_left = attn.draft_commit(s["k_pages"], s["v_pages"], s["table"], s["held"], s["lens"], s["path"],
                                            s["n_path"], s["free"], s["n_free"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "seqlens": seqlens, "free": s["free"],
                "n_left": n_left}
    pairing = "half" if case["half"] else "adjacent"
    if case["op"] == "prefill":
        out, _ = attn.prefill_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"],
                                    s["positions"], rope_base=case["base"], pairing=pairing)
    else:
        out, _ = attn.decode_tree(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], s["positions"],
                                  s["visible"], rope_base=case["base"], pairing=pairing)
    return {"out": out}


# ------------------------------------------------------------------------------------------ plain forms
def _rotate(x, positions, base, half):
    """x [n, heads, d] in 32 bits, rotated at the positions [n] (the angle in 64 bits: positions are large)."""
    if base <= 0:
        return x
    d = x.shape[-1]
    theta = base ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    a = positions.double()[:, None] * theta[None, :]
    c, s = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    if half:
        x0, x1 = x[..., : d // 2], x[..., d // 2:]
        return torch.cat([x0 * c - x1 * s, x0 * s + x1 * c], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], -1).flatten(-2)


def _plain_attend(case, s):
    n_h, n_kv, d, page = case["n_h"], case["n_kv"], case["d"], case["page"]
    G = n_h // n_kv
    q = _rotate(s["q"].float(), torch.clamp(s["positions"], min=0), case["base"], case["half"]) / math.sqrt(d)
    out = torch.zeros(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    first = 0
    for b, (n, ctx) in enumerate(s["host"]):
        L = n + ctx
        pages = s["table"][b, : _pages_of(L, page)].long()
        k = s["k_pages"][pages].flatten(0, 1)[:L].float().permute(1, 2, 0)  # [n_kv, d, L]
        v = s["v_pages"][pages].flatten(0, 1)[:L].float().permute(1, 0, 2)  # [n_kv, L, d]
        rows = max(1, (1 << 31) // (n_h * L))  # new tokens at a time
        for i in range(0, n, rows):
            m = min(rows, n - i)
            x = q[first + i:first + i + m].view(m, n_kv, G, d).permute(1, 2, 0, 3).reshape(n_kv, G * m, d)
            score = (x @ k).view(n_kv, G, m, L)
            at = torch.arange(L, device=DEV)[None, :]
            if case["op"] == "prefill":
                seen = at <= ctx + torch.arange(i, i + m, device=DEV)[:, None]
            else:
                draft = (at - ctx).clamp(min=0)
                word = s["visible"][first + i:first + i + m].gather(1, (draft // 32).expand(m, L).long())
                seen = (at < ctx) | (((word >> (draft % 32)) & 1) != 0)
            score.masked_fill_(~seen, -math.inf)
            p = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
            o = (p.view(n_kv, G * m, L) @ v).view(n_kv, G, m, d) / p.sum(-1, keepdim=True)
            out[first + i:first + i + m] = o.permute(2, 0, 1, 3).reshape(m, n_h, d).to(out.dtype)
        first += n
    return {"out": out}


def _plain_plan(case, s):
    cu, places, parents = s["cu"].long(), s["places"].long(), s["parents"].long()
    N, W = places.numel(), _words(case)
    t = torch.arange(N, device=DEV)
    owner = torch.searchsorted(cu, t, right=True) - 1
    live = (t < cu[-1]) & (places >= 0)
    first = cu[torch.clamp(owner, max=cu.numel() - 2)]
    depth = torch.full((N,), -1, dtype=torch.long, device=DEV)
    seen = torch.zeros(N, W * 32, dtype=torch.int64, device=DEV)
    at = torch.where(live, t - first, -1)  # the token, its parent, ... within its request; -1 past the root
    for _ in range(W * 32):
        on = at >= 0
        seen.scatter_add_(1, at.clamp(min=0)[:, None], on.long()[:, None])
        depth += on
        at = torch.where(on, parents[torch.clamp(first + at, 0, N - 1)], -1)
    bits = (seen.view(N, W, 32) << torch.arange(32, device=DEV)).sum(-1)
    visible = torch.where(bits >= 1 << 31, bits - (1 << 32), bits)
    return {"positions": torch.where(live, places - (t - first) + depth, -1).int(), "visible": visible.int()}


def _plain_commit(case, s):
    page, table = case["page"], s["table"].long()
    held, lens, n_path = s["held"].long(), s["lens"].long(), s["n_path"].long()
    k, v = s["k_pages"].flatten(0, 1), s["v_pages"].flatten(0, 1)
    i = torch.arange(s["path"].shape[1], device=DEV)[None, :]
    live = i < n_path[:, None]

    def slots(at):
        at = torch.where(live, at, 0)
        return table.gather(1, at // page) * page + at % page

    src, dst = slots(held[:, None] + s["path"].long())[live], slots(held[:, None] + i)[live]
    k[dst], v[dst] = k[src], v[src]
    seqlens = held + n_path
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    back = (col >= ((seqlens + page - 1) // page)[:, None]) & (col < ((lens + page - 1) // page)[:, None])
    released = s["table"][back]
    n = int(released.numel())
    s["free"][2:2 + n] = released  # the stack holds two pages
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "seqlens": seqlens.int(), "free": s["free"],
            "n_left": s["n_free"] + n}


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"prefill": _exact_attend, "tree": _exact_attend, "plan": _exact_plan, "commit": _exact_commit}[case["op"]](
        case, s)


def _exact_attend(case, s):
    n_h, n_kv, d, page = case["n_h"], case["n_kv"], case["d"], case["page"]
    G = n_h // n_kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    pair = torch.arange(d // 2, device=DEV)
    x0, x1 = (pair, pair + d // 2) if case["half"] else (2 * pair, 2 * pair + 1)
    first = 0
    for b, (n, ctx) in enumerate(s["host"]):
        pages = s["table"][b, : _pages_of(n + ctx, page)].long()
        k = s["k_pages"][pages].flatten(0, 1)[: n + ctx].double()
        v = s["v_pages"][pages].flatten(0, 1)[: n + ctx].double()
        x = s["q"][first:first + n].double()
        if case["op"] == "prefill":
            place = torch.arange(ctx, ctx + n, dtype=torch.float64, device=DEV)
        else:
            lines = _lineage(s["parents"][b])
            place = torch.tensor([ctx + len(line) - 1 for line in lines], dtype=torch.float64, device=DEV)
            seen = torch.zeros(n, n, dtype=torch.bool)
            for i, line in enumerate(lines):
                seen[i, line] = True
            seen = seen.to(DEV)
        if case["base"] > 0:
            # each pair of dims as a complex number, multiplied by exp(i * position * theta)
            rate = torch.pow(torch.tensor(case["base"], dtype=torch.float64, device=DEV), -2.0 * pair.double() / d)
            turn = place[:, None] * rate[None, :]
            z = torch.complex(x[..., x0], x[..., x1]) * torch.polar(torch.ones_like(turn), turn)[:, None, :]
            x = x.clone()
            x[..., x0], x[..., x1] = z.real, z.imag
        step = max(1, (1 << 28) // (n_h * (n + ctx)))
        for i in range(0, n, step):
            m = min(step, n - i)
            last = ctx + i + m if case["op"] == "prefill" else ctx + n  # keys that these rows may see
            score = torch.einsum("igjd,ngd->gjin", x[i:i + m].view(m, n_kv, G, d), k[:last]) / math.sqrt(d)
            if case["op"] == "prefill":
                hide = torch.ones(m, last, dtype=torch.bool, device=DEV).triu(ctx + i + 1)
            else:
                hide = torch.cat([torch.zeros(m, ctx, dtype=torch.bool, device=DEV), ~seen[i:i + m]], 1)
            score = score.masked_fill_(hide, -math.inf)
            p = score.sub_(torch.logsumexp(score, -1, keepdim=True)).exp_()
            out[first + i:first + i + m] = torch.einsum("gjin,ngd->igjd", p, v[:last]).reshape(m, n_h, d)
        first += n
    return {"out": out}


def _exact_plan(case, s):
    """Token after token, as one would by hand."""
    positions, words, places = [], [], s["places"].tolist()
    for parents in s["host"]:
        base = places[len(positions)]
        for line in _lineage(parents):
            positions.append(base + len(line) - 1)
            row = [sum(1 << (j % 32) for j in line if j // 32 == w) for w in range(_words(case))]
            words.append([w - (1 << 32) if w >> 31 else w for w in row])
    positions += [-1] * case["pad"]
    words += [[0] * _words(case)] * case["pad"]
    return {"positions": torch.tensor(positions, dtype=torch.int32).to(DEV),
            "visible": torch.tensor(words, dtype=torch.int32).to(DEV)}


def _exact_commit(case, s):
    page = case["page"]
    k, v = s["k_pages"].double().flatten(0, 1), s["v_pages"].double().flatten(0, 1)
    table, held = s["table"].tolist(), s["held"].tolist()
    free, left = s["free"].tolist(), int(s["n_free"][0])
    src, dst, seqlens = [], [], []
    for b, (path, (n, ctx)) in enumerate(zip(s["paths"], s["host"])):
        assert held[b] == ctx
        for i, j in enumerate(path):
            src.append(table[b][(ctx + j) // page] * page + (ctx + j) % page)
            dst.append(table[b][(ctx + i) // page] * page + (ctx + i) % page)
        seqlens.append(ctx + len(path))
        for j in range(_pages_of(seqlens[-1], page), _pages_of(n + ctx, page)):
            free[left] = table[b][j]
            left += 1
    k[dst], v[dst] = k[src], v[src]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).to(DEV)

    return {"k_pages": k.view(s["k_pages"].shape), "v_pages": v.view(s["v_pages"].shape), "seqlens": ints(seqlens),
            "free": ints(free), "n_left": ints([left])}


def work(case):
    if case["op"] == "plan":
        tokens = sum(_spread(case["lo"], case["hi"], case["B"]))
        # parents, places and offsets in; positions and visibility out
        return {"bytes": 4 * case["B"] + (12 + 4 * _words(case)) * (tokens + case["pad"]), "flops": 10 * tokens}
    size = 2 if case["dtype"] == "bf16" else 4
    row = case["n_kv"] * case["d"] * size
    if case["op"] == "commit":
        # about a fifth of the drafts on a path, each read and written once
        moved = case["B"] * max(1, case["n"] // 5)
        return {"bytes": 4 * row * moved + 16 * case["B"], "flops": moved}
    requests = _requests(case)
    tokens, keys = sum(n for n, _ in requests), sum(n + c for n, c in requests)
    pairs = sum(n * c + (n * (n + 1) // 2 if case["op"] == "prefill" else n) for n, c in requests)
    return {"bytes": 2 * keys * row + 2 * tokens * case["n_h"] * case["d"] * size
            + 4 * _pages_of(keys, case["page"]), "flops": 4 * pairs * case["n_h"] * case["d"]}
