"""Plain references, in 64 bits, of the steps that add several tokens per request (test infrastructure)."""
from __future__ import annotations

import numpy as np

import oracle


def lineage(parents):
    """For each token its ancestors and itself; None where the walk to a root breaks."""
    lines = []
    for i, p in enumerate(parents):
        if p == -1:
            lines.append([i])
        elif 0 <= p < i and lines[p] is not None:
            lines.append(lines[p] + [i])
        else:
            lines.append(None)
    return lines


def random_tree(n, rng, back=8, roots=0.05):
    """Parents of n drafted tokens: now and then a root, else one of the `back` tokens before."""
    return [-1 if i == 0 or rng.random() < roots else max(0, i - int(rng.integers(1, back + 1))) for i in range(n)]


def draft_plan(places, cu, parents, words):
    T = len(places)
    positions, visible = np.full(T, -1, np.int64), np.zeros((T, words), np.uint32)
    for b in range(len(cu) - 1):
        lo, hi = min(cu[b], T), min(cu[b + 1], T)
        for i, line in enumerate(lineage(list(parents[lo:hi]))):
            if line is None or i >= 32 * words or places[lo + i] < 0:
                continue
            positions[lo + i] = places[lo + i] - i + len(line) - 1
            for j in line:
                visible[lo + i, j // 32] |= np.uint32(1 << (j % 32))
    return positions, visible.view(np.int32)


def causal(new, ctx):
    """bool [new, new + ctx]: what each new token of a request sees."""
    return np.arange(new + ctx)[None] <= ctx + np.arange(new)[:, None]


def tree(new, ctx, visible):
    """The same from rows of visibility bits int32 [new, words]."""
    bits = np.unpackbits(np.ascontiguousarray(visible).view(np.uint8), axis=1, bitorder="little").astype(bool)
    drafts = np.zeros((new, new), bool)
    w = min(new, bits.shape[1])
    drafts[:, :w] = bits[:, :w]
    return np.concatenate([np.ones((new, ctx), bool), drafts], 1)


def attend(q, positions, sees, k, v, *, rope_base=0.0, rope_offset=0, rope_dims=None, scale=None, pairing="adjacent"):
    """One request: q [n, n_h, D], positions [n], sees bool [n, L], k [L, n_kv, D], v [L, n_kv, D_v], in float64.

    (out, lse, spread, err): rows that see nothing or have a negative position get 0 and -inf; spread is sum p |v|,
    err a bound of a score's error when the rotated query is rounded to bf16: half a step (2^-8) of every term of
    the largest dot product."""
    n, n_h, D = q.shape
    n_kv, D_v = k.shape[1], v.shape[2]
    G = n_h // n_kv
    sc = oracle.attention.default_scale(D, scale)
    qr = q
    if rope_base > 0:
        at = np.maximum(positions, 0)
        qr = np.stack([oracle.rope_rotate(q[:, h], at, rope_base, rope_offset, rope_dims, pairing=pairing)
                       for h in range(n_h)], 1)
    sees = sees & (np.asarray(positions) >= 0)[:, None]
    out, spread = np.zeros((n, n_h, D_v)), np.zeros((n, n_h, D_v))
    lse, err = np.full((n, n_h), -np.inf), np.zeros((n, n_h))
    for h in range(n_h):
        kh, vh = k[:, h // G], v[:, h // G]
        with np.errstate(all="ignore"):
            s = np.where(sees, qr[:, h] @ kh.T * sc, -np.inf)
        top = s.max(1, initial=-np.inf)
        live = top > -np.inf
        p = np.exp(s[live] - top[live, None])
        total = p.sum(1)
        lse[live, h] = top[live] + np.log(total)
        p /= total[:, None]
        out[live, h], spread[live, h] = p @ vh, p @ np.abs(vh)
        if rope_base > 0 and kh.shape[0]:
            err[:, h] = sc * 2.0 ** -8 * (np.abs(qr[:, h]) @ np.abs(kh).T).max(1)
    return out, lse, spread, err


def commit(lens, seqlens, path, n_path, table, page, n_pages, free, n_free, cap):
    """(new_lens, moves [(from slot, to slot)] per request, free, n_left)."""
    width = len(table[0])
    new_lens, moves, free, left = [], [], list(free), None if n_free is None else max(0, min(n_free, cap))
    for b in range(len(lens)):
        held, L = max(int(lens[b]), 0), min(max(int(seqlens[b]), 0), width * page)
        mine, last = [], -1
        for i in range(min(max(int(n_path[b]), 0), len(path[b]))):
            j = int(path[b][i])
            if j <= last or j < 0 or held + j >= L:
                break
            last = j
            p, q = int(table[b][(held + j) // page]), int(table[b][(held + i) // page])
            mine.append((p * page + (held + j) % page, q * page + (held + i) % page)
                        if 0 <= p < n_pages and 0 <= q < n_pages else None)
        new_lens.append(held + len(mine))
        moves.append([m for m in mine if m is not None])
        if left is not None:
            for j in range(-(-new_lens[-1] // page), -(-L // page)):
                if left < cap:
                    free[left] = int(table[b][j])
                    left += 1
    return new_lens, moves, free, left
