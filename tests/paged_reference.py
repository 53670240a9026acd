"""Plain references of the paged-cache calls, and builders of paged caches (test infrastructure).

plan() walks the requests one after the other, as one would by hand; attend() gathers each request's
keys into one array and hands it to the fp64 oracle.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle


def plan(lens, n_new, table, free, n_free, page, n_pages, max_tokens):
    """(table, seqlens, cu_new, slots, positions, n_left) as int lists / arrays; nothing is changed in place."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    top = left = max(0, min(int(n_free), len(free)))
    seqlens, cu = [], [0]
    slots, positions = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int64)
    asked = 0
    for b, (n, more) in enumerate(zip(lens, n_new)):
        n, more = max(int(n), 0), max(int(more), 0)
        first = cu[-1]
        cu.append(first + more)
        have, want = -(-n // page), -(-(n + more) // page)
        if n + more > width * page or first + more > max_tokens:
            seqlens.append(n)
            continue
        asked += want - have
        if want > have and asked > top:
            seqlens.append(n)
            continue
        for c in range(have, want):
            left -= 1
            table[b, c] = free[left]
        for i in range(more):
            pos = n + i
            pg = int(table[b, pos // page])
            positions[first + i] = pos
            slots[first + i] = pg * page + pos % page if 0 <= pg < n_pages else -1
        seqlens.append(n + more)
    return table, seqlens, [min(c, 2**31 - 1) for c in cu], slots, positions, left


def make_cache(lens, prefix, page, n_kv, D_qk, D_v, dtype, seed=0, alias=False, spare=3, fill=float("nan")):
    """A shuffled paged cache of requests of the given lengths (the first `prefix` tokens shared; lengths of at most
    `prefix` own nothing).  Rows that hold no token, and spare pages, are filled with `fill`.

    Returns (k_pages, v_pages, table, prefix_pages, k_of, v_of): CPU tensors, and per request the float64 keys and
    values in order."""
    g = torch.Generator().manual_seed(seed)
    n_shared = prefix // page
    own = [max(0, -(-int(n) // page) - n_shared) for n in lens]
    n_pages = n_shared + sum(own) + spare
    order = torch.randperm(n_pages, generator=g)
    width = max(1, n_shared + max(own + [0]))
    table = torch.full((len(lens), width), -7, dtype=torch.int32)  # never read where no page is owned
    k = torch.full((n_pages, page, n_kv, D_qk), fill, dtype=dtype)
    v = k[..., :D_v] if alias else torch.full((n_pages, page, n_kv, D_v), fill, dtype=dtype)

    def write(page_id, n_rows):
        k[page_id, :n_rows] = torch.randn(n_rows, n_kv, D_qk, generator=g).to(dtype)
        if not alias:
            v[page_id, :n_rows] = torch.randn(n_rows, n_kv, D_v, generator=g).to(dtype)

    for j in range(n_shared):
        write(order[j], page)
    at = n_shared
    for b, n in enumerate(lens):
        for j in range(own[b]):
            write(order[at], min(page, int(n) - (n_shared + j) * page))
            table[b, n_shared + j] = order[at]
            at += 1
    prefix_pages = order[:n_shared].to(torch.int32)
    k_of, v_of = [], []
    for b, n in enumerate(lens):
        pages = torch.cat([prefix_pages, table[b, n_shared:n_shared + own[b]]]).long()
        n = int(n) if int(n) > prefix else 0
        k_of.append(k[pages].reshape(-1, n_kv, D_qk)[:n].double().numpy())
        v_of.append(v[pages].reshape(-1, n_kv, D_v)[:n].double().numpy())
    return k, v, table, prefix_pages, k_of, v_of


def attend(q, k_of, v_of, *, rope_base=0.0, rope_offset=0, rope_dims=None, scale=None, pairing="adjacent"):
    """(out, lse, err): the fp64 result per request (0 and -inf without keys), and a bound of the score's error when
    the rotated query is rounded to bf16: half a step (2^-8) of every term of the largest dot product."""
    B, n_h, D_qk = q.shape
    n_kv, D_v = k_of[0].shape[1], v_of[0].shape[2]
    out = np.zeros((B, n_h, D_v))
    lse = np.full((B, n_h), -np.inf)
    err = np.zeros((B, n_h))
    for b in range(B):
        n = k_of[b].shape[0]
        if n == 0:
            continue
        o, l = oracle.attention_decode(q[b:b + 1], k_of[b][None], v_of[b][None], np.array([n]), rope_base=rope_base,
                                       rope_offset=rope_offset, rope_dims=rope_dims, scale=scale, pairing=pairing)
        out[b], lse[b] = o[0], l[0]
        if rope_base > 0:
            qr = np.abs(oracle.rope_rotate(q[b], np.full(n_h, n - 1), rope_base, rope_offset, rope_dims,
                                           pairing=pairing))
            g = n_h // n_kv
            dots = np.einsum("gid,ngd->gin", qr.reshape(n_kv, g, D_qk), np.abs(k_of[b])).max(-1).reshape(n_h)
            err[b] = oracle.attention.default_scale(D_qk, scale) * dots * 2.0 ** -8
    return out, lse, err
