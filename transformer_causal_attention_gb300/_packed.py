"""ctypes binding of the steps that add several tokens per request (include/attn_packed.h).

As in _paged.py, every function checks the tensors it is given, allocates the outputs
the caller does not pass, and forwards raw pointers; the calls run on the device of
their tensors, on the given stream or that device's current one.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _binding as _b
from ._paged import _NO_SIZE, _TAIL, _cuda, _ints, _on, _page_dims

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_SIZES = [_i] * 9  # T, B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks

# (name, restype, argtypes) of every symbol of include/attn_packed.h
SIGNATURES = [
    ("attn_packed_workspace_size", _sz, [_i] * 9),
    ("attn_prefill_paged", _i, [_vp, _vp, _vp, _i] + [_vp] * 6 + _SIZES + _TAIL),
    ("attn_decode_tree", _i, [_vp, _vp, _vp, _i] + [_vp] * 5 + [_i, _vp, _vp] + _SIZES + _TAIL),
    ("attn_draft_plan", _i, [_vp] * 5 + [_i] * 3 + [_vp]),
    ("attn_draft_commit", _i, [_vp, _vp, _i] + [_vp] * 9 + [_i] * 10 + [_vp]),
]

_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        lib = _b.load()
        for name, res, args in SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


@functools.lru_cache(maxsize=256)  # a serving loop asks with the same sizes step after step
def _workspace_size(*sizes) -> int:
    return _lib().attn_packed_workspace_size(*sizes)


def packed_workspace_size(T, B, n_h, n_kv, D_qk, D_v, page_size, max_blocks, dtype=torch.bfloat16) -> int:
    """Bytes of scratch of prefill_paged or decode_tree."""
    n = _workspace_size(T, B, n_h, n_kv, D_qk, D_v, page_size, max_blocks,
                        _b.ATTN_BF16 if dtype == torch.bfloat16 else _b.ATTN_F32)
    if n == _NO_SIZE:
        raise ValueError("invalid packed step sizes")
    return n


def _attend(q, k_pages, v_pages, block_table, cu_new, seqlens, positions, visible, rope_base, rope_offset, rope_dims,
            scale, out, lse, workspace, pairing, stream):
    device = _cuda(q, "q", None, None)
    _cuda(k_pages, "k_pages", q.dtype, device)
    n_pages, page_size, n_kv, D_qk, D_v, ldv = _page_dims(k_pages, v_pages, device)
    if q.dim() != 3 or q.shape[2] != D_qk:
        raise ValueError(f"q must be [T, n_h, {D_qk}]")
    T, n_h, _ = q.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, max_blocks = block_table.shape
    _cuda(block_table, "block_table", torch.int32, device)
    _ints(cu_new, "cu_new", (B + 1,), device)
    _ints(seqlens, "seqlens", (B,), device)
    if positions is not None:
        _ints(positions, "positions", (T,), device)
    if visible is not None:
        if visible.dim() != 2 or not 1 <= visible.shape[1] <= 4:
            raise ValueError("visible must be int32 [T, words], 1 <= words <= 4")
        _ints(visible, "visible", (T, visible.shape[1]), device)
    rope_dims = (D_qk - rope_offset) if rope_dims is None else rope_dims
    code = _b._dtype_code(q, pairing)
    lib = _lib()
    context, st = _on(device, stream)
    with context:
        if out is None:
            out = torch.empty((T, n_h, D_v), dtype=q.dtype, device=device)
        else:
            _cuda(out, "out", q.dtype, device)
            if out.shape != (T, n_h, D_v):
                raise ValueError(f"out must be [{T}, {n_h}, {D_v}]")
        if isinstance(lse, torch.Tensor):
            _cuda(lse, "lse", torch.float32, device)
            if lse.shape != (T, n_h):
                raise ValueError(f"lse must be fp32 [{T}, {n_h}]")
            lse_t = lse
        else:
            lse_t = torch.empty((T, n_h), dtype=torch.float32, device=device) if lse else None
        if T == 0:
            return out, lse_t
        if workspace is None:
            need = _workspace_size(T, B, n_h, n_kv, D_qk, D_v, page_size, max_blocks, code & 0xff)
            # invalid sizes: the call itself says what is wrong with them
            workspace = torch.empty(16 if need == _NO_SIZE else need, dtype=torch.uint8, device=device)
        else:
            _cuda(workspace, "workspace", None, device)
        head = (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), ldv, block_table.data_ptr(), cu_new.data_ptr(),
                seqlens.data_ptr(), _b._ptr(positions))
        tail = (out.data_ptr(), _b._ptr(lse_t), T, B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks, rope_base,
                rope_offset, rope_dims, scale, code, workspace.data_ptr(), workspace.nbytes, st)
        if visible is None:
            rc = lib.attn_prefill_paged(*head, *tail)
        else:
            rc = lib.attn_decode_tree(*head, visible.data_ptr(), visible.shape[1], *tail)
    _b._check(rc, "attn_prefill_paged" if visible is None else "attn_decode_tree")
    return out, lse_t


def prefill_paged(q, k_pages, v_pages, block_table, cu_new, seqlens, positions=None, *, rope_base: float = 0.0,
                  rope_offset: int = 0, rope_dims: int | None = None, scale: float = 0.0, out=None,
                  lse: bool | torch.Tensor = False, workspace=None, pairing: str = "adjacent", stream=None):
    """Causal attention of packed new tokens against a paged cache via attn_prefill_paged.

    q [T, n_h, D_qk] (un-rotated): request b's new tokens are rows cu_new[b] .. cu_new[b+1]
    - 1 (cu_new int32 [B+1]) and, already appended, the last of its seqlens[b] tokens
    (int32 [B]) in k_pages [n_pages, page_size, n_kv, D_qk] (rotated keys) and v_pages
    [n_pages, page_size, n_kv, D_v] through block_table int32 [B, max_blocks].  positions
    int32 [T] or None (the tokens' places): where queries are rotated; negative: an empty
    row (output 0, lse -inf), like rows behind cu_new[B].
    Returns (out [T, n_h, D_v], lse [T, n_h] or None).
    """
    return _attend(q, k_pages, v_pages, block_table, cu_new, seqlens, positions, None, rope_base, rope_offset,
                   rope_dims, scale, out, lse, workspace, pairing, stream)


def decode_tree(q, k_pages, v_pages, block_table, cu_new, seqlens, positions, visible, *, rope_base: float = 0.0,
                rope_offset: int = 0, rope_dims: int | None = None, scale: float = 0.0, out=None,
                lse: bool | torch.Tensor = False, workspace=None, pairing: str = "adjacent", stream=None):
    """Attention of drafted tokens that form a tree, against a paged cache, via attn_decode_tree.

    As prefill_paged, but a new token sees what its request held before the new tokens, and
    of these the ones whose bits are set in its row of visible (int32 [T, words], words 1 to
    4: bit j % 32 of word j / 32 for the request's j-th new token).  positions and visible
    are what draft_plan returns.
    """
    if visible is None:
        raise ValueError("visible must be an int32 CUDA tensor")
    return _attend(q, k_pages, v_pages, block_table, cu_new, seqlens, positions, visible, rope_base, rope_offset,
                   rope_dims, scale, out, lse, workspace, pairing, stream)


def draft_plan(places, cu_new, parents, *, words: int = 4, positions=None, visible=None, stream=None):
    """Positions and visibility bits of drafted tokens from their parents via attn_draft_plan.

    places int32 [T] (page_plan's positions; negative: an empty row), cu_new int32 [B+1],
    parents int32 [T]: each draft's parent among its request's drafts (a smaller index), -1
    for a child of the last token before them.  words (1 to 4): 32 drafts of a request each.
    Returns (positions int32 [T], visible int32 [T, words]); the outputs may be passed in.
    """
    device = _cuda(places, "places", torch.int32, None)
    _cuda(cu_new, "cu_new", torch.int32, device)
    if places.dim() != 1 or cu_new.dim() != 1 or cu_new.shape[0] < 2:
        raise ValueError("places must be [T] and cu_new [B + 1]")
    T, B = places.shape[0], cu_new.shape[0] - 1
    _ints(parents, "parents", (T,), device)
    if not 1 <= words <= 4:
        raise ValueError("words must be 1 to 4")
    context, st = _on(device, stream)
    with context:
        if positions is None:
            positions = torch.empty(T, dtype=torch.int32, device=device)
        else:
            _ints(positions, "positions", (T,), device)
        if visible is None:
            visible = torch.empty((T, words), dtype=torch.int32, device=device)
        else:
            _ints(visible, "visible", (T, words), device)
        if T == 0:
            return positions, visible
        rc = _lib().attn_draft_plan(places.data_ptr(), cu_new.data_ptr(), parents.data_ptr(), positions.data_ptr(),
                                    visible.data_ptr(), T, B, words, st)
    _b._check(rc, "attn_draft_plan")
    return positions, visible


def draft_commit(k_pages, v_pages, block_table, lens, seqlens, path, n_path, free_pages=None, n_free=None, *,
                 new_lens=None, n_left=None, stream=None):
    """Move accepted drafts to consecutive places of a paged cache via attn_draft_commit.

    lens and seqlens int32 [B]: tokens without and with the drafts.  path int32
    [B, max_path] (max_path <= 128), n_path int32 [B]: the accepted drafts' indices, rising.
    k_pages and v_pages are updated in place (v_pages a leading slice of k_pages: its keys
    alone).  With free_pages int32 [n] and n_free int32 [1] (page_plan's stack) the pages
    that fall free are put on the stack.  Returns (new_lens int32 [B], n_left int32 [1] or
    None); the outputs may be passed in.
    """
    device = _cuda(k_pages, "k_pages", None, None)
    n_pages, page_size, n_kv, D_qk, D_v, ldv = _page_dims(k_pages, v_pages, device)
    if block_table.dim() != 2 or path.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks] and path [B, max_path]")
    B, max_blocks = block_table.shape
    _cuda(block_table, "block_table", torch.int32, device)
    _ints(lens, "lens", (B,), device)
    _ints(seqlens, "seqlens", (B,), device)
    _ints(path, "path", (B, path.shape[1]), device)
    _ints(n_path, "n_path", (B,), device)
    if (free_pages is None) != (n_free is None):
        raise ValueError("free_pages and n_free go together")
    if free_pages is None and n_left is not None:
        raise ValueError("n_left needs free_pages and n_free")
    if free_pages is not None:
        _ints(free_pages, "free_pages", (free_pages.numel(),), device)
        _ints(n_free, "n_free", (1,), device)
    code = _b._dtype_code(k_pages)
    context, st = _on(device, stream)
    with context:
        if new_lens is None:
            new_lens = torch.empty(B, dtype=torch.int32, device=device)
        else:
            _ints(new_lens, "new_lens", (B,), device)
        if free_pages is not None and n_left is None:
            n_left = torch.empty(1, dtype=torch.int32, device=device)
        elif n_left is not None:
            _ints(n_left, "n_left", (1,), device)
        rc = _lib().attn_draft_commit(
            k_pages.data_ptr(), None if ldv else v_pages.data_ptr(), 0, block_table.data_ptr(), lens.data_ptr(),
            seqlens.data_ptr(), path.data_ptr(), n_path.data_ptr(), new_lens.data_ptr(), _b._ptr(free_pages),
            _b._ptr(n_free), _b._ptr(n_left), B, path.shape[1], n_kv, D_qk, D_v, n_pages, page_size, max_blocks,
            0 if free_pages is None else free_pages.shape[0], code, st)
    _b._check(rc, "attn_draft_commit")
    return new_lens, n_left
