"""ctypes binding of the paged-cache calls of libattn.so (include/attn_paged.h).

As in _binding.py, every function checks the tensors it is given, allocates the
outputs the caller does not pass, and forwards raw pointers; the arithmetic runs
in the library's kernels.  The calls run on the device of their tensors, on the
given stream or that device's current one; what they allocate belongs to that
stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import _binding as _b

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_CACHE = [_i] * 8  # B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks
_TAIL = [_f, _i, _i, _f, _i, _vp, _sz, _vp]  # rope_base, offset, dims, scale, dtype, workspace, bytes, stream

# (name, restype, argtypes) of every symbol of include/attn_paged.h
SIGNATURES = [
    ("attn_page_plan", _i, [_vp] * 10 + [_i] * 6 + [_vp]),
    ("attn_kv_append_paged", _i, [_vp] * 4 + [_i, _vp, _vp] + [_i] * 6 + [_f, _i, _i, _i, _vp]),
    ("attn_decode_paged_workspace_size", _sz, [_i] * 9),
    ("attn_decode_paged", _i, [_vp, _vp, _vp, _i, _vp, _vp, _vp, _vp] + _CACHE + _TAIL),
    ("attn_decode_shared", _i, [_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp] + _CACHE + _TAIL),
]

_LIB = None
_NO_SIZE = ctypes.c_size_t(-1).value


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


# A small call's time is its host time, so the checks below are written out: no dicts, and no stream or
# device objects where the call runs on the current stream of the current device.
def _cuda(t, name: str, dtype, device):
    """Check that t is a contiguous CUDA tensor (of dtype, on device, unless these are None); its device."""
    if not t.is_cuda or not t.is_contiguous():
        _b._dev(t, name)
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if device is None:
        return t.device
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return device


def _ints(t, name: str, shape: tuple, device) -> None:
    _cuda(t, name, torch.int32, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be int32 {list(shape)}, not {list(t.shape)}")


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """(context, stream handle): the tensors' device made current, with the call's stream current on it."""
    if stream is None:
        index = device.index
        if index == torch.cuda.current_device():
            return _HERE, torch._C._cuda_getCurrentRawStream(index)
        return torch.cuda.device(device), torch._C._cuda_getCurrentRawStream(index)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device=device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _page_dims(k_pages, v_pages, device):
    """(n_pages, page_size, n_kv, D_qk, D_v, v_token_stride) of a cache; v_pages contiguous, or a leading slice of the
    last dim of k_pages with its one head (MLA: the values are the first D_v latent dims)."""
    ks, vs = k_pages.shape, v_pages.shape
    if len(ks) != 4 or len(vs) != 4 or vs[:3] != ks[:3]:
        raise ValueError("k_pages and v_pages must be [n_pages, page_size, n_kv, D] with the same first three sizes")
    if v_pages.dtype is not k_pages.dtype or v_pages.device != device:
        raise TypeError("k_pages and v_pages must share a dtype and a device")
    if v_pages.is_contiguous():
        ldv = 0
    elif (v_pages.data_ptr() == k_pages.data_ptr() and v_pages.stride() == k_pages.stride() and vs[3] <= ks[3]
          and ks[2] == 1):
        ldv = v_pages.stride(1)
    else:
        raise ValueError("v_pages must be contiguous or a leading slice of the last dim of k_pages (of one head)")
    return ks[0], ks[1], ks[2], ks[3], vs[3], ldv


def page_plan(lens, n_new, block_table, free_pages, n_free, *, page_size: int, n_pages: int, max_tokens: int,
              seqlens=None, cu_new=None, slots=None, positions=None, n_left=None, stream=None):
    """Block tables, slots and positions of one step's new tokens via attn_page_plan.

    lens and n_new int32 [B]: tokens that each request holds and adds.  block_table
    int32 [B, max_blocks] is updated in place with the pages taken from the top of the
    stack free_pages[: n_free] (n_free int32 [1]).  Returns (seqlens [B], cu_new [B+1],
    slots [max_tokens], positions [max_tokens], n_left [1]), all int32; requests that do
    not fit keep their length and get slots of -1.  The outputs may be passed in (for a
    captured step), but none may overlap an input.
    """
    device = _cuda(lens, "lens", torch.int32, None)
    _cuda(block_table, "block_table", torch.int32, device)
    _cuda(free_pages, "free_pages", torch.int32, device)
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [B, max_blocks] and free_pages [n]")
    B, max_blocks = block_table.shape
    _ints(lens, "lens", (B,), device)
    _ints(n_new, "n_new", (B,), device)
    _ints(n_free, "n_free", (1,), device)
    context, st = _on(device, stream)
    with context:
        def given(t, name, n):
            if t is None:
                return torch.empty(n, dtype=torch.int32, device=device)
            _ints(t, name, (n,), device)
            return t
        seqlens, cu_new = given(seqlens, "seqlens", B), given(cu_new, "cu_new", B + 1)
        slots, positions = given(slots, "slots", max_tokens), given(positions, "positions", max_tokens)
        n_left = given(n_left, "n_left", 1)
        rc = _lib().attn_page_plan(lens.data_ptr(), n_new.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(),
                                   n_free.data_ptr(), seqlens.data_ptr(), cu_new.data_ptr(), slots.data_ptr(),
                                   positions.data_ptr(), n_left.data_ptr(), B, max_blocks, page_size, n_pages,
                                   free_pages.shape[0], max_tokens, st)
    _b._check(rc, "attn_page_plan")
    return seqlens, cu_new, slots, positions, n_left


def kv_append_paged(k_new, v_new, k_pages, v_pages, slots, positions=None, *, rope_base: float = 0.0,
                    rope_offset: int = 0, rope_dims: int | None = None, pairing: str = "adjacent",
                    stream=None) -> None:
    """Write packed new tokens into a paged cache via attn_kv_append_paged.

    k_new [T, n_kv, D_qk], v_new [T, n_kv, D_v] or None (values alias the keys), k_pages
    [n_pages, page_size, n_kv, D_qk], v_pages [n_pages, page_size, n_kv, D_v], slots int32
    [T] (outside the cache: skipped), positions int32 [T] (needed when rope_base > 0).
    """
    device = _cuda(k_new, "k_new", None, None)
    _cuda(k_pages, "k_pages", k_new.dtype, device)
    n_pages, page_size, n_kv, D_qk, D_v, ldv = _page_dims(k_pages, v_pages, device)
    T = k_new.shape[0]
    if k_new.shape != (T, n_kv, D_qk):
        raise ValueError(f"k_new must be [T, {n_kv}, {D_qk}]")
    if v_new is not None:
        _cuda(v_new, "v_new", k_new.dtype, device)
        if v_new.shape != (T, n_kv, D_v):
            raise ValueError(f"v_new must be [{T}, {n_kv}, {D_v}]")
    _ints(slots, "slots", (T,), device)
    if positions is not None:
        _ints(positions, "positions", (T,), device)
    if T == 0:
        return
    rope_dims = (D_qk - rope_offset) if rope_dims is None else rope_dims
    code = _b._dtype_code(k_new, pairing)
    context, st = _on(device, stream)
    with context:
        rc = _lib().attn_kv_append_paged(k_new.data_ptr(), _b._ptr(v_new), k_pages.data_ptr(), v_pages.data_ptr(),
                                         ldv, slots.data_ptr(), _b._ptr(positions), T, n_kv, D_qk, D_v, n_pages,
                                         page_size, rope_base, rope_offset, rope_dims, code, st)
    _b._check(rc, "attn_kv_append_paged")


@functools.lru_cache(maxsize=256)  # a serving loop asks with the same sizes step after step
def _workspace_size(*sizes) -> int:
    return _lib().attn_decode_paged_workspace_size(*sizes)


def decode_paged_workspace_size(B, n_h, n_kv, D_qk, D_v, page_size, max_blocks, prefix_len=0,
                                dtype=torch.bfloat16) -> int:
    """Bytes of scratch of decode_paged (prefix_len = 0) or decode_shared."""
    n = _workspace_size(B, n_h, n_kv, D_qk, D_v, page_size, max_blocks, prefix_len,
                        _b.ATTN_BF16 if dtype == torch.bfloat16 else _b.ATTN_F32)
    if n == _NO_SIZE:
        raise ValueError("invalid paged decode sizes")
    return n


def _decode(q, k_pages, v_pages, prefix_pages, block_table, seqlens, rope_base, rope_offset, rope_dims, scale, out,
            lse, workspace, pairing, stream):
    device = _cuda(q, "q", None, None)
    _cuda(k_pages, "k_pages", q.dtype, device)
    n_pages, page_size, n_kv, D_qk, D_v, ldv = _page_dims(k_pages, v_pages, device)
    if q.dim() != 3 or q.shape[2] != D_qk:
        raise ValueError(f"q must be [B, n_h, {D_qk}]")
    B, n_h, _ = q.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    max_blocks = block_table.shape[1]
    _ints(block_table, "block_table", (B, max_blocks), device)
    _ints(seqlens, "seqlens", (B,), device)
    prefix_len = 0
    if prefix_pages is not None:
        _ints(prefix_pages, "prefix_pages", (prefix_pages.numel(),), device)
        prefix_len = prefix_pages.shape[0] * page_size
    rope_dims = (D_qk - rope_offset) if rope_dims is None else rope_dims
    code = _b._dtype_code(q, pairing)
    lib = _lib()
    context, st = _on(device, stream)
    with context:
        if out is None:
            out = torch.empty((B, n_h, D_v), dtype=q.dtype, device=device)
        else:
            _cuda(out, "out", q.dtype, device)
            if out.shape != (B, n_h, D_v):
                raise ValueError(f"out must be [{B}, {n_h}, {D_v}]")
        if isinstance(lse, torch.Tensor):
            _cuda(lse, "lse", torch.float32, device)
            if lse.shape != (B, n_h):
                raise ValueError(f"lse must be fp32 [{B}, {n_h}]")
            lse_t = lse
        else:
            lse_t = torch.empty((B, n_h), dtype=torch.float32, device=device) if lse else None
        if workspace is None:
            need = _workspace_size(B, n_h, n_kv, D_qk, D_v, page_size, max_blocks, prefix_len, code & 0xff)
            # invalid sizes: the call itself says what is wrong with them
            workspace = torch.empty(16 if need == _NO_SIZE else need, dtype=torch.uint8, device=device)
        else:
            _cuda(workspace, "workspace", None, device)
        if prefix_pages is None:
            rc = lib.attn_decode_paged(
                q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), ldv, block_table.data_ptr(), seqlens.data_ptr(),
                out.data_ptr(), _b._ptr(lse_t), B, n_h, n_kv, D_qk, D_v, n_pages, page_size, max_blocks, rope_base,
                rope_offset, rope_dims, scale, code, workspace.data_ptr(), workspace.nbytes, st)
        else:
            rc = lib.attn_decode_shared(
                q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), ldv, prefix_pages.data_ptr(), prefix_len,
                block_table.data_ptr(), seqlens.data_ptr(), out.data_ptr(), _b._ptr(lse_t), B, n_h, n_kv, D_qk, D_v,
                n_pages, page_size, max_blocks, rope_base, rope_offset, rope_dims, scale, code, workspace.data_ptr(),
                workspace.nbytes, st)
    _b._check(rc, "attn_decode_paged" if prefix_pages is None else "attn_decode_shared")
    return out, lse_t


def decode_paged(q, k_pages, v_pages, block_table, seqlens, *, rope_base: float = 0.0, rope_offset: int = 0,
                 rope_dims: int | None = None, scale: float = 0.0, out=None, lse: bool | torch.Tensor = False,
                 workspace=None, pairing: str = "adjacent", stream=None):
    """One new token per request against a paged cache via attn_decode_paged.

    q [B, n_h, D_qk] (un-rotated), k_pages [n_pages, page_size, n_kv, D_qk] (rotated keys),
    v_pages [n_pages, page_size, n_kv, D_v] contiguous or a last-dim slice of k_pages (MLA),
    block_table int32 [B, max_blocks], seqlens int32 [B] (keys incl. the new one; <= 0: an
    empty place, output 0 and lse -inf).  Returns (out [B, n_h, D_v], lse [B, n_h] or None).
    """
    return _decode(q, k_pages, v_pages, None, block_table, seqlens, rope_base, rope_offset, rope_dims, scale, out,
                   lse, workspace, pairing, stream)


def decode_shared(q, k_pages, v_pages, prefix_pages, block_table, seqlens, *, rope_base: float = 0.0,
                  rope_offset: int = 0, rope_dims: int | None = None, scale: float = 0.0, out=None,
                  lse: bool | torch.Tensor = False, workspace=None, pairing: str = "adjacent", stream=None):
    """decode_paged() for a batch whose requests all start with the tokens in prefix_pages (attn_decode_shared).

    prefix_pages int32 [n]: the n full pages that every row of block_table starts with;
    they are read and computed once for the whole batch (in the MLA-absorbed shape, values
    sliced from one 576-dim head under 128 heads, once per request).  seqlens counts them:
    request b has seqlens[b] - n * page_size >= 1 tokens of its own (fewer: an empty place).
    """
    if prefix_pages is None:
        raise ValueError("prefix_pages must be an int32 CUDA tensor")
    return _decode(q, k_pages, v_pages, prefix_pages, block_table, seqlens, rope_base, rope_offset, rope_dims, scale,
                   out, lse, workspace, pairing, stream)
