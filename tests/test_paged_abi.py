"""The paged-cache part of the C ABI without a GPU: header and binding agree, and bad arguments are
refused on the host before anything touches a device (the pointers are never dereferenced)."""
import ctypes
import os
import re

import pytest
import torch

import transformer_causal_attention_gb300 as attn
from transformer_causal_attention_gb300 import _binding, _paged
from transformer_causal_attention_gb300 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [(i + 1) << 24 for i in range(16)]  # distinct 16-byte aligned addresses, far apart
ODD = (1 << 24) + 2
NO_SIZE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _paged._lib()


def test_header_and_binding_agree(lib):
    text = open(os.path.join(ROOT, "include", "attn_paged.h"), encoding="utf-8").read()
    names = set(re.findall(r"ATTN_API\s+[\w\s\*]*?\b(attn_\w+)\s*\(", text))
    assert names == {n for n, _, _ in _paged.SIGNATURES}
    for name, _, args in _paged.SIGNATURES:
        assert hasattr(lib, name)
        decl = re.search(r"\b%s\s*\(([^;]*)\);" % name, text).group(1)
        assert len(decl.split(",")) == len(args), name


def plan(lib, lens=P[0], new=P[1], table=P[2], free=P[3], n_free=P[4], seqlens=P[5], cu=P[6], slots=P[7], pos=P[8],
         left=P[9], B=4, max_blocks=8, page=16, n_pages=64, cap=32, max_tokens=100):
    return lib.attn_page_plan(lens, new, table, free, n_free, seqlens, cu, slots, pos, left, B, max_blocks, page,
                              n_pages, cap, max_tokens, None)


def test_page_plan_refusals(lib):
    for name in ("lens", "new", "table", "free", "n_free", "seqlens", "cu", "slots", "pos", "left"):
        assert plan(lib, **{name: None}) == -1
        assert plan(lib, **{name: ODD + (40 << 24)}) == -3
    for name in ("B", "max_blocks", "n_pages", "cap", "max_tokens", "page"):
        assert plan(lib, **{name: 0}) == -1
        assert plan(lib, **{name: -5}) == -1
    assert plan(lib, lens=P[0] + 2) == -3
    assert plan(lib, left=P[9] + 1) == -3
    for page in (1, 8, 17, 24, 512):
        assert plan(lib, page=page) == -2
    assert plan(lib, B=16385, max_tokens=20000) == -2
    assert plan(lib, cap=65) == -1                                   # a stack higher than the cache has pages
    assert plan(lib, page=256, n_pages=1 << 23) == -1                # 2^31 slots
    assert plan(lib, page=256, max_blocks=1 << 23, B=1) == -1
    # outputs on top of inputs or of each other
    assert plan(lib, seqlens=P[0]) == -1
    assert plan(lib, left=P[4]) == -1
    assert plan(lib, slots=P[8] - 4 * 99) == -1
    assert plan(lib, table=P[3] - 4 * 31) == -1


def append(lib, k=P[0], v=P[1], kp=P[2], vp=P[3], ldv=0, slots=P[4], pos=P[5], T=4, n_kv=2, Dqk=64, Dv=64, n_pages=8,
           page=16, rope=1e4, roff=0, rdims=64, dtype=1):
    return lib.attn_kv_append_paged(k, v, kp, vp, ldv, slots, pos, T, n_kv, Dqk, Dv, n_pages, page, rope, roff, rdims,
                                    dtype, None)


def test_kv_append_paged_refusals(lib):
    for name in ("k", "kp", "slots", "vp", "pos"):
        assert append(lib, **{name: None}) == -1
    for name in ("T", "n_kv", "Dqk", "Dv", "n_pages", "page"):
        assert append(lib, **{name: 0}) == -1
    assert append(lib, dtype=2) == -1
    assert append(lib, page=20) == -2
    assert append(lib, Dqk=60) == -1
    assert append(lib, roff=4, rdims=56) == -1
    assert append(lib, roff=8) == -1                       # span past the head
    assert append(lib, roff=8, rdims=2**31 - 8) == -1      # offset + dims would overflow
    assert append(lib, rdims=8, dtype=1 | _binding.ATTN_ROPE_HALF) == -1
    assert append(lib, ldv=-8) == -1
    assert append(lib, ldv=64) == -1                       # slots of two heads x 64 would overlap
    assert append(lib, ldv=132) == -2
    assert append(lib, Dqk=1024, rdims=1024) == -2         # more pairs than the table holds
    assert append(lib, k=P[0] + 8) == -3
    assert append(lib, slots=P[4] + 2) == -3
    assert append(lib, n_pages=1 << 27) == -1
    for vp in (P[2], P[2] + 16, P[2] + 2 * 64 * 2 * 127):  # values over the keys
        assert append(lib, vp=vp) == -1
    assert append(lib, vp=P[2] - 2 * 64 * 2 * 16) == -1


def decode(lib, q=P[0], kp=P[1], vp=P[2], ldv=0, pages=P[3], prefix=64, table=P[4], sl=P[5], out=P[6], lse=None, B=2,
           n_h=8, n_kv=2, Dqk=128, Dv=128, n_pages=64, page=16, max_blocks=8, rope=1e4, roff=0, rdims=128, scale=0.0,
           dtype=1, ws=P[7], ws_bytes=1 << 40):
    dims = (B, n_h, n_kv, Dqk, Dv, n_pages, page, max_blocks, rope, roff, rdims, scale, dtype, ws, ws_bytes, None)
    shared = lib.attn_decode_shared(q, kp, vp, ldv, pages, prefix, table, sl, out, lse, *dims)
    if (pages, prefix) == (P[3], 64):  # the same refusal without a prefix
        assert lib.attn_decode_paged(q, kp, vp, ldv, table, sl, out, lse, *dims) == shared
    return shared


def test_decode_refusals(lib):
    for name in ("q", "kp", "vp", "table", "sl", "out", "ws"):
        assert decode(lib, **{name: None}) == -1
    for name in ("B", "n_h", "n_kv", "Dqk", "Dv", "n_pages", "page", "max_blocks"):
        assert decode(lib, **{name: 0}) == -1
    assert decode(lib, pages=None) == -1
    for prefix in (0, -16, 8, 72, 144):                    # none, negative, broken pages, past the table
        assert decode(lib, prefix=prefix) == -1
    assert decode(lib, n_h=6, n_kv=4) == -1
    assert decode(lib, dtype=7) == -1
    assert decode(lib, ldv=-8) == -1
    assert decode(lib, ldv=128) == -1                      # separate values closer than their heads
    assert decode(lib, roff=64) == -1
    assert decode(lib, rdims=3) == -1
    assert decode(lib, page=48) == -2
    assert decode(lib, Dqk=100) == -2
    assert decode(lib, Dqk=648, rdims=128) == -2
    assert decode(lib, Dv=520) == -2
    assert decode(lib, ldv=260) == -2
    assert decode(lib, q=P[0] + 4) == -3
    assert decode(lib, sl=P[5] + 1) == -3
    assert decode(lib, lse=P[8] + 2) == -3
    assert decode(lib, ws_bytes=16) == -6
    assert decode(lib, n_pages=1 << 27) == -1
    assert decode(lib, max_blocks=1 << 27) == -1
    assert decode(lib, max_blocks=(1 << 27) - 4095) == -1  # past 2^31 - 2^16 tokens
    assert decode(lib, B=1 << 20, n_h=1 << 12, n_kv=1 << 11) == -1


def test_workspace_size(lib):
    f = lib.attn_decode_paged_workspace_size
    assert 0 < f(59, 32, 8, 128, 128, 64, 128, 0, 1) < 256 << 20
    assert 0 < f(59, 32, 8, 128, 128, 64, 128, 4096, 1) < 256 << 20
    assert 0 < f(1, 1, 1, 8, 8, 16, (1 << 27) - 4096, 0, 1) < NO_SIZE
    assert 0 < f(1, 1, 1, 8, 8, 16, (1 << 27) - 4096, (1 << 31) - (1 << 16), 1) < NO_SIZE
    for bad in ((1, 1, 1, 8, 8, 16, (1 << 27) - 4095, 0, 1), (0, 32, 8, 128, 128, 64, 128, 0, 1), (4, 32, 5, 128, 128, 64, 128, 0, 1),
                (4, 32, 8, 128, 128, 60, 128, 0, 1), (4, 32, 8, 128, 128, 64, 128, 100, 1),
                (4, 32, 8, 128, 128, 64, 128, 64 * 129, 1), (4, 32, 8, 128, 128, 64, 128, 0, 9)):
        assert f(*bad) == NO_SIZE
    assert f(4, 32, 8, 128, 128, 64, 128, 0, 1) == f(4, 32, 8, 128, 128, 64, 128, 0, 1 | _binding.ATTN_ROPE_HALF)


def test_python_refuses_cpu_tensors(lib):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.page_plan(i, i, i.view(4, 1), i, i[:1], page_size=16, n_pages=4, max_tokens=4)
    x = torch.zeros(2, 16, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        attn.kv_append_paged(x[0], x[0], x, x, i)
    with pytest.raises(ValueError, match="CUDA"):
        attn.decode_paged(x[0, :1], x, x, i.view(1, 4), i[:1])
    with pytest.raises(ValueError, match="prefix_pages"):
        attn.decode_shared(x[0, :1], x, x, None, i.view(1, 4), i[:1])
