"""The packed part of the C ABI without a GPU: header and binding agree, and bad arguments are refused on the
host before anything touches a device (the pointers are never dereferenced)."""
import ctypes
import os
import re

import pytest
import torch

import transformer_causal_attention_gb300 as attn
from transformer_causal_attention_gb300 import _packed
from transformer_causal_attention_gb300 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [(i + 1) << 28 for i in range(16)]  # distinct 16-byte aligned addresses, far apart
NO_SIZE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _packed._lib()


def test_header_and_binding_agree(lib):
    text = open(os.path.join(ROOT, "include", "attn_packed.h"), encoding="utf-8").read()
    names = set(re.findall(r"ATTN_API\s+[\w\s\*]*?\b(attn_\w+)\s*\(", text))
    assert names == {n for n, _, _ in _packed.SIGNATURES}
    for name, _, args in _packed.SIGNATURES:
        assert hasattr(lib, name)
        decl = re.search(r"\b%s\s*\(([^;]*)\);" % name, text).group(1)
        assert len(decl.split(",")) == len(args), name


def attend(lib, q=P[0], kp=P[1], vp=P[2], ldv=0, table=P[3], cu=P[4], sl=P[5], pos=P[6], vis=P[7], words=2, out=P[8],
           lse=None, T=50, B=2, n_h=8, n_kv=2, Dqk=128, Dv=128, n_pages=64, page=16, max_blocks=8, rope=1e4, roff=0,
           rdims=128, scale=0.0, dtype=1, ws=P[9], ws_bytes=1 << 27):
    dims = (T, B, n_h, n_kv, Dqk, Dv, n_pages, page, max_blocks, rope, roff, rdims, scale, dtype, ws, ws_bytes, None)
    tree = lib.attn_decode_tree(q, kp, vp, ldv, table, cu, sl, pos, vis, words, out, lse, *dims)
    if (vis, words) == (P[7], 2):  # the same refusal without a tree
        assert lib.attn_prefill_paged(q, kp, vp, ldv, table, cu, sl, pos, out, lse, *dims) == tree
    return tree


def test_attention_refusals(lib):
    for name in ("q", "kp", "vp", "table", "cu", "sl", "out", "ws", "vis"):
        assert attend(lib, **{name: None}) == -1, name
    for name in ("T", "B", "n_h", "n_kv", "Dqk", "Dv", "n_pages", "page", "max_blocks"):
        assert attend(lib, **{name: 0}) == -1, name
        assert attend(lib, **{name: -3}) == -1, name
    for words in (0, 5, -1):
        assert attend(lib, words=words) == -1
    assert attend(lib, n_h=6, n_kv=4) == -1
    assert attend(lib, dtype=7) == -1
    assert attend(lib, ldv=-8) == -1
    assert attend(lib, ldv=128) == -1                      # separate values closer than their heads
    assert attend(lib, roff=64) == -1
    assert attend(lib, roff=8, rdims=2**31 - 8) == -1
    assert attend(lib, rdims=3) == -1
    assert attend(lib, page=48) == -2
    assert attend(lib, Dqk=100) == -2
    assert attend(lib, Dqk=648, rdims=128) == -2
    assert attend(lib, Dv=520) == -2
    assert attend(lib, ldv=260) == -2
    for name, i in (("q", 0), ("kp", 1), ("vp", 2), ("out", 8), ("ws", 9)):
        assert attend(lib, **{name: P[i] + 8}) == -3, name
    for name, i in (("table", 3), ("cu", 4), ("sl", 5), ("pos", 6), ("vis", 7), ("lse", 10)):
        assert attend(lib, **{name: P[i] + 2}) == -3, name
    assert attend(lib, ws_bytes=8) == -6
    assert attend(lib, n_pages=1 << 27) == -1
    assert attend(lib, max_blocks=1 << 27) == -1
    assert attend(lib, max_blocks=(1 << 27) - 4095) == -1  # past 2^31 - 2^16 tokens
    assert attend(lib, T=1 << 20, n_h=1 << 12, n_kv=1 << 11) == -1
    row, slots = 50 * 8 * 128 * 2, 64 * 16 * 2 * 128 * 2
    for name, at in (("out", P[0]), ("out", P[0] + row - 16), ("out", P[1]), ("out", P[2] + slots - 16), ("out", P[9]),
                     ("lse", P[8]), ("lse", P[6] + 4 * 49), ("ws", P[0]), ("ws", P[3]), ("out", P[4]), ("out", P[5])):
        assert attend(lib, **{name: at}) == -1, (name, hex(at))
    assert attend(lib, vis=P[8] + 64) == -1                # under the output


def test_workspace_size(lib):
    f = lib.attn_packed_workspace_size
    for dtype in (0, 1):
        for sizes in ((1, 1, 32, 8, 128, 128, 64, 128), (32768, 4, 32, 8, 128, 128, 64, 128),
                      (1888, 59, 32, 8, 128, 128, 64, 128), (64, 2, 128, 1, 576, 512, 16, 8192),
                      (1, 1, 1, 1, 8, 8, 16, (1 << 27) - 4096)):
            # partials of the blocks, and the queries once more with half of them in a second part
            assert 0 < f(*sizes, dtype) < (64 << 20) + 4 * sizes[0] * sizes[2] * sizes[4] + (96 << 20) * (dtype == 0), sizes
    for bad in ((0, 1, 32, 8, 128, 128, 64, 128, 1), (4, 0, 32, 8, 128, 128, 64, 128, 1), (4, 1, 32, 5, 128, 128, 64, 128, 1),
                (4, 1, 32, 8, 128, 128, 60, 128, 1), (4, 1, 32, 8, 100, 128, 64, 128, 1), (4, 1, 32, 8, 128, 128, 64, 128, 9),
                (1, 1, 1, 1, 8, 8, 16, (1 << 27) - 4095, 1)):
        assert f(*bad) == NO_SIZE
    # tables are as wide as a request may grow: the scratch does not follow
    assert len({f(77, 3, 32, 8, 128, 128, 64, blocks, 1) for blocks in (1 << 8, 1 << 14, 1 << 20)}) == 1


def plan(lib, places=P[0], cu=P[1], parents=P[2], pos=P[3], vis=P[4], T=40, B=3, words=2):
    return lib.attn_draft_plan(places, cu, parents, pos, vis, T, B, words, None)


def test_draft_plan_refusals(lib):
    for name, i in (("places", 0), ("cu", 1), ("parents", 2), ("pos", 3), ("vis", 4)):
        assert plan(lib, **{name: None}) == -1
        assert plan(lib, **{name: P[i] + 1}) == -3
    for name in ("T", "B", "words"):
        assert plan(lib, **{name: 0}) == -1
        assert plan(lib, **{name: -2}) == -1
    assert plan(lib, words=5) == -1
    assert plan(lib, pos=P[0]) == -1
    assert plan(lib, pos=P[2] + 4 * 39) == -1
    assert plan(lib, vis=P[1] + 12) == -1
    assert plan(lib, vis=P[3] - 8 * 40 + 4) == -1


def commit(lib, kp=P[0], vp=P[1], ldv=0, table=P[2], lens=P[3], sl=P[4], path=P[5], n_path=P[6], new=P[7], free=P[8],
           n_free=P[9], left=P[10], B=3, max_path=8, n_kv=2, Dqk=64, Dv=64, n_pages=32, page=16, max_blocks=4, cap=32,
           dtype=1):
    return lib.attn_draft_commit(kp, vp, ldv, table, lens, sl, path, n_path, new, free, n_free, left, B, max_path, n_kv,
                                 Dqk, Dv, n_pages, page, max_blocks, cap, dtype, None)


def test_draft_commit_refusals(lib):
    for name in ("kp", "table", "lens", "sl", "path", "n_path", "new", "free", "n_free", "left"):
        assert commit(lib, **{name: None}) == -1, name
    for name in ("B", "max_path", "n_kv", "Dqk", "Dv", "n_pages", "page", "max_blocks", "cap"):
        assert commit(lib, **{name: 0}) == -1, name
        assert commit(lib, **{name: -1}) == -1, name
    assert commit(lib, dtype=5) == -1
    assert commit(lib, cap=33) == -1
    assert commit(lib, ldv=-8) == -1
    assert commit(lib, ldv=64) == -1
    assert commit(lib, ldv=132) == -2
    assert commit(lib, page=24) == -2
    assert commit(lib, Dqk=60) == -2
    assert commit(lib, B=16385) == -2
    assert commit(lib, max_path=129) == -2
    assert commit(lib, n_pages=1 << 27, cap=32) == -1
    for name, i in (("kp", 0), ("vp", 1)):
        assert commit(lib, **{name: P[i] + 8}) == -3
    for name, i in (("table", 2), ("lens", 3), ("sl", 4), ("path", 5), ("n_path", 6), ("new", 7), ("free", 8),
                    ("n_free", 9), ("left", 10)):
        assert commit(lib, **{name: P[i] + 2}) == -3, name
    assert commit(lib, new=P[3]) == -1
    assert commit(lib, new=P[4] + 8) == -1
    assert commit(lib, left=P[9]) == -1
    assert commit(lib, left=P[8] + 4 * 31) == -1
    assert commit(lib, vp=P[0]) == -1
    assert commit(lib, vp=P[0] + 16) == -1
    assert commit(lib, path=P[0] + 64) == -1


def test_python_refuses(lib):
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(2, 16, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        attn.prefill_paged(x[0], x, x, i.view(1, 4), i[:2], i[:1], i)
    with pytest.raises(ValueError, match="CUDA"):
        attn.decode_tree(x[0], x, x, i.view(1, 4), i[:2], i[:1], i, i.view(4, 1))
    with pytest.raises(ValueError, match="visible"):
        attn.decode_tree(x[0], x, x, i.view(1, 4), i[:2], i[:1], i, None)
    with pytest.raises(ValueError, match="CUDA"):
        attn.draft_plan(i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        attn.draft_commit(x, x, i.view(1, 4), i[:1], i[:1], i.view(1, 4), i[:1])
    with pytest.raises(ValueError, match="invalid"):
        attn.packed_workspace_size(1, 1, 3, 2, 64, 64, 16, 4)
