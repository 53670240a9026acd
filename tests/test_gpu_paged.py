"""The paged cache on the GPU: page plan, append, decode and decode behind a shared prefix, against plain
references in 64 bits (tests/paged_reference.py), alone and as a serving loop runs them together.

Caches are filled with NaN wherever no token lives, so a read behind a request's end shows.  bf16
results are held to the parity bars of tests/tolerances.py (the same roundings as attn_decode) and
element-wise to 2^-8 |o| (the stored result) + (2^-8 + 2 e) * max|v| (each weight rounded, and off by
at most 2 e for scores off by e <= 1/2, the reference's bound for the rounded query); the
log-sum-exp to e plus 1e-5 relative (fp32 sums).
"""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.tolerances import BF16_REL_L2, FP32_MAX_ABS, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import transformer_causal_attention_gb300 as attn
    yield attn
    assert attn.device_status() == 0


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------- page plan
def check_plan(lib, lens, n_new, table, free, n_free, page, n_pages, max_tokens):
    want = ref.plan(lens, n_new, table, free, n_free, page, n_pages, max_tokens)
    t = ints(table).contiguous()
    got = lib.page_plan(ints(lens), ints(n_new), t, ints(free), ints([n_free]), page_size=page, n_pages=n_pages,
                        max_tokens=max_tokens)
    torch.cuda.synchronize()
    for name, a, b in zip(("table", "seqlens", "cu_new", "slots", "positions", "n_left"),
                          (t, *got), (*want[:5], [want[5]])):
        np.testing.assert_array_equal(a.cpu().numpy(), np.asarray(b), err_msg=name)
    return t, got


def random_plan(seed, B, hi, new, page, room=None, slack=4):
    rng = np.random.default_rng(seed)
    lens, n_new = rng.integers(0, hi + 1, B), rng.integers(0, new + 1, B)
    have, want = -(-lens // page), -(-(lens + n_new) // page)
    held, need = int(have.sum()), int((want - have).sum())
    free_n = need + slack if room is None else max(1, int(need * room))
    order = rng.permutation(held + free_n)
    table = np.full((B, int(want.max()) + 1), -1)
    table[np.arange(table.shape[1])[None] < have[:, None]] = order[:held]
    return lens, n_new, table, order[held:], free_n, page, held + free_n, int(n_new.sum()) + 5


@pytest.mark.parametrize("B,hi,new,page,room", [
    (1, 0, 1, 16, None), (1, 500, 900, 32, None), (59, 8192, 1, 64, None), (257, 40, 3, 16, None),
    (1024, 300, 30, 128, None), (1025, 300, 30, 16, 0.5), (5000, 20, 20, 16, 0.7), (33, 4000, 2000, 256, 0.9),
    (2, 100000, 60000, 16, None), (7, 100, 0, 16, None), (16384, 9, 2, 16, 0.99),
])
def test_page_plan(lib, B, hi, new, page, room):
    for seed in range(2):
        check_plan(lib, *random_plan(seed, B, hi, new, page, room))


def test_page_plan_corners(lib):
    table = [[0, -1, -1], [1, 2, -1], [3, -1, -1], [-1, -1, -1]]
    free = [9, 8, 7, 6, 5, 4]
    common = dict(page=16, n_pages=10, max_tokens=40)
    check_plan(lib, [16, 17, 5, 0], [1, 1, 1, 1], table, free, 6, **common)
    check_plan(lib, [16, 17, 5, 0], [33, 1, 1, 1], table, free, 6, **common)       # past the table: refused alone
    check_plan(lib, [16, 17, 5, 0], [1, 16, 30, 1], table, free, 6, **common)      # past max_tokens from row 2 on
    check_plan(lib, [16, 17, 5, 0], [1, 1, 1, 16], table, free, 1, **common)       # stack empty: row 3 refused
    check_plan(lib, [16, 17, 5, 0], [1, 1, 1, 16], table, free, 0, **common)       # only rows without a new page
    check_plan(lib, [16, 17, 5, 0], [20, 17, 1, 1], table, free, 3, **common)      # 2 + 2 pages of 3: row 1 and 3 refused
    check_plan(lib, [16, 17, 5, 0], [1, 1, 1, 1], table, free, 99, **common)       # height above the array
    check_plan(lib, [16, 17, 5, 0], [1, 1, 1, 1], table, free, -3, **common)
    check_plan(lib, [-4, 17, 5, 0], [1, -9, 0, 0], table, free, 6, **common)       # negative counts
    check_plan(lib, [16, 17, 5, 0], [0, 0, 0, 0], table, free, 6, **common)        # nothing to do
    check_plan(lib, [0, 0, 0, 0], [2**31 - 1] * 4, table, free, 6, **common)       # sums past 32 bits
    check_plan(lib, [2**31 - 1, 17, 5, 0], [1, 1, 1, 1], table, free, 6, **common)
    # page indices outside the cache, in the table and in the stack
    check_plan(lib, [3, 17, 5, 0], [1, 1, 1, 1], [[-5, 0, 0], [1, 10, 0], [3, 0, 0], [0, 0, 0]], free, 6, **common)
    check_plan(lib, [16, 17, 5, 0], [1, 1, 1, 1], table, [9, 8, 7, 6, 1 << 30, -1], 6, **common)


def test_page_plan_given_outputs_and_stream(lib):
    args = random_plan(3, 40, 200, 50, 16)
    want = ref.plan(*args)
    lens, n_new, table, free, n_free, page, n_pages, max_tokens = args
    st = torch.cuda.Stream()
    out = {k: torch.full((n,), -77, dtype=torch.int32, device=DEV) for k, n in
           (("seqlens", 40), ("cu_new", 41), ("slots", max_tokens), ("positions", max_tokens), ("n_left", 1))}
    t, src = ints(table), [ints(lens), ints(n_new), ints(free), ints([n_free])]
    torch.cuda.synchronize()
    got = lib.page_plan(src[0], src[1], t, src[2], src[3], page_size=page, n_pages=n_pages, max_tokens=max_tokens,
                        stream=st, **out)
    st.synchronize()
    for g, o, w in zip(got, out.values(), (*want[1:5], [want[5]])):
        assert g is o
        np.testing.assert_array_equal(g.cpu().numpy(), np.asarray(w))
    with pytest.raises(lib.AttnError):   # seqlens on top of lens
        lib.page_plan(src[0], src[1], t, src[2], src[3], page_size=page, n_pages=n_pages, max_tokens=max_tokens,
                      seqlens=src[0])
    with pytest.raises(ValueError):
        lib.page_plan(src[0], src[1][:-1], t, src[2], src[3], page_size=page, n_pages=n_pages, max_tokens=max_tokens)
    with pytest.raises(TypeError):
        lib.page_plan(src[0].long(), src[1], t, src[2], src[3], page_size=page, n_pages=n_pages, max_tokens=max_tokens)


# ---------------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("T,n_kv,Dqk,Dv,page,rope,roff,rdims,pairing,alias,dtype", [
    (1, 1, 64, 64, 16, 1e4, 0, 64, "adjacent", False, "bf16"),
    (59, 8, 128, 128, 64, 5e5, 0, 128, "adjacent", False, "bf16"),
    (300, 8, 128, 128, 64, 5e5, 0, 128, "half", False, "bf16"),
    (37, 3, 72, 40, 32, 0.0, 0, 72, "adjacent", False, "bf16"),
    (37, 5, 64, 128, 256, 1e4, 16, 32, "half", False, "f32"),
    (40, 1, 576, 512, 16, 1e4, 512, 64, "adjacent", True, "bf16"),
    (9000, 12, 64, 64, 16, 1e4, 0, 64, "adjacent", False, "f32"),
    (20000, 8, 128, 128, 128, 5e5, 0, 128, "adjacent", False, "bf16"),
    (20001, 4, 128, 128, 16, 5e5, 0, 128, "half", False, "bf16"),
])
def test_kv_append_paged(lib, T, n_kv, Dqk, Dv, page, rope, roff, rdims, pairing, alias, dtype):
    import oracle
    dt = TYPES[dtype]
    g = torch.Generator().manual_seed(T)
    n_pages = -(-T // page) + 2
    k = torch.randn(T, n_kv, Dqk, generator=g).to(dt)
    v = torch.randn(T, n_kv, Dv, generator=g).to(dt)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[T // 2] = (-1, n_pages * page, 2**31 - 1, -2**31)[T % 4]  # outside the cache: skipped
    pos = torch.randint(0, 100000, (T,), generator=g).to(torch.int32)
    kp = torch.randn(n_pages, page, n_kv, Dqk, generator=g).to(dt)
    vp = kp[..., :Dv] if alias else torch.randn(n_pages, page, n_kv, Dv, generator=g).to(dt)
    live = torch.arange(T) != T // 2
    rot = k.double().numpy()
    if rope > 0:
        rot = oracle.rope_rotate(rot, pos.numpy()[:, None], rope, roff, rdims, pairing=pairing)
    want_k = kp.double().flatten(0, 1).numpy().copy()
    want_k[slots[live].long().numpy()] = rot[live.numpy()]
    kd = kp.to(DEV)
    vd = kd[..., :Dv] if alias else vp.to(DEV)
    lib.kv_append_paged(k.to(DEV), None if alias else v.to(DEV), kd, vd, slots.to(DEV),
                        pos.to(DEV) if rope > 0 else None, rope_base=rope, rope_offset=roff, rope_dims=rdims,
                        pairing=pairing)
    torch.cuda.synchronize()
    got = kd.double().flatten(0, 1).cpu().numpy()
    # half a step of the stored type, and 1e-6 of the pair's norm for the fp32 rotation
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = eps * np.abs(want_k) + 1e-6 * np.sqrt(2) * 6
    assert np.all(np.abs(got - want_k) <= tol)
    untouched = np.ones(n_pages * page, bool)
    untouched[slots[live].long().numpy()] = False
    np.testing.assert_array_equal(got[untouched], want_k[untouched])
    if not alias:
        want_v = vp.flatten(0, 1).clone()
        want_v[slots[live].long()] = v[live]
        assert torch.equal(vd.flatten(0, 1).cpu(), want_v)


# ---------------------------------------------------------------------------------------------- decode
def check_decode(lib, lens, prefix, page, n_h, n_kv, Dqk, Dv, rope=0.0, roff=0, rdims=None, scale=0.0,
                 pairing="adjacent", dtype="bf16", alias=False, seed=0, shared=None, **call):
    """decode_shared (prefix > 0) or decode_paged against the fp64 reference; returns the output."""
    dt = TYPES[dtype]
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, page, n_kv, Dqk, Dv, dt, seed=seed, alias=alias)
    q = torch.randn(len(lens), n_h, Dqk, generator=torch.Generator().manual_seed(seed + 1)).to(dt)
    want, want_lse, err = ref.attend(q, k_of, v_of, rope_base=rope, rope_offset=roff, rope_dims=rdims, scale=scale,
                                     pairing=pairing)
    kd = k.to(DEV)
    vd = kd[..., :Dv] if alias else v.to(DEV)
    args = dict(rope_base=rope, rope_offset=roff, rope_dims=rdims, scale=scale, pairing=pairing, lse=True, **call)
    if prefix:
        out, lse = lib.decode_shared(q.to(DEV), kd, vd, pre.to(DEV), table.to(DEV), ints(lens), **args)
    else:
        out, lse = lib.decode_paged(q.to(DEV), kd, vd, table.to(DEV), ints(lens), **args)
    torch.cuda.synchronize()
    check_result(to_np(out), to_np(lse), want, want_lse, err, v_of, dtype)
    return out, lse


def check_result(got, got_lse, want, want_lse, err, v_of, dtype):
    empty = np.isneginf(want_lse)
    assert np.all(np.isneginf(got_lse[empty])) and np.all(got[empty] == 0)
    live = ~empty
    if not live.any():
        return
    diff = np.abs(got - want)
    if dtype == "f32":
        assert np.max(diff[live]) <= FP32_MAX_ABS
        assert np.max(np.abs(got_lse[live] - want_lse[live])) <= FP32_MAX_ABS
        return
    vmax = np.array([np.abs(x).max() if x.size else 0.0 for x in v_of])[:, None, None]
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * err[..., None]) * vmax + 1e-6
    assert np.all(diff[live] <= tol[live]), (diff[live] - tol[live]).max()
    rel = np.linalg.norm(diff[live]) / np.linalg.norm(want[live])
    assert rel <= BF16_REL_L2, rel
    assert np.all(np.abs(got_lse[live] - want_lse[live]) <= (err + 1e-5 * np.abs(want_lse) + 1e-5)[live])


DECODE = [
    # lens, prefix, page, n_h, n_kv, Dqk, Dv, options
    ([1], 0, 16, 1, 1, 64, 64, {}),
    ([333], 0, 16, 32, 8, 128, 128, dict(rope=5e5)),
    ([128, 129, 127, 1, 255, 257], 0, 32, 8, 2, 128, 128, dict(rope=1e4)),
    ([700, 1, 0, 64, -3, 2100], 0, 64, 32, 8, 128, 128, dict(rope=5e5, pairing="half")),
    ([1000, 17, 4000], 0, 16, 12, 12, 64, 64, {}),
    ([300, 40], 0, 128, 28, 4, 128, 128, dict(rope=1e4)),       # 7 heads per KV head
    ([513, 30, 255], 0, 256, 8, 1, 64, 64, dict(rope=1e4, pairing="half", scale=0.3)),
    ([300, 1, 77], 0, 16, 20, 1, 128, 128, {}),                 # 20 heads per KV head
    ([200, 65], 0, 16, 128, 1, 64, 64, {}),                     # 128 heads per KV head
    ([1030, 12], 0, 32, 6, 3, 128, 64, {}),                     # unequal head dims: CUDA cores
    ([100, 333], 0, 32, 6, 2, 96, 96, dict(rope=1e4)),
    ([100, 333], 0, 32, 6, 2, 128, 128, dict(rope=1e4, roff=64, rdims=64)),  # RoPE on half of the head
    ([50, 300], 0, 16, 6, 2, 256, 256, dict(rope=1e4)),
    ([300, 129], 0, 64, 16, 1, 576, 512, dict(rope=1e4, roff=512, rdims=64, alias=True)),
    ([1, 2, 100, 0, 1024], 0, 32, 12, 12, 64, 64, dict(dtype="f32")),
    ([700, 33], 0, 16, 10, 2, 128, 128, dict(dtype="f32", rope=5e5, pairing="half")),
    ([5000], 0, 16, 3, 1, 40, 24, dict(dtype="f32")),
    # 128 heads over one latent head (the MLA-absorbed shape, on CTA pairs), values in front of the keys
    ([300, 129, 1, 0, 1030, 256], 0, 16, 128, 1, 576, 512, dict(rope=1e4, roff=512, rdims=64, alias=True)),
    ([513, 40], 0, 64, 128, 1, 576, 512, dict(scale=0.0722, alias=True)),
    ([2000, 100, 257], 0, 256, 128, 1, 576, 512, dict(rope=1e4, roff=512, rdims=64, pairing="half", alias=True)),
    ([900, 600, 513, 3, 512, 1300], 512, 32, 128, 1, 576, 512, dict(rope=1e4, roff=512, rdims=64, alias=True)),
    ([4000 + 300 * i for i in range(5)], 3968, 128, 128, 1, 576, 512, dict(alias=True)),
    ([300, 40], 0, 64, 128, 1, 576, 512, {}),                   # values apart from the keys: CUDA cores
    # behind a shared prefix
    ([17], 16, 16, 1, 1, 64, 64, {}),
    ([65, 128, 100, 64, 0], 64, 64, 32, 8, 128, 128, dict(rope=5e5)),
    ([2049, 2100, 3000, 2500], 2048, 64, 32, 8, 128, 128, dict(rope=5e5, pairing="half")),
    ([1041 + 7 * i for i in range(40)], 1040, 16, 32, 8, 128, 128, dict(rope=1e4)),   # 160 rows: a pair of tiles
    ([273 + i for i in range(33)], 272, 16, 32, 8, 64, 64, dict(rope=1e4)),           # 132 rows
    ([545 + 3 * i for i in range(100)], 544, 32, 16, 2, 128, 128, {}),                # 800 rows
    ([300 + i for i in range(97)], 256, 256, 28, 4, 64, 64, dict(rope=1e4)),          # 679 rows
    ([1100, 1024, 1025, 1030], 1024, 128, 12, 12, 64, 64, {}),
    ([400, 390], 384, 32, 128, 1, 128, 128, dict(rope=1e4)),
    ([130, 150, 129], 128, 32, 6, 2, 96, 96, dict(rope=1e4)),
    ([1100, 1025, 1030], 1024, 16, 16, 1, 576, 512, dict(rope=1e4, roff=512, rdims=64, alias=True)),
    ([1030, 1025, 10, 1200, 1999, 1026], 1024, 32, 12, 12, 64, 64, dict(dtype="f32")),
    ([600, 700, 513], 512, 16, 10, 2, 128, 128, dict(dtype="f32", rope=5e5)),
]


@pytest.mark.parametrize("lens,prefix,page,n_h,n_kv,Dqk,Dv,opts", DECODE)
def test_decode(lib, lens, prefix, page, n_h, n_kv, Dqk, Dv, opts):
    check_decode(lib, lens, prefix, page, n_h, n_kv, Dqk, Dv, **opts)


@pytest.mark.parametrize("prefix", [0, 64])
def test_decode_of_empty_batch_places_only(lib, prefix):
    check_decode(lib, [prefix, 0, -1, -2**31], prefix, 16, 8, 2, 128, 128)
    check_decode(lib, [prefix, 0, -1, -2**31], prefix, 16, 6, 2, 96, 96)


@pytest.mark.parametrize("prefix,D,dtype", [(0, 128, "bf16"), (64, 128, "bf16"), (64, 64, "bf16"), (64, 96, "bf16"),
                                            (64, 64, "f32")])
def test_lowest_lengths_are_empty_places(lib, prefix, D, dtype):
    """Between live requests: the lowest lengths less a prefix do not fit 32 bits."""
    low = -2**31
    check_decode(lib, [400, low, 700, low + 1, low + prefix, 0, 300], prefix, 16, 8, 2, D, D, dtype=dtype)


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "bf16"), (96, "bf16"), (64, "f32")])
def test_lengths_above_the_table_are_clamped(lib, D, dtype):
    dt = TYPES[dtype]
    k, v, table, pre, k_of, v_of = ref.make_cache([80, 80], 32, 16, 2, D, D, dt)
    q = torch.randn(2, 8, D, generator=torch.Generator().manual_seed(9)).to(dt)
    want, want_lse, err = ref.attend(q, k_of, v_of, scale=0.1)
    for n in (81, 2**31 - 1):
        out, lse = lib.decode_shared(q.to(DEV), k.to(DEV), v.to(DEV), pre.to(DEV), table.to(DEV), ints([80, n]),
                                     scale=0.1, lse=True)
        check_result(to_np(out), to_np(lse), want, want_lse, err, v_of, dtype)


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "bf16"), (96, "bf16"), (64, "f32"), (576, "bf16")])
def test_pages_outside_the_cache_read_as_zero(lib, D, dtype):
    dt = TYPES[dtype]
    lens, prefix, page = [200, 150, 90], 64, 16
    mla = D == 576
    n_kv, n_h, Dv = (1, 128, 512) if mla else (2, 8, D)
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, page, n_kv, D, Dv, dt, alias=mla)
    q = torch.randn(3, n_h, D, generator=torch.Generator().manual_seed(9)).to(dt)
    n_pages = k.shape[0]
    for (b, j), bad in (((0, 5), -1), ((0, 12), n_pages), ((1, 4), 2**31 - 1), ((1, 9), -2**31), ((2, 5), 1 << 27)):
        table[b, j] = bad
        k_of[b][j * page:(j + 1) * page] = 0
        v_of[b][j * page:(j + 1) * page] = 0
    pre[2] = n_pages + 5
    for b in range(3):
        k_of[b][2 * page:3 * page] = 0
        v_of[b][2 * page:3 * page] = 0
    want, want_lse, err = ref.attend(q, k_of, v_of)
    kd = k.to(DEV)
    vd = kd[..., :Dv] if mla else v.to(DEV)
    out, lse = lib.decode_shared(q.to(DEV), kd, vd, pre.to(DEV), table.to(DEV), ints(lens), lse=True)
    check_result(to_np(out), to_np(lse), want, want_lse, err, v_of, dtype)
    # the same cache read as one without a prefix
    whole = torch.cat([pre.repeat(3, 1), table[:, 4:]], 1).contiguous()
    out, lse = lib.decode_paged(q.to(DEV), kd, vd, whole.to(DEV), ints(lens), lse=True)
    check_result(to_np(out), to_np(lse), want, want_lse, err, v_of, dtype)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_large_scores(lib, dtype, D):
    """Scores of a few hundred: one key takes nearly all the weight, and the running maximum moves often."""
    dt = TYPES[dtype]
    lens, prefix = [900, 700, 1300], 512
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 32, 2, D, D, dt, seed=4)
    q = (20 * torch.randn(3, 8, D, generator=torch.Generator().manual_seed(9))).to(dt)
    want, want_lse, _ = ref.attend(q, k_of, v_of)
    out, lse = lib.decode_shared(q.to(DEV), k.to(DEV), v.to(DEV), pre.to(DEV), table.to(DEV), ints(lens), lse=True)
    # fp32 dot products of |terms| summing to at most ~20 * D: off by a few 2^-24 of that, times scale
    e = 20 * D * 8 * 2.0 ** -24
    vmax = max(np.abs(x).max() for x in v_of)
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert np.max(np.abs(to_np(out) - want)) <= (2 * eps + 2 * e) * vmax
    assert np.max(np.abs(to_np(lse) - want_lse)) <= e + 1e-5 * np.max(np.abs(want_lse))


@pytest.mark.parametrize("B,G,D,dtype", [(4, 4, 128, "bf16"), (40, 4, 128, "bf16"), (80, 4, 64, "bf16"), (4, 4, 96, "bf16"),
                                         (3, 2, 96, "bf16"), (3, 2, 64, "f32"), (20, 2, 64, "f32"), (3, 1, 256, "f32")])
@pytest.mark.parametrize("prefix", [0, 128])
def test_nan_of_a_live_token_shows(lib, B, G, D, dtype, prefix):
    """A NaN in a query, a key or a value reaches the rows that see it, and no other."""
    dt = TYPES[dtype]
    lens = [prefix + 40 + 150 * (b % 3) for b in range(B)]
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 16, 2, D, D, dt, seed=8)
    q = torch.randn(B, 2 * G, D, generator=torch.Generator().manual_seed(5)).to(dt)
    want, want_lse, err = ref.attend(q, k_of, v_of)
    own = table[:, prefix // 16:]
    q[1, 0] = float("nan")                         # head 0 of request 1
    k[own[0, 1], 3, 1, 7] = float("nan")           # a key of request 0, KV head 1
    v[own[2, 2], 15, 0, 9] = float("nan")          # a value of request 2, KV head 0, dim 9
    if prefix:
        out, lse = lib.decode_shared(q.to(DEV), k.to(DEV), v.to(DEV), pre.to(DEV), table.to(DEV), ints(lens), lse=True)
    else:
        out, lse = lib.decode_paged(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV), ints(lens), lse=True)
    out, lse = to_np(out), to_np(lse)
    bad = np.zeros(out.shape, bool)
    bad[1, 0] = bad[0, G:] = bad[2, :G, 9] = True
    np.testing.assert_array_equal(np.isnan(out), bad)
    np.testing.assert_array_equal(np.isnan(lse), bad.all(-1))
    out[bad], lse[bad.all(-1)] = want[bad], want_lse[bad.all(-1)]
    check_result(out, lse, want, want_lse, err, v_of, dtype)


# The rows of a piece on the tensor cores: in groups of eight with the rests of their queries (own keys of up to
# 64 heads per KV head; a prefix's of up to eight groups), or one after the other.
ROWS = [
    # lens, prefix, heads per KV head
    ([70, 300, 129, 128, 1] * 3, 0, 1),
    ([70, 300], 0, 8), ([70, 300], 0, 9), ([140, 33, 600], 0, 31), ([140, 33], 0, 32), ([300, 140, 33], 0, 33),
    ([300, 140, 33], 0, 64), ([300, 140], 0, 65), ([300, 140], 0, 96),
    ([70 + i for i in range(64)], 64, 1), ([70 + i for i in range(65)], 64, 1),     # 8 groups of 8 requests, 9
    ([400 + i for i in range(16)], 256, 3), ([400 + i for i in range(17)], 256, 3),  # 8 groups of 2 requests, 9
    ([400 + i for i in range(8)], 256, 5), ([400 + i for i in range(9)], 256, 5),
    ([200, 129, 0, 400], 128, 16), ([200, 129, 130, 0, 400], 128, 16),              # 8 groups, 10
    ([200, 129, 400], 128, 12), ([200, 400], 128, 32), ([200, 0, 400], 128, 32), ([400], 128, 64), ([129], 128, 128),
]


@pytest.mark.parametrize("lens,prefix,G", ROWS)
@pytest.mark.parametrize("D,rope", [(128, 1e4), (64, 1e4), (128, 0.0)])
def test_rows_of_a_piece(lib, lens, prefix, G, D, rope):
    check_decode(lib, lens, prefix, 16, 2 * G, 2, D, D, rope=rope, pairing="half" if G & 1 else "adjacent")


@pytest.mark.parametrize("lens,prefix,G", [([1000, 30, 300], 0, 4), ([1000, 300], 0, 64), ([1000, 30, 300], 16, 20),
                                           ([1000, 30], 16, 20),
                                           ([500 + i for i in range(16)], 480, 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_grouped_rows_keep_their_rests(lib, lens, prefix, G, D):
    """Rows in groups are as good as fp32 but for the stored result: queries and weights to 17 bits, so that a score
    is off by at most e = 2^-16 |q| |k| / sqrt(D) and a weight by 2 e + 2^-16, fp32 sums and the rotation's angles
    (positions below 2^10, fp32 sine and cosine) by some 2^-16 more.  Three requests' 20 heads are 3 x 3 = 9 groups,
    one too many for the prefix: there e has the 2^-8 of a bf16 query, and a weight another 2^-8."""
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 16, 2, D, D, torch.bfloat16, seed=6)
    q = torch.randn(len(lens), 2 * G, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    want, want_lse, _ = ref.attend(q, k_of, v_of, rope_base=1e4)
    out, lse = lib.decode_shared(q.to(DEV), k.to(DEV), v.to(DEV), pre.to(DEV), table.to(DEV), ints(lens), rope_base=1e4,
                                 lse=True) if prefix else \
        lib.decode_paged(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV), ints(lens), rope_base=1e4, lse=True)
    norm = max(np.linalg.norm(x, axis=-1).max() for x in k_of if x.size)
    groups = -(-len(lens) // (8 // G)) if G <= 8 else len(lens) * -(-G // 8)
    bits = 2.0 ** -8 if prefix and groups > 8 else 2.0 ** -16
    e = bits * q.double().norm(dim=-1).max().item() * norm / D ** 0.5
    vmax = max(np.abs(x).max() for x in v_of if x.size)
    got = to_np(out)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2 * e + bits + 2.0 ** -16) * vmax)
    live = np.isfinite(want_lse)
    assert np.max(np.abs(to_np(lse) - want_lse)[live]) <= e + 2.0 ** -16 * np.max(np.abs(want_lse[live])) + 2.0 ** -16


@pytest.mark.parametrize("n_h,n_kv,D,Dv,dtype,slots", [
    (32, 8, 128, 128, "bf16", 2_300_032), (12, 6, 96, 96, "bf16", 3_900_032), (8, 8, 128, 128, "f32", 2_300_032),
    (128, 1, 576, 512, "bf16", 3_900_032)])
def test_offsets_past_32_bits(lib, n_h, n_kv, D, Dv, dtype, slots):
    """A cache of more than 2^31 elements: pages at its far end, written and read, give what a small cache gives."""
    dt, page, mla = TYPES[dtype], 64, D == 576
    lens, prefix = [200, 130, 64 + 1], 64
    assert slots * n_kv * D > 2**31
    k, v, table, pre, _, _ = ref.make_cache(lens, prefix, page, n_kv, D, Dv, dt, alias=mla)
    n = k.shape[0]
    shift = slots // page - n
    rope = dict(rope_base=1e4, rope_offset=512, rope_dims=64) if mla else dict(rope_base=1e4)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(3, n_h, D, generator=g).to(dt).to(DEV)
    k_new = torch.randn(3, n_kv, D, generator=g).to(dt).to(DEV)
    v_new = None if mla else torch.randn(3, n_kv, Dv, generator=g).to(dt).to(DEV)

    def run(k, v, first):
        last = [int(table[b, (L - 1) // page]) * page + (L - 1) % page for b, L in enumerate(lens)]
        lib.kv_append_paged(k_new, v_new, k, v, ints([first * page + x for x in last]), ints([L - 1 for L in lens]), **rope)
        t, p = (table + first).to(DEV), (pre + first).to(DEV)
        whole = torch.cat([p.repeat(3, 1), t[:, 1:]], 1).contiguous()
        return (lib.decode_shared(q, k, v, p, t, ints(lens), **rope, lse=True) +
                lib.decode_paged(q, k, v, whole, ints(lens), **rope, lse=True))

    ks, big_k = k.to(DEV), torch.empty(slots // page, page, n_kv, D, dtype=dt, device=DEV)
    big_k[-n:] = ks
    if mla:
        vs, big_v = ks[..., :Dv], big_k[..., :Dv]
    else:
        vs, big_v = v.to(DEV), torch.empty(slots // page, page, n_kv, Dv, dtype=dt, device=DEV)
        big_v[-n:] = vs
    for a, b in zip(run(ks, vs, 0), run(big_k, big_v, shift)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_shared_equals_paged(lib):
    """The same batch with and without the prefix computed once: equal up to rounding."""
    lens, prefix, page = [3000 + 37 * i for i in range(24)], 2944, 64
    k, v, table, pre, _, _ = ref.make_cache(lens, prefix, page, 8, 128, 128, torch.bfloat16, seed=2)
    q = torch.randn(24, 32, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    k, v = k.to(DEV), v.to(DEV)
    a, la = lib.decode_shared(q, k, v, pre.to(DEV), table.to(DEV), ints(lens), rope_base=5e5, lse=True)
    whole = torch.cat([pre.repeat(24, 1), table[:, prefix // page:]], 1).contiguous().to(DEV)
    b, lb = lib.decode_paged(q, k, v, whole, ints(lens), rope_base=5e5, lse=True)
    assert (a.float() - b.float()).norm() / b.float().norm() <= BF16_REL_L2
    # Only the prefix's 96 rows a KV head have their queries rounded (a request's own 4 rows, and all of b's, keep
    # the rest): components off by at most 2^-8 of themselves move a score by at most 2^-8 |q| |k| / sqrt(128),
    # and a log-sum-exp by no more than its scores.  fp32 sums: 1e-4.
    moved = 2.0 ** -8 * q.float().norm(dim=-1).max() * k[~k.isnan().any(-1)].float().norm(dim=-1).max() / 128 ** 0.5
    assert (la - lb).abs().max() <= moved + 1e-4


def test_repeated_calls_give_the_same_bits(lib):
    for opts in (dict(), dict(dtype="f32")):
        lens, prefix = [1100 + 61 * i for i in range(30)], 1024
        a = check_decode(lib, lens, prefix, 32, 16, 4, 64, 64, **opts)
        for _ in range(3):
            b = check_decode(lib, lens, prefix, 32, 16, 4, 64, 64, **opts)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_workspace_contents_and_size(lib):
    lens, prefix, page = [600, 513, 900], 512, 64
    n = lib.decode_paged_workspace_size(3, 8, 2, 128, 128, page, 15, prefix)
    a = check_decode(lib, lens, prefix, page, 8, 2, 128, 128)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)  # NaN everywhere
    b = check_decode(lib, lens, prefix, page, 8, 2, 128, 128, workspace=ws)
    assert torch.equal(a[0], b[0])
    with pytest.raises(lib.AttnError, match="workspace"):
        check_decode(lib, lens, prefix, page, 8, 2, 128, 128, workspace=ws[:1024])


def test_outputs_given_and_rows_around_them(lib):
    lens, page = [100, 300], 16
    buf = torch.full((4, 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, 8), 7.0, device=DEV)
    k, v, table, _, k_of, v_of = ref.make_cache(lens, 0, page, 2, 64, 64, torch.bfloat16)
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    want, want_lse, err = ref.attend(q, k_of, v_of)
    out, l2 = lib.decode_paged(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV), ints(lens), out=buf[1:3], lse=lse[1:3])
    check_result(to_np(out), to_np(l2), want, want_lse, err, v_of, "bf16")
    assert torch.all(buf[0] == 7) and torch.all(buf[3] == 7) and torch.all(lse[0] == 7) and torch.all(lse[3] == 7)


def test_on_another_stream(lib):
    st = torch.cuda.Stream()
    check_decode(lib, [600, 513, 900], 512, 64, 8, 2, 128, 128, stream=st)
    check_decode(lib, [600, 513, 900], 0, 64, 6, 2, 96, 96, stream=st)


def test_two_calls_on_two_streams(lib):
    """Calls that overlap, each with the scratch that it allocates itself."""
    lens, prefix = [2100 + 100 * i for i in range(8)], 2048
    k, v, table, pre, _, _ = (x.to(DEV) if torch.is_tensor(x) else x for x in
                              ref.make_cache(lens, prefix, 64, 8, 128, 128, torch.bfloat16))
    q = [torch.randn(8, 32, 128, device=DEV).to(torch.bfloat16) for _ in range(2)]
    sl = ints(lens)
    want = [lib.decode_shared(x, k, v, pre, table, sl)[0].clone() for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [lib.decode_shared(x, k, v, pre, table, sl, stream=s)[0] for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# -------------------------------------------------------------------------------------- used together
class Server:
    """The buffers of a serving loop over one paged cache, B requests behind one shared prompt."""

    def __init__(self, lib, B, prefix, page, n_h, n_kv, D, dtype, steps, rope):
        self.lib, self.page, self.prefix, self.rope = lib, page, prefix, rope
        self.n_pages = prefix // page + B * (-(-steps // page) + 1)
        self.k_pages = torch.full((self.n_pages, page, n_kv, D), float("nan"), dtype=dtype, device=DEV)
        self.v_pages = torch.full_like(self.k_pages, float("nan"))
        self.free = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(3)).int().to(DEV)
        self.n_free = [ints([self.n_pages]), ints([0])]
        self.lens = [ints([prefix] * B), ints([0] * B)]
        self.table = torch.full((B, prefix // page + -(-steps // page) + 1), -1, dtype=torch.int32, device=DEV)
        self.one = ints([1] * B)

    def prompt(self, k, v):
        """Writes the shared prompt's pages (taken by a plan of one request) and puts them into every row."""
        n = k.shape[0]
        row = torch.full((1, self.table.shape[1]), -1, dtype=torch.int32, device=DEV)
        _, _, slots, pos, left = self.lib.page_plan(ints([0]), ints([n]), row, self.free, self.n_free[0],
                                                    page_size=self.page, n_pages=self.n_pages, max_tokens=n)
        self.lib.kv_append_paged(k, v, self.k_pages, self.v_pages, slots, pos, rope_base=self.rope)
        self.n_free[0].copy_(left)
        self.pre = row[0, :n // self.page].contiguous()
        self.table[:, :n // self.page] = self.pre

    def step(self, i, q, k, v):
        """One decode step: plan, append, attend (the two copies of the state take turns)."""
        a, b = i % 2, 1 - i % 2
        _, _, slots, pos, _ = self.lib.page_plan(self.lens[a], self.one, self.table, self.free, self.n_free[a],
                                                 page_size=self.page, n_pages=self.n_pages, max_tokens=q.shape[0],
                                                 seqlens=self.lens[b], n_left=self.n_free[b])
        self.lib.kv_append_paged(k, v, self.k_pages, self.v_pages, slots, pos, rope_base=self.rope)
        out, _ = self.lib.decode_shared(q, self.k_pages, self.v_pages, self.pre, self.table, self.lens[b],
                                        rope_base=self.rope)
        return out


@pytest.mark.parametrize("dtype,n_h,n_kv,D,graph", [("bf16", 32, 8, 128, False), ("bf16", 32, 8, 128, True),
                                                    ("bf16", 12, 12, 64, True), ("f32", 8, 2, 64, False)])
def test_serving_loop(lib, dtype, n_h, n_kv, D, graph):
    """A prompt shared by five requests, then decode steps that cross page ends - eagerly, or as two captured
    steps replayed in turn - against attention over contiguous caches in 64 bits."""
    import oracle
    dt, rope, B, page, prefix, steps = TYPES[dtype], 1e4, 5, 16, 160, 36
    g = torch.Generator().manual_seed(11)
    pk, pv = (torch.randn(prefix, n_kv, D, generator=g).to(dt) for _ in range(2))
    qs, ks, vs = (torch.randn(steps, B, h, D, generator=g).to(dt) for h in (n_h, n_kv, n_kv))
    s = Server(lib, B, prefix, page, n_h, n_kv, D, dt, steps + 4, rope)
    s.prompt(pk.to(DEV), pv.to(DEV))
    outs = []
    if graph:
        q, k, v = (torch.empty_like(x[0]).to(DEV) for x in (qs, ks, vs))
        for x, y in zip((q, k, v), (qs, ks, vs)):
            x.copy_(y[0])
        graphs, results = [], []
        keep = [x.clone() for x in (*s.lens, *s.n_free, s.table)]
        s.step(0, q, k, v)                    # warm-up of both steps, then back to the start
        s.step(1, q, k, v)
        for x, y in zip((*s.lens, *s.n_free, s.table), keep):
            x.copy_(y)
        torch.cuda.synchronize()
        for i in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                results.append(s.step(i, q, k, v))
        for i in range(steps):
            for x, y in zip((q, k, v), (qs, ks, vs)):
                x.copy_(y[i])
            graphs[i % 2].replay()
            outs.append(results[i % 2].clone())
    else:
        for i in range(steps):
            outs.append(s.step(i, qs[i].to(DEV), ks[i].to(DEV), vs[i].to(DEV)))
    torch.cuda.synchronize()
    pos = np.arange(prefix + steps)
    for b in range(B):
        kk = np.concatenate([pk.double().numpy(), ks[:, b].double().numpy()])
        vv = np.concatenate([pv.double().numpy(), vs[:, b].double().numpy()])
        kk = oracle.rope_rotate(kk, pos[:, None], rope)
        for i in (0, 1, 15, 16, 17, 31, 35):
            n = prefix + i + 1
            want, _ = oracle.attention_decode(qs[i, b:b + 1], kk[None, :n], vv[None, :n], np.array([n]),
                                              rope_base=rope)
            diff = np.abs(to_np(outs[i][b]) - want[0])
            if dtype == "f32":
                assert diff.max() <= FP32_MAX_ABS
            else:
                assert np.linalg.norm(diff) / np.linalg.norm(want) <= BF16_REL_L2 * 1.5  # cached keys rounded as well


def test_calls_refuse_what_does_not_fit(lib):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV)
    t, sl = ints([[0, 1], [2, 3]]), ints([5, 6])
    for bad in (dict(q=q.float()), dict(q=q[..., ::2]), dict(k=k[:, ::2]), dict(v=k.clone()[..., :32]), dict(v=k[:3]),
                dict(t=t[:1]), dict(t=t.long()), dict(sl=sl[:1]), dict(sl=sl.cpu()), dict(out=q.float()),
                dict(out=q[:1]), dict(lse=torch.zeros(2, 4, device=DEV)), dict(pairing="other")):
        a = dict(q=q, k=k, v=k.clone(), t=t, sl=sl)
        a.update({x: y for x, y in bad.items() if x in a})
        rest = {x: y for x, y in bad.items() if x not in a}
        with pytest.raises((ValueError, TypeError)):
            lib.decode_paged(a["q"], a["k"], a["v"], a["t"], a["sl"], **rest)
    with pytest.raises(ValueError, match="slice"):     # the slice's heads are not D_v apart
        lib.decode_paged(q, k, k[..., :32], t, sl)
    with pytest.raises(lib.AttnError):                 # values over the keys
        lib.kv_append_paged(k[0, :2], k[0, :2], k, k, ints([0, 1]))
    with pytest.raises(lib.AttnError):
        lib.decode_shared(q, k, k.clone(), ints([0, 1, 2]), t, sl)   # a prefix longer than the table
    with pytest.raises(lib.AttnError):
        lib.decode_shared(q, k, k.clone(), ints([]), t, sl)
    with pytest.raises(lib.AttnError):
        lib.kv_append_paged(k[0, :2], k[0, :2], k, k.clone(), ints([0, 1]), None, rope_base=1e4)
    with pytest.raises((ValueError, TypeError)):
        lib.kv_append_paged(k[0, :2].float(), k[0, :2], k, k.clone(), ints([0, 1]))
    lib.kv_append_paged(k[0, :0], k[0, :0], k, k.clone(), ints([]))  # nothing to write
