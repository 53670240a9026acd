"""The paged cache at the ends of its arguments' ranges: tables that end with the prefix, infinities, positions of more
than 24 bits, tables far wider than their requests, single-token appends.

Tolerances are those of tests/test_gpu_paged.py where a test names none of its own.
"""
import numpy as np
import pytest
import torch

import oracle
from tests import paged_reference as ref
from tests.test_gpu_paged import DEV, TYPES, check_decode, check_result, ints, lib  # noqa: F401 (lib is a fixture)
from tests.tolerances import to_np

pytestmark = pytest.mark.gpu

# one shape per path: n_h, n_kv, D_qk, D_v, dtype; 576: the MLA-absorbed shape, values in front of the keys
SHAPES = [(8, 2, 128, 128, "bf16"), (8, 2, 64, 64, "bf16"), (8, 2, 96, 96, "bf16"), (8, 2, 64, 64, "f32"),
          (128, 1, 576, 512, "bf16")]


def normal(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def to64(t):
    return t.double().numpy()


# ------------------------------------------------------------------------------- lengths above the table
@pytest.mark.parametrize("n_h,n_kv,D,Dv,dtype", SHAPES)
def test_lengths_above_a_table_that_ends_with_the_prefix_are_empty_places(lib, n_h, n_kv, D, Dv, dtype):
    """They are clamped to the table, the prefix, so that they own no token."""
    dt, prefix, page = TYPES[dtype], 64, 16
    k, v, _, pre, _, _ = ref.make_cache([prefix], prefix, page, n_kv, D, Dv, dt, alias=D == 576)
    lens = [prefix + 1, prefix, 2**31 - 1, 0, prefix + 300]
    table = pre.repeat(len(lens), 1).contiguous()
    kd = k.to(DEV)
    vd = kd[..., :Dv] if D == 576 else v.to(DEV)
    out, lse = lib.decode_shared(normal((len(lens), n_h, D), dt, 1).to(DEV), kd, vd, pre.to(DEV), table.to(DEV),
                                 ints(lens), lse=True)
    assert torch.all(out == 0) and torch.all(lse == -torch.inf)


@pytest.mark.parametrize("n_h,n_kv,D,Dv,dtype", SHAPES)
def test_lengths_above_a_longer_table_are_clamped(lib, n_h, n_kv, D, Dv, dtype):
    dt = TYPES[dtype]
    k, v, table, pre, k_of, v_of = ref.make_cache([80, 80, 80], 32, 16, n_kv, D, Dv, dt, alias=D == 576)
    q = normal((3, n_h, D), dt, 9)
    want, want_lse, err = ref.attend(q, k_of, v_of, scale=0.1)
    kd = k.to(DEV)
    vd = kd[..., :Dv] if D == 576 else v.to(DEV)
    out, lse = lib.decode_shared(q.to(DEV), kd, vd, pre.to(DEV), table.to(DEV), ints([81, 80, 2**31 - 1]), scale=0.1,
                                 lse=True)
    check_result(to_np(out), to_np(lse), want, want_lse, err, v_of, dtype)


# --------------------------------------------------------------------------------------------- infinities
# B, heads per KV head, D, dtype: rows in groups with the rests of their roundings, one after the other, CUDA cores
NON_FINITE = [(4, 4, 128, "bf16"), (4, 4, 64, "bf16"), (40, 4, 128, "bf16"), (4, 4, 96, "bf16"), (3, 2, 64, "f32"),
              (20, 2, 64, "f32")]


@pytest.mark.parametrize("prefix", [0, 128])
@pytest.mark.parametrize("rope", [0.0, 1e4])
@pytest.mark.parametrize("B,G,D,dtype", NON_FINITE)
def test_infinite_values_reach_their_rows(lib, B, G, D, dtype, rope, prefix):
    """A weight above 0 times an infinite value is that infinity; both infinities in one dim give NaN.  (Scores of
    these inputs lie within some 30 of each other, so that no weight is 0.)"""
    dt = TYPES[dtype]
    lens = [prefix + (1, 40, 190, 340)[b % 4] for b in range(B)]
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 16, 2, D, D, dt, seed=8)
    q = normal((B, 2 * G, D), dt, 5)
    want, want_lse, err = ref.attend(q, k_of, v_of, rope_base=rope)
    own = table[:, prefix // 16:]
    inf = float("inf")
    v[own[0, 0], 0, 0, 9] = inf        # request 0's first own token, without a prefix its only one: KV head 0, dim 9
    v[own[1, 2], 3, 1, 0] = -inf       # request 1, KV head 1
    v[own[2, 3], 15, 0, D - 1] = inf   # request 2: two of one sign, two of both
    v[own[2, 9], 1, 0, D - 1] = inf
    v[own[2, 0], 2, 1, 8] = inf
    v[own[2, 11], 0, 1, 8] = -inf
    for h, want_inf in ((slice(0, G), (0, 9, inf)), (slice(G, None), (1, 0, -inf)), (slice(0, G), (2, D - 1, inf)),
                        (slice(G, None), (2, 8, float("nan")))):
        b, d, x = want_inf
        want[b, h, d] = x
    if prefix:
        v[pre[3], 5, 1, 3] = -inf      # a shared token: every request's rows of KV head 1
        want[:, G:, 3] = -inf
        call, first = lib.decode_shared, (pre.to(DEV), table.to(DEV))
    else:
        call, first = lib.decode_paged, (table.to(DEV),)
    out, lse = call(q.to(DEV), k.to(DEV), v.to(DEV), *first, ints(lens), rope_base=rope, lse=True)
    check_non_finite(to_np(out), to_np(lse), want, want_lse, err, v_of, dtype)


def check_non_finite(out, lse, want, want_lse, err, v_of, dtype):
    odd = ~np.isfinite(want)
    np.testing.assert_array_equal(out[odd], want[odd])
    odd_lse = ~np.isfinite(want_lse)
    np.testing.assert_array_equal(lse[odd_lse], want_lse[odd_lse])
    assert np.isfinite(out[~odd]).all() and np.isfinite(lse[~odd_lse]).all()
    check_result(np.where(odd, 0, out), np.where(odd_lse, 0, lse), np.where(odd, 0, want),
                 np.where(odd_lse, 0, want_lse), err, v_of, dtype)


@pytest.mark.parametrize("prefix", [0, 128])
@pytest.mark.parametrize("rope", [0.0, 1e4])
@pytest.mark.parametrize("B,G,D,dtype", NON_FINITE)
def test_keys_with_a_score_of_minus_infinity_have_no_weight(lib, B, G, D, dtype, rope, prefix):
    """An infinite component of a key makes its score -inf for the heads whose (rotated) query has the other sign
    there - their rows are those without that key - and inf for the others, whose softmax is NaN."""
    dt = TYPES[dtype]
    lens = [prefix + (2, 40, 190, 340)[b % 4] for b in range(B)]
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 16, 2, D, D, dt, seed=8)
    q = normal((B, 2 * G, D), dt, 5)
    own = table[:, prefix // 16:]
    turned = to64(q) if rope <= 0 else np.stack([oracle.rope_rotate(to64(q[b]), np.full(2 * G, lens[b] - 1), rope)
                                                 for b in range(B)])
    hit = np.zeros((B, 2 * G), int)     # the sign of the infinite score that a row sees

    def spoil(b, g, key, d, sign):      # key of request b's own, KV head g
        n = prefix + key
        k[own[b, key // 16], key % 16, g, d] = sign * float("inf")
        rows = slice(g * G, (g + 1) * G)
        assert np.abs(turned[b, rows, d]).min() > 1e-3  # the sign hangs on no rounding
        hit[b, rows] = np.sign(sign * turned[b, rows, d])
        k_of[b][n, g] = 0               # for the rows of score -inf: as if the key were not there
        gone.append((b, g, n))
    gone = []
    spoil(0, 1, 0, 7, 1)
    spoil(1, 0, 33, D // 2, -1)
    spoil(2, 1, 128, 0, 1)
    want, want_lse = np.zeros((B, 2 * G, D)), np.zeros((B, 2 * G))
    err = np.zeros((B, 2 * G))
    for g in range(2):                  # each KV head of each request with its own set of keys
        rows = slice(g * G, (g + 1) * G)
        keep = [np.setdiff1d(np.arange(lens[b]), [n for bb, gg, n in gone if (bb, gg) == (b, g)]) for b in range(B)]
        for b in range(B):
            s = turned[b, rows] @ k_of[b][keep[b], g].T / np.sqrt(D)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            want[b, rows] = p @ v_of[b][keep[b], g] / p.sum(-1, keepdims=True)
            want_lse[b, rows] = top[:, 0] + np.log(p.sum(-1))
            if rope > 0:
                err[b, rows] = (np.abs(turned[b, rows]) @ np.abs(k_of[b][:, g]).T).max(-1) / np.sqrt(D) * 2.0 ** -8
    if prefix:
        call, first = lib.decode_shared, (pre.to(DEV), table.to(DEV))
    else:
        call, first = lib.decode_paged, (table.to(DEV),)
    out, lse = call(q.to(DEV), k.to(DEV), v.to(DEV), *first, ints(lens), rope_base=rope, lse=True)
    out, lse = to_np(out), to_np(lse)
    assert (hit > 0).any() and (hit < 0).any()
    assert np.isnan(out[hit > 0]).all() and not np.isfinite(lse[hit > 0]).any()
    out[hit > 0], lse[hit > 0] = want[hit > 0], want_lse[hit > 0]
    check_result(out, lse, want, want_lse, err, v_of, dtype)


@pytest.mark.parametrize("prefix", [0, 128])
def test_latent_rows_with_a_score_of_minus_infinity_have_no_weight(lib, prefix):
    """The same in the MLA-absorbed shape, in the dims behind the values (0 times an infinite value would be NaN)."""
    lens = [prefix + n for n in (2, 340, 700)]
    k, _, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 16, 1, 576, 512, torch.bfloat16, seed=8, alias=True)
    q = normal((3, 128, 576), torch.bfloat16, 5)
    own = table[:, prefix // 16:]
    spoilt = [(0, 1, 570), (1, 300, 512), (2, 129, 575)]  # request, own key, dim
    hit = np.zeros((3, 128), bool)
    for b, key, d in spoilt:
        k[own[b, key // 16], key % 16, 0, d] = float("inf")
        hit[b] = to64(q)[b, :, d] > 0
        k_of[b], v_of[b] = (np.delete(x, prefix + key, 0) for x in (k_of[b], v_of[b]))
    want, want_lse, err = ref.attend(q, k_of, v_of, scale=0.0722)
    kd = k.to(DEV)
    call, first = (lib.decode_shared, (pre.to(DEV), table.to(DEV))) if prefix else (lib.decode_paged, (table.to(DEV),))
    out, lse = call(q.to(DEV), kd, kd[..., :512], *first, ints(lens), scale=0.0722, lse=True)
    out, lse = to_np(out), to_np(lse)
    assert np.isnan(out[hit]).all() and not np.isfinite(lse[hit]).any()
    out[hit], lse[hit] = want[hit], want_lse[hit]
    check_result(out, lse, want, want_lse, err, v_of, "bf16")


@pytest.mark.parametrize("prefix", [0, 128])
@pytest.mark.parametrize("far", [False, True])
def test_nan_of_a_live_latent_row_shows(lib, prefix, far):
    """The MLA-absorbed shape, whose keys' first dims are the values: a NaN in a query reaches its head's row, a NaN in
    a latent row (in its values, in its rotary part) all heads of the request, and neither any other row.  far: the
    key's score lies so far below the others' that its piece's weight is 0, and 0 times NaN is NaN."""
    lens = [prefix + n for n in (40, 4190, 340, 700, 90)]
    k, _, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 16, 1, 576, 512, torch.bfloat16, seed=8, alias=True)
    q = normal((5, 128, 576), torch.bfloat16, 5)
    own = table[:, prefix // 16:]
    if far:  # request 1's first 2048 own keys score far below the others
        rows = k[own[1, :128].long()]
        k[own[1, :128].long()] = (-40 * q[1, 0] + rows * 0).to(torch.bfloat16)
        k_of[1][prefix:prefix + 2048] = v_of[1][prefix:prefix + 2048] = 0
    want, want_lse, err = ref.attend(q, k_of, v_of, scale=0.0722)
    q[3, 77, 500] = float("nan")
    k[own[1, 2], 3, 0, 7] = float("nan")
    k[own[2, 5], 15, 0, 570] = float("nan")
    kd = k.to(DEV)
    if prefix:
        call, first = lib.decode_shared, (pre.to(DEV), table.to(DEV))
    else:
        call, first = lib.decode_paged, (table.to(DEV),)
    out, lse = call(q.to(DEV), kd, kd[..., :512], *first, ints(lens), scale=0.0722, lse=True)
    out, lse = to_np(out), to_np(lse)
    bad = np.zeros((5, 128), bool)
    bad[3, 77] = bad[1] = bad[2] = True
    np.testing.assert_array_equal(np.isnan(out), np.broadcast_to(bad[..., None], out.shape))
    np.testing.assert_array_equal(np.isnan(lse), bad)
    out[bad], lse[bad] = want[bad], want_lse[bad]
    check_result(out, lse, want, want_lse, err, v_of, "bf16")


# ------------------------------------------------------------------------- positions of more than 24 bits
FAR = [2**24 - 1, 2**24, 2**24 + 1, 2**24 + 3, 2**25 + 1, 2**27 + 5, 2**30 + 63, 2**31 - 2**16 - 1, 2**31 - 1, -1,
       -2**24 - 1, -2**31, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairing", ["adjacent", "half"])
@pytest.mark.parametrize("D,roff,rdims", [(128, 0, 128), (64, 0, 64), (128, 64, 64), (576, 512, 64)])
def test_append_at_far_positions(lib, D, roff, rdims, pairing, dtype):
    """Frequencies f (in turns, at most 0.16) are held to 2^-48 of themselves, so that an angle is off by |pos| 2^-48
    from there - doubled for the power that f comes from -, by some 1e-6 from fp32 sums of turns below 2, and by 1e-6
    from sine and cosine; the result is rounded once."""
    dt, T = TYPES[dtype], len(FAR)
    k = normal((T, 2, D), dt, 3)
    kp = torch.zeros(2, 16, 2, D, dtype=dt, device=DEV)
    lib.kv_append_paged(k.to(DEV), k[..., :8].contiguous().to(DEV), kp, torch.zeros(2, 16, 2, 8, dtype=dt, device=DEV),
                        ints(range(T)), ints(FAR), rope_base=1e4, rope_offset=roff, rope_dims=rdims, pairing=pairing)
    got = to_np(kp.flatten(0, 1)[:T])
    pos = np.array(FAR, dtype=np.float64)[:, None]
    want = oracle.rope_rotate(to64(k), np.broadcast_to(pos, (T, 2)), 1e4, roff, rdims, pairing=pairing)
    half_step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    angle = 2 * np.abs(pos[..., None]) * 2.0 ** -48 + 4e-6
    longest = 2 ** 0.5 * k.double().abs().max().item()  # of a pair
    assert np.all(np.abs(got - want) <= half_step * np.abs(want) + angle * longest)


@pytest.mark.parametrize("n", [2**24 + 2, 2**25 + 4])
@pytest.mark.parametrize("n_h,n_kv,D,Dv,roff,dtype,pairing,shared", [
    (4, 1, 128, 128, 0, "bf16", "adjacent", False), (4, 1, 64, 64, 0, "bf16", "half", False),
    (4, 1, 64, 64, 32, "bf16", "adjacent", False), (2, 1, 64, 64, 0, "f32", "adjacent", False),
    (2, 1, 64, 64, 0, "f32", "half", True), (16, 1, 64, 64, 0, "f32", "adjacent", True),
    (128, 1, 576, 512, 512, "bf16", "adjacent", False), (128, 1, 576, 512, 512, "bf16", "half", True)])
def test_decode_at_far_positions(lib, n, n_h, n_kv, D, Dv, roff, dtype, pairing, shared):
    """n keys in four pages that the table lists over and over: the softmax over 1024 distinct keys, each as often as
    it occurs.  The query's fastest pair is long, and the
    values repeat the keys', so that the angle decides where the output points."""
    dt, page = TYPES[dtype], 256
    kp = normal((4, page, 1, D), dt, 7)
    q = normal((1, n_h, D), dt, 9) / 4
    rope = dict(rope_base=1e4, rope_offset=roff, rope_dims=D - roff, pairing=pairing)
    first = [roff, roff + 1] if pairing == "adjacent" else [roff, roff + (D - roff) // 2]
    q[..., first] = q[..., first] * 64
    if D == 576:
        kp[..., :2] = kp[..., first]
    vp = kp[..., :Dv].contiguous()
    blocks = -(-n // page)
    table = (torch.arange(blocks, dtype=torch.int32) % 4)[None].to(DEV)
    times = np.bincount(np.arange(n) % (4 * page), minlength=4 * page)
    turned = oracle.rope_rotate(to64(q[0]), np.full(n_h, n - 1), 1e4, roff, D - roff, pairing=pairing)
    s = turned @ to64(kp).reshape(-1, D).T / np.sqrt(D) + np.log(times)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    want = (p @ to64(vp).reshape(-1, Dv) / p.sum(-1, keepdims=True))[None]
    want_lse = (top[:, 0] + np.log(p.sum(-1)))[None]
    err = ((np.abs(turned) @ np.abs(to64(kp).reshape(-1, D)).T).max(-1) / np.sqrt(D))[None]
    kd, qd = kp.to(DEV), q.to(DEV)
    vd = kd[..., :Dv] if D == 576 else vp.to(DEV)
    if shared:
        out, lse = lib.decode_shared(qd, kd, vd, table[0, :blocks - 1].contiguous(), table, ints([n]), lse=True, **rope)
    else:
        out, lse = lib.decode_paged(qd, kd, vd, table, ints([n]), lse=True, **rope)
    # angles are off by some 4e-6 (see above), a score by as much of err's dot product of absolute values
    moved = err * (4e-6 if dtype == "f32" else 2.0 ** -8 + 4e-6)
    diff, vmax = np.abs(to_np(out) - want), np.abs(to64(vp)).max()
    weights = 2 * moved[..., None] + (2.0 ** -8 if dtype == "bf16" else 1e-5)  # fp32 sums over 2^24 and more keys: 1e-5
    assert np.all(diff <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(want) + weights * vmax)
    assert np.all(np.abs(to_np(lse) - want_lse) <= moved + 1e-5 * np.abs(want_lse) + 1e-5)


# ---------------------------------------------------------------------- tables wider than their requests
@pytest.mark.parametrize("prefix", [0, 64])
@pytest.mark.parametrize("n_h,n_kv,D,Dv,dtype,opts", [
    (12, 12, 64, 64, "f32", {}), (32, 8, 128, 128, "bf16", dict(rope_base=1e4, rope_offset=64)),
    (6, 2, 96, 96, "bf16", {}), (16, 1, 576, 512, "bf16", {}), (32, 8, 128, 128, "bf16", {}), (10, 2, 256, 256, "f32", {}),
    (128, 1, 576, 512, "bf16", {})])
def test_a_wider_table_changes_nothing(lib, n_h, n_kv, D, Dv, dtype, opts, prefix):
    """Work is cut by the requests' lengths: not a bit depends on how many blocks a table row has room for."""
    dt = TYPES[dtype]
    lens = [1000, 0, 700, 65, 1900]
    alias = D == 576
    k, v, table, pre, k_of, v_of = ref.make_cache(lens, prefix, 16, n_kv, D, Dv, dt, alias=alias)
    q = normal((5, n_h, D), dt, 1).to(DEV)
    kd = k.to(DEV)
    vd = kd[..., :Dv] if alias else v.to(DEV)
    wide = torch.full((5, 64 * table.shape[1]), -7, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    results = []
    for t in (table, wide):
        if prefix:
            results.append(lib.decode_shared(q, kd, vd, pre.to(DEV), t.to(DEV), ints(lens), lse=True, **opts))
        else:
            results.append(lib.decode_paged(q, kd, vd, t.to(DEV), ints(lens), lse=True, **opts))
    (a, la), (b, lb) = results
    assert torch.equal(a, b) and torch.equal(la, lb)
    want, want_lse, err = ref.attend(q.cpu(), k_of, v_of, **opts)
    check_result(to_np(a), to_np(la), want, want_lse, err, v_of, dtype)


# requests, prefix, lengths of their own: from one key each to a single request among empty places
MIXES = [(1, 0, [4097]), (1, 0, [70000]), (2, 0, [1, 30000]), (40, 0, [5000] + [1] * 39), (300, 0, [1 + i % 130 for i in range(300)]),
         (33, 0, [0] * 32 + [9000]), (33, 0, [9000] + [0] * 32), (64, 256, [0, 1, 64, 65] * 16), (1, 1024, [3]),
         (9, 2048, [300] * 9), (2500, 0, [1 + i % 3 for i in range(2500)])]


@pytest.mark.parametrize("B,prefix,own", MIXES)
@pytest.mark.parametrize("n_h,n_kv,D,Dv,dtype", [(6, 2, 96, 96, "bf16"), (4, 4, 64, 64, "f32"), (5, 1, 256, 192, "f32")])
def test_mixes_of_lengths_on_cuda_cores(lib, B, prefix, own, n_h, n_kv, D, Dv, dtype):
    check_decode(lib, [prefix + n for n in own], prefix, 32, n_h, n_kv, D, Dv, dtype=dtype)


# ----------------------------------------------------------------------------------- single-token appends
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairing", ["adjacent", "half"])
@pytest.mark.parametrize("n_kv,D,Dv,rope,roff,rdims,alias", [
    (1, 64, 64, 1e4, 0, 64, False), (8, 128, 128, 5e5, 0, 128, False), (3, 128, 64, 1e4, 64, 64, False),
    (2, 72, 40, 0.0, 0, 72, False), (1, 576, 512, 1e4, 512, 64, True)])
def test_append_of_one_token(lib, n_kv, D, Dv, rope, roff, rdims, alias, pairing, dtype):
    """One token to one slot, and nothing else; to a slot outside the cache, nothing at all."""
    dt, page, n_pages = TYPES[dtype], 16, 3
    k, v = normal((1, n_kv, D), dt, 1), normal((1, n_kv, Dv), dt, 2)
    kp = normal((n_pages, page, n_kv, D), dt, 3)
    vp = kp[..., :Dv] if alias else normal((n_pages, page, n_kv, Dv), dt, 4)
    want = oracle.rope_rotate(to64(k), np.full((1, n_kv), 777), rope, roff, rdims, pairing=pairing) if rope > 0 else to64(k)
    for slot in (0, 17, n_pages * page - 1, -1, n_pages * page):
        kd = kp.to(DEV)
        vd = kd[..., :Dv] if alias else vp.to(DEV)
        lib.kv_append_paged(k.to(DEV), None if alias else v.to(DEV), kd, vd, ints([slot]), ints([777]) if rope > 0 else None,
                            rope_base=rope, rope_offset=roff, rope_dims=rdims, pairing=pairing)
        got, others = kd.flatten(0, 1).cpu(), torch.arange(n_pages * page) != slot
        assert torch.equal(got[others], kp.flatten(0, 1)[others])
        if not alias:
            assert torch.equal(vd.flatten(0, 1).cpu()[others], vp.flatten(0, 1)[others])
        if 0 <= slot < n_pages * page:
            # half a step of the stored type, and 1e-6 of the pair's norm for the fp32 rotation
            eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
            assert np.all(np.abs(to_np(got[slot]) - want[0]) <= eps * np.abs(want[0]) + 1e-6 * np.sqrt(2) * 6)
            if not alias:
                assert torch.equal(vd.flatten(0, 1)[slot].cpu(), v[0])


# --------------------------------------------------------------------------------- captured and side by side
@pytest.mark.parametrize("prefix", [0, 64])
@pytest.mark.parametrize("n_h,n_kv,D,Dv,dtype", SHAPES)
def test_a_captured_call_follows_the_lengths(lib, n_h, n_kv, D, Dv, dtype, prefix):
    """A graph is captured once; what it computes is cut by the lengths that it finds when it runs."""
    dt, most = TYPES[dtype], [2500, 1000, 300, 90, 1700]
    k, v, table, pre, _, _ = ref.make_cache([prefix + n for n in most], prefix, 16, n_kv, D, Dv, dt, alias=D == 576,
                                            fill=0.5)
    kd, td, pd = k.to(DEV), table.to(DEV), pre.to(DEV)
    vd = kd[..., :Dv] if D == 576 else v.to(DEV)
    q, lens = normal((5, n_h, D), dt, 1).to(DEV), ints([prefix + n for n in most])

    def call():
        if prefix:
            return lib.decode_shared(q, kd, vd, pd, td, lens, lse=True)
        return lib.decode_paged(q, kd, vd, td, lens, lse=True)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    for own in (most, [1, 1, 1, 1, 1], [0, 0, 300, 0, 0], [0] * 5, [2500, 0, 1, 64, 65]):
        lens.copy_(ints([prefix + n for n in own]))
        want, want_lse = call()
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_fp32_calls_on_two_streams(lib):
    """Calls on CUDA cores that overlap, each with the scratch that it allocates itself."""
    lens, prefix = [2100 + 100 * i for i in range(8)], 2048
    k, v, table, pre, _, _ = (x.to(DEV) if torch.is_tensor(x) else x for x in
                              ref.make_cache(lens, prefix, 64, 4, 64, 64, torch.float32))
    q = [normal((8, 16, 64), torch.float32, i).to(DEV) for i in range(2)]
    sl = ints(lens)
    want = [lib.decode_shared(x, k, v, pre, table, sl)[0].clone() for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [lib.decode_shared(x, k, v, pre, table, sl, stream=s)[0] for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
