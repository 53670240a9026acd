"""Steps of several tokens per request at the edges of their numbers: queries of zero and near it beside huge keys,
infinite values whose keys have no weight, what two-part queries and weights are worth, and table entries of no page beside
the free stack.  Inputs, references and element-wise bars are those of tests/test_gpu_packed.py.
"""
import numpy as np
import pytest
import torch

from tests import packed_reference as ref
from tests.test_gpu_packed import DEV, Step, ints, lib  # noqa: F401 (lib: the module's fixture)
from tests.tolerances import to_np

pytestmark = pytest.mark.gpu
TC = [(8, 2, 128, "bf16"), (4, 4, 64, "bf16")]
ALL = TC + [(4, 2, 64, "f32"), (4, 2, 96, "bf16")]


def set_key(s, b, places, dims, value, head=slice(None)):
    """Key elements of request b at the given places, in the cache and for the reference."""
    page = s.k.shape[1]
    for p in np.atleast_1d(places):
        for d in np.atleast_1d(dims):
            s.k[int(s.table[b, p // page]), p % page, head, d] = value
            s.k_of[b][p, head, d] = float(torch.tensor(value).to(s.k.dtype))


def set_value(s, b, place, dim, value):
    page = s.v.shape[1]
    s.v[int(s.table[b, place // page]), place % page, 0, dim] = value


# ------------------------------------------------------------------------------------------- queries of zero
@pytest.mark.parametrize("n_h,n_kv,D,dtype", ALL)
@pytest.mark.parametrize("pairing", ["adjacent", "half"])
@pytest.mark.parametrize("tree", [False, True])
def test_zero_query_elements_beside_huge_keys(lib, n_h, n_kv, D, dtype, pairing, tree):  # noqa: F811
    """Where the rotated query is 0 a finite key, however large, adds nothing: the same bits as with a key of 0."""
    dims = [6, 7] if pairing == "adjacent" else [6, 6 + D // 2]
    s = Step([70, 20, 3], [200, 0, 5], n_h, n_kv, D, dtype=dtype, tree=tree, base=1e4, pairing=pairing, seed=2)
    s.q[..., dims] = 0
    got = []
    for value in (0.0, 3e38, -3e38, 2.0 ** 90):
        set_key(s, 0, np.arange(0, 270, 3), dims, value)
        set_key(s, 1, np.arange(20), dims, value)
        got.append(s.run(lib))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("n_h,n_kv,D,dtype", ALL)
@pytest.mark.parametrize("tree", [False, True])
def test_tiny_query_elements_beside_huge_keys(lib, n_h, n_kv, D, dtype, tree):  # noqa: F811
    """Query elements that bf16 holds exactly (dims behind the rotated span, and position 0), 2^-104 against keys of
    2^106: 4 in the sum."""
    s = Step([70, 20, 3], [200, 0, 5], n_h, n_kv, D, dtype=dtype, tree=tree, base=1e4, dims=32, seed=6)
    s.q[..., 40] = s.q[..., 40].sign() * 2.0 ** -104
    sign = np.where(np.random.default_rng(1).random(270) < 0.5, -1.0, 1.0)
    for p in range(270):
        set_key(s, 0, p, 40, sign[p] * 2.0 ** 106)
    for p in range(20):
        set_key(s, 1, p, 40, sign[p] * 2.0 ** 106)
    for p in range(8):
        set_key(s, 2, p, 40, 0.0)
    s.check(lib)


@pytest.mark.parametrize("n_h,n_kv,D", [c[:3] for c in TC])
@pytest.mark.parametrize("tree", [False, True])
def test_infinite_keys_beside_exact_queries(lib, n_h, n_kv, D, tree):  # noqa: F811
    """Query elements that bf16 holds exactly, against an infinite key: -inf (no weight) or inf (NaN), by their signs."""
    for place in (3, 130, 210):
        for value in (float("inf"), float("-inf")):
            s = Step([70, 20], [200, 10], n_h, n_kv, D, tree=tree, base=1e4, dims=32, seed=7)
            s.q[::2, :, 40] = 2.0 ** -60  # a power of two: both parts differ from it
            s.q[1::4, :, 40] = -1.0
            set_key(s, 0, place, 40, value, head=0)
            out, _ = s.run(lib)
            sees = ref.causal(70, 200) if not tree else ref.tree(70, 200, s.visible[:70])
            sees = np.broadcast_to(sees[:, place][:, None], (70, n_h)) & (np.arange(n_h) < n_h // n_kv)[None]
            up = sees & (s.q[:70, :, 40].float().numpy() * value > 0)
            o = to_np(out)
            assert np.isnan(o[:70][up]).all()
            assert np.isfinite(o[:70][~up]).all() and np.isfinite(o[70:]).all()


# ------------------------------------------------------------------------------------------- values without weight
@pytest.mark.parametrize("n_h,n_kv,D,dtype", ALL)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("base", [0.0, 1e4])
def test_infinite_values_of_keys_without_weight(lib, n_h, n_kv, D, dtype, tree, base):  # noqa: F811
    """0 times an infinity is NaN, in tiles that rows see whole and in part: keys whose score is -inf, or so low that its
    exponential is 0 in 32 bits (2^-150 is half the least number there is; these scores are below -500 times log2 e).  A
    key with a weight, however small, gives the infinity."""
    sc = D ** -0.5
    for place in (3, 127, 130, 199, 205, 210):  # of request 0: 200 tokens held, 70 new ones
        for value in (float("inf"), float("-inf")):
            for score in (float("-inf"), -1000.0, -30.0):
                s = Step([70, 20], [200, 10], n_h, n_kv, D, dtype=dtype, tree=tree, base=base, dims=32 if base else None,
                         seed=8)
                s.q[..., 40] = 1.0
                clean, clean_lse = s.run(lib)
                set_key(s, 0, place, 40, score / sc, head=0)
                low, low_lse = s.run(lib)  # what the rows are with finite values
                set_value(s, 0, place, 9, value)
                out, lse = s.run(lib)
                sees = ref.causal(70, 200) if not tree else ref.tree(70, 200, s.visible[:70])
                hit = np.zeros((s.T, n_h), bool)
                hit[:70, :n_h // n_kv] = sees[:, place][:, None]
                assert hit.any() and not hit[:70].all()
                hit = torch.as_tensor(hit, device=DEV)
                x = out[hit][:, 9].float()
                assert (x == value).all() if score == -30.0 else torch.isnan(x).all(), (place, value, score)
                rest = torch.arange(D, device=DEV) != 9
                assert torch.equal(out[hit][:, rest], low[hit][:, rest]) and torch.isfinite(out[hit][:, rest]).all()
                assert torch.equal(out[~hit], clean[~hit])
                assert torch.equal(lse, low_lse) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("n_h,n_kv,D,dtype", ALL)
@pytest.mark.parametrize("tree", [False, True])
def test_infinite_values_in_parts_without_weight(lib, n_h, n_kv, D, dtype, tree):  # noqa: F811
    """The same where the key axis is cut, and a whole part has scores of -inf alone: the value is not lost."""
    n, ctx = 3, 9000
    lo, hi = 2000, 7000  # keys with a score of -inf for KV head 0
    for place in (lo, 2100, 4444, hi - 1, ctx):  # the last: of the first new token, alone with a weight of 0 in its tile
        s = Step([n], [ctx], n_h, n_kv, D, dtype=dtype, tree=tree, page=64, seed=9)
        s.q[..., 40] = 1.0
        s.k.view(-1, n_kv, D)[s.table[0].long().repeat_interleave(64)[lo:hi] * 64 + torch.arange(lo, hi) % 64, 0, 40] = -float("inf")
        set_key(s, 0, place, 40, -float("inf"), head=0)
        low, low_lse = s.run(lib)
        assert torch.isfinite(low).all() and torch.isfinite(low_lse).all()
        set_value(s, 0, place, 9, float("inf"))
        out, lse = s.run(lib)
        sees = (ref.causal(n, ctx) if not tree else ref.tree(n, ctx, s.visible))[:, place]
        hit = np.zeros((n, n_h), bool)
        hit[:, :n_h // n_kv] = sees[:, None]
        hit = torch.as_tensor(hit, device=DEV)
        rest = torch.arange(D, device=DEV) != 9
        assert torch.isnan(out[hit][:, 9]).all(), place
        assert torch.equal(out[hit][:, rest], low[hit][:, rest]) and torch.equal(out[~hit], low[~hit])
        assert torch.equal(lse, low_lse)


@pytest.mark.parametrize("n_h,n_kv,D,dtype", ALL)
def test_rows_without_any_weight_stay_zero(lib, n_h, n_kv, D, dtype):  # noqa: F811
    """All scores -inf: the row is one that sees no key, whatever the values are, in one piece or many."""
    for news, ctx in (([2, 1], 0), ([1, 5], 9000)):
        s = Step(news, [ctx, 3], n_h, n_kv, D, dtype=dtype, page=64, seed=10)
        s.q[..., 40] = 1.0
        n = news[0] + ctx
        at = s.table[0].long().repeat_interleave(64)[:n] * 64 + torch.arange(n) % 64
        s.k.view(-1, n_kv, D)[at, 0, 40] = -float("inf")
        s.v.view(-1, n_kv, D)[at[::3], 0, 9] = float("inf")
        s.v.view(-1, n_kv, D)[at[1::3], 0, 10] = float("nan")
        out, lse = s.run(lib)
        heads = n_h // n_kv
        assert not out[:news[0], :heads].any() and torch.isneginf(lse[:news[0], :heads]).all()
        assert torch.isfinite(out).all() and torch.isfinite(lse[:, heads:]).all() and torch.isfinite(lse[news[0]:]).all()


@pytest.mark.parametrize("n_h,n_kv,D,dtype", ALL)
@pytest.mark.parametrize("tree", [False, True])
def test_what_the_workspace_held_does_not_matter(lib, n_h, n_kv, D, dtype, tree):  # noqa: F811
    """Parts that hold nothing for some rows (a row tile behind its last key among them) come out alike from a workspace
    of NaN and one of zeros; the key axis is cut at other places from case to case."""
    for news, ctx in (([130], 0), ([200], 60), ([257, 3], 500), ([300], 1000), ([700], 90), ([1500, 140], 0), ([128], 3000)):
        if tree:
            news = [min(n, 128) for n in news]
        s = Step(news, [ctx] * len(news), n_h, n_kv, D, dtype=dtype, tree=tree, base=1e4, seed=ctx + news[0])
        args = s.tensors()
        n = lib.packed_workspace_size(s.T, len(news), n_h, n_kv, D, D, 16, s.table.shape[1], s.k.dtype)
        got = [s.run(lib, args, workspace=torch.full((n,), fill, dtype=torch.uint8, device=DEV)) for fill in (0, 255)]
        assert torch.isfinite(got[1][0]).all()
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ------------------------------------------------------------------------------------------- two-part queries and weights
def step_error(s, lib):  # noqa: F811
    """The error of bf16 outputs against 64 bits, over that of the reference's own rounding to bf16 (norms)."""
    out, _ = s.run(lib)
    want = s.want()[0]
    once = torch.as_tensor(want).to(torch.bfloat16).double().numpy()
    return np.linalg.norm(to_np(out) - want) / np.linalg.norm(once - want)


@pytest.mark.parametrize("D,offset,dims,pairing", [
    (64, 0, None, "adjacent"), (64, 0, None, "half"), (64, 8, 48, "half"), (128, 0, None, "adjacent"),
    (128, 0, None, "half"), (128, 8, 56, "adjacent"), (128, 64, 64, "half"), (128, 72, 48, "half")])
@pytest.mark.parametrize("tree", [False, True])
def test_error_of_two_part_queries_and_weights(lib, D, offset, dims, pairing, tree):  # noqa: F811
    """For normally distributed inputs with scores of variance 1, in units of the output's own rounding (a relative error
    of variance e^2): a weight rounded once adds e^2 of the output's variance (sum (p e)^2 over sum p^2), and so does a
    query rounded once in all dims (its scores are off by e times a normal number).  Half of the weights and 64 of the query
    dims in two parts with D = 128 leave 1 + 1/2 + 1/2 at most, all query dims with D = 64 and weights rounded once 1 + 1:
    the square root is 1.41.  Where a whole head is rotated, second parts of half of the weights or queries lost and the
    first ones rounded are sqrt(2.5) = 1.58; as the first ones are cut off, a part lost has an error of variance 4 e^2 or
    more, and a factor of sqrt(1 + 1/2 + 4/2) = 1.87.  The bar is half way between 1.41 and 1.58."""
    s = Step([40, 64], [1500, 900], 8, 2, D, page=64, base=5e5, pairing=pairing, offset=offset, dims=dims, tree=tree,
             seed=D + offset)
    assert step_error(s, lib) <= 1.5


@pytest.mark.parametrize("D,offset,dims", [(64, 0, 64), (64, 16, 32), (128, 0, 64), (128, 8, 48), (128, 64, 64), (128, 72, 48)])
@pytest.mark.parametrize("pairing", ["adjacent", "half"])
@pytest.mark.parametrize("tree", [False, True])
def test_second_parts_of_queries(lib, D, offset, dims, pairing, tree):  # noqa: F811
    """Queries within the 64 dims that have second parts (from the start of the rotated span on, down to a multiple of
    16): scores are as of 16 bits.  Each term of a score is off by 2^-8 of what one bf16 leaves, at most 2^-7 of it where
    that is cut off: 2^-15; the rotation in fp32 with the hardware's sines (2^-21 each, two terms) and the sums add less
    than 2^-17 of the terms.  So the log-sum-exp is off by 2^-14 of the largest sum of |terms| at most, and a hundredth
    of what one rounding of every term may be."""
    s = Step([40, 64], [700, 3], 8, 2, D, page=64, base=5e5, pairing=pairing, offset=offset, dims=dims, tree=tree,
             seed=D + offset + 1)
    first = min(offset // 16 * 16, D - 64)
    keep = torch.zeros(D, dtype=torch.bool)
    keep[first:first + 64] = True
    s.q[..., ~keep] = 0
    _, lse = s.run(lib)
    _, want, _, err = s.want()  # err: with 2^-8 of every term
    d = np.abs(to_np(lse) - want)
    assert (d <= err * 2.0 ** -6 + 1e-6 * (1 + np.abs(want))).all(), float((d / err).max())


@pytest.mark.parametrize("tree", [False, True])
def test_second_parts_of_weights(lib, tree):  # noqa: F811
    """D = 128 with RoPE: values in the last 64 keys of each 128 alone.  Their weights are in two parts, off by 2^-15 (as above)
    and 2^-20, and so are the queries, here within their 64 dims; what is left is the output's rounding, half a step."""
    s = Step([40, 64], [700, 300], 8, 2, 128, page=64, base=5e5, dims=64, tree=tree, seed=5)
    s.q[..., 64:] = 0
    for b, n in enumerate(s.lens):
        at = s.table[b].long().repeat_interleave(64)[:n] * 64 + torch.arange(n) % 64
        first = torch.arange(n) % 128 < 64
        s.v.view(-1, 2, 128)[at[first]] = 0
        s.v_of[b][first.numpy()] = 0
    out, _ = s.run(lib)
    want, _, spread, err = s.want()
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -14 + np.expm1(2 * (err * 2.0 ** -6 + 1e-6))[..., None] + 1e-5) * spread
    d = np.abs(to_np(out) - want)
    assert (d <= tol).all(), float((d / tol).max())


# ------------------------------------------------------------------------------------------- the free stack
def freed(table, lens, seqlens, kept, page, n_pages):
    """Pages that fall free, from the definition: those of the cache among each row's surplus entries."""
    pages = []
    for b in range(len(lens)):
        for j in range(-(-kept[b] // page), -(-seqlens[b] // page)):
            if 0 <= table[b, j] < n_pages:
                pages.append(int(table[b, j]))
    return pages


@pytest.mark.parametrize("B,page,most", [(3, 16, 40), (300, 16, 90), (700, 32, 200), (2, 16, 20000), (40, 16, 3000)])
def test_pages_outside_the_cache_do_not_reach_the_stack(lib, B, page, most):  # noqa: F811
    """Entries of no page (behind those that a request owns, or anywhere) among what a commit gives back."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, most // 2, B)
    drafts = rng.integers(0, most // 2, B)
    lens[B // 2], drafts[B // 2] = 0, most
    seqlens = np.minimum(lens + drafts, most)
    width = -(-most // page)
    n_pages = B * width + 3
    table = rng.permutation(n_pages)[:B * width].reshape(B, width)
    bad = rng.random((B, width))
    table[bad < 0.15] = -1
    table[bad < 0.05] = n_pages
    table[bad < 0.03] = 2 ** 31 - 1
    table[bad < 0.01] = -2 ** 31
    table[0] = -1  # a request that owns nothing
    k = torch.zeros(n_pages, page, 1, 8, dtype=torch.bfloat16, device=DEV)
    path, n_path = np.zeros((B, 1)), rng.integers(0, 2, B)
    kept = lens + np.minimum(n_path, seqlens - lens)
    want = freed(table, lens, seqlens, kept, page, n_pages)
    for cap in sorted({n_pages, min(n_pages, 5 + len(want) // 2)}):
        stack = np.full(cap, -7)
        stack[:3] = [11, 12, 13]
        stack_t = ints(stack)
        new, left = lib.draft_commit(k, k.clone(), ints(table), ints(lens), ints(seqlens), ints(path), ints(n_path),
                                     stack_t, ints([3]))
        np.testing.assert_array_equal(new.cpu().numpy(), kept)
        stack[3:3 + len(want)] = want[:cap - 3]
        np.testing.assert_array_equal(stack_t.cpu().numpy(), stack)
        assert int(left) == min(cap, 3 + len(want))


def test_a_commit_of_lengths_above_the_table(lib):  # noqa: F811
    """seqlens is cut to the table, whose entries behind the request's pages are -1: the next plan hands out real pages."""
    page, n_pages, width = 16, 8, 6
    table = ints([[4, 2, -1, -1, -1, -1], [5, 1, 0, -1, -1, -1]])
    k = torch.zeros(n_pages, page, 1, 8, dtype=torch.bfloat16, device=DEV)
    free = ints([3, 6, 7, -7, -7, -7, -7, -7])
    lens, left = lib.draft_commit(k, k.clone(), table, ints([10, 30]), ints([2 ** 31 - 1, 40]), ints([[0], [0]]), ints([1, 1]),
                                  free, ints([3]))
    assert lens.tolist() == [11, 31] and int(left) == 5 and free.tolist() == [3, 6, 7, 2, 0, -7, -7, -7]
    _, _, slots, positions, left = lib.page_plan(lens, ints([10, 30]), table, free, left, page_size=page, n_pages=n_pages,
                                                 max_tokens=40)
    assert (slots >= 0).all() and (positions >= 0).all()
