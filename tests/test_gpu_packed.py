"""Steps that add several tokens per request on the GPU - packed prefill over pages, trees of drafted tokens, their
plan and commit - against plain references in 64 bits (tests/packed_reference.py), alone and as a speculative
serving loop runs them together.

Caches are filled with NaN wherever no token lives, and outputs with NaN before each call, so a read behind a
request's end and a row left as it was both show.  bf16 results are held to the parity bars of tests/tolerances.py
and element-wise to 2^-8 |o| (the stored result) + (2^-8 + exp(2 e) - 1) * sum p |v|: each weight rounded to bf16
(half a step, 2^-8 of it), and off by a factor of at most exp(2 e) for scores off by e, the reference's bound for a
rotated query rounded to bf16 (numerator and sum each by exp(e)); fp32 sums add 1e-5 of sum p |v|.  The
log-sum-exp is held to e + 1e-5 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

from tests import packed_reference as ref
from tests import paged_reference
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


class Step:
    """Inputs of one attention call: requests with news[b] new tokens behind ctxs[b], pad rows behind the last."""

    def __init__(self, news, ctxs, n_h, n_kv, D_qk, D_v=None, page=16, dtype="bf16", pad=0, seed=0, alias=False,
                 tree=False, words=None, masks=None, base=0.0, scale=None, pairing="adjacent", offset=0, dims=None):
        D_v = D_qk if D_v is None else D_v
        self.news, self.ctxs, self.n_h, self.D_v, self.dtype = news, ctxs, n_h, D_v, dtype
        lens = [n + c for n, c in zip(news, ctxs)]
        rng = np.random.default_rng(seed)
        self.k, self.v, self.table, _, self.k_of, self.v_of = paged_reference.make_cache(
            lens, 0, page, n_kv, D_qk, D_v, TYPES[dtype], seed=seed, alias=alias)
        self.cu = np.concatenate([[0], np.cumsum(news)])
        T = int(self.cu[-1]) + pad
        self.T = T
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(T, n_h, D_qk, generator=g).to(TYPES[dtype])
        self.positions = np.full(T, -1)
        self.visible = None
        if tree:
            words = words or max(1, -(-max(news) // 32))
            self.parents = [ref.random_tree(n, rng) for n in news]
            places = np.full(T, -1)
            for b, (n, c) in enumerate(zip(news, ctxs)):
                places[self.cu[b]:self.cu[b + 1]] = c + np.arange(n)
            flat = np.concatenate([np.asarray(p, np.int64) for p in self.parents] + [np.full(pad, -1)])
            self.positions, self.visible = ref.draft_plan(places, self.cu, flat, words)
            if masks is not None:
                self.visible = masks(rng, self.visible.shape).astype(np.uint32).view(np.int32)
        else:
            for b, (n, c) in enumerate(zip(news, ctxs)):
                self.positions[self.cu[b]:self.cu[b + 1]] = c + np.arange(n)
        self.lens = lens
        self.kw = dict(rope_base=base, pairing=pairing, rope_offset=offset, rope_dims=dims)
        self.scale = scale

    def tensors(self):
        k = self.k.to(DEV)
        v = k[..., :self.D_v] if self.v.data_ptr() == self.k.data_ptr() else self.v.to(DEV)
        return (self.q.to(DEV), k, v, self.table.to(DEV), ints(self.cu), ints(self.lens), ints(self.positions))

    def run(self, lib, args=None, **kw):
        args = args or self.tensors()
        out = torch.full((self.T, self.n_h, self.D_v), float("nan"), dtype=TYPES[self.dtype], device=DEV)
        lse = torch.full((self.T, self.n_h), float("nan"), device=DEV)
        kw = dict(self.kw, scale=self.scale or 0.0, out=out, lse=lse, **kw)
        if self.visible is None:
            got = lib.prefill_paged(*args, **kw)
        else:
            got = lib.decode_tree(*args, torch.as_tensor(self.visible).contiguous().to(DEV), **kw)
        assert got[0] is out and got[1] is lse
        return out, lse

    def want(self):
        T = self.T
        out, lse = np.zeros((T, self.n_h, self.D_v)), np.full((T, self.n_h), -np.inf)
        spread, err = np.zeros_like(out), np.zeros((T, self.n_h))
        for b, (n, c) in enumerate(zip(self.news, self.ctxs)):
            r = slice(int(self.cu[b]), int(self.cu[b + 1]))
            sees = ref.causal(n, c) if self.visible is None else ref.tree(n, c, self.visible[r])
            out[r], lse[r], spread[r], err[r] = ref.attend(
                self.q[r].double().numpy(), self.positions[r], sees, self.k_of[b], self.v_of[b], scale=self.scale,
                **self.kw)
        return out, lse, spread, err

    def check(self, lib, **kw):
        got, lse = self.run(lib, **kw)
        compare(got, lse, *self.want(), self.dtype)
        return got, lse


def compare(got, lse, want, want_lse, spread, err, dtype):
    o, l = to_np(got), to_np(lse)
    empty = np.isneginf(want_lse)
    np.testing.assert_array_equal(np.isneginf(l), empty)
    assert np.isfinite(o).all() and not o[empty].any()
    d = np.abs(o - want)
    if dtype == "f32":
        assert d.max(initial=0.0) <= FP32_MAX_ABS
        tol_l = np.full_like(want_lse, 1e-5)
    else:
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + np.expm1(2 * err)[..., None] + 1e-5) * spread
        assert (d <= tol + 1e-30).all(), float((d - tol).max())
        assert np.linalg.norm(o - want) <= BF16_REL_L2 * np.linalg.norm(want)
        tol_l = err + 1e-5
    with np.errstate(invalid="ignore"):
        assert (np.abs(l - want_lse)[~empty] <= (tol_l + 1e-5 * np.abs(want_lse))[~empty]).all()


# ------------------------------------------------------------------------------------------- packed prefill
RAGGED = [5, 0, 1, 64, 33, 129, 2, 31, 200]
HEADS = [(8, 2, 128), (4, 4, 64), (32, 8, 128), (6, 2, 64), (14, 2, 128), (8, 1, 64), (3, 3, 128), (40, 8, 64),
         (24, 1, 128), (96, 1, 64), (128, 1, 128)]


@pytest.mark.parametrize("n_h,n_kv,D", HEADS)
@pytest.mark.parametrize("base,pairing", [(0.0, "adjacent"), (1e4, "adjacent"), (5e5, "half")])
def test_prompts_of_different_lengths(lib, n_h, n_kv, D, base, pairing):
    Step(RAGGED, [0] * len(RAGGED), n_h, n_kv, D, page=16, pad=3, base=base, pairing=pairing, seed=n_h).check(lib)


@pytest.mark.parametrize("n_h,n_kv,D", HEADS[:5])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_chunks_behind_a_cache(lib, n_h, n_kv, D, page):
    """New tokens that start just before, at and behind the borders of key tiles."""
    Step([1, 40, 64, 3, 130, 17, 1, 1], [127, 128, 129, 255, 1000, 0, 0, 777], n_h, n_kv, D, page=page, base=1e4,
         seed=page).check(lib)


@pytest.mark.parametrize("n", [1, 2, 15, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("n_h,n_kv,D", [(8, 2, 128), (2, 2, 64)])
def test_one_prompt(lib, n, n_h, n_kv, D):
    Step([n], [0], n_h, n_kv, D, base=1e4, seed=n).check(lib)
    Step([n], [300 - n], n_h, n_kv, D, base=0.0, seed=n + 1).check(lib)


@pytest.mark.parametrize("n_h,n_kv,D_qk,D_v,dtype,offset,dims", [
    (4, 2, 64, 64, "f32", 0, None), (12, 12, 64, 64, "f32", 0, 32), (4, 1, 96, 96, "bf16", 0, None),
    (4, 2, 128, 128, "f32", 0, None), (4, 2, 192, 128, "bf16", 128, 64), (2, 1, 40, 72, "f32", 8, 16),
    (160, 1, 64, 64, "bf16", 0, None), (4, 2, 128, 128, "bf16", 64, 64), (4, 2, 64, 64, "bf16", 16, 16),
    (2, 2, 640, 512, "f32", 0, 256), (4, 2, 128, 64, "bf16", 0, None), (4, 2, 128, 128, "bf16", 2, 60)])
@pytest.mark.parametrize("pairing", ["adjacent", "half"])
def test_other_shapes(lib, n_h, n_kv, D_qk, D_v, dtype, offset, dims, pairing):
    kw = dict(page=32, dtype=dtype, base=1e4, offset=offset, dims=dims, pairing=pairing)
    Step([7, 1, 70, 0, 33], [0, 90, 5, 20, 64], n_h, n_kv, D_qk, D_v, pad=1, **kw).check(lib)
    Step([5, 40, 9], [70, 0, 130], n_h, n_kv, D_qk, D_v, tree=True, **kw).check(lib)


@pytest.mark.parametrize("n_h,n_kv,D_qk,D_v", [
    (3, 1, 96, 40), (5, 1, 40, 24), (6, 2, 8, 8), (4, 4, 64, 72), (14, 2, 128, 128), (7, 7, 64, 64), (2, 1, 120, 64),
    (100, 1, 32, 128), (4, 2, 136, 64), (4, 2, 64, 136)])
@pytest.mark.parametrize("tree", [False, True])
def test_f32_shapes(lib, n_h, n_kv, D_qk, D_v, tree):
    """Key parts of several tiles and of none, tiles that hold rows of several tokens or of part of one."""
    kw = dict(page=16, dtype="f32", base=1e4, tree=tree)
    Step([100, 1, 64, 0, 17], [0, 700, 5, 20, 333], n_h, n_kv, D_qk, D_v, pad=2, **kw).check(lib)
    Step([3], [1500], n_h, n_kv, D_qk, D_v, **kw).check(lib)
    Step([128] * 20, [64 * i for i in range(20)], n_h, n_kv, D_qk, D_v, **kw).check(lib)


def test_mla_latent_rows(lib):
    """128 heads over one latent head whose first dims are the values."""
    for tree in (False, True):
        Step([3, 1, 10], [50, 0, 200], 128, 1, 576, 512, page=64, alias=True, base=1e4, offset=512, dims=64,
             scale=192 ** -0.5, tree=tree).check(lib)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_keys_for_few_rows(lib, dtype):
    """The key axis is split."""
    D, lens = (128, [20000, 7001]) if dtype == "bf16" else (64, [6000, 1])
    Step([16, 3], lens, 8, 2, D, page=64, base=5e5, dtype=dtype).check(lib)
    Step([40, 64], lens, 8, 2, D, page=16, base=5e5, dtype=dtype, tree=True).check(lib)
    Step([1], lens[:1], 4, 4, D, page=128, dtype=dtype).check(lib)


def test_long_prompts(lib):
    Step([2000, 700, 1], [0, 1500, 3000], 4, 2, 128, page=64, base=5e5).check(lib)
    Step([1500], [0], 4, 4, 64, page=32, base=1e4).check(lib)


def test_many_requests(lib):
    rng = np.random.default_rng(5)
    news, ctxs = rng.integers(0, 4, 700).tolist(), rng.integers(0, 40, 700).tolist()
    for n_h, n_kv, D in ((8, 2, 128), (4, 4, 64)):
        Step(news, ctxs, n_h, n_kv, D, base=1e4, pad=9).check(lib)
    Step(news, ctxs, 4, 2, 64, base=1e4, dtype="f32").check(lib)


def test_padded_batches(lib):
    """Thousands of places without new tokens, with and without a cache, between a few that have some."""
    news, ctxs = [0] * 2500, [0] * 2500
    for b, n, c in ((0, 3, 0), (31, 40, 100), (32, 1, 5), (33, 70, 0), (1700, 129, 20), (2499, 2, 300)):
        news[b], ctxs[b] = n, c
    ctxs[40], ctxs[2000] = 500, 77
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 2, 64, "f32")):
        for tree in (False, True):
            Step(news, ctxs, n_h, n_kv, D, dtype=dtype, base=1e4, pad=4, tree=tree, words=4).check(lib)


def test_decode_is_the_single_token_case(lib):
    s = Step([1] * 6, [0, 5, 127, 128, 400, 2000], 8, 2, 128, base=5e5)
    args = s.tensors()
    out, lse = s.run(lib, args)
    one, one_lse = lib.decode_paged(args[0], args[1], args[2], args[3], args[5], rope_base=5e5, lse=True)
    o, l, spread, err = s.want()
    compare(out, lse, o, l, spread, err, "bf16")
    compare(one, one_lse, o, l, spread, err, "bf16")


def test_positions_are_the_rotations(lib):
    """Other positions than the places, far ones among them, and none at all."""
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 2, 64, "f32")):
        s = Step([9, 30], [4, 0], n_h, n_kv, D, base=1e4, dtype=dtype)
        s.positions = np.arange(39) * 55_000_001 % (2 ** 31)
        s.check(lib)
        plain = Step([9, 30], [4, 0], n_h, n_kv, D, base=1e4, dtype=dtype)
        args = plain.tensors()
        a, b = plain.run(lib, args), plain.run(lib, (*args[:6], None))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refused_requests_and_broken_offsets(lib):
    """What the page plan leaves for a request that does not fit, and rows past the end of q."""
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 2, 64, "f32")):
        s = Step([20, 30, 40], [100, 10, 0], n_h, n_kv, D, base=1e4, dtype=dtype)
        s.positions[20:50] = -1
        s.check(lib)
        # the last request's rows pass T: those that exist are its first ones
        s = Step([20, 30, 40], [100, 10, 7], n_h, n_kv, D, base=1e4, dtype=dtype)
        want = [x[:75] for x in s.want()]
        args = list(s.tensors())
        s.T = 75
        args[0], args[6] = args[0][:75].contiguous(), args[6][:75].contiguous()
        compare(*s.run(lib, args), *want, dtype)
        for cu in ([0, -5, 75, 10], [2 ** 31 - 1] * 4, [-1, 2 ** 31 - 1, 0, 2 ** 31 - 1], [75, 50, 25, 0]):
            args[4] = ints(cu)
            s.run(lib, args)  # no meaning, and no fault


def test_more_new_tokens_than_tokens(lib):
    """Tokens at places below 0 see nothing; lengths above the table are cut to it."""
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 2, 64, "f32")):
        for tree in (False, True):
            s = Step([40, 5], [0, 3], n_h, n_kv, D, dtype=dtype, tree=tree)
            args = list(s.tensors())
            args[5] = ints([25, 8])  # as if 15 tokens were missing in front
            if tree:
                s.visible[:] = -1
            out, lse = s.run(lib, args)
            k, v, q = s.k_of[0][:25], s.v_of[0][:25], s.q[:40].double().numpy()
            sees = np.arange(25)[None] <= np.arange(40)[:, None] - 15
            if tree:
                sees = np.broadcast_to((np.arange(40) >= 15)[:, None], (40, 25))
                # token j is at place j - 15, behind bit j: bits 32.. belong to words the row does not have
                sees = sees & (np.arange(25) + 15 < 32 * s.visible.shape[1])[None]
            o, l, spread, err = ref.attend(q, s.positions[:40], sees, k, v)
            compare(out[:40], lse[:40], o, l, spread, err, dtype)
    s = Step([20], [28], 8, 2, 128, page=16)
    args = list(s.tensors())
    a = s.run(lib, args)
    args[5] = ints([2 ** 31 - 1])  # 48 tokens fill the table's three pages
    b = s.run(lib, args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pages_outside_the_cache_read_as_zero(lib):
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 2, 64, "f32")):
        for tree in (False, True):
            s = Step([30, 20], [200, 0], n_h, n_kv, D, dtype=dtype, tree=tree)
            s.table[0, 3], s.table[0, 7], s.table[1, 0] = -1, s.k.shape[0], 2 ** 31 - 1
            for b, j in ((0, 3), (0, 7), (1, 0)):
                s.k_of[b][16 * j:16 * j + 16] = 0
                s.v_of[b][16 * j:16 * j + 16] = 0
            s.check(lib)


def test_nan_and_infinities_reach_their_rows_only(lib):
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 4, 64, "bf16"), (4, 2, 64, "f32")):
        for tree in (False, True):
            for what in ("k", "v", "q"):
                for value in (float("nan"), float("inf"), float("-inf")):
                    s = Step([70, 20, 64], [100, 10, 0], n_h, n_kv, D, dtype=dtype, tree=tree, seed=3)
                    clean, clean_lse = s.run(lib)
                    place = 140  # of request 0: its 40th new token
                    page, row = int(s.table[0, place // 16]), place % 16
                    if what == "q":
                        s.q[33, 1, 5] = value
                        touched = np.zeros(s.T, bool)
                        touched[33] = True
                        heads = [1]
                    else:
                        (s.k if what == "k" else s.v)[page, row, 0, 7] = value
                        sees = ref.causal(70, 100) if not tree else ref.tree(70, 100, s.visible[:70])
                        touched = np.zeros(s.T, bool)
                        touched[:70] = sees[:, place]
                        heads = list(range(n_h // n_kv))
                    assert touched.any() and not touched.all()
                    got, lse = s.run(lib)
                    hit = torch.zeros(s.T, n_h, dtype=torch.bool, device=DEV)
                    for h in heads:
                        hit[:, h] = torch.as_tensor(touched, device=DEV)
                    assert torch.equal(got[~hit], clean[~hit]), (what, value, tree)
                    assert torch.equal(lse[~hit], clean_lse[~hit])
                    if what == "v":
                        x = got[hit][:, 7]
                        assert torch.isnan(x).all() if value != value else (x == value).all()
                        rest = torch.ones(D, dtype=torch.bool)
                        rest[7] = False
                        assert torch.equal(got[hit][:, rest], clean[hit][:, rest])
                    elif value != value:
                        assert torch.isnan(got[hit]).all()


@pytest.mark.parametrize("n_h,n_kv,D,dtype", [(8, 2, 128, "bf16"), (4, 4, 64, "bf16"), (4, 2, 64, "f32")])
@pytest.mark.parametrize("tree", [False, True])
def test_infinities_behind_a_rotation(lib, n_h, n_kv, D, dtype, tree):
    """Values, keys and queries that are infinite, in tiles that rows see whole and in part, with rotated queries: the
    results are the reference's infinities, and NaN where it has NaN.  (A key with a score of -inf has no weight, one
    with inf makes its rows NaN.)"""
    for place in (3, 70, 127, 130, 141, 210):  # of request 0: 200 tokens held, 70 new ones
        for value in (float("inf"), float("-inf")):
            s = Step([70, 20], [200, 10], n_h, n_kv, D, dtype=dtype, tree=tree, seed=5, base=1e4)
            page, row = int(s.table[0, place // 16]), place % 16
            for what in ("v", "k"):
                x, of = (s.v, s.v_of) if what == "v" else (s.k, s.k_of)
                kept, kept_of = x[page, row, 0, 7].clone(), of[0][place, 0, 7]
                x[page, row, 0, 7], of[0][place, 0, 7] = value, value
                got, lse = s.run(lib)
                with np.errstate(all="ignore"):
                    if what == "v":  # weights are what they were
                        sees = ref.causal(70, 200) if not tree else ref.tree(70, 200, s.visible[:70])
                        hit = np.zeros((s.T, n_h), bool)
                        hit[:70, :n_h // n_kv] = sees[:, place][:, None]
                        o = to_np(got)
                        assert (o[hit][:, 7] == value).all()
                        assert np.isfinite(o[~hit]).all() and np.isfinite(np.delete(o[hit], 7, 1)).all()
                    else:  # a score of inf or -inf, by the sign of the rotated query's element
                        q = s.q[:70].double().numpy()
                        turned = np.stack([ref.oracle.rope_rotate(q[:, h], s.positions[:70], 1e4) for h in range(n_h)], 1)
                        sees = ref.causal(70, 200) if not tree else ref.tree(70, 200, s.visible[:70])
                        sees = np.broadcast_to(sees[:, place][:, None], (70, n_h)) & (np.arange(n_h) < n_h // n_kv)[None]
                        up = sees & (turned[:, :, 7] * value > 0)
                        o = to_np(got)
                        assert np.isnan(o[:70][up]).all()
                        assert np.isfinite(o[:70][~up]).all() and np.isfinite(o[70:]).all()
                x[page, row, 0, 7], of[0][place, 0, 7] = kept, kept_of


def test_values_in_rows_of_no_token(lib):
    """What lies behind the last token, or in pages of others, may be anything."""
    s = Step([70, 20], [31, 0], 8, 2, 128, seed=4)
    a = s.run(lib)
    for fill in (float("inf"), 3e38, 0.0):
        for t in (s.k, s.v):
            t[torch.isnan(t)] = fill
        b = s.run(lib)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        for t in (s.k, s.v):
            t[t == torch.tensor(fill).to(t.dtype)] = float("nan")


def test_scores_far_apart(lib):
    """Maxima that rise by hundreds from tile to tile, and rows of equal scores."""
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 2, 64, "f32")):
        s = Step([300], [200], n_h, n_kv, D, dtype=dtype)
        ramp = torch.linspace(-40, 40, 500)
        slot = s.table[0].long()[torch.arange(500) // 16] * 16 + torch.arange(500) % 16
        s.k.view(-1, n_kv, D)[slot, :, 0] = ramp[:, None].to(s.k.dtype)
        s.k_of[0][:, :, 0] = s.k.view(-1, n_kv, D)[slot, :, 0].double().numpy()
        s.check(lib, )
        s.q[:] = 0
        s.check(lib)


@pytest.mark.parametrize("n_h", [1 << 22, (1 << 22) + 3])
def test_heads_of_more_than_two_to_the_31_elements(lib, n_h):
    """One KV head whose query heads' outputs pass 32 bits in a row: a token, and a row behind the last."""
    D_v = 512
    q = torch.zeros(2, n_h, 8, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, 16, 1, 8, dtype=torch.bfloat16, device=DEV)
    v = torch.randn(1, 16, 1, D_v, dtype=torch.bfloat16, device=DEV)
    out = torch.full((2, n_h, D_v), float("nan"), dtype=torch.bfloat16, device=DEV)
    _, lse = lib.prefill_paged(q, k, v, ints([[0]]), ints([0, 1]), ints([1]), out=out, lse=True)
    assert (out[0] == v[0, 0, 0]).all() and not lse[0].any()  # the one key's value, score 0
    assert not out[1].any() and torch.isneginf(lse[1]).all()


def test_caches_of_more_than_two_to_the_31_elements(lib):
    """Pages at the end of a cache whose offsets pass 32 bits, attended and committed to."""
    n_pages, page, n_kv, D = 33000, 64, 8, 128
    k, v = (torch.zeros(n_pages, page, n_kv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert k.numel() > 2 ** 31
    s = Step([20, 9], [100, 0], 32, n_kv, D, page=page, base=1e4)
    n = s.k.shape[0]
    small = s.run(lib)
    k[-n:], v[-n:] = s.k.to(DEV), s.v.to(DEV)
    args = list(s.tensors())
    far = args[3] + (n_pages - n) * (args[3] >= 0).int()
    args[1], args[2], args[3] = k, v, far
    big = s.run(lib, args)
    assert torch.equal(small[0], big[0]) and torch.equal(small[1], big[1])
    before = k[-n:].clone()
    new, _ = lib.draft_commit(k, v, far, ints([100, 0]), ints([120, 9]), ints([[3, 19], [0, 2]]), ints([2, 2]))
    assert new.tolist() == [102, 2]
    rows = k[-n:].view(-1, n_kv, D)
    table = s.table.long()
    for b, src, dst in ((0, 103, 100), (0, 119, 101), (1, 2, 1)):
        at = [int(table[b, p // page]) * page + p % page for p in (src, dst)]
        assert torch.equal(rows[at[1]], before.view(-1, n_kv, D)[at[0]])


# ------------------------------------------------------------------------------------------- trees
@pytest.mark.parametrize("n_h,n_kv,D", HEADS)
@pytest.mark.parametrize("base,pairing", [(1e4, "adjacent"), (5e5, "half")])
def test_trees(lib, n_h, n_kv, D, base, pairing):
    Step([1, 25, 64, 0, 7, 32, 33, 128], [900, 128, 63, 40, 0, 1, 127, 500], n_h, n_kv, D, page=16, pad=2, base=base,
         pairing=pairing, tree=True, words=4, seed=n_h).check(lib)


@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 96, 127, 128, 129, 191, 255, 256])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 100, 128])
def test_tree_across_tile_borders(lib, ctx, n):
    Step([n, 3], [ctx, ctx + 5], 8, 2, 128, page=32, tree=True, seed=ctx + n).check(lib)
    Step([n, 3], [ctx, ctx + 5], 4, 4, 64, page=32, tree=True, seed=ctx + n).check(lib)


def test_any_masks(lib):
    """Masks that are no trees, rows that see no draft, and rows that see nothing at all."""
    def masks(rng, shape):
        m = rng.integers(0, 2 ** 32, shape, dtype=np.uint64)
        m[rng.random(shape[0]) < 0.3] = 0
        return m
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 4, 64, "bf16"), (4, 2, 64, "f32")):
        for words in (1, 2, 4):
            Step([100, 30, 5, 128], [0, 200, 0, 90], n_h, n_kv, D, dtype=dtype, tree=True, words=words, masks=masks,
                 seed=words).check(lib)


def test_a_chain_is_causal(lib):
    s = Step([60, 7, 128], [100, 0, 333], 8, 2, 128, base=1e4)
    parents = np.concatenate([np.arange(n) - 1 for n in s.news])
    args = s.tensors()
    positions, visible = lib.draft_plan(args[6], args[4], ints(parents))
    assert torch.equal(positions, args[6])
    causal, lse = s.run(lib, args)
    s.visible = visible.cpu().numpy()
    tree, tree_lse = s.run(lib, args)
    o, l, spread, err = s.want()
    compare(causal, lse, o, l, spread, err, "bf16")
    compare(tree, tree_lse, o, l, spread, err, "bf16")


def test_more_drafts_than_bits(lib):
    """Drafts behind the last bit are seen by none; their own rows see what their bits say."""
    for n_h, n_kv, D, dtype in ((8, 2, 128, "bf16"), (4, 2, 64, "f32")):
        s = Step([200, 40], [50, 0], n_h, n_kv, D, dtype=dtype, tree=True, words=1,
                 masks=lambda rng, shape: np.full(shape, 2 ** 32 - 1, np.uint64))
        s.positions[:] = 7
        s.check(lib)


# ------------------------------------------------------------------------------------------- how calls are made
def test_streams_and_workspaces(lib):
    """Two calls that overlap on two streams, each with its own workspace; and a workspace with garbage in it."""
    a, b = Step([50, 900], [700, 0], 8, 2, 128, base=1e4), Step([64] * 8, [3000] * 8, 8, 2, 128, base=1e4, tree=True)
    ta, tb = a.tensors(), b.tensors()
    alone = a.run(lib, ta), b.run(lib, tb)

    def space(s):
        n = lib.packed_workspace_size(s.T, len(s.news), s.n_h, 2, 128, 128, 16, s.table.shape[1])
        return torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    wa, wb = space(a), space(b)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        ra, rb = a.run(lib, ta, workspace=wa, stream=sa), b.run(lib, tb, workspace=wb, stream=sb.cuda_stream)
        torch.cuda.synchronize()
        for got, want in ((ra, alone[0]), (rb, alone[1])):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(lib.AttnError):
        a.run(lib, ta, workspace=wa[:8].clone())


def test_captured_calls_follow_the_lengths(lib):
    """A captured step is replayed with other lengths, offsets and tables in its buffers."""
    for dtype, D in (("bf16", 128), ("f32", 64)):
        for tree in (False, True):
            steps = [Step([20, 40, 4], [200, 0, 60], 8, 2, D, dtype=dtype, tree=tree, words=2, base=1e4, seed=1),
                     Step([0, 1, 60], [90, 300, 150], 8, 2, D, dtype=dtype, tree=tree, words=2, base=1e4, seed=2, pad=3),
                     Step([64, 0, 0], [7, 0, 0], 8, 2, D, dtype=dtype, tree=tree, words=2, base=1e4, seed=3)]
            pages = max(s.k.shape[0] for s in steps)
            width = max(s.table.shape[1] for s in steps)
            q = torch.zeros(64, 8, D, dtype=TYPES[dtype], device=DEV)
            k, v = (torch.zeros(pages, 16, 2, D, dtype=TYPES[dtype], device=DEV) for _ in range(2))
            table, cu, lens = ints(np.zeros((3, width))), ints(np.zeros(4)), ints(np.zeros(3))
            positions, visible = ints(np.zeros(64)), ints(np.zeros((64, 2)))
            out, lse = torch.empty_like(q), torch.empty(64, 8, device=DEV)
            ws = torch.empty(lib.packed_workspace_size(64, 3, 8, 2, D, D, 16, width, TYPES[dtype]), dtype=torch.uint8,
                             device=DEV)

            def call():
                kw = dict(rope_base=1e4, out=out, lse=lse, workspace=ws)
                if tree:
                    lib.decode_tree(q, k, v, table, cu, lens, positions, visible, **kw)
                else:
                    lib.prefill_paged(q, k, v, table, cu, lens, positions, **kw)
            call()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            for s in steps + steps[:1]:
                a = s.tensors()
                q.zero_()
                q[:s.T], k[:a[1].shape[0]], v[:a[2].shape[0]] = a[0], a[1], a[2]
                table[:, :a[3].shape[1]] = a[3]
                cu.copy_(a[4])
                lens.copy_(a[5])
                positions.fill_(-1)
                positions[:s.T] = a[6]
                if tree:
                    visible[:s.T] = torch.as_tensor(s.visible).to(DEV)
                out.fill_(float("nan"))
                lse.fill_(float("nan"))
                graph.replay()
                compare(out[:s.T], lse[:s.T], *s.want(), dtype)
                assert not out[s.T:].any() and torch.isneginf(lse[s.T:]).all()


def test_same_bits_every_time(lib):
    for s in (Step([700, 33, 1], [0, 4000, 900], 8, 2, 128, base=1e4), Step([32] * 5, [6000] * 5, 8, 2, 128, tree=True),
              Step([40] * 3, [500] * 3, 4, 2, 64, dtype="f32")):
        args = s.tensors()
        a = s.run(lib, args)
        for _ in range(3):
            b = s.run(lib, args)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_rows_and_python_checks(lib):
    s = Step([3], [5], 8, 2, 128)
    q, k, v, table, cu, lens, positions = s.tensors()
    out, lse = lib.prefill_paged(q[:0], k, v, table, ints([0, 0]), lens, positions[:0], lse=True)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    for bad in (dict(cu_new=cu.long()), dict(cu_new=cu[:1]), dict(seqlens=lens.repeat(2)), dict(positions=positions[:2]),
                dict(q=q.float()), dict(q=q[:, :, :64].contiguous()), dict(q=q.transpose(0, 1))):
        args = dict(q=q, k_pages=k, v_pages=v, block_table=table, cu_new=cu, seqlens=lens, positions=positions)
        with pytest.raises((ValueError, TypeError)):
            lib.prefill_paged(**dict(args, **bad))
    with pytest.raises(ValueError):
        lib.decode_tree(q, k, v, table, cu, lens, positions, ints(np.zeros((3, 5))))
    with pytest.raises(lib.AttnError):
        lib.prefill_paged(q, k, v, table, cu, lens, positions, out=q)


# ------------------------------------------------------------------------------------------- plan and commit
@pytest.mark.parametrize("words", [1, 2, 3, 4])
def test_draft_plan(lib, words):
    rng = np.random.default_rng(words)
    news = [1, 0, 32, 33, 128, 5, 200, 64, 96, 17]
    cu = np.concatenate([[0], np.cumsum(news)])
    T = int(cu[-1]) + 11
    parents = np.concatenate([np.asarray(ref.random_tree(n, rng), np.int64) for n in news] + [np.full(11, 3)])
    places = np.concatenate([c + np.arange(n) for n, c in zip(news, rng.integers(0, 5000, len(news)))] + [np.full(11, 9)])
    broken = rng.random(T) < 0.02
    parents[broken] = rng.integers(-9, 300, int(broken.sum()))
    places[cu[7]:cu[8]] = -1
    places[cu[9] + 3] = -5
    for fill in (-1, 12345):
        positions = torch.full((T,), fill, dtype=torch.int32, device=DEV)
        visible = torch.full((T, words), fill, dtype=torch.int32, device=DEV)
        lib.draft_plan(ints(places), ints(cu), ints(parents), words=words, positions=positions, visible=visible)
        want = ref.draft_plan(places, cu, parents, words)
        np.testing.assert_array_equal(positions.cpu().numpy(), want[0])
        np.testing.assert_array_equal(visible.cpu().numpy(), want[1])


def test_draft_plan_long_chains_and_broken_offsets(lib):
    n = 128
    cu = ints([0, n])
    positions, visible = lib.draft_plan(ints(1000 + np.arange(n)), cu, ints(np.arange(n) - 1))
    want = ref.draft_plan(1000 + np.arange(n), [0, n], np.arange(n) - 1, 4)
    np.testing.assert_array_equal(positions.cpu().numpy(), want[0])
    np.testing.assert_array_equal(visible.cpu().numpy(), want[1])
    # rows past T do not exist
    positions, visible = lib.draft_plan(ints(np.arange(50)), ints([0, 40, 80]), ints([-1] + [0] * 49), words=2)
    want = ref.draft_plan(np.arange(50), [0, 40, 80], [-1] + [0] * 49, 2)
    np.testing.assert_array_equal(positions.cpu().numpy(), want[0])
    np.testing.assert_array_equal(visible.cpu().numpy(), want[1])
    for bad in ([0, -7, 2 ** 31 - 1], [2 ** 31 - 1, 5, -3]):
        lib.draft_plan(ints(np.arange(50)), ints(bad), ints([-1] + [0] * 49), words=2)  # no meaning, and no fault
    assert lib.draft_plan(ints([]), ints([0, 0]), ints([]))[0].shape == (0,)


def commit_case(seed, B, page, max_path, n_kv, D_qk, D_v, dtype, alias=False):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 100, B)
    drafts = rng.integers(0, max_path + 3, B)
    seqlens = lens + drafts
    pages = -(-seqlens // page)
    n_pages = int(pages.sum()) + 4
    order = rng.permutation(n_pages)
    table = np.full((B, int(pages.max(initial=1)) + 1), -1)
    table[np.arange(table.shape[1])[None] < pages[:, None]] = order[:pages.sum()]
    path = np.full((B, max_path), -1)
    n_path = np.zeros(B, np.int64)
    for b in range(B):
        p = np.sort(rng.permutation(int(drafts[b]))[:rng.integers(0, min(max_path, drafts[b]) + 1)])
        path[b, :len(p)] = p
        n_path[b] = len(p)
        if len(p) > 2 and rng.random() < 0.2:  # paths that break
            path[b, rng.integers(0, len(p))] = rng.choice([-1, 0, 500, path[b, 0]])
    n_path[rng.random(B) < 0.1] = 500
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(n_pages, page, n_kv, D_qk, generator=g).to(TYPES[dtype])
    v = k[..., :D_v] if alias else torch.randn(n_pages, page, n_kv, D_v, generator=g).to(TYPES[dtype])
    return lens, seqlens, table, path, n_path, n_pages, list(order[pages.sum():]), k, v


@pytest.mark.parametrize("seed,B,page,max_path,n_kv,D_qk,D_v,dtype,alias", [
    (0, 7, 16, 8, 8, 128, 128, "bf16", False), (1, 60, 16, 33, 2, 64, 64, "f32", False),
    (2, 300, 32, 128, 1, 64, 72, "bf16", False), (3, 5, 64, 12, 1, 576, 512, "bf16", True),
    (4, 1, 16, 1, 3, 40, 8, "f32", False), (5, 600, 16, 5, 12, 64, 64, "bf16", False)])
def test_draft_commit(lib, seed, B, page, max_path, n_kv, D_qk, D_v, dtype, alias):
    lens, seqlens, table, path, n_path, n_pages, spare, k, v = commit_case(seed, B, page, max_path, n_kv, D_qk, D_v,
                                                                           dtype, alias)
    if seed == 1:  # pages outside the cache
        table[3, 0], table[10, 1] = n_pages, -4
    for cap in {n_pages, min(n_pages, len(spare) + 2)}:
        free = (spare + [-7] * n_pages)[:cap]
        new, moves, free_want, left = ref.commit(lens, seqlens, path, n_path, table, page, n_pages, free, len(spare), cap)
        kd = k.to(DEV).clone()
        vd = kd[..., :D_v] if alias else v.to(DEV).clone()
        free_t = ints(free)
        got, n_left = lib.draft_commit(kd, vd, ints(table), ints(lens), ints(seqlens), ints(path), ints(n_path), free_t,
                                       ints([len(spare)]))
        np.testing.assert_array_equal(got.cpu().numpy(), new)
        np.testing.assert_array_equal(free_t.cpu().numpy(), free_want)
        assert int(n_left) == left
        for x, d, heads in ((k, kd, D_qk), (v, vd, D_v)):
            flat = x.reshape(-1, n_kv, heads)
            want = flat.clone()
            for mine in moves:
                for src, dst in mine:
                    want[dst] = flat[src]
            assert torch.equal(d.reshape(-1, n_kv, heads).cpu(), want)
    kd, vd = k.to(DEV).clone(), v.to(DEV).clone()
    if not alias:  # without the stack
        got, n_left = lib.draft_commit(kd, vd, ints(table), ints(lens), ints(seqlens), ints(path), ints(n_path))
        np.testing.assert_array_equal(got.cpu().numpy(), new)
        assert n_left is None


def test_draft_commit_of_odd_lengths(lib):
    k = torch.zeros(4, 16, 1, 64, device=DEV)
    for lens, seqlens, want in ((-5, 3, 1), (10, 4, 10), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (3, 2 ** 31 - 1, 4)):
        new, _ = lib.draft_commit(k, k.clone(), ints([[0, 1]]), ints([lens]), ints([seqlens]), ints([[0]]), ints([1]))
        assert int(new) == want, (lens, seqlens)


# ------------------------------------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_speculative_serving_loop(lib, dtype, D):
    """Prompts are admitted, then trees of drafts are planned, appended, attended and committed for some steps; every
    attention is checked against the tokens that the requests hold by then, and pages return to the stack."""
    rng = np.random.default_rng(11)
    B, n_h, n_kv, page, n_pages, width = 5, 8, 2, 16, 90, 20
    base = 1e4
    k_pages, v_pages = (torch.full((n_pages, page, n_kv, D), float("nan"), dtype=TYPES[dtype], device=DEV) for _ in range(2))
    table = ints(np.full((B, width), -1))
    free, n_free = ints(rng.permutation(n_pages)), ints([n_pages])
    lens = ints(np.zeros(B))
    held_k, held_v, held_pos = [[] for _ in range(B)], [[] for _ in range(B)], [[] for _ in range(B)]

    def rotated(k, positions):
        x = torch.stack([torch.as_tensor(ref.oracle.rope_rotate(k[:, h].double().numpy(), positions, base))
                         for h in range(n_kv)], 1)
        return x.to(TYPES[dtype]).double().numpy()

    for step in range(6):
        prompt = step == 0
        news = rng.integers(1, 70, B) if prompt else rng.integers(1, 33, B)
        T = int(news.sum()) + 3
        parents = [list(np.arange(n) - 1) if prompt else ref.random_tree(n, rng) for n in news]
        g = torch.Generator().manual_seed(step)
        q = torch.randn(T, n_h, D, generator=g).to(TYPES[dtype])
        k, v = (torch.randn(T, n_kv, D, generator=g).to(TYPES[dtype]) for _ in range(2))
        seqlens, cu, slots, places, left = lib.page_plan(lens, ints(news), table, free, n_free, page_size=page,
                                                         n_pages=n_pages, max_tokens=T)
        flat = ints(np.concatenate([np.asarray(p) for p in parents] + [np.full(3, -1)]))
        positions, visible = (places, None) if prompt else lib.draft_plan(places, cu, flat, words=1)
        lib.kv_append_paged(k.to(DEV), v.to(DEV), k_pages, v_pages, slots, positions, rope_base=base)
        if prompt:
            out, lse = lib.prefill_paged(q.to(DEV), k_pages, v_pages, table, cu, seqlens, positions, rope_base=base, lse=True)
        else:
            out, lse = lib.decode_tree(q.to(DEV), k_pages, v_pages, table, cu, seqlens, positions, visible, rope_base=base,
                                       lse=True)
        # what each row should see, from the tokens themselves
        pos = positions.cpu().numpy()
        first = 0
        want = [np.zeros((T, n_h, D)), np.full((T, n_h), -np.inf), np.zeros((T, n_h, D)), np.zeros((T, n_h))]
        for b, n in enumerate(news):
            r = slice(first, first + n)
            lines = ref.lineage(parents[b])
            ctx = len(held_pos[b])
            assert pos[r].tolist() == [ctx + len(x) - 1 for x in lines]
            kr = rotated(k[r], pos[r])
            sees = np.zeros((n, ctx + n), bool)
            sees[:, :ctx] = True
            for i, x in enumerate(lines):
                sees[i, ctx + np.asarray(x)] = True
            keys = np.concatenate([np.asarray(held_k[b]).reshape(-1, n_kv, D), kr])
            values = np.concatenate([np.asarray(held_v[b]).reshape(-1, n_kv, D), v[r].double().numpy()])
            for w, x in zip(want, ref.attend(q[r].double().numpy(), pos[r], sees, keys, values, rope_base=base)):
                w[r] = x
            accepted = list(range(n)) if prompt else lines[int(rng.integers(0, n))]
            for i in accepted:
                held_k[b].append(kr[i])
                held_v[b].append(v[first + i].double().numpy())
                held_pos[b].append(int(pos[first + i]))
            parents[b] = accepted
            first += n
        # the keys in the cache are rotated in 32 bits, the reference's in 64: bf16 may round the other way
        want[3] += 0 if dtype == "f32" else 2.0 ** -8 * D ** -0.5 * np.abs(q.double().numpy()).sum(-1) * 4
        compare(out, lse, *want, dtype)
        if prompt:
            lens, n_free = seqlens, left
        else:
            width_p = max(len(p) for p in parents)
            path = ints([p + [0] * (width_p - len(p)) for p in parents])
            lens, n_free = lib.draft_commit(k_pages, v_pages, table, lens, seqlens, path, ints([len(p) for p in parents]),
                                            free, left)
        assert lens.cpu().tolist() == [len(x) for x in held_pos]
        in_use = sum(-(-len(x) // page) for x in held_pos)
        assert int(n_free) == n_pages - in_use
        owned = np.concatenate([table[b, : -(-len(held_pos[b]) // page)].cpu().numpy() for b in range(B)])
        assert sorted(owned.tolist() + free[: int(n_free)].cpu().tolist()) == list(range(n_pages))
