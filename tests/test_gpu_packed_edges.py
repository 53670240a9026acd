"""Steps of several tokens per request at the edges of their numbers: queries of zero and near it beside huge keys.
Inputs, references and element-wise bars are those of tests/test_gpu_packed.py.
"""
import numpy as np
import pytest
import torch

from tests import packed_reference as ref
from tests.test_gpu_packed import Step, lib  # noqa: F401 (lib: the module's fixture)
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
