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
