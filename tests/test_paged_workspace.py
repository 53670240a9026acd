"""The scratch of paged decode: what a call's rows and the card's blocks need, whatever the tables' width (no GPU)."""
import pytest
import torch

import transformer_causal_attention_gb300 as attn
from transformer_causal_attention_gb300 import build as build_mod

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()


def size(B, n_h, n_kv, Dqk, Dv, tokens, prefix, dtype, page=64):
    return attn.decode_paged_workspace_size(B, n_h, n_kv, Dqk, Dv, page, tokens // page, prefix, TYPES[dtype])


@pytest.mark.parametrize("B,n_h,n_kv,Dqk,Dv,prefix,dtype", [
    (256, 32, 8, 128, 128, 0, "bf16"), (256, 64, 8, 128, 128, 16384, "bf16"), (8, 12, 12, 64, 64, 0, "f32"),
    (59, 32, 8, 128, 128, 0, "f32"), (64, 128, 1, 576, 512, 0, "bf16"), (1, 6, 2, 96, 96, 1024, "bf16")])
def test_size_does_not_depend_on_the_tables_width(B, n_h, n_kv, Dqk, Dv, prefix, dtype):
    sizes = {size(B, n_h, n_kv, Dqk, Dv, prefix + own, prefix, dtype) for own in (1 << 17, 1 << 20, 1 << 23)}
    assert len(sizes) == 1


@pytest.mark.parametrize("B,n_h,n_kv,Dqk,Dv,tokens,prefix,dtype,megabytes", [
    (256, 32, 8, 128, 128, 16640, 16384, "bf16", 60), (256, 32, 8, 128, 128, 16640, 16384, "f32", 60),
    (1024, 32, 8, 128, 128, 131072, 0, "bf16", 60), (1024, 32, 8, 128, 128, 131072, 0, "f32", 60),
    (256, 64, 8, 128, 128, 1 << 20, 0, "bf16", 60), (64, 128, 1, 576, 512, 131072, 0, "bf16", 60),
    (64, 32, 8, 128, 128, 1 << 20, 1 << 19, "f32", 60)])
def test_size_stays_small(B, n_h, n_kv, Dqk, Dv, tokens, prefix, dtype, megabytes):
    assert 0 < size(B, n_h, n_kv, Dqk, Dv, tokens, prefix, dtype) < megabytes * 1e6


def test_size_holds_a_partial_of_every_row():
    for B, n_h, n_kv, D in ((1, 1, 1, 8), (3, 6, 2, 96), (300, 32, 8, 128)):
        assert size(B, n_h, n_kv, D, D, 4096, 0, "f32") >= 4 * B * n_h * (D + 1)
