"""Host side of the decoder operators at the limits of what their descriptions allow (no GPU
needed)."""
from __future__ import annotations

import pytest
import torch

import bit_groupwise_weight_gb300 as lb
from bit_groupwise_weight_gb300 import build as lbuild
from bit_groupwise_weight_gb300 import decoder
from test_decoder_host import ATTN, CACHE, EINVAL, SEQS, call, descriptor


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return lb.abi()


def workspace(lib, heads=ATTN["heads"], cache=None, seqs=None):
    return lib.lowbit_attention_workspace(heads, descriptor("cache", CACHE | (cache or {})), descriptor("seqs", SEQS | (seqs or {})))


@pytest.mark.parametrize("heads,cache,seqs", [
    (8, dict(head_dim=96), {}), (8, dict(head_dim=256), {}), (8, dict(page=48), {}), (8, dict(page=8), {}), (8, dict(page=512), {}),
    (8, dict(pages=0), {}), (8, dict(pages=-1), {}), (8, dict(kv_heads=3), {}), (8, dict(kv_heads=0), {}), (0, {}, {}), (9, {}, {}),
    (8, {}, dict(tokens=7)), (8, {}, dict(tokens=-1)), (8, {}, dict(batch=-1)), (8, {}, dict(width=0)), (8, {}, dict(width=-1)),
    (8, {}, dict(cu_q=0x42000, max_q=0)), (8, {}, dict(tokens=3 << 28)), (8, {}, dict(width=1 << 28, table_stride=1 << 28))])
def test_no_workspace_for_sizes_that_attention_refuses(lib, heads, cache, seqs):
    assert call(lib, "attention", dict(heads=heads), cache, seqs) == EINVAL
    assert workspace(lib, heads, cache, seqs) == 0


@pytest.mark.parametrize("seqs", [dict(tokens=0), dict(batch=0), dict(batch=0, tokens=0)])
def test_no_workspace_for_empty_calls(lib, seqs):
    assert workspace(lib, seqs=seqs) == 0


def test_workspace_follows_from_the_sizes_alone(lib):
    """It can be asked for before there is a cache or a table."""
    nothing = dict(k=None, v=None, k_exp=None, v_exp=None, page_stride=0, head_stride=0)
    assert workspace(lib, cache=nothing, seqs=dict(page_table=None, lens=None, table_stride=0)) == workspace(lib) > 0


def test_extension_module_of_another_pytorch_is_not_used(lib, monkeypatch):
    """It is compiled against PyTorch's C++ headers: after an upgrade it has to be built again."""
    assert lbuild.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert not lbuild.up_to_date()
    monkeypatch.setattr(decoder, "_hot", None)
    with pytest.raises(ImportError, match="not built"):
        decoder._load()
