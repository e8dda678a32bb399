"""Attention over the 4-bit cache on both sides of the rule that divides its kernels by the query
rows of a sequence."""
from __future__ import annotations

import pytest
import torch

import cache4_ref as ref4

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_attention4 as whole  # noqa: E402


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sequences", [15, 16])
@pytest.mark.parametrize("new", [12, 13, 16, 17])
def test_same_rows_of_every_sequence(sequences, new, dim):
    """44 to 68 rows a sequence: with 128 values 48 are the last of the kernel for few in batches of 64 sequences
    times kv heads and more, 64 in smaller ones and with 64 values."""
    b = ref4.make_batch(101, [new + 37 * i for i in range(sequences)], [new] * sequences, 4, dim, 32)
    whole.check(b, whole.queries(102, new * sequences, 16, dim))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sequences", [15, 16])
@pytest.mark.parametrize("window", [0, 90])
def test_sequences_on_both_sides(sequences, window, dim):
    """11, 12 and 13 new tokens of 4 heads a group (44, 48 and 52 rows), and 15, 16 and 17, in one batch."""
    news = ([11, 12, 13, 1, 15, 16, 17, 0] * 2)[:sequences]
    b = ref4.make_batch(103, [n + 41 * i for i, n in enumerate(news)], news, 4, dim, 64)
    whole.check(b, whole.queries(104, sum(news), 16, dim), window=window)
