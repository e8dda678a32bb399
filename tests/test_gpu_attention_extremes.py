"""Attention over both kinds of cache where scores leave the sizes that models have: far from
zero (next to which fp32 holds no fractions), at fp32's ends, rows of q near the largest number."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import cache4_ref as ref4
import decoder_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_groupwise_weight_gb300 as lb  # noqa: E402
from bit_groupwise_weight_gb300 import build as lbuild  # noqa: E402

lbuild.build()

HEADS = 4                                                 # over one kv head: 1 new token is 4 rows, 80 are 320
FEW_AND_MANY = "n", [1, 80]


def batch(bits, seed, n, dim, keys, power, lens=(300, 131)):
    """Two sequences whose keys are rows of `keys` (whole numbers of up to 7) times 2^power, chosen at random, all
    kinds of them among the first.  Returns the batch and each sequence's choice."""
    lens = list(lens)
    make = (ref4 if bits == 4 else ref).make_batch
    b = make(seed, lens, [n, n], 1, dim, 32)
    rng = np.random.default_rng([seed, 1])
    kinds = [np.concatenate([np.arange(len(keys)), rng.integers(0, len(keys), m - len(keys))]) for m in lens]
    if bits == 8:
        b.k_exp[:], b.v_exp[:] = power, -6                                    # (v's exponent is added to the scores)
    for s, m in enumerate(lens):
        at = np.arange(m)
        page, slot = b.table[s, at // 32], at % 32
        if bits == 4:
            b.k[page, 0, slot] = keys[kinds[s]] + 8
            b.k_scale[page, 0, slot] = (power + 15) << 2                      # 2^power as e5m2
        else:
            b.k[page, 0, slot] = ref.e4m3_round(keys[kinds[s]].astype(float))
    return b, kinds


def run(b, q, scale):
    cache, table, lens, cu = b.device()
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    out = lb.attention(q.cuda(), *cache, table, lens, cu_q=cu, max_q=max(b.news), scale=scale, lse=lse)
    assert lb.wait_timeouts() == 0
    return ref.f64(out), ref.f64(lse)


def seen_values(bits, b, s):
    """(v fp64 [len, dim], how many keys each of the sequence's new rows sees)."""
    v = ref4.cached(b, s, 0, "v")[0] if bits == 4 else ref.cached(b, s, 0, "v")
    return v, b.lens[s] - b.news[s] + np.arange(b.news[s]) + 1


def check(bits, b, kinds, q, keys, power, scale):
    """Kinds of keys whose scores are so far apart that the best one has all of the weight: the mean of its values.
    Equal keys have equal scores and so equal weights, rounded to fp16 (2^-11 of themselves) for the product and not for
    their sum; sums and products are fp32's (2^-16 of the magnitudes covers 300 of them in a row; more are divided), out is rounded to bf16; scores
    are some ten roundings of sums of up to 16 |q| 2^power a value over 4 bits (2^-20 of that), the logarithm is off by
    2 units and lse by one.
    Of the few rows for which two kinds come near each other only sizes are looked at."""
    out, lse = run(b, q, scale)
    x, checked = ref.f64(q), 0
    for s, n in enumerate(b.news):
        v, sees = seen_values(bits, b, s)
        for i in range(n):
            row, mine = b.starts[s] + i, kinds[s][:sees[i]]
            for h in range(HEADS):
                scores = keys.astype(float) @ x[row, h] * 2.0 ** power * scale
                mag = np.abs(x[row, h]).sum() * 16 * 2.0 ** power * abs(scale)
                order = np.argsort(-scores)
                best = mine == order[0]
                assert np.all(np.abs(out[row, h]) <= np.abs(v).max() * (1 + 2.0 ** -8)), (row, h)
                assert abs(lse[row, h] - scores[order[0]]) <= 2.0 ** -19 * mag + 10, (row, h, lse[row, h], scores[order[0]])
                if len(keys) > 1 and scores[order[0]] - scores[order[1]] < max(2.0 ** -14 * mag, 200):
                    continue
                checked += 1
                want, mean = v[:sees[i]][best].mean(0), np.abs(v[:sees[i]][best]).mean(0)
                assert np.all(np.abs(out[row, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * mean + 2.0 ** -16 * np.abs(v).max()), (row, h)
                want = scores[order[0]] + np.log(best.sum())
                assert abs(lse[row, h] - want) <= 2.0 ** -20 * mag + 2.0 ** -21 * abs(want) + 2.0 ** -18, (row, h, lse[row, h], want)
    assert checked >= 0.8 * out.shape[0] * HEADS


def make_keys(seed, count, dim):
    return np.random.default_rng([seed, 2]).integers(-7, 8, (count, dim))


def make_q(seed, n, dim, size):
    """Rows whose largest magnitude is in [size, 2 size)."""
    x = np.random.default_rng([seed, 3]).uniform(-1, 1, (2 * n, HEADS, dim))
    x *= 1.5 * size / np.abs(x).max(-1, keepdims=True)
    return ref.bf16(x)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize(*FEW_AND_MANY)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("far", [20, 23, 24, 26, 27, 30, 60, 118])
def test_scores_far_from_zero(bits, n, dim, far):
    """A score's fraction is lost in fp32: its product, rounded and not, must not be taken for different scores."""
    keys, q = make_keys(far, 3, dim), make_q(far, n, dim, 2.0 ** (far // 2))
    b, kinds = batch(bits, far, n, dim, keys, 0)
    for sign in (1, -1):
        check(bits, b, kinds, q, keys, 0, sign * 2.0 ** (far - far // 2) / 100)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize(*FEW_AND_MANY)
@pytest.mark.parametrize("unit", [1, 2, 4, 8, 16, 32])
def test_scores_some_units_apart_far_from_zero(bits, n, unit):
    """Scores of 2^23 units and 0 to 21 more, a unit being what fp32 holds there: weights of a unit are e^unit, and
    what comes out lies between the values that went in."""
    rng = np.random.default_rng([unit, 5])
    keys = np.zeros((64, 64), int)
    keys[:, 0] = 4
    keys[:, [33, 40, 50]] = rng.integers(0, 8, (64, 3))
    b, kinds = batch(bits, 70 + unit, n, 64, keys, 0)
    q = torch.zeros(2 * n, HEADS, 64)
    q[..., 0], q[..., [33, 40, 50]] = 2.0 ** 21 * unit, float(unit)
    out, lse = run(b, q.to(torch.bfloat16), float(np.log(2.0)))
    for s in range(2):
        v, sees = seen_values(bits, b, s)
        for i in range(n):
            row = b.starts[s] + i
            low, high = v[:sees[i]].min(0), v[:sees[i]].max(0)
            slack = 2.0 ** -8 * np.abs(v).max()
            assert np.all((low - slack <= out[row]) & (out[row] <= high + slack)), row
            want = 2.0 ** 23 * unit * np.log(2.0)
            assert np.all(np.abs(lse[row] - want) <= 2.0 ** -18 * want + 30), (row, lse[row], want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize(*FEW_AND_MANY)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [119, 121, 123, 125, 127])
def test_rows_of_q_near_the_largest_number(bits, n, dim, size):
    """What turns codes into scores stays a number for every row of q: with small keys the scores are."""
    keys, q = make_keys(size, 3, dim), make_q(size, n, dim, 2.0 ** (size if size < 127 else 126.9))
    b, kinds = batch(bits, size, n, dim, keys, -14)
    for scale in (dim ** -0.5, -dim ** -0.5, 1.0):
        check(bits, b, kinds, q, keys, -14, scale)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize(*FEW_AND_MANY)
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_at_the_ends_of_fp32(bits, n, sign):
    """Times log2 e within a tenth of the largest number, on either side of 0."""
    keys = np.zeros((1, 64), int)
    keys[0, 5] = 7
    b, kinds = batch(bits, 90, n, 64, keys, 10)
    q = torch.zeros(2 * n, HEADS, 64)
    q[..., 5] = sign * 3.2e38 / np.log2(np.e) / 7 / 2.0 ** 10 * 8
    check(bits, b, kinds, q.to(torch.bfloat16), keys, 10, 0.125)


@pytest.mark.parametrize(*FEW_AND_MANY)
@pytest.mark.parametrize("scale", [64.0, -1e6, 9e29])
def test_zero_keys_have_zero_scores_whatever_the_row_of_q(n, scale):
    keys = np.zeros((1, 64), int)
    b, kinds = batch(4, 91, n, 64, keys, 0)
    out, lse = run(b, make_q(91, n, 64, 2.0 ** 126.9), scale)
    for s in range(2):
        v, sees = seen_values(4, b, s)
        for i in range(n):
            row, want, mean = b.starts[s] + i, v[:sees[i]].mean(0), np.abs(v[:sees[i]]).mean(0)
            assert np.all(np.abs(out[row] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * mean + 2.0 ** -16 * np.abs(v).max())
            assert np.all(np.abs(lse[row] - np.log(sees[i])) <= 2.0 ** -20)


@pytest.mark.parametrize("n", [1, 3, 64, 150])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("by", [2.0 ** 24, -2.0 ** 40, 2.0 ** 90])
def test_rows_beside_others_far_from_zero_are_the_same(n, dim, by):
    """To the bit, over 4 bits: rows of the same tiles, warps and sequences."""
    b = ref4.make_batch(98, [700], [n], 1, dim, 64)
    q = ref.bf16(np.random.default_rng([99, n]).standard_normal((n, 8, dim)))
    alone, alone_lse = run(b, q, dim ** -0.5)
    loud = q.clone()
    loud[:, ::2] *= by
    got, lse = run(b, loud, dim ** -0.5)
    assert np.array_equal(got[:, 1::2], alone[:, 1::2]) and np.array_equal(lse[:, 1::2], alone_lse[:, 1::2])
    assert np.isfinite(got).all() and np.isfinite(lse).all() and not np.array_equal(got[:, ::2], alone[:, ::2])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize(*FEW_AND_MANY)
@pytest.mark.parametrize("far", [25, 60])
def test_scores_far_from_zero_in_parts(bits, n, far):
    """Keys divided between CTAs, whose parts are joined."""
    keys, q = make_keys(far, 3, 128), make_q(far, n, 128, 2.0 ** (far // 2))
    b, kinds = batch(bits, far, n, 128, keys, 0, lens=(9000, 2500))
    check(bits, b, kinds, q, keys, 0, 2.0 ** (far - far // 2) / 100)
