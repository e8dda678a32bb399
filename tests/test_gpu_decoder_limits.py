"""The decoder operators at the limits of what their descriptions allow, against the same
64-bit definitions as test_gpu_decoder."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import decoder_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_groupwise_weight_gb300 as lb  # noqa: E402
from bit_groupwise_weight_gb300 import build as lbuild  # noqa: E402

lbuild.build()


def queries(seed, T, heads, dim):
    return ref.bf16(np.random.default_rng([seed, T, heads, dim]).standard_normal((T, heads, dim)))


def attend(b, q, scale=None, window=0, max_q=None):
    """(out, lse) in fp64 of a batch, with rows that the call does not write left as 7."""
    cache, table, lens, cu = b.device()
    out = torch.full_like(q.cuda(), 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    lb.attention(q.cuda(), *cache, table, lens, cu_q=cu, max_q=max(b.news) if max_q is None else max_q, scale=scale, window=window,
                 out=out, lse=lse)
    assert lb.wait_timeouts() == 0
    return ref.f64(out), ref.f64(lse)


def close(got, want, bound):
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound)
    bad &= ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {want[bad][0]}"


# ---------------------------------------------------------------------------
# More new tokens than max_q
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("news,max_q", [([10, 3, 1, 7], 4), ([100, 90, 1, 300], 80)])
@pytest.mark.parametrize("window", [0, 6])
def test_attention_leaves_tokens_past_max_q_out(news, max_q, window):
    """The tokens before keep their positions, len - n + i with all n of the sequence counted."""
    lens = [n + e for n, e in zip(news, [0, 40, 5, 200])]
    b = ref.make_batch(100, lens, news, 2, 64, 16)
    q = queries(101, sum(news), 8, 64)
    out, lse = attend(b, q, window=window, max_q=max_q)
    want, want_lse, bound, lse_bound = ref.attention(ref.f64(q), b, 0.125, window)
    kept = np.concatenate([np.arange(n) < max_q for n in news])
    close(out[kept], want[kept], bound[kept])
    close(lse[kept], want_lse[kept], lse_bound[kept])
    assert (out[~kept] == 7).all() and (lse[~kept] == 7).all()


@pytest.mark.parametrize("page,news,lens,max_q", [(16, [10, 2], [10, 33], 4), (32, [150, 70, 1], [170, 70, 8], 65),
                                                  (16, [30, 5], [12, 5], 21)])
def test_append_leaves_tokens_past_max_q_out(page, news, lens, max_q):
    """The cache and the rotated rows are those of the call without these tokens."""
    heads, kv_heads, dim = 4, 2, 64
    b = ref.make_batch(102, lens, news, kv_heads, dim, page)
    x = queries(103, sum(news), heads + 2 * kv_heads, dim).cuda()
    turns = lb.rotary_turns(dim, device="cuda")
    kept = torch.from_numpy(np.concatenate([np.arange(n) < max_q for n in news])).cuda()

    def append(rows, cu, lens, max_q):
        cache, table, _, _ = b.device()
        q, k, v = rows.split([heads, kv_heads, kv_heads], 1)
        out = torch.full((rows.shape[0], heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        ints = dict(dtype=torch.int32, device="cuda")
        lb.kv_append(q, k, v, *cache, table, torch.tensor(lens, **ints), cu_q=torch.tensor(cu, **ints), max_q=max_q, turns=turns, out=out)
        return out, [c.view(torch.uint8) for c in cache]
    out, cache = append(x, b.starts.tolist(), lens, max_q)
    fewer = [min(n, max_q) for n in news]
    want, want_cache = append(x[kept].contiguous(), [0] + np.cumsum(fewer).tolist(),
                              [m - n + f for m, n, f in zip(lens, news, fewer)], max_q)
    assert torch.equal(out[kept], want) and (out[~kept] == 7).all()
    assert all(torch.equal(c, w) for c, w in zip(cache, want_cache))


# ---------------------------------------------------------------------------
# Windows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,news", [([5, 40, 0], [10, 10, 10]), ([60, 300, 3], [200, 200, 200]), ([40, 2000], [400, 333])])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 7, 1 << 30])
def test_largest_windows_hide_nothing(lens, news, window):
    """As no window, also for rows before position 0."""
    b = ref.make_batch(104, lens, news, 2, 64, 32)
    q = queries(105, sum(news), 4, 64)
    want, want_lse, bound, lse_bound = ref.attention(ref.f64(q), b, 0.125, 0)
    out, lse = attend(b, q, window=window)
    close(out, want, bound)
    close(lse, want_lse, lse_bound)
