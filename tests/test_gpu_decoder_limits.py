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
    want = np.broadcast_to(want, got.shape)
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


# ---------------------------------------------------------------------------
# Page exponents of V
# ---------------------------------------------------------------------------

def definition(b, q, scale):
    """(out, its bound, lse).

    Weights are held to 2^-11 of themselves, or to 2^-32 of the row's largest product of weight
    and page scale of V where that is more; scores and 2^x are off by 2^-16 here (sizes below 30),
    l by 2^-18.  So |error| <= 2^-8 |out| (bf16) + 2^-10 sum p |v| + 2^-32 max(p 2^e) sum |codes|."""
    T, heads, dim = q.shape
    group = heads // b.k.shape[1]
    out, bound, lse = np.zeros_like(q), np.zeros_like(q), np.zeros((T, heads))
    for s, n in enumerate(b.news):
        rows = slice(b.starts[s], b.starts[s] + n)
        seen = np.arange(b.lens[s])[None] <= b.lens[s] - n + np.arange(n)[:, None]
        for h in range(heads):
            k, v = ref.cached(b, s, h // group, "k"), ref.cached(b, s, h // group, "v")
            x = np.where(seen, q[rows, h] @ k.T * scale, -np.inf)
            m = x.max(1, keepdims=True)
            w = np.exp(x - m)
            z = w.sum(1, keepdims=True)
            p = w / z
            e = 2.0 ** np.repeat(b.v_exp[b.table[s], h // group].astype(float), b.page)[:b.lens[s]]
            floor = np.max(p * e, 1, keepdims=True) * (seen @ np.abs(v / e[:, None])) * 2.0 ** -32
            out[rows, h] = p @ v
            bound[rows, h] = 2.0 ** -8 * np.abs(p @ v) + 2.0 ** -10 * (p @ np.abs(v)) + floor
            lse[rows, h] = (np.log(z) + m)[:, 0]
    return out, bound, lse


@pytest.mark.parametrize("n", [1, 5, 80])
@pytest.mark.parametrize("order", ["high first", "low first", "in turn"])
@pytest.mark.parametrize("scores", ["equal", "random"])
def test_v_exponents_at_both_limits(n, order, scores):
    """Half of the weight lies on pages whose scale is 2^-64, the other half on pages of 2^64."""
    b = ref.make_batch(106, [256, 192], [n, n], 2, 64, 32, garbage=False)
    b.k_exp[:] = -9
    for s in range(2):
        pages = -(-b.lens[s] // 32)
        at = np.arange(pages)
        high = {"high first": at < pages // 2, "low first": at >= pages // 2, "in turn": at % 2 == 0}[order]
        b.v_exp[b.table[s, :pages]] = np.where(high, 64, -64)[:, None]
    q = queries(107, 2 * n, 4, 64)
    if scores == "equal":
        q = torch.zeros_like(q)
    want, bound, want_lse = definition(b, ref.f64(q), 1.0)
    out, lse = attend(b, q, scale=1.0)
    close(lse, want_lse, 2.0 ** -15)
    close(out, want, bound)


@pytest.mark.parametrize("n,copies", [(1, 64), (5, 64), (80, 8)])
@pytest.mark.parametrize("at", [3, 2000])
@pytest.mark.parametrize("apart", [0, 7, 14])
def test_v_exponent_of_one_page_above_the_others(n, copies, at, apart):
    """One key with half of the weight on a page of a large scale and small codes, among 4000
    alike with the other half, which may not be lost.  As many sequences over the same pages as
    leave no one's keys split between CTAs: one running maximum serves them all."""
    length, page, dim, heads = 4000, 64, 64, 16
    b = ref.make_batch(108, [length], [n], heads, dim, page, garbage=False)
    b.k[:] = 0
    b.k_exp[:], b.v_exp[:] = 0, -6
    b.k[b.table[0, at // page], :, at % page, 0] = 0x38                      # 1.0
    b.v[:] &= 0x7F                                                           # one sign: nothing cancels
    b.v[b.table[0, at // page]] = 0x01
    b.v_exp[b.table[0, at // page]] += apart
    q = torch.zeros(n, heads, dim, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    scale = float(np.log(length - 1.0))
    want, bound, want_lse = definition(b, ref.f64(q), scale)
    many = ref.Batch([length] * copies, [n] * copies, np.repeat(b.table, copies, 0), b.k, b.v, b.k_exp, b.v_exp)
    out, lse = attend(many, q.repeat(copies, 1, 1), scale=scale)
    close(lse.reshape(copies, n, heads), want_lse, 2.0 ** -15)
    close(out.reshape(copies, n, heads, dim), want, bound)


# ---------------------------------------------------------------------------
# Lengths at the end of 32 bits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("page", [16, 256])
def test_append_rotates_at_the_last_positions(n, page):
    """Past the page table: rotated, not stored."""
    heads, kv_heads, dim = 4, 2, 64
    last = 2 ** 31 - 1
    b = ref.make_batch(111, [20], [n], kv_heads, dim, page)
    cache, table, _, _ = b.device()
    before = [c.view(torch.uint8).clone() for c in cache]
    x = queries(112, n, heads + 2 * kv_heads, dim)
    q, k, v = x.cuda().split([heads, kv_heads, kv_heads], 1)
    turns = lb.rotary_turns(dim)
    out = torch.full((n, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lb.kv_append(q, k, v, *cache, table, torch.tensor([last], dtype=torch.int32, device="cuda"), turns=turns.cuda(), out=out)
    want, mag = ref.rotate(ref.f64(x)[:, :heads], [last - n + i for i in range(n)], turns.tolist(), False, 1.0)
    close(ref.f64(out), want, 2.0 ** (np.frexp(want)[1] - 9.0) + mag * 2.0 ** -20)
    assert all(torch.equal(c.view(torch.uint8), o) for c, o in zip(cache, before))


# ---------------------------------------------------------------------------
# Signs of the scale
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 5, 80])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("scale", [-0.125, 0.0, -0.0])
def test_negative_and_zero_scales(n, window, scale):
    """As -q with a positive scale; zero: the mean of what a row sees."""
    b = ref.make_batch(109, [200, 129], [n, n], 2, 64, 32)
    q = queries(110, 2 * n, 8, 64)
    out, lse = attend(b, q, scale=scale, window=window)
    x = ref.f64(q) * (np.sign(scale) if scale else 0.0)
    want, want_lse, bound, lse_bound = ref.attention(x, b, 0.125, window)
    close(out, want, bound)
    close(lse, want_lse, lse_bound)
