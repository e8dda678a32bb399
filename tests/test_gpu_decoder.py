"""The decoder operators on the GPU against their plain 64-bit definitions
(decoder_ref): the cache append, attention over the 8-bit cache, and sampling, at
the sizes and masks where they can go wrong.  Tolerances are derived beside the
definitions."""
from __future__ import annotations

import math

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


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def run_attention(b, q, scale=None, window=0, **kw):
    """q bf16 on the CPU [T, heads, dim]."""
    cache, table, lens, cu = b.device()
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    out = lb.attention(q.cuda(), *cache, table, lens, cu_q=cu, max_q=max(b.news), scale=scale, window=window, lse=lse, **kw)
    assert lb.wait_timeouts() == 0
    return ref.f64(out), ref.f64(lse)


def check_attention(b, q, scale=None, window=0, **kw):
    out, lse = run_attention(b, q, scale, window, **kw)
    s = q.shape[2] ** -0.5 if scale is None else scale
    want, want_lse, bound, lse_bound = ref.attention(ref.f64(q), b, s, window)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(out), nan)
    err = np.abs(out - want)
    assert np.all((err <= bound)[~nan]), (f"worst {np.nanmax((err - bound)[~nan])}, at "
                                          f"{np.argwhere((err > bound) & ~nan)[:4].tolist()}")
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    ok = ~empty & ~np.isnan(want_lse)
    assert np.all(np.abs(lse[ok] - want_lse[ok]) <= lse_bound[ok])
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse))


def queries(seed, T, heads, dim, spread=1.0):
    rng = np.random.default_rng([seed, T, heads, dim])
    return ref.bf16(rng.standard_normal((T, heads, dim)) * spread)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (8, 2), (6, 2), (9, 1), (16, 1), (32, 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_decode_lengths(dim, heads, kv_heads, page):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1000]
    b = ref.make_batch(1, lens, [1] * len(lens), kv_heads, dim, page)
    check_attention(b, queries(2, len(lens), heads, dim))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("n", [2, 3, 5, 16, 33, 64, 130])
def test_several_tokens_a_sequence(dim, page, n):
    lens = [n, n + 1, n + 63, n + 200]
    b = ref.make_batch(3, lens, [n] * 4, 2, dim, page)
    check_attention(b, queries(4, 4 * n, 6, dim))


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (16, 1, 128), (5, 1, 64)])
def test_ragged_prompts_and_single_tokens_together(heads, kv_heads, dim):
    lens = [1, 40, 300, 129, 700, 64, 257, 5]
    news = [1, 40, 1, 128, 333, 64, 2, 0]
    b = ref.make_batch(5, lens, news, kv_heads, dim, 64)
    check_attention(b, queries(6, sum(news), heads, dim))


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("window", [0, 700])
def test_prompts_behind_lengths_far_apart(heads, kv_heads, dim, window):
    """Some tiles' keys are split between CTAs, others' are not, some sequences have none."""
    lens, news = [5000, 90, 0, 2100, 1300, 300], [100, 90, 0, 70, 1, 300]
    b = ref.make_batch(80, lens, news, kv_heads, dim, 64)
    check_attention(b, queries(81, sum(news), heads, dim), window=window)


def test_prompts_of_many_sequences():
    """More sequences than lanes, a few of them long."""
    lens = [20 + 3 * i for i in range(40)] + [3000, 0, 1500]
    news = [20] * 40 + [33, 0, 21]
    b = ref.make_batch(82, lens, news, 1, 64, 32)
    check_attention(b, queries(83, sum(news), 4, 64))


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 1000])
@pytest.mark.parametrize("n", [1, 7, 150])
@pytest.mark.parametrize("dim", [64, 128])
def test_window(window, n, dim):
    lens = [n, n + 64, n + 300]
    b = ref.make_batch(7, lens, [n] * 3, 2, dim, 16)
    check_attention(b, queries(8, 3 * n, 8, dim), window=window)


def test_window_leaves_earlier_pages_unread():
    """Pages wholly before the window may have been given away (table entry -1)."""
    b = ref.make_batch(9, [1000], [1], 2, 128, 64)
    q = queries(10, 1, 8, 128)
    whole, whole_lse = run_attention(b, q, window=100)
    b.table[0, :(1000 - 100) // 64] = -1
    cut, cut_lse = run_attention(b, q, window=100)
    assert np.array_equal(whole, cut) and np.array_equal(whole_lse, cut_lse)


@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_rows_that_see_nothing(n):
    """Empty sequences, and new tokens before position 0 (more of them than the length)."""
    lens, news = [0, 5, n, 0], [n, n, n, n]
    b = ref.make_batch(11, lens, news, 2, 128, 16)
    check_attention(b, queries(12, 4 * n, 4, 128))


@pytest.mark.parametrize("n", [4, 100])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_reaches_only_the_rows_that_see_it(n, window, which):
    b = ref.make_batch(13, [150, 130], [n, n], 2, 128, 32)
    codes = b.k if which == "k" else b.v
    for seq, at, d in ((0, 148, 5), (0, 100, 77), (1, 127, 0)):
        codes[b.table[seq, at // 32], :, at % 32, d] = 0x7F
    check_attention(b, queries(14, 2 * n, 8, 128), window=window)


@pytest.mark.parametrize("n", [1, 64])
def test_infinite_and_nan_queries_keep_to_their_rows(n):
    b = ref.make_batch(15, [200] * 3, [n] * 3, 2, 128, 64)
    q = queries(16, 3 * n, 8, 128)
    clean, _ = run_attention(b, q)
    bad = q.clone()
    bad[0, 1, 3], bad[n, 2, 9] = float("nan"), float("inf")
    got, _ = run_attention(b, bad)
    hit = np.zeros(got.shape[:2], bool)
    hit[0, 1] = hit[n, 2] = True
    assert np.isnan(got[hit]).all()
    assert np.array_equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("spread", [1e-30, 1e-3, 30.0, 1e4, 1e30])
@pytest.mark.parametrize("n", [1, 80])
def test_query_sizes(spread, n):
    """Rows are brought to fp16 by a power of two of their own: any bf16 size will do."""
    b = ref.make_batch(17, [333, 100], [n] * 2, 1, 64, 64)
    scale = 0.125 / spread
    check_attention(b, queries(18, 2 * n, 4, 64, spread), scale=scale)


@pytest.mark.parametrize("n", [1, 80])
@pytest.mark.parametrize("k_exps,v_exps", [((-64, -40), (-64, -60)), ((0, 1), (40, 64)), ((-14, -2), (-30, 20))])
def test_page_exponents_far_apart(n, k_exps, v_exps):
    b = ref.make_batch(19, [400, 257], [n] * 2, 2, 128, 32)
    rng = np.random.default_rng(20)
    b.k_exp[:] = rng.integers(k_exps[0], k_exps[1] + 1, b.k_exp.shape)
    b.v_exp[:] = rng.integers(v_exps[0], v_exps[1] + 1, b.v_exp.shape)
    top = 2.0 ** int(b.k_exp.max())
    check_attention(b, queries(21, 2 * n, 4, 128), scale=0.02 / top)


def test_long_sequence_is_split_and_joined():
    b = ref.make_batch(22, [20000, 3], [1, 1], 1, 64, 256)
    check_attention(b, queries(23, 2, 8, 64))


def test_many_sequences():
    rng = np.random.default_rng(24)
    lens = rng.integers(1, 90, 400).tolist()
    b = ref.make_batch(24, lens, [1] * 400, 1, 64, 16)
    check_attention(b, queries(25, 400, 3, 64))


def test_strided_cache_and_rows():
    """k and v as views of one tensor, pages with a gap, q a slice of a projection, out and lse views."""
    b = ref.make_batch(26, [77, 200], [3, 3], 2, 128, 64)
    (k, v, ke, ve), table, lens, _ = b.device()
    pages = k.shape[0]
    both = torch.full((pages, 3, 2, 64, 128), 0x7F, dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 2] = k.view(torch.uint8), v.view(torch.uint8)
    both = both.view(torch.float8_e4m3fn)
    wide = torch.full((2, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = queries(27, 6, 8, 128)
    proj = torch.randn(6, 12, 128, device="cuda").to(torch.bfloat16)
    proj[:, :8] = q.cuda()
    out = torch.zeros(6, 10, 132, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(6, 11, device="cuda")
    got = lb.attention(proj[:, :8], both[:, 0], both[:, 2], ke, ve, wide[:, :table.shape[1]], lens,
                       out=out[:, 1:9, 4:], lse=lse[:, 2:10])
    want, want_lse = run_attention(b, q)
    assert np.array_equal(ref.f64(got), want) and np.array_equal(ref.f64(lse[:, 2:10]), want_lse)
    assert not out[:, 0].any() and not out[:, 9].any() and not out[..., :4].any() and not lse[:, :2].any()


def test_cache_beyond_32_bit_offsets():
    """Pages past 2^32 bytes from the cache's start."""
    pages, page, dim = (1 << 32) // (64 * 128) + 3, 64, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 10 * (1 << 30):
        pytest.skip("needs 10 GiB")
    k = torch.zeros(pages, 1, page, dim, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    exps = torch.zeros(pages, 1, dtype=torch.int8, device="cuda")
    small = ref.make_batch(28, [100], [1], 1, dim, page, spare=0)
    far = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    for i in range(2):
        k[far[0, i].item()] = torch.from_numpy(small.k[small.table[0, i]]).cuda()
        v[far[0, i].item()] = torch.from_numpy(small.v[small.table[0, i]]).cuda()
        exps[far[0, i].item()] = int(small.k_exp[small.table[0, i], 0])
    small.v_exp[:] = small.k_exp
    q = queries(29, 1, 4, dim)
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    got = lb.attention(q.cuda(), k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), exps, exps, far, lens)
    want, _ = run_attention(small, q)
    assert np.array_equal(ref.f64(got), want)
    # And the append reaches them.
    x = torch.randn(1, 1, dim, device="cuda").to(torch.bfloat16)
    lb.kv_append(q.cuda(), x, x, k, v, exps, exps.clone(), far, lens)
    assert k[pages - 2, 0, 99 % 64].any() and not k[:2].any()


def test_same_result_every_time_and_on_another_stream():
    b = ref.make_batch(30, [5000, 17, 900], [2, 2, 2], 2, 128, 64)
    q = queries(31, 6, 8, 128).cuda()
    cache, table, lens, _ = b.device()
    ws = torch.empty(lb.attention_workspace(q, *cache, table, lens), dtype=torch.uint8, device="cuda")
    first = lb.attention(q, *cache, table, lens, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = lb.attention(q, *cache, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, second)
    for _ in range(20):
        assert torch.equal(first, lb.attention(q, *cache, table, lens, workspace=ws))


def test_captured_step_follows_the_lengths():
    """A CUDA graph of append and attention, replayed as the sequences grow."""
    heads, kv_heads, dim, page = 8, 2, 128, 16
    b = ref.make_batch(32, [64, 64], [1, 1], kv_heads, dim, page)
    cache, table, lens, _ = b.device()
    turns = lb.rotary_turns(dim, device="cuda")
    qkv = torch.randn(2, heads + 2 * kv_heads, dim, device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
    lens.copy_(torch.tensor([30, 60]))

    def step():
        return lb.attention(lb.kv_append(q, k, v, *cache, table, lens, turns=turns), *cache, table, lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    start = [c.view(torch.uint8).clone() for c in cache]
    with torch.cuda.graph(graph):
        o = step()
    got = []
    for _ in range(3):
        lens += 1
        graph.replay()
        got.append(o.clone())
    after = [c.view(torch.uint8).clone() for c in cache]
    for c, s in zip(cache, start):
        c.view(torch.uint8).copy_(s)
    lens.copy_(torch.tensor([30, 60]))
    for i in range(3):
        lens += 1
        assert torch.equal(step(), got[i])
    assert all(torch.equal(c.view(torch.uint8), a) for c, a in zip(cache, after))


# ---------------------------------------------------------------------------
# kv_append
# ---------------------------------------------------------------------------

def append_inputs(seed, T, heads, kv_heads, dim, size=1.0):
    rng = np.random.default_rng([seed, T, heads, dim])
    return ref.bf16(rng.standard_normal((T, heads + 2 * kv_heads, dim)) * size)


def check_append(b, qkv, heads, turns, interleaved=False, factor=1.0, in_place=False, split=None):
    kv_heads, page, T = b.k.shape[1], b.page, qkv.shape[0]
    cache, table, lens, cu = b.device()
    dev = qkv.cuda() if split is None else split(qkv)
    q, k, v = dev.split([heads, kv_heads, kv_heads], 1)
    t = None if turns is None else torch.tensor(turns, dtype=torch.int64, device="cuda")
    got = lb.kv_append(q, k, v, *cache, table, lens, cu_q=cu, max_q=max(b.news), turns=t, interleaved=interleaved,
                       factor=factor, out=q if in_place else None)
    x = ref.f64(qkv)
    turns = [] if turns is None else turns
    pos = np.concatenate([n - m + np.arange(m) for n, m in zip(b.lens, b.news)]) if T else np.zeros(0, int)
    want_q, mag = ref.rotate(x[:, :heads], pos, turns, interleaved, factor)
    # fp32 rotation (angle to 2^-23, three roundings), one rounding to bf16: half a unit in
    # the last of its 8 bits.
    bound = 2.0 ** (np.frexp(want_q)[1] - 9.0) + mag * 2.0 ** -20
    assert np.all(np.abs(ref.f64(got) - want_q) <= bound)
    fresh_k, mag_k = ref.rotate(x[:, heads:heads + kv_heads], pos, turns, interleaved, factor)
    for which, fresh, mag, before, exp_before, codes, exps in (
            ("k", fresh_k, mag_k, b.k, b.k_exp, cache[0], cache[2]),
            ("v", x[:, heads + kv_heads:], np.abs(x[:, heads + kv_heads:]), b.v, b.v_exp, cache[1], cache[3])):
        codes, exps = codes.view(torch.uint8).cpu().numpy(), exps.cpu().numpy()
        touched = np.zeros(codes.shape[:1] + codes.shape[2:3], bool)          # [pages, page]
        paged = np.zeros(codes.shape[0], bool)
        for s, (n, m) in enumerate(zip(b.lens, b.news)):
            for slot in range(max(n - m, 0) // page, -(-n // page)):
                lo, hi = max(slot * page, n - m, 0), min(slot * page + page, n)
                if lo >= hi or slot >= b.table.shape[1]:
                    continue
                pg = b.table[s, slot]
                if not 0 <= pg < codes.shape[0]:
                    continue
                paged[pg] = True
                older = lo - slot * page
                touched[pg, :hi - slot * page] = True
                rows = slice(b.starts[s] + lo - (n - m), b.starts[s] + hi - (n - m))
                for h in range(kv_heads):
                    new, slack = fresh[rows, h], mag[rows, h] * 2.0 ** -20
                    size = np.where(np.isfinite(new), np.abs(new), 0.0)
                    lo_e = ref.page_exponent((size - slack).max())
                    hi_e = ref.page_exponent((size + np.nan_to_num(slack, posinf=0.0)).max())
                    e, was = int(exps[pg, h]), int(exp_before[pg, h])
                    if older:
                        assert max(lo_e, was) <= e <= max(hi_e, was)
                        moved = ref.e4m3_round(ref.E4M3[before[pg, h, :older]] * 2.0 ** (was - e))
                        assert np.array_equal(codes[pg, h, :older], moved if e != was else before[pg, h, :older])
                    else:
                        assert lo_e <= e <= hi_e
                    val = ref.E4M3[codes[pg, h, older:hi - slot * page]]
                    want = np.clip(new * 2.0 ** -e, -448, 448)
                    assert np.array_equal(np.isnan(val), np.isnan(want))
                    # The stored value is the nearest, up to the fp32 error of the rotation.
                    near = np.abs(ref.E4M3[ref.e4m3_round(want)] - want)
                    ok = np.abs(val - want) <= near + 2 * np.nan_to_num(slack, posinf=0.0) * 2.0 ** -e + 1e-300
                    assert np.all(ok | np.isnan(want)), (which, s, slot, h)
        # Everything else is untouched.
        assert np.array_equal(np.where(touched[:, None, :, None], 0, codes), np.where(touched[:, None, :, None], 0, before))
        assert np.array_equal(exps[~paged], exp_before[~paged])
    return cache


def turns_of(dim, base=10000.0):
    return lb.rotary_turns(dim, base).tolist()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 32), (128, 128), (128, 96), (128, 64), (128, 10), (64, 2), (128, 0)])
def test_append_rotary_forms(interleaved, dim, rotary):
    lens, news = [40, 3, 130, 65], [7, 3, 100, 1]
    b = ref.make_batch(40, lens, news, 2, dim, 32)
    check_append(b, append_inputs(41, sum(news), 6, 2, dim), 6, turns_of(rotary) if rotary else None, interleaved, 1.1)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("news", [[1, 1, 1, 1], [5, 0, 300, 2], [64, 64, 64, 64], [257, 1, 33, 600]])
def test_append_pages_and_lengths(page, news):
    lens = [n + e for n, e in zip(news, [0, 15, 31, 255])]
    b = ref.make_batch(42, lens, news, 3, 64, page)
    check_append(b, append_inputs(43, sum(news), 3, 3, 64), 3, turns_of(64))


@pytest.mark.parametrize("size", [1e-6, 1.0, 300.0, 1e20])
def test_append_older_codes_move_with_the_scale(size):
    """One token after another into the same page: its scale grows with the largest value."""
    b = ref.make_batch(44, [9, 33], [1, 1], 2, 128, 16, exps=(-3, 9))
    check_append(b, append_inputs(45, 2, 4, 2, 128, size), 4, turns_of(128))


def test_append_far_positions_are_as_exact_as_near_ones():
    """Position 10^6 with the fastest frequencies: an fp32 angle would be off by 0.03."""
    b = ref.make_batch(46, [20], [4], 1, 64, 16)
    b.lens = [1_000_000]
    b.table = np.full((1, 62500), -1, np.int32)
    b.table[0, -1] = 0
    check_append(b, append_inputs(47, 4, 2, 1, 64), 2, turns_of(64))


def test_append_infinite_and_nan_values():
    b = ref.make_batch(48, [20, 5], [3, 5], 1, 64, 16)
    x = append_inputs(49, 8, 1, 1, 64)
    x[1, 2, 5], x[3, 2, 9], x[4, 2, 1] = float("inf"), float("-inf"), float("nan")     # in v
    cache = check_append(b, x, 1, None)
    assert ref.E4M3[cache[1].view(torch.uint8).cpu().numpy()[b.table[1, 0], 0, 0, 9]] == -448


def test_append_outside_the_cache_is_left_out():
    """New tokens before position 0, past the page table, or on a page that is not in the cache."""
    b = ref.make_batch(50, [3, 40, 33], [10, 40, 2], 2, 64, 16)
    b.table[1, 1] = -5
    b.table[2, 2] = b.k.shape[0] + 7
    check_append(b, append_inputs(51, 52, 2, 2, 64), 2, turns_of(64))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [64, 10])
def test_append_in_place_and_unaligned(interleaved, rotary):
    b = ref.make_batch(52, [40, 80], [40, 5], 2, 64, 64)
    x = append_inputs(53, 45, 4, 2, 64)
    check_append(b, x, 4, turns_of(rotary), interleaved, in_place=True)

    def odd(t):                                        # rows that start on odd elements
        wide = torch.zeros(t.shape[0], t.shape[1], 67, dtype=torch.bfloat16, device="cuda")
        wide[..., 3:] = t.cuda()
        return wide[..., 3:]
    check_append(b, x, 4, turns_of(rotary), interleaved, split=odd)


def test_appending_a_prompt_in_parts_gives_the_same_cache():
    """Chunks that end on page boundaries, and all at once: the same codes and exponents."""
    x = append_inputs(54, 150, 2, 2, 64).cuda()
    turns = lb.rotary_turns(64, device="cuda")
    table = torch.arange(5, dtype=torch.int32, device="cuda")[None]

    def fill(cuts):
        cache = lb.empty_cache(5, 2, 64, 32)
        for a, e in zip(cuts[:-1], cuts[1:]):
            q, k, v = x[a:e].split([2, 2, 2], 1)
            lb.kv_append(q, k, v, *cache, table, torch.tensor([e], dtype=torch.int32, device="cuda"), turns=turns)
        return [c.view(torch.uint8) for c in cache]
    assert all(torch.equal(a, b) for a, b in zip(fill([0, 150]), fill([0, 32, 96, 128, 150])))


@pytest.mark.parametrize("scaling", [None, "linear", "base", "wavelength"])
def test_rotary_scaling_reaches_the_rotation(scaling):
    turns = lb.rotary_turns(64, 10000.0, scaling=scaling, factor=4.0, original_length=512).tolist()
    b = ref.make_batch(55, [300], [2], 1, 64, 64)
    check_append(b, append_inputs(56, 2, 2, 1, 64), 2, turns, factor=0.9)


# ---------------------------------------------------------------------------
# sample
# ---------------------------------------------------------------------------

def run_sample(logits, u, temperature, top_k, top_p, min_p, per_row=True):
    B = logits.shape[0]
    if per_row:
        def dev(x, dt):
            return torch.tensor(np.broadcast_to(np.asarray(x), (B,)).copy(), dtype=dt, device="cuda")
        temperature, top_p, min_p = (dev(x, torch.float32) for x in (temperature, top_p, min_p))
        top_k = dev(top_k, torch.int32)
    logprob = torch.empty(B, device="cuda")
    token = lb.sample(logits.cuda(), torch.tensor(u, dtype=torch.float32, device="cuda"), temperature, top_k, top_p, min_p,
                      logprob=logprob)
    return token.cpu().numpy(), ref.f64(logprob)


def check_rows(logits, u, temperature, top_k, top_p, min_p):
    B = logits.shape[0]
    token, logprob = run_sample(logits, u, temperature, top_k, top_p, min_p)
    rows = ref.f64(logits)
    args = [np.broadcast_to(np.asarray(x), (B,)) for x in (temperature, top_k, top_p, min_p)]
    for b in range(B):
        t, k, p, m = (float(np.float32(a[b])) if i != 1 else int(a[b]) for i, a in enumerate(args))
        ref.check_sample(rows[b], float(np.float32(u[b])), t, k, p, m, int(token[b]), float(logprob[b]))


def make_logits(seed, B, V, dtype, spread=3.0):
    rng = np.random.default_rng([seed, B, V])
    return torch.from_numpy((rng.standard_normal((B, V)) * spread).astype(np.float32)).to(dtype)


SETTINGS = [dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), dict(temperature=0.7, top_k=40, top_p=1.0, min_p=0.0),
            dict(temperature=1.2, top_k=0, top_p=0.9, min_p=0.0), dict(temperature=0.9, top_k=0, top_p=1.0, min_p=0.05),
            dict(temperature=0.8, top_k=300, top_p=0.95, min_p=0.001), dict(temperature=5.0, top_k=3, top_p=0.5, min_p=0.0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4097, 32000, 70001])
@pytest.mark.parametrize("s", range(len(SETTINGS)))
def test_sample_sizes(dtype, V, s):
    B = 5
    u = np.random.default_rng([60, V, s]).random(B)
    u[0], u[1] = 0.0, 1 - 2.0 ** -24
    check_rows(make_logits(61, B, V, dtype), u, **SETTINGS[s])


@pytest.mark.parametrize("B", [1, 2, 40, 300])
def test_sample_batches_with_settings_of_their_own(B):
    rng = np.random.default_rng([62, B])
    check_rows(make_logits(63, B, 9000, torch.float32), rng.random(B), rng.choice([0.0, 0.5, 1.0, 2.0], B),
               rng.choice([0, 1, 2, 17, 8999, 9000, 20000], B), rng.choice([1.0, 0.0, 0.3, 0.99], B),
               rng.choice([0.0, 0.01, 1.0], B))


@pytest.mark.parametrize("V", [700, 20000])
def test_sample_equal_logits(V):
    """All equal, and many equal at the cut: kept in index order."""
    flat = torch.zeros(4, V)
    check_rows(flat, np.array([0.0, 0.31, 0.77, 0.9999]), 1.0, [0, 10, 0, 100], [1.0, 1.0, 0.25, 0.5], 0.0)
    steps = torch.from_numpy((np.arange(4 * V).reshape(4, V) * 7919 % 5).astype(np.float32))
    check_rows(steps, np.array([0.1, 0.5, 0.9, 0.99]), 1.0, [0, V // 5 + 13, 0, V // 5 + 13], [0.9, 1.0, 0.7, 0.99], 0.0)


def test_sample_signed_zeros_are_equal():
    x = torch.zeros(1, 64)
    x[0, ::2] = -0.0
    for k in (1, 3, 33):
        assert run_sample(x, [0.999], 1.0, k, 1.0, 0.0)[0][0] == k - 1


def test_sample_infinities_nan_and_empty_rows():
    x = make_logits(64, 6, 5000, torch.float32)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf
    x[3, 7], x[3, 4000] = math.inf, math.inf
    x[4, ::2] = math.nan
    x[5, 100:] = -3.4e38
    token, logprob = run_sample(x, [0.5] * 6, 1.0, 0, 1.0, 0.0)
    assert token[0] == -1 and token[1] == -1 and logprob[0] == -math.inf
    assert token[2] == 0 and logprob[2] == 0
    assert token[3] == 4000 and abs(logprob[3] + math.log(2)) < 1e-6
    rows = ref.f64(x)
    for b in (4, 5):
        ref.check_sample(rows[b], 0.5, 1.0, 0, 1.0, 0.0, int(token[b]), float(logprob[b]))
    assert run_sample(x, [0.5] * 6, 0.0, 0, 1.0, 0.0)[0].tolist()[:4] == [-1, -1, 0, 7]
    assert run_sample(x, [0.1] * 6, 1.0, 1, 1.0, 0.0)[0].tolist()[:4] == [-1, -1, 0, 7]


@pytest.mark.parametrize("temperature", [0.01, 0.1, 10.0, 1000.0])
def test_sample_temperatures(temperature):
    u = np.random.default_rng(65).random(8)
    check_rows(make_logits(66, 8, 3000, torch.float32, 5.0), u, temperature, [0, 0, 50, 50, 0, 0, 0, 2], [1.0, 0.9] * 4, 0.0)


def test_sample_wide_range_of_logits():
    """Values over many binades on both sides of zero."""
    rng = np.random.default_rng(67)
    x = torch.from_numpy((np.sign(rng.standard_normal((4, 6000))) * 10.0 ** rng.uniform(-30, 1, (4, 6000))).astype(np.float32))
    check_rows(x, rng.random(4), 1.0, [0, 2500, 0, 2999], [0.6, 1.0, 0.9, 0.9], 0.0)


def test_sample_rows_apart_scalars_and_repeat():
    x = make_logits(68, 6, 3001, torch.bfloat16).cuda()
    wide = torch.full((6, 3100), 50.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 33:33 + 3001] = x
    u = torch.rand(6, device="cuda")
    a = lb.sample(x, u, 0.8, 30, 0.9, 0.01)
    assert torch.equal(a, lb.sample(wide[:, 33:33 + 3001], u, 0.8, 30, 0.9, 0.01))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = lb.sample(x, u, torch.full((6,), 0.8, device="cuda"), 30, 0.9, torch.full((6,), 0.01, device="cuda"))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, c)
    for _ in range(20):
        assert torch.equal(a, lb.sample(x, u, 0.8, 30, 0.9, 0.01))


def test_sample_draws_follow_the_distribution():
    """Over an even grid of u the draws' counts are the weights, to one step each."""
    n, V = 4096, 50
    x = make_logits(69, 1, V, torch.float32, 1.0)
    u = (np.arange(n) + 0.5) / n
    token, _ = run_sample(x.expand(n, V).contiguous(), u, 1.0, 0, 1.0, 0.0)
    p = np.exp(ref.f64(x)[0])
    assert np.all(np.abs(np.bincount(token, minlength=V) - n * p / p.sum()) <= 1.01)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [900, 3000, 50_000])
def test_sample_many_kept_tokens(V, dtype):
    """Flat rows: lists of all lengths up to the longest and beyond, with many equal logits."""
    u = np.random.default_rng([74, V]).random(10)
    x = make_logits(75, 10, V, dtype, 0.3)
    check_rows(x, u, 1.0, [33, 100, 400, 880, 0, 0, 500, 0, 0, 31], [1.0, 0.9, 0.5, 0.99, 0.02, 0.3, 1.0, 0.9, 0.999, 0.5],
               [0.0] * 9 + [0.9])


def test_sample_top_p_at_its_ends():
    """Zero, and what is below it: the first token.  One, and what is above it: all."""
    x = make_logits(76, 6, 5000, torch.float32)
    first = [int(i) for i in x.argmax(1)]
    token, logprob = run_sample(x, [0.99] * 6, 1.0, 0, [0.0, -0.5, -1e30, 1e-38, 1.0, 2.0], 0.0)
    assert token[:4].tolist() == first[:4] and (logprob[:4] == 0).all()
    for b in (4, 5):
        ref.check_sample(ref.f64(x)[b], float(np.float32(0.99)), 1.0, 0, 1.0, 0.0, int(token[b]), float(logprob[b]))


def test_sample_row_sizes_in_turn():
    """Large rows, small ones, large ones again: each launch has the shared memory it needs."""
    for V in (90_000, 100, 90_000, 3000, 300_000, 40_000):
        check_rows(make_logits(73, 3, V, torch.float32), np.array([0.2, 0.6, 0.95]), 1.0, [0, 50, 0], [0.9, 1.0, 1.0], 0.0)


def test_sample_large_vocabulary_beyond_what_is_held():
    check_rows(make_logits(70, 2, 400_003, torch.float32), np.array([0.2, 0.95]), 1.0, [0, 1000], [0.95, 1.0], 0.0)
