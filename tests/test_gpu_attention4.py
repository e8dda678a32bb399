"""Attention over the 4-bit cache on the GPU against its plain 64-bit definition (cache4_ref),
at the sizes and masks where it can go wrong, and the operators of a decode step together."""
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
from bit_groupwise_weight_gb300 import decoder  # noqa: E402

lbuild.build()


def run(b, q, scale=None, window=0, **kw):
    """q bf16 on the CPU [T, heads, dim]."""
    cache, table, lens, cu = b.device()
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    out = lb.attention(q.cuda(), *cache, table, lens, cu_q=cu, max_q=max(b.news), scale=scale, window=window, lse=lse, **kw)
    assert lb.wait_timeouts() == 0
    return ref.f64(out), ref.f64(lse)


def check(b, q, scale=None, window=0, **kw):
    out, lse = run(b, q, scale, window, **kw)
    s = q.shape[2] ** -0.5 if scale is None else scale
    want, want_lse, bound, lse_bound = ref4.attention(ref.f64(q), b, s, window)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(out), nan)
    err = np.abs(out - want)
    assert np.all((err <= bound)[~nan]), f"worst {np.nanmax((err - bound)[~nan])}, at {np.argwhere((err > bound) & ~nan)[:4].tolist()}"
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    ok = ~empty & ~np.isnan(want_lse)
    assert np.all(np.abs(lse[ok] - want_lse[ok]) <= lse_bound[ok]), np.max(np.abs(lse[ok] - want_lse[ok]) - lse_bound[ok])
    assert np.array_equal(np.isnan(lse), np.isnan(want_lse))


def queries(seed, T, heads, dim, spread=1.0):
    rng = np.random.default_rng([seed, T, heads, dim])
    return ref.bf16(rng.standard_normal((T, heads, dim)) * spread)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (8, 2), (7, 1), (9, 1), (16, 1), (32, 1)])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_lengths(dim, heads, kv_heads, page):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1000]
    b = ref4.make_batch(1, lens, [1] * len(lens), kv_heads, dim, page)
    check(b, queries(2, len(lens), heads, dim))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("n", [2, 3, 5, 16, 33, 64, 130])
def test_several_tokens_a_sequence(dim, page, n):
    lens = [n, n + 1, n + 63, n + 200]
    b = ref4.make_batch(3, lens, [n] * 4, 2, dim, page)
    check(b, queries(4, 4 * n, 6, dim))


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (16, 1, 128), (5, 1, 64)])
def test_ragged_prompts_and_single_tokens_together(heads, kv_heads, dim):
    lens = [1, 40, 300, 129, 700, 64, 257, 5]
    news = [1, 40, 1, 128, 333, 64, 2, 0]
    b = ref4.make_batch(5, lens, news, kv_heads, dim, 64)
    check(b, queries(6, sum(news), heads, dim))


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("window", [0, 700])
def test_prompts_behind_lengths_far_apart(heads, kv_heads, dim, window):
    """Some tiles' keys are split between CTAs, others' are not, some sequences have none."""
    lens, news = [5000, 90, 0, 2100, 1300, 300], [100, 90, 0, 70, 1, 300]
    b = ref4.make_batch(7, lens, news, kv_heads, dim, 64)
    check(b, queries(8, sum(news), heads, dim), window=window)


def test_prompts_of_many_sequences():
    """More sequences than lanes, a few of them long."""
    lens = [20 + 3 * i for i in range(40)] + [2700, 0, 1500]
    news = [20] * 40 + [33, 0, 21]
    b = ref4.make_batch(9, lens, news, 1, 64, 32)
    check(b, queries(10, sum(news), 4, 64))


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 1000])
@pytest.mark.parametrize("n", [1, 7, 150])
@pytest.mark.parametrize("dim", [64, 128])
def test_window(window, n, dim):
    lens = [n, n + 64, n + 300]
    b = ref4.make_batch(11, lens, [n] * 3, 2, dim, 16)
    check(b, queries(12, 3 * n, 8, dim), window=window)


def test_window_leaves_earlier_pages_unread():
    """Pages wholly before the window may have been given away (table entry -1)."""
    b = ref4.make_batch(13, [1000], [1], 2, 128, 64)
    q = queries(14, 1, 8, 128)
    whole, whole_lse = run(b, q, window=100)
    b.table[0, :(1000 - 100) // 64] = -1
    cut, cut_lse = run(b, q, window=100)
    assert np.array_equal(whole, cut) and np.array_equal(whole_lse, cut_lse)


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_outside_the_cache_read_as_zeros(n, page):
    b = ref4.make_batch(15, [300, 280], [n, n], 2, 128, page)
    b.table[0, 1], b.table[1, 0] = -1, b.k.shape[0] + 5
    check(b, queries(16, 2 * n, 8, 128))


@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_rows_that_see_nothing(n):
    """Empty sequences, and new tokens before position 0 (more of them than the length)."""
    lens, news = [0, 5, n, 0], [n, n, n, n]
    b = ref4.make_batch(17, lens, news, 2, 128, 16)
    check(b, queries(18, 4 * n, 4, 128))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 100])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_reaches_only_the_rows_that_see_it(n, window, which, dim):
    """A scale that is no number: in v its 32 values of the rows that see the key, in k all of such rows."""
    b = ref4.make_batch(19, [150, 130], [n, n], 2, dim, 32)
    scales = b.k_scale if which == "k" else b.v_scale
    for seq, at, j in ((0, 148, 1), (0, 100, 0), (1, 127, dim // 32 - 1)):
        scales[b.table[seq, at // 32], :, at % 32, j] = 0x7F
    check(b, queries(20, 2 * n, 8, dim), window=window)


@pytest.mark.parametrize("n", [1, 64])
def test_infinite_and_nan_queries_keep_to_their_rows(n):
    b = ref4.make_batch(21, [200] * 3, [n] * 3, 2, 128, 64)
    q = queries(22, 3 * n, 8, 128)
    clean, _ = run(b, q)
    bad = q.clone()
    bad[0, 1, 3], bad[n, 2, 9] = float("nan"), float("inf")
    got, _ = run(b, bad)
    hit = np.zeros(got.shape[:2], bool)
    hit[0, 1] = hit[n, 2] = True
    assert np.isnan(got[hit]).all()
    assert np.array_equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("spread", [1e-30, 1e-3, 30.0, 1e4, 1e30])
@pytest.mark.parametrize("n", [1, 80])
def test_query_sizes(spread, n):
    """Rows are brought to fp16 by a power of two of their own: any bf16 size will do."""
    b = ref4.make_batch(23, [333, 100], [n] * 2, 1, 64, 64)
    check(b, queries(24, 2 * n, 4, 64, spread), scale=0.125 / spread)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
@pytest.mark.parametrize("n", [1, 80])
def test_scales_of_the_scores(scale, n):
    b = ref4.make_batch(25, [333, 100], [n] * 2, 2, 128, 64)
    check(b, queries(26, 2 * n, 4, 128), scale=scale)


@pytest.mark.parametrize("n", [1, 80])
@pytest.mark.parametrize("size", [1e-5, 1e-3, 1e3, 2e5])
def test_cache_sizes(n, size):
    """Scales at both of their limits: products with q and v stay in range."""
    b = ref4.make_batch(27, [400, 257], [n] * 2, 2, 128, 32, size=size)
    check(b, queries(28, 2 * n, 4, 128), scale=0.05 / size)


@pytest.mark.parametrize("n", [1, 80])
def test_scales_far_apart_and_every_code(n):
    """Any scale beside any other, subnormal ones among them, and codes 0 to 15."""
    b = ref4.make_batch(29, [400, 257], [n] * 2, 2, 128, 32)
    rng = np.random.default_rng(30)
    for scales, codes in ((b.k_scale, b.k), (b.v_scale, b.v)):
        scales[:] = rng.integers(0, 0x7C, scales.shape)
        codes[:] = rng.integers(0, 16, codes.shape)
    check(b, queries(31, 2 * n, 4, 128), scale=1e-6)


def test_long_sequence_is_split_and_joined():
    b = ref4.make_batch(32, [20000, 3], [1, 1], 1, 64, 256)
    check(b, queries(33, 2, 8, 64))


def test_many_sequences():
    rng = np.random.default_rng(34)
    lens = rng.integers(1, 90, 400).tolist()
    b = ref4.make_batch(34, lens, [1] * 400, 1, 64, 16)
    check(b, queries(35, 400, 3, 64))


def test_more_tokens_than_max_q_and_rows_behind_the_last_sequence():
    """Tokens past max_q, and rows of no sequence, are left as they were."""
    b = ref4.make_batch(36, [70, 90], [6, 9], 2, 64, 16)
    cache, table, lens, _ = b.device()
    q = queries(37, 20, 4, 64).cuda()
    cu = torch.tensor([0, 6, 15], dtype=torch.int32, device="cuda")
    for window in (0, 20):
        whole = lb.attention(q, *cache, table, lens, cu_q=cu, max_q=9, window=window, out=torch.full_like(q, 7.0))
        part = lb.attention(q, *cache, table, lens, cu_q=cu, max_q=4, window=window, out=torch.full_like(q, 7.0))
        assert (whole[15:] == 7).all()
        live = torch.zeros(20, dtype=torch.bool, device="cuda")
        live[:4] = live[6:10] = True
        assert torch.equal(part[live], whole[live]) and (part[~live] == 7).all()


def test_strided_cache_and_rows():
    """k and v as views of one tensor, their scales too, q a slice of a projection, out and lse views."""
    b = ref4.make_batch(38, [77, 200], [3, 3], 2, 128, 64)
    (k, v, ks, vs), table, lens, _ = b.device()
    pages = k.shape[0]
    codes = torch.full((pages, 3, 2, 64, 64), 0x7F, dtype=torch.uint8, device="cuda")
    codes[:, 0], codes[:, 2] = k, v
    scales = torch.full((pages, 2, 2, 64, 4), 0x7F, dtype=torch.uint8, device="cuda")
    scales[:, 0], scales[:, 1] = ks.view(torch.uint8), vs.view(torch.uint8)
    wide = torch.full((2, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = queries(39, 6, 8, 128)
    proj = torch.randn(6, 12, 128, device="cuda").to(torch.bfloat16)
    proj[:, :8] = q.cuda()
    out = torch.zeros(6, 10, 132, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(6, 11, device="cuda")
    got = lb.attention(proj[:, :8], codes[:, 0], codes[:, 2], scales[:, 0], scales[:, 1], wide[:, :table.shape[1]], lens,
                       out=out[:, 1:9, 4:], lse=lse[:, 2:10])
    want, want_lse = run(b, q)
    assert np.array_equal(ref.f64(got), want) and np.array_equal(ref.f64(lse[:, 2:10]), want_lse)
    assert not out[:, 0].any() and not out[:, 9].any() and not out[..., :4].any() and not lse[:, :2].any()


@pytest.mark.parametrize("n", [1, 90])
def test_cache_beyond_32_bit_offsets(n):
    """Pages past 2^32 bytes from the cache's start."""
    pages, page, dim = (1 << 32) // (64 * 64) + 3, 64, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    cache = lb.empty_cache(pages, 1, dim, page, bits=4)
    small = ref4.make_batch(40, [100], [n], 1, dim, page, spare=0)
    far = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    for i in range(2):
        for c, s in zip(cache, small.cache()):
            c.view(torch.uint8)[far[0, i].item()] = s.view(torch.uint8)[small.table[0, i]]
    q = queries(41, n, 4, dim)
    got = lb.attention(q.cuda(), *cache, far, torch.tensor([100], dtype=torch.int32, device="cuda"))
    want, _ = run(small, q)
    assert np.array_equal(ref.f64(got), want)


@pytest.mark.parametrize("n", [2, 100])
def test_same_result_every_time_and_on_another_stream(n):
    b = ref4.make_batch(42, [5000, 117, 900], [n] * 3, 2, 128, 64)
    q = queries(43, 3 * n, 8, 128).cuda()
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
    for other in (lb.attention(q[:1, :4], cache[0][:, :1], cache[1][:, :1], cache[2][:, :1], cache[3][:, :1], table[:1], lens[:1], workspace=ws),
                  lb.attention(q, *cache, table, lens, workspace=ws)):          # a workspace of another call's leavings
        assert torch.isfinite(other).all()
    assert torch.equal(first, other)


@pytest.mark.parametrize("bits", [4, 8])
def test_decode_step_together(bits):
    """Norms, rotation with two axes, cache write and attention, a prompt and then single tokens as
    replays of a graph, against attention in fp64 over what the cache holds."""
    heads, kv_heads, dim, page, n = 8, 2, 128, 32, 70
    gen = torch.Generator(device="cuda").manual_seed(44)
    cache = lb.empty_cache(12, kv_heads, dim, page, bits=bits)
    table = torch.randperm(12, generator=gen, device="cuda").to(torch.int32).view(2, 6)
    turns, w = lb.rotary_turns(dim, device="cuda"), torch.rand(2, dim, generator=gen, device="cuda") + 0.5
    axes = (torch.arange(dim // 2, device="cuda") % 2).to(torch.uint8)

    def expected(q, lens, news):
        k, v = (x.double() for x in lb.cache_values(*cache))
        out, at = torch.empty(q.shape, dtype=torch.float64, device="cuda"), 0
        for s, (length, new) in enumerate(zip(lens, news)):
            ks, vs = (x[table[s].long()].transpose(0, 1).reshape(kv_heads, -1, dim)[:, :length].repeat_interleave(heads // kv_heads, 0)
                      for x in (k, v))
            scores = torch.einsum("thd,hkd->htk", q[at:at + new].double(), ks) * dim ** -0.5
            hidden = torch.arange(length, device="cuda") > torch.arange(length - new, length, device="cuda")[:, None]
            out[at:at + new] = torch.einsum("htk,hkd->thd", scores.masked_fill(hidden, -torch.inf).softmax(-1), vs)
            at += new
        return out
    news = [n, 33]
    lens = torch.tensor(news, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n, n + 33], dtype=torch.int32, device="cuda")

    def step(qkv, cu_q, max_q, positions):
        q, k, v = qkv.split([heads, kv_heads, kv_heads], 1)
        q = lb.kv_append(q, k, v, *cache, table, lens, cu_q, max_q, turns=turns, q_norm=w[0], k_norm=w[1], positions=positions, axes=axes)
        return q, lb.attention(q, *cache, table, lens, cu_q, max_q)

    def near(out, want):
        # scores to 2^-20 of sums of 128 products of up to 8 x 8, weights to 2^-11, out to 2^-8 of itself
        assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * want.abs().amax(-1, keepdim=True) + 1e-3).all()
    qkv = torch.randn(n + 33, heads + 2 * kv_heads, dim, generator=gen, device="cuda").to(torch.bfloat16)
    places = torch.cat((torch.arange(n), torch.arange(33))).to(torch.int32).cuda()
    q, out = step(qkv, cu, n, torch.stack((places, places // 7), 1).contiguous())
    near(out, expected(q, news, news))
    one, where = torch.zeros(2, heads + 2 * kv_heads, dim, device="cuda", dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lens += 1
        step(one, None, None, where)
    torch.cuda.current_stream().wait_stream(side)
    lens -= 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, out = step(one, None, None, where)
    for i in range(1, 5):
        lens += 1
        one.copy_(torch.randn(one.shape, generator=gen, device="cuda"))
        where.copy_(torch.stack((lens, lens // 7), 1))
        graph.replay()
        near(out, expected(q, [m + i for m in news], [1, 1]))


def test_both_sides_of_the_binding_make_the_same_call(monkeypatch):
    class Nothing:
        attention = staticmethod(lambda *a: None)
    b = ref4.make_batch(45, [40, 90], [3, 3], 2, 64, 16)
    cache, table, lens, _ = b.device()
    q, lse = queries(46, 6, 4, 64).cuda(), torch.zeros(2, 6, 4, device="cuda")
    a = lb.attention(q, *cache, table, lens, window=33, lse=lse[0])
    need = lb.attention_workspace(q, *cache, table, lens)
    monkeypatch.setattr(decoder, "_hot", Nothing)
    c = lb.attention(q, *cache, table, lens, window=33, lse=lse[1], workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a, c) and torch.equal(lse[0], lse[1])
    with pytest.raises(lb.LowbitError):
        lb.attention(q, *cache, table, lens, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("n", [1, 3, 64])
def test_a_row_does_not_depend_on_the_others(n):
    """Other rows of the same sequence and heads with far larger scores, to the bit."""
    b = ref4.make_batch(47, [700], [n], 1, 128, 64)
    q = queries(48, n, 8, 128)
    few, _ = run(b, q)
    loud = q.clone()
    loud[:, ::2] *= 30
    got, _ = run(b, loud)
    assert np.array_equal(got[:, 1::2], few[:, 1::2]) and not np.array_equal(got[:, ::2], few[:, ::2])


def test_full_batch_of_few_and_many_rows():
    """Sequences times kv heads enough that 32 rows, and not 64, divide the two kernels; sequences on both sides of it."""
    news = [1, 8, 9, 16, 17, 2, 40, 0] * 2
    lens = [n + 37 * i for i, n in enumerate(news)]
    b = ref4.make_batch(49, lens, news, 4, 128, 32)
    check(b, queries(50, sum(news), 16, 128))
    b = ref4.make_batch(51, [60 + i for i in range(16)], [8] * 16, 4, 128, 64)
    check(b, queries(52, 128, 16, 128))


@pytest.mark.parametrize("n", [1, 30])
def test_table_far_wider_than_the_lengths(n):
    """What is planned by the table's width, more CTAs and a second launch, changes no result beyond rounding."""
    b = ref4.make_batch(53, [66, 300], [n, n], 2, 128, 64)
    b.table = np.concatenate([b.table, np.full((2, 2000), -1, np.int32)], 1)
    check(b, queries(54, 2 * n, 8, 128))


def test_lengths_below_nothing_and_past_the_table():
    b = ref4.make_batch(55, [64, 64], [3, 3], 1, 64, 16)
    cache, table, _, _ = b.device()
    q = queries(56, 6, 4, 64).cuda()
    lse = torch.zeros(6, 4, device="cuda")
    out = lb.attention(q, *cache, table, torch.tensor([-7, 64], dtype=torch.int32, device="cuda"), lse=lse)
    assert not out[:3].any() and torch.isneginf(lse[:3]).all() and out[3:].any()
    # past the table: counted as the table's 64 tokens
    past = lb.attention(q, *cache, table, torch.tensor([2 ** 31 - 1, 64], dtype=torch.int32, device="cuda"))
    whole = lb.attention(q, *cache, table, torch.tensor([64, 64], dtype=torch.int32, device="cuda"))
    assert torch.equal(past, whole)


def test_two_calls_at_once():
    """Decode, prompts and cache writes on two streams at the same time, each with its own outputs."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for i, (lens, n) in enumerate((([5000, 700], 1), ([900, 300], 90))):
        b = ref4.make_batch(57 + i, lens, [n, n], 2, 128, 64)
        cache, table, lens, _ = b.device()
        q = queries(59 + i, 2 * n, 8, 128).cuda()
        kv = queries(61 + i, 2 * n, 4, 128).cuda()
        work.append((q, kv, cache, table, lens, lb.attention(q, *cache, table, lens)))
    torch.cuda.synchronize()
    results = [[], []]
    for _ in range(20):
        for side, (q, kv, cache, table, lens, _), got in zip(sides, work, results):
            with torch.cuda.stream(side):
                got.append(lb.attention(q, *cache, table, lens))
                fresh = lb.empty_cache(cache[0].shape[0], 2, 128, 64, bits=4)
                lb.kv_append(q, kv[:, :2], kv[:, 2:], *fresh, table, lens)
                got.append(fresh[0])
    torch.cuda.synchronize()
    for got, (*_, want) in zip(results, work):
        assert all(torch.equal(x, want) for x in got[::2]) and all(torch.equal(x, got[1]) for x in got[3::2])


def test_two_graphs_with_one_workspace():
    """Replayed in turn, also after calls outside of them."""
    b = ref4.make_batch(63, [3000, 80], [2, 2], 2, 128, 64)
    cache, table, lens, _ = b.device()
    qs = [queries(64 + i, 4, 8, 128).cuda() for i in range(2)]
    ws = torch.empty(lb.attention_workspace(qs[0], *cache, table, lens), dtype=torch.uint8, device="cuda")
    want = [lb.attention(q, *cache, table, lens, workspace=ws) for q in qs]
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lb.attention(q, *cache, table, lens, workspace=ws))
        graphs.append(g)
    for _ in range(5):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            assert torch.equal(o, w)
        assert torch.equal(lb.attention(qs[0], *cache, table, lens, workspace=ws), want[0])
