"""The write into a cache with head norms and positions of several axes, into the 4-bit cache
and the 8-bit one, on the GPU against plain 64-bit definitions (cache4_ref, decoder_ref).
Tolerances are derived beside the checks."""
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

# A value normed and rotated in fp32 is off by this of the magnitudes behind it: the sum of
# squares by 8 roundings (halved by the root), the mean, root, reciprocal and two products by one
# each; the angle by 2^-24 of half a turn, cosine and sine by 2 units, two products and a sum.
SLACK = 2.0 ** -20


def inputs(seed, T, heads, kv_heads, dim, size=1.0):
    rng = np.random.default_rng([seed, T, heads, dim])
    return ref.bf16(rng.standard_normal((T, heads + 2 * kv_heads, dim)) * size)


def turns_of(dim, base=10000.0):
    return lb.rotary_turns(dim, base).tolist()


def weight_of(seed, dim, dtype):
    return (1 + 0.5 * torch.randn(dim, generator=torch.Generator().manual_seed(seed))).to(dtype)


def slots(b):
    """(row of q, page, slot) of each new token that the cache holds, page and slot -1 for others."""
    page, slot = [], []
    for s, (n, m) in enumerate(zip(b.lens, b.news)):
        for pos in range(n - m, n):
            at = pos // b.page
            pg = b.table[s, at] if 0 <= pos and at < b.table.shape[1] else -1
            ok = 0 <= pg < b.k.shape[0]
            page.append(pg if ok else -1)
            slot.append(pos % b.page if ok else -1)
    return np.array(page, int), np.array(slot, int)


def expected(b, qkv, heads, turns, interleaved, factor, norms, eps, positions, axes):
    """(rows of q, k, v in fp64, how far fp32 may be from them)."""
    x, Hk = ref.f64(qkv), b.k.shape[1]
    pos = b.positions if positions is None else positions
    out = []
    for part, w in ((x[:, :heads], norms[0]), (x[:, heads:heads + Hk], norms[1])):
        y, mag = ref4.rotated(ref4.normed(part, None if w is None else ref.f64(w), eps), pos, turns, axes, interleaved, factor)
        out.append((y, mag * SLACK))
    out.append((x[:, heads + Hk:], np.zeros_like(x[:, heads + Hk:])))
    return out


def check_q(got, want, slack):
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    # one rounding to bf16: half a unit in the last of its 8 bits
    with np.errstate(invalid="ignore"):
        bound = 2.0 ** (np.frexp(np.abs(want) + slack)[1] - 9.0) + slack
        assert np.all((np.abs(got - want) <= bound)[~nan])


def call(b, qkv, heads, turns=None, interleaved=False, factor=1.0, norms=(None, None), eps=1e-6, positions=None, axes=None,
         split=None, cache=None, **kw):
    cache = cache or b.device()[0]
    _, table, lens, cu = b.device()
    dev = qkv.cuda() if split is None else split(qkv)
    q, k, v = dev.split([heads, b.k.shape[1], b.k.shape[1]], 1)
    t = None if turns is None else torch.tensor(turns, dtype=torch.int64, device="cuda")
    got = lb.kv_append(q, k, v, *cache, table, lens, cu_q=cu, max_q=max(b.news), turns=t, interleaved=interleaved, factor=factor,
                       q_norm=None if norms[0] is None else norms[0].cuda(), k_norm=None if norms[1] is None else norms[1].cuda(),
                       eps=eps, positions=None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda"),
                       axes=None if axes is None else torch.tensor(axes, dtype=torch.uint8, device="cuda"), **kw)
    return got, cache


def check(b, qkv, heads, turns=None, interleaved=False, factor=1.0, norms=(None, None), eps=1e-6, positions=None, axes=None, **kw):
    got, cache = call(b, qkv, heads, turns, interleaved, factor, norms, eps, positions, axes, **kw)
    rows = expected(b, qkv, heads, turns or [], interleaved, factor, norms, eps, positions, axes)
    check_q(ref.f64(got), *rows[0])
    page, slot = slots(b)
    held = page >= 0
    for (fresh, slack), codes, scales, before, scales_before in (
            (rows[1], cache[0], cache[2], b.k, b.k_scale), (rows[2], cache[1], cache[3], b.v, b.v_scale)):
        codes, scales = ref4.unpacked(codes.cpu().numpy()), scales.view(torch.uint8).cpu().numpy()
        want_codes, want_scales = before.copy(), scales_before.copy()
        want_codes[page[held], :, slot[held]] = 255
        want_scales[page[held], :, slot[held]] = 255
        touched = want_codes == 255
        assert np.array_equal(codes[~touched], want_codes[~touched])          # everything else is as it was
        c = codes[page[held], :, slot[held]].astype(np.float64) - 8           # [tokens, heads, dim]
        s = scales[page[held], :, slot[held]]
        x = fresh[held].reshape(*c.shape[:2], -1, ref4.GROUP)
        d = np.nan_to_num(slack[held].reshape(x.shape), nan=0.0, posinf=0.0)
        size = np.where(np.isfinite(x), np.abs(x), 0.0)
        nan = np.isnan(x).any(-1)
        assert np.array_equal(s[nan], np.full(nan.sum(), 0x7F))
        lo, hi = ref4.scale_byte(np.maximum(size - d, 0).max(-1)), ref4.scale_byte((size + d).max(-1))
        assert np.all(((lo <= s) & (s <= hi))[~nan])
        step = ref4.E5M2[np.where(nan, 4, s)][..., None]
        least, most = (np.clip(np.rint((x + sign * d) / step), -7, 7) for sign in (-1, 1))
        c = c.reshape(x.shape)
        assert np.all(((least <= c) & (c <= most))[~nan])
    return cache


BOTH = "bits", [4, 8]


# ---------------------------------------------------------------------------
# Into the 4-bit cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 32), (128, 128), (128, 96), (128, 64), (128, 10), (64, 2), (128, 0), (128, 120)])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_forms(norm, interleaved, dim, rotary):
    lens, news = [40, 3, 130, 65], [7, 3, 100, 1]
    b = ref4.make_batch(40, lens, news, 2, dim, 32)
    norms = (weight_of(1, dim, torch.bfloat16), weight_of(2, dim, torch.bfloat16)) if norm else (None, None)
    check(b, inputs(41, sum(news), 6, 2, dim), 6, turns_of(rotary) if rotary else None, interleaved, 1.1, norms)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("news", [[1, 1, 1, 1], [5, 0, 300, 2], [64, 64, 64, 64], [257, 1, 33, 600]])
def test_pages_and_lengths(page, news):
    lens = [n + e for n, e in zip(news, [0, 15, 31, 255])]
    b = ref4.make_batch(42, lens, news, 3, 64, page)
    check(b, inputs(43, sum(news), 3, 3, 64), 3, turns_of(64))


@pytest.mark.parametrize("heads,kv_heads,dim", [(32, 8, 128), (28, 4, 128), (16, 1, 128), (5, 5, 64), (7, 1, 64), (1, 1, 128)])
@pytest.mark.parametrize("n", [1, 40])
def test_heads(heads, kv_heads, dim, n):
    b = ref4.make_batch(44, [n + 3, n + 70], [n, n], kv_heads, dim, 64)
    check(b, inputs(45, 2 * n, heads, kv_heads, dim), heads, turns_of(dim), norms=(weight_of(3, dim, torch.float32),) * 2)


def test_more_tokens_than_fill_the_gpu():
    """Several tokens a CTA, and a last one with fewer."""
    n = 8 * 152 * 4 + 3
    b = ref4.make_batch(46, [n], [n], 1, 64, 256)
    check(b, inputs(47, n, 1, 1, 64), 1, turns_of(64), norms=(None, weight_of(4, 64, torch.bfloat16)))


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-6, 1e-3, 300.0, 1e5, 1e30])
def test_sizes(size):
    """Scales at both of their limits."""
    b = ref4.make_batch(48, [20], [6], 2, 128, 16)
    check(b, inputs(49, 6, 4, 2, 128, size), 4, turns_of(128))


def test_borders():
    """Values of v at the border between two codes, between two scales, and one unit beside them."""
    s = ref4.SCALES[40:60:3]
    rows = []
    for a in s:
        row = np.concatenate([(np.arange(15) - 7.0) * a, (np.arange(15) - 7.5) * a, [0.0, 7.5 * a]])
        rows.append(row)
        rows.append(row * (1 + 2.0 ** -7))                                    # amax past 7.5 s
        rows.append(np.concatenate([row[:31] * (1 - 2.0 ** -7), [7.5 * a]]))
    x = np.stack(rows + rows[:1])[:22].reshape(11, 1, 64)
    qkv = torch.cat((torch.zeros(11, 2, 64, dtype=torch.bfloat16), ref.bf16(x)), 1)
    b = ref4.make_batch(50, [11], [11], 1, 64, 16)
    cache = check(b, qkv, 1)
    want, scales = ref4.coded(ref.f64(qkv[:, 2]))
    assert np.array_equal(ref4.unpacked(cache[1].cpu().numpy())[b.table[0, 0], 0, :11], want)
    assert np.array_equal(cache[3].view(torch.uint8).cpu().numpy()[b.table[0, 0], 0, :11], scales)


def test_infinite_and_nan_values():
    b = ref4.make_batch(51, [20, 5], [3, 5], 1, 64, 16)
    x = inputs(52, 8, 1, 1, 64)
    x[1, 2, 5], x[3, 2, 9], x[4, 2, 1] = float("inf"), float("-inf"), float("nan")     # in v
    x[5, 1, 40], x[6, 1, 2], x[7, 0, 1] = float("nan"), float("inf"), float("nan")     # in k and q
    x[2, 2] = float("inf")
    cache = check(b, x, 1)
    k, v = lb.cache_values(*cache)
    assert torch.isnan(v[b.table[1, 0], 0, 1, :32]).all() and torch.isfinite(v[b.table[1, 0], 0, 1, 32:]).all()
    assert torch.isnan(k[b.table[1, 0], 0, 2, 32:]).all() and torch.isfinite(k[b.table[1, 0], 0, 3]).all()


def test_norms_of_infinite_nan_and_zero_rows():
    """x / inf = 0, inf / inf and NaN: what the formula gives, in that head alone; a row of zeros stays zeros."""
    b = ref4.make_batch(53, [8], [8], 2, 128, 16)
    x = inputs(54, 8, 2, 2, 128)
    x[1, 0, 5], x[2, 2, 9], x[3, 1, 100], x[4, 3, 1] = float("inf"), float("-inf"), float("nan"), float("nan")
    x[5, :4] = 0
    x[6, 2] = 3e38                                                            # squares past fp32: divided by infinity
    w = weight_of(5, 128, torch.float16)
    got, cache = call(b, x, 2, norms=(w, w))
    k, _ = lb.cache_values(*cache)
    page = b.table[0, 0]
    assert torch.isnan(got[1, 0, 5]) and not got[1, 0, :5].any() and not got[1, 0, 6:].any() and torch.isfinite(got[1, 1]).all()
    assert torch.isnan(got[3, 1]).all() and torch.isfinite(got[3, 0]).all()
    assert torch.isnan(k[page, 0, 2, :32]).all() and not k[page, 0, 2, 32:].any()
    assert torch.isnan(k[page, 1, 4]).all() and not k[page, :, 5].any() and not k[page, 0, 6].any()
    assert torch.isfinite(k[page, :, 7]).all() and torch.isfinite(got[7]).all()


@pytest.mark.parametrize("norms", [("q",), ("k",), ("q", "k")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_norms(norms, dtype, eps):
    b = ref4.make_batch(55, [33, 90], [5, 5], 2, 64, 32)
    w = tuple(weight_of(i, 64, dtype) if n in norms else None for i, n in enumerate("qk"))
    check(b, inputs(56, 10, 6, 2, 64, 0.3), 6, turns_of(64), norms=w, eps=eps)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [64, 40])
@pytest.mark.parametrize("axes", [1, 2, 3, 7])
def test_positions_of_several_axes(interleaved, rotary, axes):
    b = ref4.make_batch(57, [20, 80], [20, 9], 2, 64, 16)
    rng = np.random.default_rng([58, axes])
    positions = rng.integers(-50, 100_000, (29, axes)).astype(np.int32)
    positions[0], positions[1] = 2 ** 31 - 1, -2 ** 31
    which = rng.integers(0, axes, rotary // 2).astype(np.uint8)
    check(b, inputs(59, 29, 4, 2, 64), 4, turns_of(rotary), interleaved, 1.0, positions=positions, axes=which,
          norms=(weight_of(6, 64, torch.bfloat16), None))


def test_positions_without_axes_and_axes_past_the_last():
    b = ref4.make_batch(60, [20], [5], 1, 64, 16)
    x, turns = inputs(61, 5, 2, 1, 64), turns_of(64)
    check(b, x, 2, turns, positions=np.array([7, 0, -3, 12345, 7], np.int32))
    two = np.array([[1, 9], [2, 8], [3, 7], [4, 6], [5, 5]], np.int32)
    past = np.full(32, 200, np.uint8)                                         # counts as the last
    assert torch.equal(call(b, x, 2, turns, positions=two, axes=past)[0], call(b, x, 2, turns, positions=two[:, 1].copy())[0])


def test_strided_positions():
    b = ref4.make_batch(60, [20], [5], 1, 64, 16)
    x, turns = inputs(61, 5, 2, 1, 64).cuda(), lb.rotary_turns(64, device="cuda")
    wide = torch.arange(50, dtype=torch.int32, device="cuda").view(5, 10)
    axes = (torch.arange(32, device="cuda") % 3).to(torch.uint8)
    cache, table, lens, _ = b.device()
    q, k, v = x.split([2, 1, 1], 1)
    a = lb.kv_append(q, k, v, *cache, table, lens, turns=turns, positions=wide[:, 4:7], axes=axes)
    c = lb.kv_append(q, k, v, *cache, table, lens, turns=turns, positions=wide[:, 4:7].contiguous(), axes=axes)
    d = lb.kv_append(q, k, v, *cache, table, lens, turns=turns, positions=wide[:, 4])
    e = lb.kv_append(q, k, v, *cache, table, lens, turns=turns, positions=wide[:, 4].contiguous())
    assert torch.equal(a, c) and torch.equal(d, e) and not torch.equal(a, d)


def test_outside_the_cache_is_left_out():
    """New tokens before position 0, past the page table, or on a page that is not in the cache."""
    b = ref4.make_batch(62, [3, 40, 33], [10, 40, 2], 2, 64, 16)
    b.table[1, 1] = -5
    b.table[2, 2] = b.k.shape[0] + 7
    check(b, inputs(63, 52, 2, 2, 64), 2, turns_of(64))
    b = ref4.make_batch(64, [16], [16], 1, 64, 16)
    b.lens = [24]                                                             # 8 past the table
    check(b, inputs(65, 16, 2, 1, 64), 2, turns_of(64))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [64, 10])
@pytest.mark.parametrize("norm", [False, True])
def test_in_place_and_unaligned(norm, interleaved, rotary):
    b = ref4.make_batch(66, [40, 80], [40, 5], 2, 64, 64)
    x = inputs(67, 45, 4, 2, 64)
    norms = (weight_of(7, 64, torch.float32), weight_of(8, 64, torch.float32)) if norm else (None, None)
    dev = x.cuda()
    want, cache = call(b, x, 4, turns_of(rotary), interleaved, norms=norms)
    got, again = call(b, x, 4, turns_of(rotary), interleaved, norms=norms, split=lambda t: dev, out=dev[:, :4])
    assert torch.equal(got, want) and got.data_ptr() == dev.data_ptr()
    assert all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip(cache, again))

    def odd(t):                                        # rows that start on odd elements
        wide = torch.zeros(t.shape[0], t.shape[1], 67, dtype=torch.bfloat16, device="cuda")
        wide[..., 3:] = t.cuda()
        return wide[..., 3:]
    check(b, x, 4, turns_of(rotary), interleaved, norms=norms, split=odd)


def test_more_new_tokens_than_max_q_and_rows_behind_the_last_sequence():
    """Tokens past max_q, and rows of no sequence, are left as they were; those before keep their positions."""
    b = ref4.make_batch(68, [30, 40], [6, 9], 2, 64, 16)
    x, turns = inputs(69, 20, 4, 2, 64).cuda(), lb.rotary_turns(64, device="cuda")
    cache, table, lens, _ = b.device()
    start = [c.view(torch.uint8).clone() for c in cache]
    cu = torch.tensor([0, 6, 15], dtype=torch.int32, device="cuda")
    q, k, v = x.split([4, 2, 2], 1)
    whole = lb.kv_append(q, k, v, *cache, table, lens, cu_q=cu, max_q=9, turns=turns, out=torch.full_like(q, 7.0))
    full = [c.view(torch.uint8).clone() for c in cache]
    assert (whole[15:] == 7).all() and not (whole[:15] == 7).all(-1).any()
    for c, s in zip(cache, start):
        c.view(torch.uint8).copy_(s)
    part = lb.kv_append(q, k, v, *cache, table, lens, cu_q=cu, max_q=4, turns=turns, out=torch.full_like(q, 7.0))
    live = torch.zeros(20, dtype=torch.bool, device="cuda")
    live[:4] = live[6:10] = True
    assert torch.equal(part[live], whole[live]) and (part[~live] == 7).all()
    for c, s, f in zip(cache, start, full):
        c = c.view(torch.uint8)
        for seq, (n, m) in enumerate(zip(b.lens, b.news)):
            for i in range(m):
                at = int(b.table[seq, (n - m + i) // 16]), slice(None), (n - m + i) % 16
                assert torch.equal(c[at], f[at] if i < 4 else s[at])


def test_tokens_one_at_a_time_give_the_same_cache():
    x = inputs(70, 50, 2, 2, 64).cuda()
    turns, w = lb.rotary_turns(64, device="cuda"), weight_of(9, 64, torch.bfloat16).cuda()
    table = torch.arange(2, dtype=torch.int32, device="cuda")[None]

    def fill(cuts):
        cache = lb.empty_cache(2, 2, 64, 32, bits=4)
        for a, e in zip(cuts[:-1], cuts[1:]):
            q, k, v = x[a:e].split([2, 2, 2], 1)
            lb.kv_append(q, k, v, *cache, table, torch.tensor([e], dtype=torch.int32, device="cuda"), turns=turns, k_norm=w)
        return [c.view(torch.uint8) for c in cache]
    assert all(torch.equal(a, b) for a, b in zip(fill([0, 50]), fill(list(range(51)))))


def test_cache_beyond_32_bit_offsets():
    """Pages past 2^32 bytes from the cache's start."""
    pages, page, dim = (1 << 32) // (64 * 64) + 3, 64, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    cache = lb.empty_cache(pages, 1, dim, page, bits=4)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    x = inputs(71, 100, 1, 1, dim).cuda()
    q, k, v = x.split([1, 1, 1], 1)
    lb.kv_append(q, k, v, *cache, table, torch.tensor([100], dtype=torch.int32, device="cuda"))
    for c, s, fresh in ((cache[0], cache[2], k), (cache[1], cache[3], v)):
        want, scales = ref4.coded(ref.f64(fresh[:, 0]))
        got = torch.cat((c[pages - 1, 0], c[pages - 2, 0, :36])).cpu().numpy()
        assert np.array_equal(ref4.unpacked(got), want)
        got = torch.cat((s.view(torch.uint8)[pages - 1, 0], s.view(torch.uint8)[pages - 2, 0, :36])).cpu().numpy()
        assert np.array_equal(got, scales)
        assert not c[:pages - 2].any() and not c[pages - 2, 0, 36:].any()


def test_captured_and_on_another_stream():
    b = ref4.make_batch(72, [30, 60], [1, 1], 2, 128, 16)
    x = inputs(73, 2, 8, 2, 128).cuda()
    q, k, v = x.split([8, 2, 2], 1)
    turns, w = lb.rotary_turns(128, device="cuda"), weight_of(10, 128, torch.bfloat16).cuda()
    cache, table, lens, _ = b.device()
    positions = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    axes = (torch.arange(64, device="cuda") // 32).to(torch.uint8)

    def step():
        return lb.kv_append(q, k, v, *cache, table, lens, turns=turns, q_norm=w, k_norm=w, positions=positions, axes=axes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    graph.replay()
    assert torch.equal(o, first)
    positions += torch.tensor([[5, 9], [400, 70]], dtype=torch.int32, device="cuda")
    lens -= 7
    graph.replay()
    got, held = o.clone(), [c.view(torch.uint8).clone() for c in cache]
    assert torch.equal(step(), got) and not torch.equal(got, first)
    assert all(torch.equal(c.view(torch.uint8), h) for c, h in zip(cache, held))


# ---------------------------------------------------------------------------
# Into the 8-bit cache
# ---------------------------------------------------------------------------

def check8(b, qkv, heads, turns, interleaved, norms, eps=1e-6, positions=None, axes=None, split=None):
    got, cache = call(b, qkv, heads, turns, interleaved, 1.0, norms, eps, positions, axes, split=split)
    class Places:                                       # what `expected` and `slots` look at
        k, table, page, lens, news = b.k, b.table, b.page, b.lens, b.news
        positions = np.concatenate([n - m + np.arange(m) for n, m in zip(b.lens, b.news)]).astype(np.int64)
    rows = expected(Places, qkv, heads, turns or [], interleaved, 1.0, norms, eps, positions, axes)
    check_q(ref.f64(got), *rows[0])
    page, slot = slots(Places)
    for (fresh, slack), codes, exps, before in ((rows[1], cache[0], cache[2], b.k_exp), (rows[2], cache[1], cache[3], b.v_exp)):
        codes, exps = codes.view(torch.uint8).cpu().numpy(), exps.cpu().numpy()
        for pg in set(page[page >= 0].tolist()):
            new = page == pg
            shared = slot[new].min() > 0                # the page holds older tokens
            for h in range(b.k.shape[1]):
                size, d = np.abs(fresh[new, h]), slack[new, h]
                lo, hi = ref.page_exponent((size - d).max()), ref.page_exponent((size + d).max())
                e, was = int(exps[pg, h]), int(before[pg, h])
                assert (max(lo, was) <= e <= max(hi, was)) if shared else lo <= e <= hi
                want = np.clip(fresh[new, h] * 2.0 ** -e, -448, 448)
                val = ref.E4M3[codes[pg, h, slot[new]]]
                near = np.abs(ref.E4M3[ref.e4m3_round(want)] - want)
                assert np.all(np.abs(val - want) <= near + 2 * d * 2.0 ** -e + 1e-300)
    return cache


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (128, 128), (128, 64), (128, 10), (64, 0)])
@pytest.mark.parametrize("news", [[1, 1, 1], [7, 0, 100], [300, 64, 1]])
def test_8_bits_norms_and_axes(interleaved, dim, rotary, news):
    lens = [n + e for n, e in zip(news, [33, 15, 255])]
    b = ref.make_batch(74, lens, news, 2, dim, 32)
    rng = np.random.default_rng([75, sum(news)])
    T = sum(news)
    norms = (weight_of(11, dim, torch.bfloat16), weight_of(12, dim, torch.bfloat16))
    positions, axes = rng.integers(0, 5000, (T, 3)).astype(np.int32), rng.integers(0, 3, rotary // 2).astype(np.uint8)
    x = inputs(76, T, 6, 2, dim)
    if rotary:
        check8(b, x, 6, turns_of(rotary), interleaved, norms, positions=positions, axes=axes)
        check8(b, x, 6, turns_of(rotary), interleaved, (None, None), positions=positions[:, 0].copy())
    check8(b, x, 6, turns_of(rotary) if rotary else None, interleaved, (norms[0], None))
    check8(b, x, 6, turns_of(rotary) if rotary else None, interleaved, (None, norms[1]), eps=0.3)


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("rotary", [64, 6])
def test_8_bits_unaligned_rows_and_large_pages(page, rotary):
    """Rows that start on odd elements; pages of more tokens than a CTA holds at once."""
    def odd(t):
        wide = torch.zeros(t.shape[0], t.shape[1], 67, dtype=torch.bfloat16, device="cuda")
        wide[..., 3:] = t.cuda()
        return wide[..., 3:]
    b = ref.make_batch(77, [300, 257], [300, 200], 2, 64, page)
    norms = (weight_of(13, 64, torch.float32), weight_of(14, 64, torch.float32))
    x = inputs(78, 500, 4, 2, 64)
    check8(b, x, 4, turns_of(rotary), False, norms)
    check8(b, x, 4, turns_of(rotary), False, norms, split=odd)


def test_8_bits_positions_of_the_places_change_nothing():
    b = ref.make_batch(79, [50, 20], [9, 9], 2, 128, 16)
    x, turns = inputs(80, 18, 4, 2, 128), turns_of(128)
    plain, cache = call(b, x, 4, turns)
    places = np.concatenate([n - 9 + np.arange(9) for n in b.lens]).astype(np.int32)
    ones = torch.ones(128)
    given, same = call(b, x, 4, turns, positions=places)
    assert torch.equal(plain, given) and all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip(cache, same))
    assert not torch.equal(plain, call(b, x, 4, turns, norms=(ones, ones))[0])


# ---------------------------------------------------------------------------
# The values of a cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 256])
def test_values_of_4_bits(dim, page):
    """Any codes and scales, negative and subnormal ones among them."""
    b = ref4.make_batch(81, [40], [1], 3, dim, page, spare=5)
    rng = np.random.default_rng(82)
    b.k_scale[:] = rng.integers(0, 256, b.k_scale.shape)
    k, v = lb.cache_values(*b.cache())
    for got, codes, scales in ((k, b.k, b.k_scale), (v, b.v, b.v_scale)):
        s = np.repeat(ref4.E5M2[scales], 32, -1)
        with np.errstate(invalid="ignore"):
            assert np.array_equal(ref.f64(got), (codes.astype(np.float64) - 8) * s, equal_nan=True)


@pytest.mark.parametrize("dim", [64, 128])
def test_values_of_8_bits(dim):
    b = ref.make_batch(83, [40], [1], 3, dim, 32, spare=3)
    b.k_exp[:] = np.random.default_rng(84).integers(-64, 65, b.k_exp.shape)
    cache = b.device()[0]
    out = tuple(torch.empty(*b.k.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = lb.cache_values(*cache, out=out)
    assert k.data_ptr() == out[0].data_ptr() and v.data_ptr() == out[1].data_ptr()
    for got, codes, exps in ((k, b.k, b.k_exp), (v, b.v, b.v_exp)):
        assert np.array_equal(ref.f64(got), ref.E4M3[codes] * 2.0 ** exps[..., None, None].astype(float), equal_nan=True)


def test_values_of_strided_caches_and_of_none():
    b = ref4.make_batch(85, [70], [1], 2, 128, 16)
    k, v, ks, vs = b.cache()
    wide = torch.zeros(k.shape[0], 5, 16, 64, dtype=torch.uint8, device="cuda")
    wide[:, :2], wide[:, 3:] = k, v
    scales = torch.zeros(k.shape[0], 4, 16, 4, dtype=torch.uint8, device="cuda")
    scales[:, :2], scales[:, 2:] = ks.view(torch.uint8), vs.view(torch.uint8)
    a = lb.cache_values(k, v, ks, vs)
    c = lb.cache_values(wide[:, :2], wide[:, 3:], scales[:, :2], scales[:, 2:])
    assert all(torch.equal(x.nan_to_num(7), y.nan_to_num(7)) for x, y in zip(a, c))
    assert [t.shape for t in lb.cache_values(*lb.empty_cache(0, 2, 128, 16, bits=4))] == [(0, 2, 16, 128)] * 2


# ---------------------------------------------------------------------------
# Refusals, and the two sides of the binding
# ---------------------------------------------------------------------------

def arguments(bits=4):
    x = inputs(86, 6, 4, 2, 64).cuda()
    q, k, v = x.split([4, 2, 2], 1)
    cache = lb.empty_cache(9, 2, 64, 16, bits=bits)
    return dict(q=q, k=k, v=v, k_cache=cache[0], v_cache=cache[1], k_exp=cache[2], v_exp=cache[3],
                page_table=torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3),
                lens=torch.tensor([5, 40, 17], dtype=torch.int32, device="cuda"), cu_q=None, max_q=None,
                turns=lb.rotary_turns(64, device="cuda"), interleaved=False, factor=1.0, out=None,
                q_norm=torch.ones(64, device="cuda"), k_norm=torch.ones(64, device="cuda") * 2, eps=1e-5,
                positions=torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2),
                axes=(torch.arange(32, device="cuda") % 2).to(torch.uint8))


def apart(t):
    return torch.stack((t, t), -1).flatten(-2)[..., ::2]


BAD = [
    ("k_cache", lambda t: t.view(torch.int8)), ("k_cache", lambda t: t.view(torch.float8_e4m3fn)), ("k_cache", lambda t: t.cpu()),
    ("k_cache", lambda t: t[..., :16]), ("k_cache", lambda t: t[:8]), ("v_cache", lambda t: t[:, :1]), ("v_cache", None),
    ("k_cache", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)),
    ("k_exp", lambda t: t.view(torch.float8_e4m3fn)), ("k_exp", lambda t: t[:, :, :8]), ("k_exp", lambda t: t[..., :1]), ("k_exp", lambda t: t.cpu()),
    ("k_exp", lambda t: t[:, :, 0]), ("v_exp", lambda t: t[:5]), ("v_exp", lambda t: t[:, :, 0, 0]), ("v_exp", None),
    ("v_exp", lambda t: t.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2)),
    ("q_norm", lambda t: t[:63]), ("q_norm", lambda t: t.double()), ("q_norm", lambda t: t.cpu()), ("q_norm", apart), ("q_norm", 1.0),
    ("q_norm", lambda t: t.half()), ("k_norm", lambda t: t[None]), ("k_norm", lambda t: t.to(torch.bfloat16)), ("eps", "x"), ("eps", None),
    ("positions", lambda t: t.long()), ("positions", lambda t: t[:5]), ("positions", lambda t: t.cpu()), ("positions", lambda t: t[..., None]),
    ("positions", apart), ("positions", lambda t: t[:, :0]), ("positions", None), ("positions", [1, 2]),
    ("axes", lambda t: t[:31]), ("axes", lambda t: t.int()), ("axes", apart), ("axes", lambda t: t.cpu()), ("axes", None)]


@pytest.mark.parametrize("name,change", BAD, ids=[f"{n}-{i}" for i, (n, _) in enumerate(BAD)])
def test_refused_with_a_reason(name, change):
    args = arguments()
    args[name] = change(args[name]) if callable(change) else change
    before = {n: t.clone() for n, t in args.items() if isinstance(t, torch.Tensor)}
    assert decoder._load().kv_append(*args.values()) is None
    with pytest.raises(ValueError) as why:
        lb.kv_append(**args)
    assert str(why.value) and not isinstance(why.value, lb.LowbitError)
    for n, t in before.items():
        assert torch.equal(args[n].contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)), n


@pytest.mark.parametrize("change", [dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                    dict(turns=lb.rotary_turns(128, device="cuda"), axes=torch.zeros(64, dtype=torch.uint8, device="cuda"))])
@pytest.mark.parametrize(*BOTH)
def test_refused_by_the_library(bits, change):
    with pytest.raises(lb.LowbitError):
        lb.kv_append(**(arguments(bits) | change))


@pytest.mark.parametrize("change", [
    {}, dict(q_norm=None), dict(k_norm=None, positions=None, axes=None), dict(q_norm=None, k_norm=None, axes=None,
                                                                              positions=torch.arange(6, dtype=torch.int32, device="cuda")),
    dict(turns=None, axes=torch.zeros(0, dtype=torch.uint8, device="cuda"))])
@pytest.mark.parametrize(*BOTH)
def test_both_sides_of_the_binding_make_the_same_call(bits, change, monkeypatch):
    class Nothing:
        kv_append = cache_values = staticmethod(lambda *a: None)
    results = []
    for stub in (False, True):
        args = arguments(bits) | change
        cache = [args[n] for n in ("k_cache", "v_cache", "k_exp", "v_exp")]
        if stub:
            monkeypatch.setattr(decoder, "_hot", Nothing)
        results.append([lb.kv_append(**args), *(c.view(torch.uint8) for c in cache), *lb.cache_values(*cache)])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("out", [(torch.empty(9, 2, 16, 64), None), (None, torch.empty(9, 2, 16, 32, dtype=torch.bfloat16)),
                                 (torch.empty(9, 2, 16, 128, dtype=torch.bfloat16)[..., ::2], None), (5, None)])
def test_values_refused(out):
    out = tuple(t.cuda() if isinstance(t, torch.Tensor) else t for t in out)
    if isinstance(out[0], torch.Tensor) and out[0].dtype == torch.bfloat16:
        out = (apart(out[0].contiguous()), None)
    with pytest.raises(ValueError):
        lb.cache_values(*lb.empty_cache(9, 2, 64, 16, bits=4), out=out)


@pytest.mark.parametrize(*BOTH)
def test_empty_calls(bits):
    args = arguments(bits)
    for n in ("q", "k", "v", "positions"):
        args[n] = args[n][:0]
    assert lb.kv_append(**args).shape == (0, 4, 64)
    assert not any(args[n].view(torch.uint8).any() for n in ("k_cache", "v_cache", "k_exp", "v_exp"))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norms_to_the_bit(dim, eps):
    """Norms alone, as fp32 operations one by one: squares added in pairs, root and reciprocal rounded to nearest."""
    T = 20000
    gen = torch.Generator(device="cuda").manual_seed(87)
    x = torch.randn(T, 4, dim, generator=gen, device="cuda") * torch.exp(torch.randn(T, 4, 1, generator=gen, device="cuda") * 8)
    x, w = x.to(torch.bfloat16), torch.randn(dim, generator=gen, device="cuda")
    cache, pages = lb.empty_cache(-(-T // 64), 1, dim, 64, bits=4), torch.arange(-(-T // 64), dtype=torch.int32, device="cuda")[None]
    q, k, v = x.split([2, 1, 1], 1)
    out = lb.kv_append(q, k, v, *cache, pages, torch.tensor([T], dtype=torch.int32, device="cuda"), q_norm=w, eps=eps)
    s = q.float() * q.float()
    while s.shape[-1] > 1:
        s = s[..., 0::2] + s[..., 1::2]
    want = q.float() * torch.reciprocal(torch.sqrt(s * (1.0 / dim) + eps)) * w
    assert torch.equal(out, want.to(torch.bfloat16))
