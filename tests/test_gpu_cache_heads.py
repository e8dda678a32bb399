"""The write into the 8-bit cache with norms or positions where a CTA takes several heads one
after another, a cache's values where a thread takes several vectors, and the norms' last bit."""
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
import test_gpu_cache4 as whole  # noqa: E402


def odd(t):
    """Rows that start on odd elements."""
    wide = torch.zeros(t.shape[0], t.shape[1], t.shape[2] + 3, dtype=torch.bfloat16, device="cuda")
    wide[..., 3:] = t.cuda()
    return wide[..., 3:]


def older(b, cache):
    """Codes that were there before, of pages that new tokens share with them: moved to the page's new exponent, and how
    many (page, head) have moved."""
    moved = stayed = 0
    for codes, exps, before, was in ((cache[0], cache[2], b.k, b.k_exp), (cache[1], cache[3], b.v, b.v_exp)):
        codes, exps = codes.view(torch.uint8).cpu().numpy(), exps.cpu().numpy()
        for s, (n, m) in enumerate(zip(b.lens, b.news)):
            at = n - m
            if at % b.page == 0:
                continue
            page, held = b.table[s, at // b.page], slice(0, at % b.page)
            for h in range(codes.shape[1]):
                by = int(was[page, h]) - int(exps[page, h])
                assert by <= 0
                want = before[page, h, held] if by == 0 else ref.e4m3_round(ref.E4M3[before[page, h, held]] * 2.0 ** by)
                assert np.array_equal(ref.E4M3[codes[page, h, held]], ref.E4M3[want])
                moved, stayed = moved + (by < 0), stayed + (by == 0)
    return moved, stayed


# kv heads, values, tokens of a page, new tokens: heads of a CTA are as many as leave a few CTAs an SM.
# 3, 3 and 2 of 8; 2, 2 and 1 of 5; 4, 4 and 1 of 9; of pages of more tokens than a CTA holds at once 2 of 8 and 2 of 16.
@pytest.mark.parametrize("kv_heads,dim,page,new,form", [(8, 128, 16, 2000, f) for f in ("halves", "neighbours", "unaligned", "part", "none")] + [
    (5, 64, 16, 2001, "halves"), (5, 64, 16, 2001, "neighbours"), (9, 128, 16, 2300, "halves"),
    (8, 128, 128, 9701, "halves"), (16, 64, 256, 9700, "neighbours")])
def test_8_bits_several_heads_of_a_cta(kv_heads, dim, page, new, form):
    news, past = [new // 3, 1, new - new // 3 - 6, 5], [page // 2 + 1, 3, 0, 7]
    b = ref.make_batch(92, [n + o for n, o in zip(news, past)], news, kv_heads, dim, page, exps=(-6, 5))
    x = whole.inputs(93, new, kv_heads, kv_heads, dim)
    x[:, kv_heads:] *= torch.exp2(torch.arange(2 * kv_heads) % 4 * 3.0 - 6).to(torch.bfloat16)[:, None]      # pages' exponents grow for some heads
    rng = np.random.default_rng(94)
    turns = None if form == "none" else whole.turns_of(dim // 2 + 4 if form == "part" else dim)
    where = dict(positions=rng.integers(0, 3000, (new, 3)).astype(np.int32), axes=rng.integers(0, 3, len(turns)).astype(np.uint8)) if turns else {}
    norms = (whole.weight_of(95, dim, torch.float32), whole.weight_of(96, dim, torch.float32) if form != "part" else None)
    cache = whole.check8(b, x, kv_heads, turns, form == "neighbours", norms, split=odd if form == "unaligned" else None, **where)
    moved, stayed = older(b, cache)
    assert moved > 0 and stayed > 0


@pytest.mark.parametrize("dim,page,heads", [(128, 256, 1), (64, 16, 5)])
@pytest.mark.parametrize("bits", [4, 8])
def test_values_of_many_pages(bits, dim, page, heads):
    """More than 152 x 128 x 256 vectors of 8: a thread takes a second one; the last pages among what is compared."""
    pages = 152 * 128 * 256 * 8 // (heads * page * dim) + 7
    gen = torch.Generator(device="cuda").manual_seed(97)
    cache = lb.empty_cache(pages, heads, dim, page, bits=bits)
    for c in cache[:2]:
        c.view(torch.uint8).random_(0, 256, generator=gen)
    if bits == 4:
        for s in cache[2:]:
            s.view(torch.uint8).random_(0, 0x7C, generator=gen)
    else:
        for c, e in zip(cache[:2], cache[2:]):
            c.view(torch.uint8)[c.view(torch.uint8) & 0x7F == 0x7F] = 0
            e.random_(-64, 65, generator=gen)
    for got, codes, scales in zip(lb.cache_values(*cache), cache[:2], cache[2:]):
        for part in (slice(0, 3), slice(pages // 2, pages // 2 + 3), slice(pages - 9, pages)):
            if bits == 4:
                c = torch.stack((codes[part] & 15, codes[part] >> 4), -1).flatten(-2).float() - 8
                want = c * scales[part].float().repeat_interleave(32, -1)
            else:
                want = codes[part].float() * torch.exp2(scales[part].float())[..., None, None]
            assert torch.equal(got[part], want.to(torch.bfloat16))
