"""Head norms on the way into a cache to the bit: codes and scales are those of fp32 operations
rounded to nearest one by one, where keys are not turned."""
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

F = np.float32


def root(x, eps):
    """fp32 [..., dim] -> [..., 1]: squares added in pairs, mean, root and reciprocal, each rounded to nearest."""
    with np.errstate(over="ignore", divide="ignore"):
        s = x * x
        while s.shape[-1] > 1:
            s = s[..., 0::2] + s[..., 1::2]
        return F(1) / np.sqrt(s * F(1.0 / x.shape[-1]) + F(eps))


def append(x, weight, eps, bits, page=64):
    """x bf16 [tokens, heads, dim] through the norm into a cache of its own: its tensors, pages in order."""
    T, heads, dim = x.shape
    pages = -(-T // page)
    cache = lb.empty_cache(pages, heads, dim, page, bits=bits)
    k = x.cuda()
    lb.kv_append(k, k, torch.zeros_like(k), *cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                 torch.tensor([T], dtype=torch.int32, device="cuda"), k_norm=weight.cuda(), eps=eps)
    return cache


def tokens(t, T):
    """[pages, heads, page, n] -> [T, heads, n]."""
    t = t.view(torch.uint8).cpu().numpy().swapaxes(1, 2)
    return t.reshape(-1, *t.shape[2:])[:T]


def check4(x, weight, eps):
    y = x.float().numpy()
    y = (y * root(y, eps)) * weight.numpy()
    cache = append(x, weight, eps, 4)
    want, scales = ref4.coded(y.astype(np.float64))
    assert np.array_equal(tokens(cache[2], len(x)), scales)
    assert np.array_equal(ref4.unpacked(tokens(cache[0], len(x))), want)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("four", [-10, 0, 9])
@pytest.mark.parametrize("bits", [0x3FBDEC0D, 0x3F9FB52F, 0x3F7FFFFE, 0x3F7FFFFF, 0x40000000, 0x3F800001])
def test_roots_that_are_hard_to_round(bits, four, dim):
    """A mean square of this float (all of it eps), and weights that bring values to the borders between codes: what
    is a unit beside falls to the other code.  The first two roots' reciprocals lie next to the middle of two floats, the
    next two roots are mantissas of ones."""
    eps = np.array(bits, np.uint32).view(F) * F(4.0 ** four)
    x = F(2.0 ** -60)
    by = x * (F(1) / np.sqrt(eps))
    weights = []
    for border in np.arange(0.5, 7.0):
        w = F(border / by)
        near = (w.view(np.uint32) + np.arange(-4, 5)).astype(np.uint32).view(F)
        weights += [n for n in near if by * n == F(border)][:1]
    assert len(weights) >= 3
    weight = np.resize(np.array(weights, F), dim) * np.resize(F([1, 1, -1]), dim)
    weight[::32] = F(7 / by)                                                  # the groups' largest: a scale of 1
    check4(torch.full((3, 2, dim), float(x)).to(torch.bfloat16), torch.from_numpy(weight), float(eps))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_codes_of_4_bits(dim, eps):
    gen = torch.Generator().manual_seed(105)
    x = torch.randn(20000, 2, dim, generator=gen) * torch.exp(torch.randn(20000, 2, 1, generator=gen) * 8)
    check4(x.to(torch.bfloat16), torch.randn(dim, generator=gen), eps)


@pytest.mark.parametrize("dim", [64, 128])
def test_codes_of_8_bits(dim):
    """Pages' exponents too; single tokens' kernel and the prompts'."""
    gen = torch.Generator().manual_seed(106)
    for T in (3, 12800):
        x = (torch.randn(T, 2, dim, generator=gen) * torch.exp(torch.randn(T, 2, 1, generator=gen) * 3)).to(torch.bfloat16)
        weight = torch.randn(dim, generator=gen)
        y = x.float().numpy()
        y = ((y * root(y, 1e-6)) * weight.numpy()).astype(np.float64)
        cache = append(x, weight, 1e-6, 8)
        exps = cache[2].cpu().numpy()
        for page in range(-(-T // 64)):
            for h in range(2):
                assert exps[page, h] == ref.page_exponent(np.abs(y[page * 64:page * 64 + 64, h]).max())
        e = np.repeat(exps, 64, 0)[:T].astype(float)
        assert np.array_equal(tokens(cache[0], T), ref.e4m3_round(y * 2.0 ** -e[..., None]))
