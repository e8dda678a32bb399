"""Host side of the decoder operators (no GPU needed): refusals of the C ABI and of the
binding, frequencies, and the tests' own definitions checked against themselves."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import bit_groupwise_weight_gb300 as lb
import decoder_ref as ref
from bit_groupwise_weight_gb300 import build as lbuild
from bit_groupwise_weight_gb300 import decoder

EINVAL = 1


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return lb.abi()


def packed(pack, names, values):
    assert set(values) <= set(names), set(values) - set(names)
    return pack(*(values[n] or 0 for n in names))


def descriptor(what, values):
    pack, names = {
        "cache": (decoder._CACHE, "k v k_exp v_exp page_stride head_stride pages kv_heads head_dim page"),
        "seqs": (decoder._SEQUENCES, "page_table lens cu_q table_stride width batch tokens max_q"),
        "append": (decoder._KV_APPEND, "q k v q_out q_token q_head k_token k_head v_token v_head o_token o_head turns factor "
                                       "heads rotary_dim interleaved"),
        "attention": (decoder._ATTENTION, "q out lse q_token q_head o_token o_head lse_token workspace workspace_bytes scale "
                                          "heads window"),
        "sample": (decoder._SAMPLE, "logits u temperature top_p min_p top_k token logprob row_stride temperature_all "
                                    "top_p_all min_p_all top_k_all rows vocab dtype"),
    }[what]
    return packed(pack, names.split(), values)


# Addresses that are never touched: every call below is rejected before CUDA, or empty.
CACHE = dict(k=0x10000, v=0x20000, k_exp=0x30000, v_exp=0x31000, page_stride=2 * 64 * 128, head_stride=64 * 128, pages=9,
             kv_heads=2, head_dim=128, page=64)
SEQS = dict(page_table=0x40000, lens=0x41000, cu_q=None, table_stride=4, width=4, batch=3, tokens=6, max_q=0)
APPEND = dict(q=0x50000, k=0x60000, v=0x70000, q_out=0x80000, q_token=1024, q_head=128, k_token=256, k_head=128,
              v_token=256, v_head=128, o_token=1024, o_head=128, turns=0x90000, factor=1.0, heads=8, rotary_dim=128,
              interleaved=0)
ATTN = dict(q=0x50000, out=0x80000, lse=None, q_token=1024, q_head=128, o_token=1024, o_head=128, lse_token=8,
            workspace=0xa0000, workspace_bytes=1 << 40, scale=0.1, heads=8, window=0)
SAMPLE = dict(logits=0x50000, u=0x60000, temperature=None, top_p=None, min_p=None, top_k=None, token=0x70000,
              logprob=None, row_stride=1000, temperature_all=1.0, top_p_all=1.0, min_p_all=0.0, top_k_all=0, rows=2,
              vocab=1000, dtype=1)


def call(lib, what, args, cache=None, seqs=None):
    cache, seqs = descriptor("cache", CACHE | (cache or {})), descriptor("seqs", SEQS | (seqs or {}))
    if what == "append":
        return lib.lowbit_kv_append(descriptor(what, APPEND | args), cache, seqs, None)
    if what == "attention":
        return lib.lowbit_attention(descriptor(what, ATTN | args), cache, seqs, None)
    return lib.lowbit_sample(descriptor(what, SAMPLE | args), None)


@pytest.mark.parametrize("what", ["append", "attention"])
@pytest.mark.parametrize("cache", [
    dict(k=None), dict(v=None), dict(k_exp=None), dict(v_exp=None), dict(k=0x10008), dict(v=0x20004), dict(pages=0),
    dict(pages=-1), dict(kv_heads=0), dict(kv_heads=3), dict(head_dim=96), dict(head_dim=256), dict(page=8), dict(page=48),
    dict(page=512), dict(head_stride=64 * 128 - 16), dict(page_stride=100), dict(head_stride=64 * 128 + 8),
    dict(page_stride=1 << 40)])
def test_caches_that_are_refused(lib, what, cache):
    assert call(lib, what, {}, cache=cache) == EINVAL


@pytest.mark.parametrize("what", ["append", "attention"])
@pytest.mark.parametrize("seqs", [
    dict(page_table=None), dict(lens=None), dict(page_table=0x40002), dict(lens=0x41001), dict(width=0), dict(width=-1),
    dict(table_stride=3), dict(batch=-1), dict(tokens=-1), dict(tokens=7), dict(cu_q=0x42000, max_q=0),
    dict(cu_q=0x42002, max_q=2), dict(tokens=3 << 28), dict(width=1 << 28, table_stride=1 << 28)])
def test_sequences_that_are_refused(lib, what, seqs):
    assert call(lib, what, {}, seqs=seqs) == EINVAL


@pytest.mark.parametrize("args", [
    dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(q=0x50001), dict(turns=None), dict(turns=0x90004),
    dict(rotary_dim=-2), dict(rotary_dim=130), dict(rotary_dim=7), dict(heads=0), dict(heads=7)])
def test_appends_that_are_refused(lib, args):
    assert call(lib, "append", args) == EINVAL


@pytest.mark.parametrize("args", [
    dict(q=None), dict(out=None), dict(q=0x50004), dict(out=0x80002), dict(lse=0xb0002), dict(q_token=1022), dict(q_head=2),
    dict(o_token=1), dict(o_head=127), dict(workspace=None), dict(workspace=0xa0008), dict(workspace_bytes=100),
    dict(scale=math.nan), dict(scale=math.inf), dict(window=-1), dict(heads=0), dict(heads=9)])
def test_attentions_that_are_refused(lib, args):
    assert call(lib, "attention", args) == EINVAL


@pytest.mark.parametrize("args", [
    dict(logits=None), dict(u=None), dict(token=None), dict(logits=0x50001), dict(dtype=0, logits=0x50002), dict(u=0x60002),
    dict(token=0x70004), dict(logprob=0x70002), dict(temperature=0x70002), dict(top_p=1), dict(min_p=2), dict(top_k=3),
    dict(rows=-1), dict(vocab=0), dict(vocab=-5), dict(vocab=(1 << 19) + 1), dict(dtype=3), dict(dtype=-1)])
def test_samples_that_are_refused(lib, args):
    assert call(lib, "sample", args) == EINVAL


def test_null_descriptors_are_refused(lib):
    cache, seqs = descriptor("cache", CACHE), descriptor("seqs", SEQS)
    for fn, args in ((lib.lowbit_kv_append, descriptor("append", APPEND)), (lib.lowbit_attention, descriptor("attention", ATTN))):
        assert fn(None, cache, seqs, None) == EINVAL
        assert fn(args, None, seqs, None) == EINVAL
        assert fn(args, cache, None, None) == EINVAL
    assert lib.lowbit_sample(None, None) == EINVAL
    assert lib.lowbit_attention_workspace(8, None, seqs) == 0


@pytest.mark.parametrize("seqs", [dict(tokens=0), dict(batch=0), dict(batch=0, tokens=0)])
def test_empty_calls_do_nothing(lib, seqs):
    nothing = dict(page_table=None, lens=None)
    no_cache = dict(k=None, v=None, k_exp=None, v_exp=None, pages=0)
    assert call(lib, "append", dict(q=None, k=None, v=None, q_out=None, turns=None, rotary_dim=0), no_cache, seqs | nothing) == 0
    assert call(lib, "attention", dict(q=None, out=None, workspace=None, workspace_bytes=0), no_cache, seqs | nothing) == 0
    assert call(lib, "sample", dict(rows=0, logits=None, u=None, token=None)) == 0


def test_workspace_is_enough_for_what_the_call_asks(lib):
    need = lib.lowbit_attention_workspace(8, descriptor("cache", CACHE), descriptor("seqs", SEQS))
    assert need > 0
    assert call(lib, "attention", dict(workspace_bytes=need - 1)) == EINVAL


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------

def test_binding_wants_cuda_tensors():
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    cache = lb.empty_cache(3, 2, 64, 16, device="cpu")
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lb.kv_append(q, kv, kv, *cache, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        lb.attention(q, *cache, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        lb.sample(torch.zeros(2, 10), torch.zeros(2))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        lb.sample(torch.zeros(2, 10, dtype=torch.float64), torch.zeros(2))
    with pytest.raises(ValueError, match="3 dimensions"):
        lb.attention(q[0], *cache, table, lens)


def test_empty_cache_shapes():
    k, v, ke, ve = lb.empty_cache(5, 3, 128, 32, device="cpu")
    assert k.shape == v.shape == (5, 3, 32, 128) and k.dtype == v.dtype == torch.float8_e4m3fn
    assert ke.shape == ve.shape == (5, 3) and ke.dtype == torch.int8


def test_rotary_turns_against_the_definition():
    for dim, base in ((64, 10000.0), (128, 500000.0), (10, 1e6)):
        t = lb.rotary_turns(dim, base)
        assert t.dtype == torch.int64 and t.shape == (dim // 2,)
        want = [base ** (-2 * j / dim) / (2 * math.pi) for j in range(dim // 2)]
        assert np.allclose([x / 2.0 ** 64 for x in t.tolist()], want, rtol=1e-14)
    assert lb.rotary_turns(0).shape == (0,)


def test_rotary_scaling():
    plain = np.array(lb.rotary_turns(128, 500000.0).tolist(), float)

    def ratio(**kw):
        return plain / np.array(lb.rotary_turns(128, 500000.0, **kw).tolist(), float)
    assert np.allclose(ratio(scaling="linear", factor=8.0), 8.0)
    r = ratio(scaling="base", factor=8.0)
    assert abs(r[0] - 1) < 1e-12 and abs(r[-1] - 8.0) < 1e-9 and np.all(np.diff(r) > 0)
    r = ratio(scaling="wavelength", factor=8.0, original_length=8192)
    over = plain / 2.0 ** 64 * 8192                       # turns over the original length
    assert np.allclose(r[over >= 4.0], 1.0) and np.allclose(r[over <= 1.0], 8.0)
    mid = (over > 1.0) & (over < 4.0)
    blend = (over[mid] - 1.0) / 3.0
    assert mid.any() and np.allclose(1.0 / r[mid], blend + (1 - blend) / 8.0)


@pytest.mark.parametrize("kw", [dict(dim=3), dict(dim=-2), dict(dim=8, base=1.0), dict(dim=8, scaling="other"),
                                dict(dim=8, scaling="linear", factor=0.5), dict(dim=8, low=4.0, high=4.0),
                                dict(dim=8, original_length=0)])
def test_rotary_turns_refusals(kw):
    with pytest.raises(ValueError):
        lb.rotary_turns(**kw)


# ---------------------------------------------------------------------------
# The definitions that the GPU tests compare with
# ---------------------------------------------------------------------------

def test_reference_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.E4M3, vals, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.integers(-4, 3, 20000), (ref.GRID[:-1] + ref.GRID[1:]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32).astype(np.float64)
    got = torch.from_numpy(x).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_round(x), got)


def test_reference_exponent():
    assert ref.page_exponent(448.0) == 0 and ref.page_exponent(448.0001) == 1 and ref.page_exponent(224.0) == -1
    assert ref.page_exponent(0.0) == -64 and ref.page_exponent(1e30) == 64


def test_reference_attention_by_differences():
    """The definition's out is the gradient of lse in the direction of v: d lse(s + h v) / dh."""
    b = ref.make_batch(1, [20], [3], 1, 64, 16)
    q = ref.f64(ref.bf16(np.random.default_rng(2).standard_normal((3, 2, 64))))
    out, lse, _, _ = ref.attention(q, b, 0.125)
    k, v = ref.cached(b, 0, 0, "k"), ref.cached(b, 0, 0, "v")
    h = 1e-5
    for r in range(3):
        x = q[r, 1] @ k[:18 + r].T * 0.125
        up, down = (np.log(np.exp(x + sgn * h * v[:18 + r, 7]).sum()) for sgn in (1, -1))
        assert abs((up - down) / (2 * h) - out[r, 1, 7]) < 1e-6 and abs(np.log(np.exp(x).sum()) - lse[r, 1]) < 1e-12


def test_reference_sample_finds_a_planted_mistake():
    row = np.log(np.array([0.5, 0.25, 0.125, 0.125]))
    ref.check_sample(row, 0.6, 1.0, 0, 1.0, 0.0, 1, math.log(0.25))
    with pytest.raises(AssertionError):
        ref.check_sample(row, 0.6, 1.0, 0, 1.0, 0.0, 2, math.log(0.125))
    with pytest.raises(AssertionError):
        ref.check_sample(row, 0.6, 1.0, 0, 1.0, 0.0, 1, math.log(0.2))
    with pytest.raises(AssertionError):
        ref.check_sample(row, 0.9, 1.0, 2, 1.0, 0.0, 2, math.log(0.2))
