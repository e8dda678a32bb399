"""Host side of the 4-bit cache, head norms and positions of several axes (no GPU needed):
refusals of the C ABI, sizes, and the tests' own definitions checked against themselves."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import bit_groupwise_weight_gb300 as lb
import cache4_ref as ref4
from bit_groupwise_weight_gb300 import build as lbuild
from bit_groupwise_weight_gb300 import decoder

EINVAL, EUNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return lb.abi()


# Addresses that are never touched: every call below is rejected before CUDA, or empty.
DEFAULTS = {
    "cache4": dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x31000, page_stride=2 * 64 * 64, head_stride=64 * 64,
                   scale_page_stride=2 * 64 * 4, scale_head_stride=64 * 4, pages=9, kv_heads=2, head_dim=128, page=64),
    "cache": dict(k=0x10000, v=0x20000, k_exp=0x30000, v_exp=0x31000, page_stride=2 * 64 * 128, head_stride=64 * 128, pages=9,
                  kv_heads=2, head_dim=128, page=64),
    "seqs": dict(page_table=0x40000, lens=0x41000, cu_q=None, table_stride=4, width=4, batch=3, tokens=6, max_q=0),
    "append": dict(q=0x50000, k=0x60000, v=0x70000, q_out=0x80000, q_token=1024, q_head=128, k_token=256, k_head=128,
                   v_token=256, v_head=128, o_token=1024, o_head=128, turns=0x90000, factor=1.0, heads=8, rotary_dim=128,
                   interleaved=0),
    "before": dict(q_norm=0xb0000, k_norm=0xb1000, positions=0xb2000, axis=0xb3000, positions_token=3, eps=1e-6, axes=3, norm_dtype=1),
    "attention": dict(q=0x50000, out=0x80000, lse=None, q_token=1024, q_head=128, o_token=1024, o_head=128, lse_token=8,
                      workspace=0xa0000, workspace_bytes=1 << 40, scale=0.1, heads=8, window=0),
}
PACK = {"cache4": decoder._CACHE4, "cache": decoder._CACHE, "seqs": decoder._SEQUENCES, "append": decoder._KV_APPEND,
        "before": decoder._PROLOGUE, "attention": decoder._ATTENTION}


def descriptor(what, **changes):
    values = DEFAULTS[what] | changes
    assert len(values) == len(DEFAULTS[what])
    return PACK[what](*(v or 0 for v in values.values()))


def append(lib, bits, args={}, before={}, cache={}, seqs={}):
    fn = lib.lowbit_kv_append4 if bits == 4 else lib.lowbit_kv_append_ex
    return fn(descriptor("append", **args), None if before is None else descriptor("before", **before),
              descriptor("cache4" if bits == 4 else "cache", **cache), descriptor("seqs", **seqs), None)


def attention(lib, args={}, cache={}, seqs={}):
    return lib.lowbit_attention4(descriptor("attention", **args), descriptor("cache4", **cache), descriptor("seqs", **seqs), None)


BAD_CACHES = [
    dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=0x10008), dict(v=0x20004), dict(k_scale=0x30008),
    dict(v_scale=0x31001), dict(pages=-1), dict(kv_heads=0), dict(kv_heads=1 << 16), dict(head_dim=96), dict(head_dim=32),
    dict(page=8), dict(page=48), dict(page=512), dict(head_stride=64 * 64 - 16), dict(page_stride=100), dict(head_stride=64 * 64 + 8),
    dict(page_stride=1 << 40), dict(scale_head_stride=64 * 4 - 16), dict(scale_head_stride=64 * 4 + 4), dict(scale_page_stride=1 << 40),
    dict(scale_page_stride=8)]


@pytest.mark.parametrize("cache", BAD_CACHES + [dict(pages=0), dict(kv_heads=3)])
def test_caches_that_are_refused(lib, cache):
    assert append(lib, 4, cache=cache) == EINVAL
    assert attention(lib, cache=cache) == EINVAL


@pytest.mark.parametrize("cache", BAD_CACHES)
def test_caches_whose_values_are_refused(lib, cache):
    assert lib.lowbit_cache4_values(descriptor("cache4", **cache), 0x100000, 0x200000, None) == EINVAL


@pytest.mark.parametrize("outs", [(0, 0x200000), (0x100000, 0), (0x100008, 0x200000), (0x100000, 0x200002)])
def test_outputs_of_values_that_are_refused(lib, outs):
    assert lib.lowbit_cache4_values(descriptor("cache4"), *outs, None) == EINVAL
    assert lib.lowbit_cache_values(descriptor("cache"), *outs, None) == EINVAL
    assert lib.lowbit_cache_values(None, 0x100000, 0x200000, None) == EINVAL
    assert lib.lowbit_cache4_values(descriptor("cache4", pages=1 << 30, kv_heads=4), 0x100000, 0x200000, None) == EINVAL
    assert lib.lowbit_cache4_values(descriptor("cache4", pages=0), *outs, None) == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("before", [
    dict(q_norm=0xb0001), dict(k_norm=0xb1003), dict(norm_dtype=0, q_norm=0xb0002), dict(norm_dtype=3), dict(norm_dtype=-1),
    dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(positions=0xb2002), dict(axes=0), dict(axes=-1), dict(axes=256)])
def test_prologues_that_are_refused(lib, bits, before):
    assert append(lib, bits, before=before) == EINVAL


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("before", [
    None, {}, dict(q_norm=None, k_norm=None, norm_dtype=9, eps=math.nan), dict(positions=None, axes=-3), dict(axis=None, axes=255)])
def test_what_is_not_used_is_not_looked_at(lib, bits, before):
    """Accepted: an empty call does nothing, any other gets as far as the device."""
    assert append(lib, bits, before=before, seqs=dict(tokens=0)) == 0
    if not torch.cuda.is_available():
        assert append(lib, bits, before=before) != EINVAL


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("args", [
    dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(q=0x50001), dict(turns=None), dict(turns=0x90004),
    dict(rotary_dim=-2), dict(rotary_dim=130), dict(rotary_dim=7), dict(heads=0), dict(heads=7)])
def test_appends_that_are_refused(lib, bits, args):
    assert append(lib, bits, args) == EINVAL


@pytest.mark.parametrize("args", [
    dict(q=None), dict(out=None), dict(q=0x50004), dict(out=0x80002), dict(lse=0xb0002), dict(q_token=1022), dict(q_head=2),
    dict(o_token=1), dict(o_head=127), dict(workspace=None), dict(workspace=0xa0008), dict(workspace_bytes=100),
    dict(scale=math.nan), dict(scale=math.inf), dict(window=-1), dict(heads=0), dict(heads=9)])
def test_attentions_that_are_refused(lib, args):
    assert attention(lib, args) == EINVAL


@pytest.mark.parametrize("seqs", [
    dict(page_table=None), dict(lens=None), dict(page_table=0x40002), dict(lens=0x41001), dict(width=0), dict(width=-1),
    dict(table_stride=3), dict(batch=-1), dict(tokens=-1), dict(tokens=7), dict(cu_q=0x42000, max_q=0),
    dict(cu_q=0x42002, max_q=2), dict(tokens=3 << 28), dict(width=1 << 28, table_stride=1 << 28)])
def test_sequences_that_are_refused(lib, seqs):
    assert append(lib, 4, seqs=seqs) == EINVAL
    assert append(lib, 8, seqs=seqs) == EINVAL
    assert attention(lib, seqs=seqs) == EINVAL


def test_null_descriptors_are_refused(lib):
    a, c, s = descriptor("append"), descriptor("cache4"), descriptor("seqs")
    assert lib.lowbit_kv_append4(None, None, c, s, None) == EINVAL
    assert lib.lowbit_kv_append4(a, None, None, s, None) == EINVAL
    assert lib.lowbit_kv_append4(a, None, c, None, None) == EINVAL
    t = descriptor("attention")
    assert lib.lowbit_attention4(None, c, s, None) == EINVAL
    assert lib.lowbit_attention4(t, None, s, None) == EINVAL
    assert lib.lowbit_attention4(t, c, None, None) == EINVAL
    assert lib.lowbit_attention4_workspace(8, None, s) == 0


@pytest.mark.parametrize("seqs", [dict(tokens=0), dict(batch=0), dict(batch=0, tokens=0)])
def test_empty_calls_do_nothing(lib, seqs):
    assert append(lib, 4, seqs=seqs) == 0
    assert attention(lib, seqs=seqs) == 0
    assert lib.lowbit_attention4_workspace(8, descriptor("cache4"), descriptor("seqs", **seqs)) == 0


def test_workspace_follows_from_the_sizes_alone(lib):
    nothing = dict(k=None, v=None, k_scale=None, v_scale=None, page_stride=0, head_stride=0, scale_page_stride=0, scale_head_stride=0)
    seqs = descriptor("seqs")
    assert lib.lowbit_attention4_workspace(8, descriptor("cache4", **nothing), seqs) == lib.lowbit_attention4_workspace(
        8, descriptor("cache4"), seqs) > 0
    for bad in (dict(head_dim=96), dict(page=48), dict(pages=0), dict(kv_heads=3)):
        assert lib.lowbit_attention4_workspace(8, descriptor("cache4", **bad), seqs) == 0


def test_empty_caches():
    k, v, ks, vs = lb.empty_cache(3, 2, 128, 16, device="cpu", bits=4)
    assert k.shape == v.shape == (3, 2, 16, 64) and k.dtype == torch.uint8 and not k.any()
    assert ks.shape == vs.shape == (3, 2, 16, 4) and ks.dtype == torch.float8_e5m2 and not ks.view(torch.uint8).any()
    assert [tuple(t.shape) for t in lb.empty_cache(3, 2, 64, 16, device="cpu")] == [(3, 2, 16, 64)] * 2 + [(3, 2)] * 2
    for bad in (dict(bits=3), dict(bits=4, head_dim=96)):
        with pytest.raises(ValueError):
            lb.empty_cache(**(dict(pages=1, kv_heads=1, head_dim=64, device="cpu") | bad))


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(6, 4, 64, dtype=torch.bfloat16)), dict(k_exp=torch.zeros(9, 2, 16, 2, dtype=torch.uint8))])
def test_the_binding_refuses_tensors_of_the_cpu(change):
    k, v, ks, vs = lb.empty_cache(9, 2, 64, 16, device="cpu", bits=4)
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    args = dict(q=q, k_cache=k, v_cache=v, k_exp=ks, v_exp=vs, page_table=torch.zeros(3, 3, dtype=torch.int32),
                lens=torch.zeros(3, dtype=torch.int32)) | change
    with pytest.raises(ValueError, match="CUDA"):
        lb.attention(**args)
    with pytest.raises(ValueError, match="CUDA"):
        lb.kv_append(**(args | dict(k=q[:, :2], v=q[:, :2], q_norm=torch.ones(64))))
    with pytest.raises(ValueError, match="CUDA"):
        lb.cache_values(k, v, ks, vs)


# ---------------------------------------------------------------------------
# The definitions
# ---------------------------------------------------------------------------

def test_scale_bytes_are_e5m2():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e5m2).to(torch.float64).numpy()
    assert np.array_equal(t, ref4.E5M2, equal_nan=True)


def test_scales_are_the_smallest_that_do():
    rng = np.random.default_rng(1)
    amax = np.concatenate([np.exp(rng.uniform(-25, 14, 5000)), ref4.SCALES * 7.5, np.nextafter(ref4.SCALES * 7.5, 0), [0.0, 1e30]])
    byte = ref4.scale_byte(amax)
    s = ref4.E5M2[byte]
    assert np.all((amax <= 7.5 * s) | (s == 57344)) and np.all((amax > 7.5 * ref4.E5M2[byte - 1]) | (s == 2.0 ** -14))


def test_codes_are_the_nearest_and_survive():
    """Within half a step; coding values again changes nothing, even where the largest code is below 7."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((50, 3, 128)) * np.exp(rng.standard_normal((50, 3, 128)))
    codes, scales = ref4.coded(x)
    y = ref4.values(codes, scales)
    step = np.repeat(ref4.E5M2[scales], 32, -1)
    assert np.all(np.abs(y - x) <= step / 2 * (1 + 1e-12)) and codes.min() >= 1 and codes.max() <= 15
    assert np.array_equal(ref4.unpacked(ref4.packed(codes)), codes)
    assert np.array_equal(y, y.astype(np.float16).astype(np.float64))                     # exact in fp16
    assert torch.equal(torch.from_numpy(y), torch.from_numpy(y).to(torch.bfloat16).double())     # and in bf16


def test_definition_of_attention_against_a_softmax():
    b = ref4.make_batch(3, [20, 9], [3, 1], 2, 64, 16)
    q = np.random.default_rng(4).standard_normal((4, 4, 64))
    out, lse, _, _ = ref4.attention(q, b, 0.2, window=6)
    k, v = ref4.cached(b, 0, 1, "k")[0], ref4.cached(b, 0, 1, "v")[0]
    for i, pos in enumerate((17, 18, 19)):
        s = q[i, 3] @ k[pos - 5:pos + 1].T * 0.2
        p = np.exp(s - s.max())
        assert np.allclose(out[i, 3], p @ v[pos - 5:pos + 1] / p.sum(), atol=1e-12)
        assert np.isclose(lse[i, 3], np.log(np.exp(s).sum()))


def test_definitions_of_norm_and_rotation():
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((4, 2, 64)), rng.standard_normal(64)
    y = ref4.normed(x, w, 0.0)
    assert np.allclose(((y / w) ** 2).mean(-1), 1)
    turns = lb.rotary_turns(64).tolist()
    place = np.array([3, 7, 100, 5])
    axes = np.arange(32) % 2
    both, _ = ref4.rotated(x, np.stack((place, place), 1), turns, axes, False, 1.0)
    one, _ = ref4.rotated(x, place, turns, None, False, 1.0)
    assert np.allclose(both, one) and np.allclose((one ** 2).sum(-1), (x ** 2).sum(-1))
    theta = place[1] * turns[5] / 2.0 ** 64 * 2 * math.pi
    assert np.isclose(one[1, 0, 5], x[1, 0, 5] * math.cos(theta) - x[1, 0, 37] * math.sin(theta))
    apart, _ = ref4.rotated(x, np.stack((place, 0 * place), 1), turns, axes, False, 1.0)
    assert np.allclose(apart[..., 1:32:2], x[..., 1:32:2]) and np.allclose(apart[..., 0:32:2], one[..., 0:32:2])
