"""What the decoder operators' binding refuses of tensors on the GPU: the extension module does
not accept it, and the Python side says why.  And the two agree on what is accepted."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_groupwise_weight_gb300 as lb  # noqa: E402
from bit_groupwise_weight_gb300 import build as lbuild  # noqa: E402
from bit_groupwise_weight_gb300 import decoder  # noqa: E402

lbuild.build()

HEADS, KV_HEADS, DIM, PAGE, BATCH, NEW = 4, 2, 64, 16, 3, 2
T = BATCH * NEW


def ints(*values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def floats(*shape):
    return torch.rand(*shape, generator=torch.Generator(device="cuda").manual_seed(sum(shape)), device="cuda")


def rows(heads, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + heads)
    return torch.randn(T, heads, DIM, generator=gen, device="cuda").to(torch.bfloat16)


def cached():
    """A cache of 9 pages with something in it, and where it is."""
    k, v, ke, ve = lb.empty_cache(9, KV_HEADS, DIM, PAGE)
    for i, c in enumerate((k, v)):
        gen = torch.Generator(device="cuda").manual_seed(i)
        c.view(torch.uint8).copy_(torch.randint(0, 0x60, c.shape, generator=gen, device="cuda", dtype=torch.uint8))
    return dict(k_cache=k, v_cache=v, k_exp=ke - 3, v_exp=ve - 3, page_table=torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3),
                lens=ints(5, 40, 17), cu_q=None, max_q=None)


def attention_args():
    return dict(q=rows(HEADS)) | cached() | dict(scale=None, window=0, out=None, lse=None, workspace=None)


def append_args():
    return dict(q=rows(HEADS), k=rows(KV_HEADS, 1), v=rows(KV_HEADS, 2)) | cached() | dict(
        turns=lb.rotary_turns(DIM, device="cuda"), interleaved=False, factor=1.0, out=None)


def sample_args():
    return dict(logits=floats(5, 300) * 8, u=floats(5), temperature=0.9, top_k=20, top_p=0.9, min_p=0.01, out=None, logprob=None)


ARGS = {"attention": attention_args, "kv_append": append_args, "sample": sample_args}


def apart(t):
    """The same values, every second of a tensor twice as wide."""
    return torch.stack((t, t), -1).flatten(-2)[..., ::2]


CACHE = [
    ("k_cache", lambda t: t.view(torch.int8)), ("k_cache", lambda t: t.cpu()), ("k_cache", lambda t: t[0]),
    ("k_cache", lambda t: t[..., :32]), ("k_cache", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)), ("k_cache", None),
    ("v_cache", lambda t: t.to(torch.bfloat16)), ("v_cache", lambda t: t[:5]), ("v_cache", lambda t: t.cpu()),
    ("v_cache", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)),
    ("k_exp", lambda t: t.int()), ("k_exp", lambda t: t[:5]), ("k_exp", lambda t: t.t().contiguous().t()), ("k_exp", lambda t: t.cpu()),
    ("v_exp", lambda t: t.view(torch.uint8)), ("v_exp", lambda t: t[:, :1]), ("v_exp", None),
    ("page_table", lambda t: t.long()), ("page_table", lambda t: t[0]), ("page_table", lambda t: t.t()),
    ("page_table", lambda t: t[:1].expand(3, 3)), ("page_table", lambda t: t.cpu()),
    ("lens", lambda t: t.long()), ("lens", lambda t: t[:2]), ("lens", apart), ("lens", lambda t: t.cpu()), ("lens", None),
    ("cu_q", lambda t: ints(0, 2, 4, 6, dtype=torch.int64)), ("cu_q", lambda t: ints(0, 3, 6)), ("cu_q", lambda t: apart(ints(0, 2, 4, 6))),
    ("cu_q", lambda t: [0, 2, 4, 6])]
ROWS = [
    ("q", lambda t: t.cpu()), ("q", lambda t: t.half()), ("q", lambda t: t[0]), ("q", apart), ("q", lambda t: t[:5]),
    ("q", lambda t: t[..., :32]), ("q", lambda t: None),
    ("out", lambda t: rows(HEADS).float()), ("out", lambda t: rows(HEADS)[:5]), ("out", lambda t: apart(rows(HEADS))),
    ("out", lambda t: rows(HEADS).cpu()), ("out", lambda t: "out")]
BAD = [("attention", n, f) for n, f in CACHE + ROWS] + [("kv_append", n, f) for n, f in CACHE + ROWS] + [
    ("attention", "max_q", 1 << 40), ("attention", "max_q", 1.5), ("attention", "scale", "x"), ("attention", "window", 1.5),
    ("attention", "window", 1 << 40),
    ("attention", "lse", lambda t: floats(T, HEADS).double()), ("attention", "lse", lambda t: floats(T, HEADS + 1)),
    ("attention", "lse", lambda t: apart(floats(T, HEADS))), ("attention", "lse", lambda t: floats(T, HEADS).cpu()),
    ("attention", "workspace", lambda t: torch.empty(1 << 20, dtype=torch.int8, device="cuda")),
    ("attention", "workspace", lambda t: torch.empty(1 << 10, 1 << 10, dtype=torch.uint8, device="cuda")),
    ("attention", "workspace", lambda t: torch.empty(1 << 21, dtype=torch.uint8, device="cuda")[::2]),
    ("attention", "workspace", lambda t: torch.empty(1 << 20, dtype=torch.uint8)),
    ("kv_append", "k", lambda t: t.float()), ("kv_append", "k", lambda t: t[:, :1]), ("kv_append", "v", apart),
    ("kv_append", "v", lambda t: t.cpu()), ("kv_append", "turns", lambda t: t.int()), ("kv_append", "turns", lambda t: t[None]),
    ("kv_append", "turns", lambda t: apart(t)), ("kv_append", "turns", lambda t: t.cpu()), ("kv_append", "factor", "x"),
    ("kv_append", "max_q", 1 << 40),
    ("sample", "logits", lambda t: t.double()), ("sample", "logits", lambda t: t[0]), ("sample", "logits", apart),
    ("sample", "logits", lambda t: t.cpu()), ("sample", "u", lambda t: t.double()), ("sample", "u", lambda t: t[:4]),
    ("sample", "u", apart), ("sample", "u", 0.5), ("sample", "temperature", lambda t: floats(4)), ("sample", "temperature", "x"),
    ("sample", "temperature", lambda t: floats(5).half()), ("sample", "temperature", lambda t: floats(5).cpu()),
    ("sample", "top_p", lambda t: floats(5, 1)), ("sample", "top_p", None), ("sample", "min_p", lambda t: apart(floats(5))),
    ("sample", "top_k", lambda t: ints(1, 2, 3, 4, 5, dtype=torch.int64)), ("sample", "top_k", 2.5), ("sample", "top_k", 1 << 40),
    ("sample", "out", lambda t: ints(1, 2, 3, 4, 5)), ("sample", "out", lambda t: ints(1, 2, dtype=torch.int64)),
    ("sample", "logprob", lambda t: floats(5).double()), ("sample", "logprob", lambda t: floats(6))]


@pytest.mark.parametrize("op,name,change", BAD, ids=[f"{o}-{n}-{i}" for i, (o, n, _) in enumerate(BAD)])
def test_refused_with_a_reason(op, name, change):
    args = ARGS[op]()
    args[name] = change(args[name]) if callable(change) else change
    if name == "max_q":                                    # counts with cu_q only
        args["cu_q"] = ints(0, 2, 4, 6)
    before = {n: t.clone() for n, t in args.items() if isinstance(t, torch.Tensor)}
    assert getattr(decoder._load(), op)(*args.values()) is None
    with pytest.raises(ValueError) as why:
        getattr(lb, op)(**args)
    assert str(why.value) and not isinstance(why.value, lb.LowbitError)
    for n, t in before.items():
        assert torch.equal(args[n].contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)), n


@pytest.mark.parametrize("op,change", [
    ("attention", dict(window=-1)), ("attention", dict(scale=float("nan"))), ("attention", dict(cu_q=ints(0, 2, 4, 6), max_q=0)),
    ("attention", dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ("kv_append", dict(turns=lb.rotary_turns(2 * DIM, device="cuda"))), ("kv_append", dict(cu_q=ints(0, 2, 4, 6), max_q=-1))])
def test_refused_by_the_library(op, change):
    with pytest.raises(lb.LowbitError):
        getattr(lb, op)(**(ARGS[op]() | change))


@pytest.mark.parametrize("op,change", [
    ("attention", {}), ("attention", dict(cu_q=ints(0, 1, 5, 6), max_q=4, scale=0.3, window=7)), ("attention", dict(cu_q=ints(0, 1, 5, 6))),
    ("attention", dict(out=rows(HEADS), workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))),
    ("kv_append", {}), ("kv_append", dict(turns=None, out=rows(HEADS))),
    ("kv_append", dict(cu_q=ints(0, 1, 5, 6), max_q=4, interleaved=True, factor=0.5, turns=lb.rotary_turns(32, device="cuda"))),
    ("sample", {}), ("sample", dict(temperature=floats(5) + 0.5, top_p=floats(5), min_p=floats(5) * 0.1, top_k=ints(0, 1, 7, 300, -1))),
    ("sample", dict(logits=floats(5, 301).to(torch.bfloat16), out=torch.empty(5, dtype=torch.int64, device="cuda")))])
def test_both_sides_of_the_binding_make_the_same_call(op, change, monkeypatch):
    class Nothing:
        attention = kv_append = sample = staticmethod(lambda *a: None)
    results = []
    for stub in (False, True):
        args = ARGS[op]() | change
        extra = {"attention": "lse", "sample": "logprob"}.get(op)
        if extra:
            args[extra] = torch.zeros((T, HEADS) if extra == "lse" else (5,), device="cuda")
        if stub:
            monkeypatch.setattr(decoder, "_hot", Nothing)
        result = [getattr(lb, op)(**args).clone()] + ([args[extra]] if extra else [])
        if op == "kv_append":
            result += [args[n].view(torch.uint8) for n in ("k_cache", "v_cache", "k_exp", "v_exp")]
        results.append(result)
    assert len(results[0]) == len(results[1]) and all(torch.equal(a, b) for a, b in zip(*results))
