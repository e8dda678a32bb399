"""What the decoder operators allocate for their callers: as torch's own operators do where
torch has something to say about new tensors (deterministic algorithms, modes, subclasses)."""
from __future__ import annotations

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_groupwise_weight_gb300 as lb  # noqa: E402
from bit_groupwise_weight_gb300 import build as lbuild  # noqa: E402

lbuild.build()


def calls(bits, wrap=lambda t: t):
    """Each operator that makes an output, over 20 rows of which sequences have 15: (name, call)."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(20, 8, 64, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = (t.contiguous() for t in x.split([4, 2, 2], 1))
    cache = lb.empty_cache(9, 2, 64, 16, bits=bits)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    lens, cu = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([30, 40], [0, 6, 15]))
    logits, u = torch.randn(3, 1000, generator=gen, device="cuda"), torch.tensor([0.1, 0.5, 0.9], device="cuda")
    q, logits, first = wrap(q), wrap(logits), wrap(cache[0])
    return {"kv_append": lambda: lb.kv_append(q, k, v, *cache, table, lens, cu_q=cu, max_q=9),
            "attention": lambda: lb.attention(q, *cache, table, lens, cu_q=cu, max_q=9),
            "cache_values": lambda: lb.cache_values(first, *cache[1:]),
            "sample": lambda: lb.sample(logits, u)}


@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("name", ["kv_append", "attention"])
def test_rows_of_no_sequence_are_nan_with_deterministic_algorithms(bits, name, deterministic):
    """New outputs are filled before anything is written, so that rows left out do not hold what was there before."""
    call = calls(bits)[name]
    for _ in range(3):
        used = [torch.full((20, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        del used
        out = call()
        assert torch.isnan(out[15:]).all() and not torch.isnan(out[:15]).any()
        del out


@pytest.mark.parametrize("name", ["kv_append", "attention", "cache_values", "sample"])
def test_same_results_with_deterministic_algorithms(name):
    plain = calls(4)[name]()
    torch.use_deterministic_algorithms(True)
    try:
        filled = calls(4)[name]()
    finally:
        torch.use_deterministic_algorithms(False)
    for a, b in zip(*((t if isinstance(t, tuple) else (t,)) for t in (plain, filled))):
        assert torch.equal(a[:15], b[:15]) and a.stride() == b.stride() and a.dtype == b.dtype


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("name,new", [("kv_append", 1), ("attention", 2), ("cache_values", 2), ("sample", 1)])
def test_modes_see_what_is_allocated(bits, name, new):
    """attention: the workspace too."""
    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.names = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(str(func))
            return func(*args, **(kwargs or {}))
    call = calls(bits)[name]
    with Seen() as seen:
        call()
    assert sum("empty" in n for n in seen.names) == new, seen.names


class Marked(torch.Tensor):
    """A subclass of which torch's operators make more."""
    made = 0

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        with torch._C._DisableTorchDispatch():
            out = func(*args, **(kwargs or {}))
        if "empty_like" not in str(func):
            return out
        Marked.made += 1
        return out.as_subclass(cls)


@pytest.mark.parametrize("name", ["kv_append", "attention"])
def test_a_subclass_of_q_says_what_comes_out(name):
    Marked.made = 0
    out = calls(8, lambda t: t.as_subclass(Marked))[name]()
    assert Marked.made == 1 and type(out) is Marked
