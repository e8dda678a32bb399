"""The decoding example with a 4-bit cache and head norms: linears, cache, attention and sampling together."""
import sys
from pathlib import Path

import pytest
import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
pytestmark = pytest.mark.gpu

SMALL = dict(layers=2, width=256, heads=4, kv_heads=2, dim=64, hidden=512, vocab=1000, length=300, cache_bits=4, head_norms=True)
PROMPTS = [[7 * i % 1000 for i in range(n)] for n in (1, 40, 130)]


def make(page=32, seed=3):
    from examples.decode import Decoder
    return Decoder(batch=3, page=page, seed=seed, **SMALL)


def test_graph_of_a_step_equals_the_calls():
    """The same tokens from replays of a captured step as from calling it."""
    settings = dict(temperature=0.9, top_k=40, top_p=0.95, min_p=0.01)
    us = torch.rand(20, 3, generator=torch.Generator().manual_seed(5)).cuda()
    answers = []
    for captured in (False, True):
        model = make()
        answer = [model.prompt(PROMPTS, us[0], **settings)]
        u = torch.zeros(3, device="cuda")
        if captured:
            graph = model.capture(u, **settings)
        for i in range(1, 20):
            u.copy_(us[i])
            graph.replay() if captured else model.step(u, **settings)
            answer.append(model.last.clone())
        answers.append(torch.stack(answer))
        assert model.lens.tolist() == [len(p) + 19 for p in PROMPTS]
    assert torch.equal(answers[0], answers[1])
    assert int(answers[0].min()) >= 0 and int(answers[0].max()) < 1000


def test_prompt_at_once_and_token_by_token():
    """The logits after a prompt, whole and a token at a time.  A token's codes depend on no other token, but the
    linears of one row and of many round differently, and a code next to a border is a seventh of its group's largest
    value off: both ways are some per cent from each other and far nearer than two unlike prompts."""
    n = 70
    tokens = torch.tensor([11 * i % 1000 for i in range(n)], device="cuda")
    lens = torch.tensor([n, 0, 0], dtype=torch.int32, device="cuda")
    cu_q = torch.tensor([0, n, n, n], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        whole = make().logits(tokens, lens, cu_q, n)[-1].double()
        other = make().logits(tokens.flip(0), lens, cu_q, n)[-1].double()
        model = make()
        cu_1 = torch.tensor([0, 1, 1, 1], dtype=torch.int32, device="cuda")
        for i in range(n):
            one = model.logits(tokens[i:i + 1], torch.tensor([i + 1, 0, 0], dtype=torch.int32, device="cuda"), cu_1, 1)
        one = one[-1].double()
    assert (whole - one).norm() <= 0.2 * whole.norm()
    assert (whole - other).norm() >= 0.5 * whole.norm()
