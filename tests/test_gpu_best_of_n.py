"""The serving calls around a linear-attention layer, together, as examples/best_of_n.py uses them: the best branch's states,
after fork, decode, free and compact, are those of reading its tokens as one prompt."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("best_of_n", os.path.join(ROOT, "examples", "best_of_n.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_best_branch_is_its_own_prompt():
    import exact_replay_decode_gb300 as ers
    ex = _example()
    model = ex.Model(vocab=1009, width=256, heads=4, groups=2)
    prompt = torch.randint(0, 1009, (200,), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    best, score, caches, tokens = ex.best_of_n(model, prompt, branches=5, steps=6)
    winner = 1 + int(score.argmax())
    fresh = model.caches(1, 1)
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c in fresh:
        ers.pages_own(c.pages, slot)
    model(torch.cat([prompt, best]), lambda n, q, k, v: ers.linattn_prefill(fresh[n], q, k, v, model.decay, slot=slot))
    for c, f in zip(caches, fresh):
        assert int((c.pages.refs > 0).sum()) == 2                 # the prompt's and the winner's
        assert sorted(c.pages.table[[0, winner], 0].tolist()) == [0, 1]
        got, want = c.state[c.pages.table[winner, 0]], f.state[0]
        # the layers' inputs are rounded to bf16 by both, along different ways through the matrix products
        assert ((got - want).norm() / want.norm()).item() < 2e-2
    assert score.isfinite().all() and len({tuple(t) for t in tokens.tolist()}) > 1
