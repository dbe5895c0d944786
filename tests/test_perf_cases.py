"""CPU: the measured cases of draft verification can be prepared in every form that their
ranges hold, on the CPU in the place of the GPU, and the plain form agrees with the
definition."""
import itertools
import os
import random
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cases():
    with open(os.path.join(ROOT, "perf", "more_operators.py")) as f:
        text = f.read().replace('"cuda"', '"cpu"')
    module = types.ModuleType("cases_on_the_cpu")
    exec(compile(text, "more_operators.py", "exec"), module.__dict__)
    return module


@pytest.mark.parametrize("q,drafts,dtype", list(itertools.product([1, 2, 3, 4, 5, 8], ["sampled", "fixed"], ["fp32", "bf16"])))
def test_verification_in_every_form(cases, q, drafts, dtype):
    case = dict(op="verify", batch=3, q=q, vocab=1000, dtype=dtype, drafts=drafts)
    state = cases.prepare(case, 11)
    assert state["tokens"].shape == (3, q - 1) and ((state["tokens"] >= 0) & (state["tokens"] < 1000)).all()
    assert state["draft"] is None if drafts == "fixed" else state["draft"].shape == (3, q - 1, 1000)
    again, other = cases.prepare(case, 11), cases.prepare(case, 12)
    for name in ("target", "tokens", "u", "lens_d"):
        assert torch.equal(state[name], again[name])
    assert not torch.equal(state["target"], other["target"])
    got, want = cases.run(state), cases.exact(case, 11)
    for name in ("accepted", "lens", "tokens"):
        assert torch.equal(got[name], want[name]), name


def test_drawn_cases_of_verification_hold_single_tokens(cases):
    rng = random.Random(0)
    drawn = [cases.draw(rng) for _ in range(2000)]
    forms = {(c["q"] > 1, c["drafts"], c["dtype"]) for c in drawn if c["op"] == "verify"}
    assert len(forms) == 8
