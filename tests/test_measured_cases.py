"""The measured cases of the step's inputs: what one pass returns belongs to that pass."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def cases():
    spec = importlib.util.spec_from_file_location("operators_cases", os.path.join(ROOT, "perf", "operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class RaisingPlan:
    """Raises s_max to the largest logit of its current inputs, as the forward pass does."""

    def __init__(self, s_max, logits):
        self.s_max, self.logits = s_max, logits

    def forward(self):
        self.s_max.copy_(torch.maximum(self.s_max, self.logits.amax(1)))


def test_a_pass_of_the_forward_case_starts_s_max_anew(cases):
    """The forward pass raises s_max and never lowers it: a pass on smaller logits returns their
    maximum, not that of the passes before it."""
    s_max = torch.full((2,), -math.inf)
    logits = torch.tensor([[3.0, 5.0], [-2.0, -1.0]])
    state = dict(case=dict(op="attention"), plan=RaisingPlan(s_max, logits), o=torch.zeros(1), lse=torch.zeros(1),
                 s_max=s_max)
    cases.own = True
    assert torch.equal(cases.run(state)[2], torch.tensor([5.0, -1.0]))
    logits.sub_(10.0)
    assert torch.equal(cases.run(state)[2], torch.tensor([-5.0, -11.0]))


@pytest.mark.gpu
def test_a_pass_of_the_forward_case_follows_its_inputs(cases):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    case = dict(op="attention", lengths="5,70", k_lengths="5,70", heads=4, kv_heads=2, dim=64, causal=True)
    cases.own = True
    state = cases.prepare(case, 1)
    first = cases.run(state)[2].clone()
    state["q"].mul_(0.25)                                       # exact in bf16: logits by a quarter
    second = cases.run(state)[2].clone()
    assert bool((first > 0).all()) and torch.equal(second, first * 0.25)
