"""GPU: the operators together, as examples/speculative_step.py runs them."""
import importlib.util
import os

import pytest

import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(bsf8_lib):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_greedy_tokens_are_those_of_a_plain_pass(example):
    """A cache that commits and appends left wrong, a mask or a position off, would give logits that have
    nothing to do with the tokens' (3 to 4 standard deviations below the best).  bf16 logits and the
    layer's roundings (2^-9 of values of a few standard deviations, a handful of times) move a logit by
    less than 0.1."""
    model, prompts = example.Model(), example.prompts()
    got = example.speculative(model, prompts, 12)
    assert all(len(t) >= 12 for t in got) and any(len(t) > 12 for t in got)
    for prompt, tokens in zip(prompts, got):
        assert max(example.shortfall(model, prompt, tokens)) < 0.1
    assert bsf8.device_status() == 0


def test_sampled_steps_repeat(example):
    model, prompts = example.Model(), example.prompts()
    a, b = (example.speculative(model, prompts, 6, sample=True) for _ in range(2))
    assert a == b and all(0 <= x < example.VOCAB for t in a for x in t)
    assert bsf8.device_status() == 0
