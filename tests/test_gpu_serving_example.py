"""GPU: the operators around a decode step together, as examples/batched_serving.py runs them."""
import importlib.util
import os

import pytest
import torch

import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(bsf8_lib):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "batched_serving.py")
    spec = importlib.util.spec_from_file_location("batched_serving", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_requests_do_not_touch_each_other(example):
    """A request's answer is the same alone as in a batch whose rows and pages are handed on: the logits of the two differ
    by roundings only (other chunks share the launches, none the sums), the greedy tokens not at all unless two logits
    are as close as those."""
    model, asked = example.Model(), example.prompts(6)
    together = example.serve(model, asked, 5, keep=0)
    assert all(len(t) == 5 for t in together)
    for p, t in list(zip(asked, together))[::2]:
        assert example.serve(model, [p], 5, keep=0)[0] == t
    assert bsf8.device_status() == 0


def test_all_pages_kept_is_attention_over_the_whole(example):
    model, asked = example.Model(), example.prompts(5, seed=7)
    whole = example.serve(model, asked, 4, keep=0)
    assert example.serve(model, asked, 4, keep=example.LONGEST // example.PAGE) == whole
    assert bsf8.device_status() == 0


def test_few_pages_and_drawn_tokens_run(example):
    model, asked = example.Model(), example.prompts(7, seed=9)
    a, b = (example.serve(model, asked, 4, keep=3, temperature=0.8) for _ in range(2))
    assert a == b and all(0 <= x < example.VOCAB for t in a for x in t)
    assert bsf8.device_status() == 0


def test_a_pool_that_is_too_small_lets_requests_wait(example):
    """Two rows of 32-token pages for one prompt: the second request is read once the first one's pages are back."""
    model = example.Model()
    server = example.Server(model, 0)
    server.book = bsf8.PageBook.empty(example.ROWS, example.LONGEST // example.PAGE, 3)
    u = torch.zeros(example.ROWS, device="cuda")
    a, b = [list(range(60)), list(range(100, 150))]
    got, _ = server.step([a, b, [], []], [False] * 4, u)
    assert got == [60, 0, 0, 0]
    got, _ = server.step([[5], b, [], []], [False] * 4, u)
    assert got == [1, 0, 0, 0]
    got, _ = server.step([[], b, [], []], [True, False, False, False], u)
    assert got == [0, 50, 0, 0] and server.book.count.tolist() == [1]
    assert bsf8.device_status() == 0
