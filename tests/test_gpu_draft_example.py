"""The example that serves with drafted tokens: steps replayed from a captured graph make the tokens that eager calls make, and
drafts that come true make several a step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_draft.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("serve_draft", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("temperature", [0.0, 0.4])
def test_graph_and_eager_steps_agree(example, temperature):
    print(f"draft example: graph and eager steps at {temperature}", flush=True)
    model = example.DraftModel(2, 256, 4, 2, 64, 500, 3, 200)
    lengths = [1, 37, 130]
    eager, steps, _ = example.serve(model, lengths, 30, temperature, graph=False)
    graph, again, _ = example.serve(model, lengths, 30, temperature, graph=True)
    assert eager == graph and steps == again
    assert all(0 <= t < 500 for line in eager for t in line)
    assert all(len(line) >= steps + 1 for line in eager)      # a token a step at least


def test_drafts_that_come_true(example):
    """Without layers a token is followed by the same one every time, so greedy lines end in a cycle, which drafts foretell."""
    print("draft example: drafts that come true", flush=True)
    model = example.DraftModel(0, 256, 4, 2, 64, 50, 2, 400)
    model.layers = example.DraftModel(1, 256, 4, 2, 64, 50, 2, 400).layers
    for layer in model.layers:
        for m in layer[1:]:
            m.codes.zero_()
    out, steps, _ = example.serve(model, [5, 9], 200)
    assert steps < 120
    follows = {}
    for line in out:
        for a, b in zip(line, line[1:]):
            assert follows.setdefault(a, b) == b
