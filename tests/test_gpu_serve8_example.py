"""The example that serves in 8 bits: steps replayed from a captured graph make the tokens that eager calls make,
whatever ran between them, and prompts read in one batch give what they give alone."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_int8.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("serve_int8", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_graph_and_eager_steps_agree(example):
    print("example: graph and eager steps", flush=True)
    model = example.Model(2, 256, 4, 2, 64, 500, 3, 200)
    lengths = [1, 37, 130]
    eager, *_ = example.serve(model, lengths, 20, graph=False)
    graph, *_ = example.serve(model, lengths, 20, graph=True)
    assert eager.shape == (21, 3)
    assert torch.equal(eager, graph)
    again, *_ = example.serve(model, lengths, 20, graph=True)
    assert torch.equal(graph, again)
    assert len(set(eager.flatten().tolist())) > 5                     # tokens that differ


def test_a_prompt_alone_and_in_a_batch(example):
    """Every operator takes each token and sequence by itself, so company changes no bit."""
    print("example: alone and in a batch", flush=True)
    lengths = [20, 5, 64]
    many = example.Model(1, 256, 4, 1, 128, 300, 3, 100)
    one = example.Model(1, 256, 4, 1, 128, 300, 1, 100)
    for a, b in zip(many.layers[0][1:], one.layers[0][1:]):
        b.codes, b.scales = a.codes, a.scales
    one.embed, one.head = many.embed, many.head
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    prompt = torch.randint(300, (sum(lengths),), device="cuda", generator=gen)
    together = example.serve(many, lengths, 0)[0][0]
    rows = torch.tensor([0, lengths[0]], dtype=torch.int32, device="cuda")
    seqs = example.qg.kv8_seqs(one.table, rows, rows[1:].clone(), lengths[0], lengths[0], 100)
    alone = one(prompt[:lengths[0]], seqs, rows[1:].long() - 1, one.workspace(seqs))
    assert int(alone[0]) == int(together[0])
