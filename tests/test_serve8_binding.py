"""CPU checks of the 8-bit serving operators' binding and example: what they refuse, what they size.  Nothing here
launches a kernel."""
import importlib.util
import os

import pytest
import torch

import block_quantized_weight_affine_amd as qg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("codes", [torch.uint8, torch.bool, torch.float8_e4m3fn, torch.float8_e5m2, torch.int16])
def test_w8a8_takes_int8_codes_only(codes):
    w, ws, x, y = torch.zeros(16, 32, dtype=codes), torch.ones(16), torch.zeros(1, 32), torch.zeros(1, 16)
    with pytest.raises(qg.QGError) as e:
        qg.qgemm_w8a8(w, ws, x, y, 16, 32, 1, stream=0)
    assert e.value.status == qg.QG_EINVAL


@pytest.mark.parametrize("scales", [torch.int32, torch.float64, torch.float16, torch.bfloat16])
def test_w8a8_takes_f32_scales_only(scales):
    w, ws, x, y = torch.zeros(16, 32, dtype=torch.int8), torch.ones(32).to(scales), torch.zeros(1, 32), torch.zeros(1, 16)
    with pytest.raises(qg.QGError) as e:
        qg.qgemm_w8a8(w, ws, x, y, 16, 32, 1, stream=0)
    assert e.value.status == qg.QG_EINVAL


@pytest.mark.parametrize("vocab,hidden,users,lengths", [(2048, 4096, 256, [2] + [1] * 255),
                                                        (500, 256, 3, [1, 37, 130])])
def test_the_example_sizes_every_call(monkeypatch, vocab, hidden, users, lengths):
    """Its buffer holds what each product needs for the rows that it gets: all tokens, or one a user at the head."""
    spec = importlib.util.spec_from_file_location("serve_int8", os.path.join(ROOT, "examples", "serve_int8.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)

    def linear(N, K):
        m = example.Linear.__new__(example.Linear)
        m.N, m.K = N, K
        return m

    model = example.Model.__new__(example.Model)
    model.users, model.q_heads = users, hidden // 64
    cache = qg.kv8_cache(*qg.kv8_pages(4, 64, 2, 64, device="cpu"), 64, 2, 64)
    products = [linear(hidden + 256, hidden), linear(hidden, hidden), linear(8 * hidden, hidden), linear(hidden, 4 * hidden)]
    model.layers, model.head = [(cache, *products)], linear(vocab, hidden)
    ints = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    seqs = qg.kv8_seqs(ints(users, 4), ints(users + 1), ints(users), sum(lengths), max(lengths), 200)
    monkeypatch.setattr(example.torch, "empty", lambda n, **kw: n)
    size = model.workspace(seqs)
    assert size >= qg.qg_attn_kv8_workspace(cache, seqs, model.q_heads)
    assert size >= max(qg.qgemm_w8a8_workspace(m.N, m.K, seqs.T) for m in products)
    assert size >= qg.qgemm_w8a8_workspace(vocab, hidden, users)


@pytest.mark.parametrize("missing", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",)])
def test_the_current_stream_without_torch_internals(monkeypatch, missing):
    """A torch that lacks the calls behind the current stream's address still gives it, by its public ones."""
    class Stream:
        cuda_stream = 4096
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 4096 if device == 3 else 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    monkeypatch.setattr(qg, "_raw_stream", None)
    assert qg._stream(None) == 4096
    assert qg._stream(None) == 4096
    assert qg._stream(17) == 17 and qg._stream(Stream()) == 4096
