"""Verification of drafted tokens at its bounds, and where a batch's numbers contradict each other: nothing outside of the outputs is
written."""
import numpy as np
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import draft as od
from test_gpu_draft import _check_verify
from test_gpu_serve8 import Batch, _dev

pytestmark = pytest.mark.gpu


def _guarded(n, room=4096):
    """(the n values of an output, all that lies around them)."""
    t = torch.full((n + 2 * room,), -9, dtype=torch.int32, device="cuda")
    return t[room:room + n], torch.cat([torch.arange(room), torch.arange(n + room, n + 2 * room)]).cuda(), t


@pytest.mark.parametrize("kind", ["chains", "drawn", "trees", "large trees"])
def test_rows_that_overlap(kind):
    """Sequences that share rows could have more rows that stay than the batch has: path holds the batch's many."""
    n, vocab = (700, 30000) if kind == "large trees" else (7, 500)
    rows = np.array([0, n, 0, n, 0, n, n + 2], np.int32)
    print(f"verify rows that overlap: {kind}", flush=True)
    seqs_n, T = len(rows) - 1, n + 2
    kv = np.full(seqs_n, 5000, np.int32)
    rng = np.random.default_rng(n)
    target = torch.from_numpy(4 * rng.normal(size=(T, vocab)).astype(np.float32)).cuda()
    best = target.argmax(1).cpu().numpy()
    par = np.arange(-1, T - 1).astype(np.int32)
    par[n:] = (-1, 0)
    tokens = np.zeros(T, np.int32)
    tokens[1:n], tokens[n + 1] = best[:n - 1], best[n]       # every row of the overlapping ones stays
    seqs = qg.kv8_seqs(torch.zeros(seqs_n, 1, dtype=torch.int32, device="cuda"), _dev(rows), _dev(kv), T, n, 5000)
    outs = [_guarded(m) for m in (seqs_n, seqs_n, seqs_n + 1, T, seqs_n)]
    size = qg.qg_draft_verify_workspace(seqs, vocab)
    work = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    kw = {}
    if kind == "drawn":
        kw = dict(draft=target.clone(), accept=torch.zeros(T, device="cuda"), sample=torch.full((T,), 0.5, device="cuda"))
    elif kind != "chains":
        kw = dict(parents=_dev(par))
    qg.qg_draft_verify(seqs, _dev(tokens), target, *(o[0] for o in outs), workspace=work[:size], **kw)
    torch.cuda.synchronize()
    assert torch.all(work[size:] == 255)
    for _, around, t in outs:
        assert torch.all(t[around] == -9)
    accepted, nxt, rows_out, path, kv_out = (o[0].cpu().numpy() for o in outs)
    assert rows_out.max() <= T and rows_out[0] == 0
    # the last sequence overlaps no other
    plain = {k: v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for k, v in kw.items()}
    sp = [(0, 0, 0)] * (seqs_n - 1) + [(n, 2, 5000)]
    want = od.verify(sp, kv, T, tokens, target.double().cpu().numpy(), **plain)
    assert (accepted[-1], nxt[-1], kv_out[-1]) == (want[0][-1], want[1][-1], want[4][-1])
    assert accepted[1] == 0 and nxt[1] == -1                 # rows that go back


@pytest.mark.parametrize("kind", ["chosen", "drawn", "none"])
def test_the_largest_vocabulary(kind):
    print(f"verify the largest vocabulary: {kind}", flush=True)
    vocab, T = 1 << 24, 3
    target = torch.randn(T, vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).mul_(3).half()
    target[:, -1] = 16.0                                     # half of the mass or so
    tokens = np.array([0, vocab - 1, 12345], np.int32)
    kw = dict(sample=np.array([0.97, 0.3, 0.5], np.float32))
    if kind == "drawn":
        kw.update(draft=target.roll(1, 0), accept=np.array([0, 0.2, 0.9], np.float32))
    if kind == "none":
        kw = {}
    _check_verify(Batch([(T, 9)], 1, 64, 16, 1), tokens, target, **kw)


@pytest.mark.parametrize("drawn", [False, True])
def test_the_most_sequences(drawn):
    print(f"verify 65535 sequences, drawn {drawn}", flush=True)
    rng = np.random.default_rng(9)
    b = Batch([(1, 5)], 1, 64, 16, 1)
    n = rng.integers(0, 3, 65535)
    b.rows = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    b.kv_len = (n + rng.integers(0, 50, 65535)).astype(np.int32)
    b.T, b.max_new, b.max_kv, b.table = int(b.rows[-1]), 2, 60, np.zeros((65535, 1), np.int32)
    target = torch.from_numpy(rng.normal(size=(b.T, 9)).astype(np.float32)).cuda()
    kw = dict(sample=rng.random(b.T).astype(np.float32))
    if drawn:
        kw.update(draft=target + 0.5, accept=rng.random(b.T).astype(np.float32))
    _check_verify(b, rng.integers(0, 9, b.T), target, **kw)


@pytest.mark.parametrize("kind", ["chain", "drawn", "tree"])
def test_kv_out_over_one_sequence_s_kv_len(kind):
    """One sequence, many workgroups, which read the length that the first to end may have replaced."""
    rng = np.random.default_rng(10)
    vocab, n = 200000, 9
    b = Batch([(n, n)], 1, 64, 16, 2)                        # no earlier tokens: fewer are left than the batch has rows
    target = torch.from_numpy(4 * rng.normal(size=(n, vocab)).astype(np.float32)).cuda()
    tokens = np.zeros(n, np.int32)
    tokens[1:4] = target.argmax(1).cpu().numpy()[:3]
    par = np.arange(-1, n - 1).astype(np.int32)
    kw = dict(parents=par) if kind == "tree" else dict(draft=target.flip(0).contiguous(), accept=np.zeros(n, np.float32),
                                                       sample=np.full(n, 0.5, np.float32)) if kind == "drawn" else {}
    plain = {k: v.double().cpu().numpy() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    want = od.verify(b.spans(), b.kv_len, n, tokens, target.double().cpu().numpy(), **plain)
    kv = _dev(b.kv_len)
    seqs = qg.kv8_seqs(_dev(b.table), _dev(b.rows), kv, n, n, n)
    work = torch.empty(qg.qg_draft_verify_workspace(seqs, vocab), dtype=torch.uint8, device="cuda")
    outs = [torch.full((m,), -9, dtype=torch.int32, device="cuda") for m in (1, 1, 2, n)] + [kv]
    dev = {k: _dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    for _ in range(20):
        kv.copy_(_dev(b.kv_len))
        qg.qg_draft_verify(seqs, _dev(tokens), target, *outs, workspace=work, **dev)
        for x, y in zip(outs, want):
            assert np.array_equal(x.cpu().numpy(), y)
