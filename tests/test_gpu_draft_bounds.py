"""Verification of drafted tokens where a batch's numbers contradict each other: nothing outside of the outputs is written."""
import numpy as np
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import draft as od
from test_gpu_serve8 import _dev

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
