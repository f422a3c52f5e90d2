"""Attention for trees whose K/V heads have so many rows that tiles of 128 or 256 take them (test_draft_tiles_host.py asks the
library's plan for every batch here): what a row sees, in every form of that kernel.  The bounds are those of
test_gpu_serve8.py, which hold for any set of tokens that a row sees."""
import numpy as np
import pytest
import torch

from draft_tiles import CASES, attend
from oracle import draft as od
from test_gpu_draft import _attend, _trees
from test_gpu_serve8 import HALF, Batch, _values

pytestmark = pytest.mark.gpu


def _check(b, q, xt, q_heads, scale, mask, window, pos, got):
    o, mean, reach = (x.cpu().numpy() for x in attend(b, q, scale, mask, window, pos, "cuda"))
    u, n, D = 2.0 ** -24, b.max_kv, b.D
    ds = ((D + 10) * u + (2.0 ** -22 if xt == "f32" else 0.0)) * reach + 2.0 ** -22
    tol = 2 * ds * mean + (2.0 ** -22 if xt == "f32" else 2.0 ** -11) * mean + \
        n * 2.0 ** -34 * 254 * np.abs(b.vs).max() + 2 * (n + 16) * u * mean + HALF[xt] * np.abs(o)
    err = np.abs(got.double().cpu().numpy() - o)
    print(f"attend: worst error / tolerance {np.max(err / np.maximum(tol, 1e-300)):.3f}", flush=True)
    bad = ~(err <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
@pytest.mark.parametrize("name", list(CASES))
def test_attend(name, kind):
    """Trees and chains, often deeper than the window, and masks of no order: rows that see nothing of the batch's, or nothing at
    all, bits past the sequence's rows, positions anywhere."""
    lens, heads, q_heads, dim, page, window, xt, _ = CASES[name]
    print(f"tree tiles {name} {kind}: {len(lens)} sequences {CASES[name][1:]}", flush=True)
    b = Batch(lens, heads, dim, page, len(name)).upload()
    words = min(32, -(-b.max_new // 32) + len(name) % 3)
    if kind == "any":
        mask = b.rng.integers(0, 1 << 32, (b.T, words), dtype=np.uint64).astype(np.uint32)
        mask[::3] = 0
        pos = b.rng.integers(-100, b.max_kv + 100, b.T).astype(np.int32)
    else:
        par = np.concatenate([_trees(b.rng, n, 1 if kind == "chain" else 9) for n, _ in lens if n]).astype(np.int32)
        mask, pos = od.plan(par, b.spans(), words, 0, b.T)
    q = _values(b.rng, (b.T, q_heads, dim), xt).cuda()
    scale = dim ** -0.5
    got = _attend(b, q, q_heads, scale, mask, window, pos if window else None)
    _check(b, q, xt, q_heads, scale, mask, window, pos, got)
    assert torch.equal(got, _attend(b, q, q_heads, scale, mask, window, pos))



@pytest.mark.parametrize("heads,group,dim,window,xt", [(2, 4, 128, 0, "bf16"), (1, 64, 64, 700, "f16"), (3, 7, 96, 0, "f32"),
                                                       (1, 2, 256, 33, "f32"), (8, 1, 192, 2000, "bf16"), (2, 65, 128, 0, "f16")])
def test_single_rows(heads, group, dim, window, xt):
    """Trees of no more than one row a sequence, that see themselves or not, over histories of any length."""
    print(f"tree single rows heads={heads} group={group} dim={dim} window={window} {xt}", flush=True)
    b = Batch([(1, 5000), (1, 1), (0, 9), (1, 300), (1, 64), (1, 1025)], heads, dim, 32, heads).upload()
    mask = np.array([[1], [0], [0xffffffff], [0xfffffffe], [1]], np.uint32)
    pos = np.array([5000, -3, 10, 63, 2 ** 31 - 1], np.int32)
    q = _values(b.rng, (b.T, heads * group, dim), xt).cuda()
    got = _attend(b, q, heads * group, 0.1, mask, window, pos if window else None)
    _check(b, q, xt, heads * group, 0.1, mask, window, pos, got)
    assert torch.all(got[1] == 0)
