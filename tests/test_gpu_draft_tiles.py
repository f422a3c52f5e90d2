"""Attention for trees whose K/V heads have so many rows that tiles of 128 or 256 take them (test_draft_tiles_host.py asks the
library's plan for every batch here): what a row sees, in every form of that kernel.  The bounds are those of
test_gpu_serve8.py and test_gpu_serve8_scales.py, which hold for any set of tokens that a row sees."""
import numpy as np
import pytest
import torch

from draft_tiles import CASES, attend, sights
from oracle import draft as od
from oracle import serve8
from test_gpu_draft import _attend, _trees
from test_gpu_serve8 import HALF, TYPES, Batch, _values

pytestmark = pytest.mark.gpu


def _check(b, q, xt, q_heads, scale, mask, window, pos, got, rows=None):
    """rows: those to look at (None: all).  The error of weights under f16's range goes by the row's own largest weight times its V
    scale, as in test_gpu_serve8_scales.py, and that of results under the type's smallest normal value by its step."""
    o, mean, reach, peak = (x.cpu().numpy() for x in attend(b, q, scale, mask, window, pos, "cuda"))
    u, n, D = 2.0 ** -24, b.max_kv, b.D
    ds = ((D + 10) * u + (2.0 ** -22 if xt == "f32" else 0.0)) * reach + 2.0 ** -22
    step = torch.finfo(TYPES[xt]).smallest_normal * torch.finfo(TYPES[xt]).eps / 2
    tol = 2 * ds * mean + (2.0 ** -22 if xt == "f32" else 2.0 ** -11) * mean + n * 2.0 ** -34 * 127 * peak + \
        2 * (n + 16) * u * mean + HALF[xt] * np.abs(o) + step
    rows = np.ones(b.T, bool) if rows is None else rows
    err, tol = np.abs(got.double().cpu().numpy() - o)[rows], tol[rows]
    print(f"attend: worst error / tolerance {np.max(err / tol):.3f}", flush=True)
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


def _batch(name, seed, window=None):
    """A case's batch with masks of no order, before it is uploaded."""
    lens, heads, q_heads, dim, page, w, xt, _ = CASES[name]
    b = Batch(lens, heads, dim, page, seed)
    mask = b.rng.integers(0, 1 << 32, (b.T, -(-b.max_new // 32)), dtype=np.uint64).astype(np.uint32)
    mask &= b.rng.integers(0, 1 << 32, mask.shape, dtype=np.uint64).astype(np.uint32)
    pos = b.rng.integers(-100, b.max_kv + 100, b.T).astype(np.int32)
    return b, mask, pos, _values(b.rng, (b.T, q_heads, dim), xt).cuda(), q_heads, w if window is None else window, xt


SOME = ["pairs", "pairs, long window", "one tile a head", "wide", "wide, odd group", "f32", "f32, heads of 256", "heads of 192"]


@pytest.mark.parametrize("name", SOME)
def test_bad_pages_and_lengths(name):
    print(f"tree tiles, bad pages: {name}", flush=True)
    b, mask, pos, q, q_heads, window, xt = _batch(name, 50)
    for s, width in enumerate((b.table >= 0).sum(1)):
        b.table[s, b.rng.permutation(width)[:max(1, width // 4)]] = (-1, b.P, 2 ** 31 - 1, -2 ** 31)[s % 4]
    bad = [1] if len(b.kv_len) < 5 else [1, 4]
    b.kv_len[bad[0]] = b.max_kv + 1
    if len(bad) > 1:
        b.kv_len[bad[1]] = b.rows[5] - b.rows[4] - 1
    b.upload()
    got = _attend(b, q, q_heads, 0.1, mask, window, pos)
    rows = np.zeros(b.T, bool)
    for r0, n, _ in b.spans():
        rows[r0:r0 + n] = True
    assert rows.any() and not rows.all()
    assert torch.all(got[torch.from_numpy(~rows).cuda()] == 9)
    _check(b, q, xt, q_heads, 0.1, mask, window, pos, got, rows)


@pytest.mark.parametrize("name", SOME)
def test_hidden_nan(name):
    """Scales that are not finite, among the earlier tokens and the batch's, reach the rows that see their blocks and no other
    (of every second sequence)."""
    print(f"tree tiles, hidden NaN: {name}", flush=True)
    window = 40
    b, mask, pos, q, q_heads, window, xt = _batch(name, 51, window)
    mask[::2] &= np.uint32(0xffff)                          # half of the rows see 16 of each 32
    odd = []
    for s, (r0, n, total) in enumerate(b.spans()):
        for j in {0, max(0, total - n - 30), total - n, total - 1} if n and s % 2 == 0 else ():
            p, o = serve8.place(b.table, b.page, b.P, s, j)
            odd.append((s, j // 16, p, o // 16))
    plain = [x.copy() for x in (b.ks, b.vs)]
    for i, (_, _, p, o) in enumerate(odd):
        (b.ks, b.vs)[i % 2][p, :, o] = (np.nan, np.inf, -np.inf)[i % 3]
    b.upload()
    b.ks, b.vs = plain
    got = _attend(b, q, q_heads, 0.1, mask, window, pos)
    sees = np.zeros(b.T, bool)
    for s, r0, seen in sights(b, mask, window, pos):
        for blk in {k for t, k, _, _ in odd if t == s}:
            sees[r0:r0 + len(seen)] |= seen[:, 16 * blk:16 * blk + 16].any(1)
    assert sees.any() and not sees.all()
    assert torch.isnan(got[torch.from_numpy(sees).cuda()]).all()
    _check(b, q, xt, q_heads, 0.1, mask, window, pos, got, ~sees)


@pytest.mark.parametrize("name", SOME)
def test_far_scales(name):
    """V scales of 0 and far from the others', among the earlier tokens and the batch's: each row keeps the precision of what it sees."""
    print(f"tree tiles, far scales: {name}", flush=True)
    b, mask, pos, q, q_heads, window, xt = _batch(name, 52, 60)
    at = b.rng.random((b.P, 1, b.page // 16))
    b.vs = np.where(at < 0.2, 0, np.where(at < 0.3, b.vs * 2.0 ** -60, np.where(at < 0.33, -b.vs, b.vs))).astype(np.float32)
    if xt == "f32":
        b.vs = np.where((at > 0.33) & (at < 0.36), b.vs * 2.0 ** 35, b.vs).astype(np.float32)
    b.ks = np.where(b.rng.random(b.ks.shape) < 0.1, -b.ks, b.ks).astype(np.float32)
    b.upload()
    got = _attend(b, q, q_heads, 0.1, mask, window, pos)
    _check(b, q, xt, q_heads, 0.1, mask, window, pos, got)
