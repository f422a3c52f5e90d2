"""Attention over the 8-bit cache where scales are extreme: each row keeps the precision of what it sees itself.

Tolerance, per element, with u = 2^-24, n tokens and half-steps h as in test_gpu_serve8.py:
  scores, weights' rounding, sums, output: 2 ds mean + (2^-11 or 2^-22) mean + 2 (n + 16) u mean + h |o| as there, all
      of the row's own weighted mean of |v|;
  weights under f16's range: an error of 2^-25 where the largest weight times its V scale stands at 2^9 or above, so
      n 2^-34 127 peak with peak the row's largest (weight / sum of weights) * |V scale|;
  results under the type's smallest normal value: half its smallest step."""
import numpy as np
import pytest
import torch

from oracle import serve8
from test_gpu_serve8 import HALF, TYPES, Batch, _attend, _values

pytestmark = pytest.mark.gpu


def _reference(b, q, scale, causal, window):
    """o, mean, reach and peak of every row and head in f64 (NaN where a row sees a scale that is not finite)."""
    T, QH, D = q.shape
    G = QH // b.H
    o, mean, reach, peak = (np.full(s, np.nan) for s in (q.shape, q.shape, (T, QH, 1), (T, QH, 1)))
    for s, (r0, n, total) in enumerate(b.spans()):
        if not n:
            continue
        j = np.arange(total)
        page, off = b.table[s][j // b.page], j % b.page
        for h in range(b.H):
            kd, vd = (x[page, h, off // 16].astype(np.float64) for x in (b.ks, b.vs))
            with np.errstate(invalid="ignore"):
                k = b.kc[page, h, off].astype(np.float64) * kd[:, None]
                v = b.vc[page, h, off].astype(np.float64) * vd[:, None]
            for i in range(n):
                pos = total - n + i
                seen = (j <= pos if causal else j >= 0) & (j > pos - window if window else j >= 0)
                if not (np.isfinite(kd[seen]).all() and np.isfinite(vd[seen]).all()):
                    continue
                x = q[r0 + i, h * G:(h + 1) * G].T
                sc = (k[seen] @ x) * scale
                w = np.exp(sc - sc.max(0))
                w /= w.sum(0)
                at = (r0 + i, slice(h * G, (h + 1) * G))
                o[at] = w.T @ v[seen]
                mean[at] = w.T @ np.abs(v[seen])
                reach[at] = abs(scale) * (np.abs(k[seen]) @ np.abs(x)).max(0)[:, None]
                peak[at] = (w * np.abs(vd[seen])[:, None]).max(0)[:, None]
    return o, mean, reach, peak


def _check(b, q, xt, scale, causal, window, got, rows=None):
    """Compares rows (of T; all that the reference gives) and returns them."""
    o, mean, reach, peak = _reference(b, q.double().cpu().numpy(), scale, causal, window)
    u, n, D = 2.0 ** -24, b.max_kv, b.D
    two = xt == "f32"
    ds = ((D + 10) * u + (2.0 ** -22 if two else 0)) * reach + 2.0 ** -22
    step = torch.finfo(TYPES[xt]).smallest_normal * torch.finfo(TYPES[xt]).eps / 2
    tol = 2 * ds * mean + (2.0 ** -22 if two else 2.0 ** -11) * mean + n * 2.0 ** -34 * 127 * peak + \
        2 * (n + 16) * u * mean + HALF[xt] * np.abs(o) + step
    if rows is None:
        rows = ~np.isnan(o).any((1, 2))
    assert rows.any()
    err = np.abs(got.double().cpu().numpy() - o)[rows]
    print(f"worst error / tolerance {np.max(np.nan_to_num(err, nan=np.inf) / tol[rows]):.3f}", flush=True)
    bad = ~(err <= tol[rows])
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5], tol[rows][bad][:5], o[rows][bad][:5])
    return rows


def _set_v(b, s, lo, hi, f):
    """Applies f to the V scales of the blocks of tokens lo..hi-1 of sequence s (lo a multiple of 16)."""
    for j in range(lo, hi, 16):
        p, o = serve8.place(b.table, b.page, b.P, s, j)
        b.vs[p, :, o // 16] = f(b.vs[p, :, o // 16])


# (rows, tokens): rows kernel in one launch and in splits, tile kernel in few and in many splits
FORMS = [(1, 900), (5, 5000), (150, 900), (90, 5000)]
ONE = (150, 250)                                       # a tile in one launch


@pytest.mark.parametrize("new", [5, 40, 150])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [np.inf, -np.inf])
@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_an_infinite_scale_makes_rows_nan(new, which, value, xt):
    """The block of the last tokens has an infinite scale; its codes and q give products of one sign, so that every
    score is -inf for one sign of a K scale."""
    print(f"infinite {which} {value} new={new} {xt}", flush=True)
    for codes in (1, -1):
        b = Batch([(new, 333)], 1, 128, 32, 41)
        q = _values(b.rng, (b.T, 4, 128), xt).abs().cuda()
        p, off = serve8.place(b.table, 32, b.P, 0, 320)
        b.kc[p, :, off:off + 16] = codes * (np.abs(b.kc[p, :, off:off + 16]) | 1)
        (b.ks if which == "k" else b.vs)[p, :, off // 16] = value
        got = _attend(b.upload(), q, 4, 0.09, True, 0)
        before = max(0, new - 13)
        assert torch.all(torch.isnan(got[before:]))
        if before:
            rows = _check(b, q, xt, 0.09, True, 0, got)
            assert np.array_equal(rows, np.arange(b.T) < before)


@pytest.mark.parametrize("new,total", FORMS + [ONE])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_values_near_the_largest(new, total, xt):
    """V up to 2^125, all of one sign, weights alike: the sums before the division would pass the largest f32."""
    print(f"large values new={new} total={total} {xt}", flush=True)
    b = Batch([(new, total)], 2, 64, 48, 42)
    b.vc = np.abs(b.vc) | 1
    b.vs *= np.float32(2.0 ** 123)
    b.upload()
    q = (_values(b.rng, (b.T, 4, 64), xt) / 16).cuda()
    got = _attend(b, q, 4, 0.125, True, 0)
    _check(b, q, xt, 0.125, True, 0, got)


@pytest.mark.parametrize("new,total", FORMS)
@pytest.mark.parametrize("size", [1.0, 1e-5, 1e-7])
@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
def test_blocks_of_zeros_before_small_values(new, total, size, xt):
    """All V before the last 250 tokens are zero, those of the last small: the weights of the zeros belong to the
    denominator and to nothing else."""
    if xt == "f16":
        size *= 64                                     # results stay in f16's normal range
    print(f"zeros new={new} total={total} {size} {xt}", flush=True)
    b = Batch([(new, total)], 2, 128, 32, 43)
    b.vs *= np.float32(size)
    _set_v(b, 0, 0, total - 250, lambda x: 0)
    b.upload()
    q = _values(b.rng, (b.T, 8, 128), xt).cuda()
    got = _attend(b, q, 8, 0.09, True, 0)
    _check(b, q, xt, 0.09, True, 0, got)


@pytest.mark.parametrize("new,total,at", [(n, t, at) for n, t in FORMS for at in (0, 416, 640)] + [ONE + (0,), ONE + (64,)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_a_block_of_zeros_that_has_the_weight(new, total, at, xt):
    """A block of V zeros scores some 20 above the rest: the result is small, and as precise as any."""
    print(f"zero block with the weight at={at} new={new} total={total} {xt}", flush=True)
    b = Batch([(new, total)], 1, 64, 16, 44)
    p, _ = serve8.place(b.table, 16, b.P, 0, at)
    b.kc[p] = 100
    b.ks[p] = 0.06
    b.vs[p] = 0
    b.upload()
    q = (_values(b.rng, (b.T, 2, 64), "f32") / 16 + 0.4).to(TYPES[xt]).cuda()
    got = _attend(b, q, 2, 0.125, True, 0)
    _check(b, q, xt, 0.125, True, 0, got)


def test_only_zeros():
    """Rows that see nothing but V zeros are zero, beside rows that see more."""
    for new, total in FORMS:
        print(f"only zeros new={new} total={total}", flush=True)
        b = Batch([(new, total)], 1, 64, 16, 45)
        b.vs[:] = 0
        b.ks[::2] = 0
        _set_v(b, 0, (total - 1) // 16 * 16, total, lambda x: 0.01)
        q = _values(b.rng, (b.T, 2, 64), "f32").cuda()
        got = _attend(b.upload(), q, 2, 0.125, True, 0)
        _check(b, q, "f32", 0.125, True, 0, got)
        first = new - ((total - 1) % 16 + 1)           # rows before the last block
        if first > 0:
            assert torch.all(got[:first] == 0)


@pytest.mark.parametrize("new,total", [(5, 370), (30, 370), (5, 5042), (150, 370), (90, 5042), (150, 178)])
@pytest.mark.parametrize("far", [20, 60, 120, 126])
@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
def test_a_hidden_block_of_another_size(new, total, far, xt):
    """The last two tokens have V scales of 2^far times the others', which causality hides from the rows before them."""
    print(f"hidden far={far} new={new} total={total} {xt}", flush=True)
    b = Batch([(new, total)], 2, 64, 16, 46)
    last = total // 16 * 16
    assert total - last == 2
    _set_v(b, 0, last, total, lambda x: np.float32(2.0 ** (far - 7)))
    b.upload()
    q = _values(b.rng, (b.T, 4, 64), xt).cuda()
    got = _attend(b, q, 4, 0.125, True, 0)
    _check(b, q, xt, 0.125, True, 0, got, np.arange(b.T) < new - 2)
    if far <= 60 and xt != "f16":                      # f16 has no such values
        _check(b, q, xt, 0.125, True, 0, got)


@pytest.mark.parametrize("new,total", FORMS)
@pytest.mark.parametrize("power", [-90, -40, 40, 90])
def test_later_blocks_of_another_size(new, total, power):
    """V scales 2^power apart between the first tokens and the last, all of them seen."""
    print(f"later blocks 2^{power} new={new} total={total}", flush=True)
    for xt in ("bf16", "f32"):
        b = Batch([(new, total)], 2, 64, 48, 47)
        _set_v(b, 0, (total - 280) // 16 * 16, total, lambda x: x * np.float32(2.0 ** power))
        b.upload()
        q = _values(b.rng, (b.T, 4, 64), xt).cuda()
        got = _attend(b, q, 4, 0.125, True, 0)
        _check(b, q, xt, 0.125, True, 0, got)


@pytest.mark.parametrize("new", [1, 6, 100])
@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
def test_heads_and_sequences_of_different_sizes(new, xt):
    """Heads and sequences whose V scales lie far below the cache's largest are as precise as the others."""
    print(f"heads of different sizes new={new} {xt}", flush=True)
    b = Batch([(new, 400), (new, 1100), (new, 130)], 3, 64, 32, 48)
    b.vs[:, 1] *= np.float32(2.0 ** -10)
    b.vs[:, 2] *= np.float32(2.0 ** (-12 if xt == "f16" else -70))
    if xt != "f16":
        _set_v(b, 1, 0, 1100, lambda x: x * np.float32(2.0 ** -30))
    unused = sorted(set(range(b.P)) - set(b.table.reshape(-1).tolist()))
    b.vs[unused] = np.float32(2.0 ** 90)
    b.upload()
    q = _values(b.rng, (b.T, 6, 64), xt).cuda()
    got = _attend(b, q, 6, 0.125, True, 0)
    _check(b, q, xt, 0.125, True, 0, got)


@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_tall_tiles(xt):
    """Tiles of 256 rows: V zeros under the first tokens, the last two of 2^120 times the others' size and hidden from the
    rows before them."""
    print(f"tall tiles {xt}", flush=True)
    b = Batch([(64, 194)] + [(i % 4, 20 + i % 4) for i in range(63)], 4, 64, 32, 49)
    _set_v(b, 0, 0, 64, lambda x: 0)
    _set_v(b, 0, 192, 194, lambda x: np.float32(2.0 ** 113))
    b.upload()
    q = _values(b.rng, (b.T, 16, 64), xt).cuda()
    got = _attend(b, q, 16, 0.125, True, 0)
    _check(b, q, xt, 0.125, True, 0, got, (np.arange(b.T) < 62) | (np.arange(b.T) >= 64))
