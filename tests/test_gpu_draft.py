"""The operators for drafted tokens on the GPU against their plain definitions (oracle/draft.py).

Rotary positions, per element, with the magnitude m = mscale (|x_a| + |x_b|) of a turned pair: sine and cosine are off by no
more than 2^-22 + 2^-52 |angle| (qgemm.h), the factor mscale, the two products and their sum round four times (2^-24 each), the
result once to its type.
Into the cache: K as the f32 rows that qg_rope gives for the same values, coded by the plain definition: equal bit for bit.
Plans and verification: whole numbers, equal.  (Verification: both sides hold probabilities in 64 bits; a draw that lies
within 2^-45 of a border between tokens could differ.)
Attention: the bounds of test_gpu_serve8.py, which hold for any set of tokens that a row sees."""
import numpy as np
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import draft as od
from oracle import serve8
from test_gpu_serve8 import HALF, TYPES, Batch, _check_cache, _dev, _values

pytestmark = pytest.mark.gpu

ROPE = [
    # T, heads, dim, rot, interleaved, type
    (1, 1, 8, 2, False, "f32"), (1, 1, 8, 8, True, "f16"), (3, 5, 64, 64, False, "bf16"), (257, 2, 96, 24, False, "f16"),
    (33, 1, 128, 128, True, "f32"), (65, 40, 128, 128, False, "bf16"), (20, 3, 80, 32, False, "f32"),
    (7, 9, 256, 62, False, "bf16"), (7, 9, 256, 62, True, "f16"), (300, 1, 64, 16, True, "bf16"), (5, 2, 1024, 1024, False, "f16"),
    (2, 300, 64, 64, False, "f32"), (9, 4, 72, 10, False, "f32"), (40, 3, 128, 0, False, "bf16"), (11, 2, 64, 4, False, "bf16"),
]


def _rotary(rot, interleaved, mscale=1.0, base=10000.0):
    freqs = base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    return freqs, qg.rotary(_dev(freqs) if rot else None, interleaved, mscale)


@pytest.mark.parametrize("i", range(len(ROPE)))
def test_rope(i):
    T, heads, dim, rot, inter, xt = ROPE[i]
    print(f"rope case {i}: {ROPE[i]}", flush=True)
    rng = np.random.default_rng(i)
    pos = rng.integers(0, [100, 5000, 1 << 20, 1 << 24][i % 4], T).astype(np.int32)
    if T > 4:
        pos[:4] = 0, 1, -1, -(1 << 20)                  # negative positions turn back
    freqs, r = _rotary(rot, inter, 1.25)
    wide = _values(rng, (T, heads + 2, dim), xt).cuda()   # inside a fused projection
    x = wide[:, 1:heads + 1]
    before = wide.clone()
    y = torch.full((heads, T, dim), 7.0, dtype=TYPES[xt], device="cuda").transpose(0, 1)   # heads first
    qg.qg_rope(r, _dev(pos), x, y)
    want, mag = od.rope(x.double().cpu().numpy(), pos, freqs, inter, 1.25)
    angle = np.abs(pos.astype(np.float64)).max() * (freqs.max() if rot else 0.0)
    tol = mag * (2.0 ** -22 + 2.0 ** -52 * angle + 4 * 2.0 ** -24) + HALF[xt] * np.abs(want)
    err = np.abs(y.double().cpu().numpy() - want)
    print(f"rope: worst error / tolerance {np.max(err / np.maximum(tol, 1e-300)):.3f}", flush=True)
    assert np.all(err <= tol)
    assert torch.equal(wide, before)
    assert torch.equal(y[..., rot:], x[..., rot:])
    qg.qg_rope(r, _dev(pos), x, x)                       # in place
    assert torch.equal(x, y)
    before[:, 1:heads + 1] = y
    assert torch.equal(wide, before)


def test_rope_specials():
    """An infinity or NaN stays within its pair; a turn of no angle changes nothing but by mscale."""
    x = torch.ones(2, 1, 64, device="cuda")
    x[0, 0, 3], x[0, 0, 40] = float("inf"), float("nan")
    _, r = _rotary(64, False, 2.0)
    y = torch.empty_like(x)
    qg.qg_rope(r, torch.zeros(2, dtype=torch.int32, device="cuda"), x, y)
    bad = ~torch.isfinite(y)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 8, 35, 40] and not bad[1].any()
    assert torch.equal(y[1], 2 * x[1])


def _trees(rng, n, wide):
    """Parents of n rows, some of them no rows before their own."""
    par = np.array([-1] + [int(rng.integers(max(0, r - wide), r)) for r in range(1, n)], np.int32)[:n]
    return par


WRITE = [
    # lens, heads, dim, page, rot, interleaved, type, q_heads
    ([(1, 1), (1, 16), (1, 17), (1, 33), (0, 20), (1, 200)], 2, 128, 64, 128, False, "bf16", 8),
    ([(5, 5), (16, 16), (17, 30), (0, 0), (40, 41), (3, 19), (100, 260)], 3, 64, 16, 32, True, "f16", 3),
    ([(7, 40), (33, 33)], 5, 96, 48, 24, False, "f32", 10),
    ([(18, 50), (1, 9)], 1, 192, 32, 192, False, "f16", 0),
    ([(9, 25), (64, 64)], 4, 256, 256, 250, False, "f32", 4),
    ([(70, 75), (2, 3)], 6, 256, 80, 128, True, "bf16", 0),
    ([(20, 37)], 2, 128, 16, 0, False, "f32", 2),
    ([(31, 31), (1, 47)], 2, 64, 48, 64, False, "bf16", 4),
]


@pytest.mark.parametrize("how", ["plain", "pos", "src"])
@pytest.mark.parametrize("i", range(len(WRITE)))
def test_write_rope(i, how):
    lens, heads, dim, page, rot, inter, xt, q_heads = WRITE[i]
    print(f"write_rope case {i} {how}: {WRITE[i]}", flush=True)
    b = Batch(lens, heads, dim, page, 50 + i).upload()
    freqs, r = _rotary(rot, inter, 1.1)
    pos = np.concatenate([np.arange(t - n, t) for n, t in lens]).astype(np.int32)
    given = src = None
    if how == "pos":
        pos = b.rng.integers(0, 100000, b.T).astype(np.int32)
        given = _dev(pos)
    R, pick = b.T, np.arange(b.T)
    if how == "src":
        R, q_heads = 2 * b.T + 3, 0
        pick = b.rng.permutation(R)[:b.T].astype(np.int32)
        src = _dev(pick)
    fused = _values(b.rng, (R, q_heads + 2 * heads, dim), xt)
    if how == "src" and b.T > 2:
        for at, bad in ((0, -1), (2, R)):                 # rows that are none: zeros
            src[at] = bad
    dev = fused.cuda()
    q, k, v = dev.split([q_heads, heads, heads], 1)
    q_out = torch.full((b.T, q_heads, dim), 5.0, dtype=TYPES[xt], device="cuda")
    qg.qg_kv8_write_rope(b.cache, b.seqs, r, k, v, q if q_heads else None, q_out if q_heads else None, given, src)
    kf, vf = (x[torch.from_numpy(pick).long().cuda()].float() for x in (k, v))
    if how == "src" and b.T > 2:
        kf[0] = vf[0] = kf[2] = vf[2] = 0
    turned = torch.empty(kf.shape, device="cuda")
    qg.qg_rope(r, _dev(pos), kf.contiguous(), turned)
    serve8.kv8_write(b.kc, b.ks, b.table, b.spans(), turned.cpu().numpy())
    serve8.kv8_write(b.vc, b.vs, b.table, b.spans(), vf.cpu().numpy())
    _check_cache(b, None, None)
    if q_heads:
        want = torch.empty_like(q_out)
        qg.qg_rope(r, _dev(pos), q, want)
        assert torch.equal(q_out, want)
        qg.qg_kv8_write_rope(b.cache, b.seqs, r, k, v, q, q, given)
        assert torch.equal(q, want)                       # in place


@pytest.mark.parametrize("new", [1, 40])
def test_write_rope_bad_tables(new):
    """Sequences whose numbers contradict each other and pages outside of the cache are left out, q's rows with the former;
    a NaN makes its block NaN."""
    print(f"write_rope bad tables new={new}", flush=True)
    b = Batch([(new, 100), (new, 90), (new, 80)], 2, 64, 32, 4, max_kv=100)
    b.table[0, (100 - new) // 32], b.kv_len[1] = b.P, 101
    b.upload()
    _, r = _rotary(64, False)
    x = _values(b.rng, (b.T, 4, 64), "f32")
    x[2 * new, 3, 5] = float("nan")
    dev = x.cuda()
    q_out = torch.full((b.T, 2, 64), 5.0, device="cuda")
    k, v = dev[:, :2], dev[:, 2:]
    qg.qg_kv8_write_rope(b.cache, b.seqs, r, k, v, k, q_out)
    pos = np.concatenate([np.arange(t - new, t) for t in (100, 90, 80)]).astype(np.int32)
    turned = torch.empty(b.T, 2, 64, device="cuda")
    qg.qg_rope(r, _dev(pos), k, turned)
    serve8.kv8_write(b.kc, b.ks, b.table, b.spans(), turned.cpu().numpy())
    serve8.kv8_write(b.vc, b.vs, b.table, b.spans(), x[:, 2:].numpy())
    _check_cache(b, None, None)
    assert torch.all(q_out[new:2 * new] == 5)
    assert torch.equal(q_out[:new], turned[:new]) and torch.equal(q_out[2 * new:], turned[2 * new:])


@pytest.mark.parametrize("lens,words,window", [
    ([(1, 1)], 1, 0), ([(25, 1025)], 1, 0), ([(32, 40), (33, 33), (0, 9), (31, 1000)], 2, 0), ([(64, 64), (65, 100)], 7, 3),
    ([(200, 5000), (1, 2), (199, 199)], 7, 1), ([(1024, 1024), (1000, 100000)], 32, 0),
    ([(1000, 1200), (5, 9), (0, 3), (8, 8)], 32, 7), ([(255, 300), (1000, 1000), (1024, 5000)], 32, 300), ([(256, 256)] * 9, 8, 255)])
def test_plan(lens, words, window):
    print(f"plan {lens} words={words} window={window}", flush=True)
    rng = np.random.default_rng(len(lens))
    b = Batch(lens, 1, 64, 65536, 3)
    par = np.concatenate([_trees(rng, n, 1 if n == 1000 else 5) for n, _ in lens]).astype(np.int32)
    if b.T > 30:
        par[3], par[7], par[11], par[20] = -5, 7, 2 ** 31 - 1, -2 ** 31   # rows that follow the cache
    mask = torch.full((b.T + 1, words), 0x55555555, dtype=torch.int32, device="cuda")
    pos = torch.full((b.T + 1,), -7, dtype=torch.int32, device="cuda")
    seqs = qg.kv8_seqs(_dev(b.table), _dev(b.rows), _dev(b.kv_len), b.T, b.max_new, b.max_kv)
    qg.qg_tree_plan(seqs, _dev(par), mask, pos, window)
    m, p = od.plan(par, b.spans(), words, window, b.T)
    assert np.array_equal(mask[:-1].cpu().numpy().view(np.uint32), m)
    assert np.array_equal(pos[:-1].cpu().numpy(), p)
    assert pos[-1] == -7 and torch.all(mask[-1] == 0x55555555)


def test_plan_leaves_out_what_contradicts():
    rows, kv = np.array([0, 4, 9, 7, 12], np.int32), np.array([3, 9, 20, 21], np.int32)
    seqs = qg.kv8_seqs(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), _dev(rows), _dev(kv), 12, 5, 20)
    mask, pos = (torch.full((12, *n), v, dtype=torch.int32, device="cuda") for n, v in (((1,), 0x55555555), ((), -7)))
    par = np.arange(-1, 11).astype(np.int32)
    qg.qg_tree_plan(seqs, _dev(par), mask, pos)
    m, p = od.plan(par, serve8.spans(rows, kv, 12, 5, 20), 1, 0, 12)
    assert np.array_equal(mask.cpu().numpy().view(np.uint32), m) and np.array_equal(pos.cpu().numpy(), p)
    assert (p == -7).sum() == 7


def _attend(b, q, q_heads, scale, mask, window, pos, fill=9.0):
    o = torch.full(q.shape, fill, dtype=q.dtype, device="cuda")
    size = qg.qg_attn_kv8_workspace(b.cache, b.seqs, q_heads)
    guard = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")   # NaN bits: nothing may be read first
    m = _dev(mask.view(np.int32))
    qg.qg_attn_kv8_tree(b.cache, b.seqs, m, q, o, q_heads, scale, window, None if pos is None else _dev(pos), guard[:size])
    torch.cuda.synchronize()
    assert torch.all(guard[size:] == 255)
    return o


def _check_attend(b, q, xt, q_heads, scale, mask, window, pos, got, rows=None):
    o, mean, reach, _ = od.attend(b.kc, b.ks, b.vc, b.vs, b.table, b.spans(), q.double().cpu().numpy(), scale, mask, window, pos)
    u, n, D = 2.0 ** -24, b.max_kv, b.D
    ds = ((D + 10) * u + (2.0 ** -22 if xt == "f32" else 0.0)) * reach + 2.0 ** -22
    tol = 2 * ds * mean + (2.0 ** -22 if xt == "f32" else 2.0 ** -11) * mean + \
        n * 2.0 ** -34 * 254 * np.nanmax(np.abs(b.vs)) + 2 * (n + 16) * u * mean + HALF[xt] * np.abs(o)
    err = np.abs(got.double().cpu().numpy() - o)
    rows = ~np.isnan(o).any((1, 2)) if rows is None else rows
    assert rows.any()
    print(f"attend: worst error / tolerance {np.max(err[rows] / np.maximum(tol[rows], 1e-300)):.3f}", flush=True)
    bad = ~(err[rows] <= tol[rows])
    assert not bad.any(), (np.argwhere(bad)[:5], err[rows][bad][:5], tol[rows][bad][:5])


ATTEND = [
    # lens, heads, q_heads, dim, page, window, type
    ([(1, 1)], 1, 1, 64, 16, 0, "f16"),
    ([(1, 1), (2, 15), (3, 16), (4, 17), (5, 63), (6, 64), (7, 65), (8, 300)], 2, 8, 128, 64, 0, "bf16"),
    ([(9, 700), (0, 0), (15, 15)], 1, 16, 256, 32, 0, "f32"),
    ([(25, 5000), (25, 1023), (25, 1049)], 2, 14, 64, 48, 0, "f16"),
    ([(13, 4500), (16, 2049)], 1, 1, 96, 80, 1500, "f32"),
    ([(61, 61), (61, 200)], 2, 2, 128, 32, 0, "bf16"),
    ([(64, 3000), (1, 5), (40, 100)], 1, 3, 192, 64, 30, "f16"),
    ([(70, 300), (33, 33)], 1, 3, 128, 64, 40, "bf16"),
    ([(130, 130), (129, 400)], 2, 2, 128, 128, 0, "bf16"),
    ([(200, 260)], 1, 5, 256, 256, 1, "f32"),
    ([(150, 2300)], 1, 7, 192, 32, 700, "bf16"),
    ([(257, 1257)], 2, 16, 64, 16, 0, "f32"),
    ([(60, 9000)], 1, 8, 128, 64, 5000, "f16"),
    ([(37, 700), (50, 63)], 2, 6, 96, 16, 0, "f32"),
    ([(1000, 1100)], 1, 1, 64, 64, 0, "f16"),
]


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attend(i, kind):
    """Trees, and masks of no order: rows that see none of the batch's, bits past the sequence's rows, positions anywhere."""
    lens, heads, q_heads, dim, page, window, xt = ATTEND[i]
    print(f"tree attend case {i} {kind}: {ATTEND[i]}", flush=True)
    b = Batch(lens, heads, dim, page, 200 + i).upload()
    words = min(32, -(-b.max_new // 32) + i % 3)
    if kind == "tree":
        par = np.concatenate([_trees(b.rng, n, 4) for n, _ in lens if n]).astype(np.int32)
        mask, pos = od.plan(par, b.spans(), words, 0, b.T)
    else:
        mask = b.rng.integers(0, 1 << 32, (b.T, words), dtype=np.uint64).astype(np.uint32)
        mask[::3] = 0
        pos = b.rng.integers(-100, b.max_kv + 100, b.T).astype(np.int32)
    q = _values(b.rng, (b.T, q_heads, dim), xt).cuda()
    scale = dim ** -0.5
    got = _attend(b, q, q_heads, scale, mask, window, pos if window else None)
    _check_attend(b, q, xt, q_heads, scale, mask, window, pos, got)
    assert torch.equal(got, _attend(b, q, q_heads, scale, mask, window, pos))


@pytest.mark.parametrize("new,xt", [(6, "bf16"), (60, "f16"), (150, "f32")])
def test_rows_that_see_nothing_and_hidden_nan(new, xt):
    """A row without history and bits gets 0; NaN in drafted rows reaches those that see them and no other."""
    print(f"tree attend hidden new={new} {xt}", flush=True)
    b = Batch([(new, new), (new, 200 + new)], 2, 128, 16, 21)
    mask = np.zeros((b.T, -(-new // 32)), np.uint32)
    for r in range(b.T):
        i = r % new
        mask[r, i // 32] |= np.uint32(1 << (i % 32))
    mask[0] = mask[new] = 0
    # the block of tokens 0..15 of sequence 1, out of every row's window, and its rows' last block
    last = 200 + new - 1
    for j in (0, last):
        p, o = serve8.place(b.table, 16, b.P, 1, j)
        b.ks[p, :, o // 16] = np.nan
    b.upload()
    clean = b.ks.copy()
    sees_last = np.zeros(b.T, bool)
    for i in range(1, new):                                # rows whose own token lies in the last block
        sees_last[new + i] = (200 + i) // 16 == last // 16
    if (200 - 1) // 16 == last // 16:
        sees_last[new:] = True                             # the last block holds history too
    b.ks = np.nan_to_num(clean, nan=0.01)
    q = _values(b.rng, (b.T, 4, 128), xt).cuda()
    window = 150
    pos = np.concatenate([np.arange(new), 200 + np.arange(new)]).astype(np.int32)
    got = _attend(b, q, 4, 0.09, mask, window, pos)
    assert torch.all(got[0] == 0)
    assert torch.isnan(got[torch.from_numpy(sees_last).cuda()]).all()
    _check_attend(b, q, xt, 4, 0.09, mask, window, pos, got, ~sees_last)


def test_attend_bad_pages_and_lengths():
    new = 20
    b = Batch([(new, 400), (new, 300), (new, 200), (new, 300)], 1, 64, 32, 8, max_kv=400)
    b.table[0, 3], b.table[0, 12], b.table[1, :] = -1, b.P, 2 ** 31 - 1
    b.kv_len[2], b.kv_len[3] = new - 1, 401
    b.upload()
    mask = np.full((b.T, 1), 0xffffffff, np.uint32)
    for q_heads in (2, 8):
        q = _values(b.rng, (b.T, q_heads, 64), "f16").cuda()
        got = _attend(b, q, q_heads, 0.125, mask, 0, None)
        _check_attend(b, q, "f16", q_heads, 0.125, mask, 0, np.zeros(b.T, int), got, np.arange(b.T) < 2 * new)
        assert torch.all(got[new:2 * new] == 0)
        assert torch.all(got[2 * new:] == 9)


@pytest.mark.parametrize("new,xt", [(2, "f16"), (12, "bf16"), (12, "f32")])
def test_attend_many_sequences(new, xt):
    """More sequences than a wavefront has lanes, of very different lengths and split."""
    print(f"attend many sequences {new} {xt}", flush=True)
    rng = np.random.default_rng(9)
    lens = [(int(n), int(n + rng.integers(0, 1 << int(rng.integers(1, 13))))) for n in rng.integers(0, new + 1, 71)]
    b = Batch(lens, 1, 64, 32, 31, max_kv=5000).upload()
    par = np.concatenate([_trees(b.rng, n, 4) for n, _ in lens if n]).astype(np.int32)
    mask, pos = od.plan(par, b.spans(), 1, 0, b.T)
    q = _values(b.rng, (b.T, 8, 64), xt).cuda()
    got = _attend(b, q, 8, 0.125, mask, 0, None)
    _check_attend(b, q, xt, 8, 0.125, mask, 0, pos, got)


def test_a_chain_of_masks_is_causal():
    """Masks of all rows up to one's own: what qg_attn_kv8 computes."""
    for new, q_heads, xt in ((7, 4, "bf16"), (90, 4, "f16")):
        b = Batch([(new, 500), (new, new)], 2, 128, 64, 31).upload()
        par = np.concatenate([np.arange(-1, new - 1)] * 2).astype(np.int32)
        mask, pos = od.plan(par, b.spans(), -(-new // 32), 0, b.T)
        q = _values(b.rng, (b.T, q_heads, 128), xt).cuda()
        got = _attend(b, q, q_heads, 0.1, mask, 0, None)
        o = torch.empty_like(q)
        ws = torch.empty(max(16, qg.qg_attn_kv8_workspace(b.cache, b.seqs, q_heads)), dtype=torch.uint8, device="cuda")
        qg.qg_attn_kv8(b.cache, b.seqs, q, o, q_heads, 0.1, True, 0, ws)
        # each is within a half step of its type and 2^-10 of the mean of |v| <= 127 * 0.02
        assert torch.all((got.float() - o.float()).abs() <= 2 * HALF[xt] * o.float().abs() + 2.0 ** -9 * 2.54)


# ---- verification -----------------------------------------------------------------------------------
def _verify(b, tokens, target, fill=-9, **kw):
    n = len(b.kv_len)
    seqs = qg.kv8_seqs(_dev(b.table), _dev(b.rows), _dev(b.kv_len), b.T, b.max_new, b.max_kv)
    outs = [torch.full((m,), fill, dtype=torch.int32, device="cuda") for m in (n, n, n + 1, b.T, n)]
    vocab = target.shape[1]
    size = qg.qg_draft_verify_workspace(seqs, vocab)
    guard = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    kw = {k: _dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items() if v is not None}
    qg.qg_draft_verify(seqs, _dev(tokens.astype(np.int32)), target, *outs, workspace=guard[:size], **kw)
    torch.cuda.synchronize()
    assert torch.all(guard[size:] == 255)
    return [x.cpu().numpy() for x in outs]


def _check_verify(b, tokens, target, **kw):
    got = _verify(b, tokens, target, **kw)
    plain = {k: v.double().cpu().numpy() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    want = od.verify(b.spans(), b.kv_len, b.T, tokens, target.double().cpu().numpy(), **plain)
    for name, x, y in zip(("accepted", "next", "rows_out", "path", "kv_out"), got, want):
        assert np.array_equal(x, y), (name, x, y)
    return got


def _inputs(rng, T, vocab, xt, noise, padded=0):
    """Logits of a target and a draft that agree but for some noise, rows apart by more than the vocabulary."""
    p = rng.normal(size=(T, vocab)) * 4
    q = p + noise * rng.normal(size=(T, vocab))
    out = []
    for x in (p, q):
        wide = torch.full((T, vocab + padded), float("nan"), dtype=TYPES[xt], device="cuda")
        wide[:, :vocab] = torch.from_numpy(x).to(TYPES[xt])
        out.append(wide[:, :vocab])
    return out


VERIFY = [
    # rows of each sequence, vocab, type, padding
    ([1], 1, "f32", 0), ([2, 1, 3], 2, "f16", 1), ([6], 32000, "f32", 0), ([5, 0, 9, 1, 4], 4096, "bf16", 0),
    ([8] * 33, 4097, "bf16", 3), ([3, 7], 12289, "f16", 0), ([4, 2], 300001, "f32", 5), ([17, 65, 30], 777, "f16", 0),
    ([300, 2], 257, "f32", 0),
]


@pytest.mark.parametrize("temp", ["one", "mixed", "cold"])
@pytest.mark.parametrize("i", range(len(VERIFY)))
def test_verify_drawn(i, temp):
    rows, vocab, xt, padded = VERIFY[i]
    print(f"verify drawn {i} {temp}: {VERIFY[i]}", flush=True)
    rng = np.random.default_rng(i)
    b = Batch([(n, n + 5) for n in rows], 1, 64, 16, i)
    target, draft = _inputs(rng, b.T, vocab, xt, 0.5, padded)
    temps = None if temp == "one" else np.where(rng.random(len(rows)) < 0.3, 0, rng.uniform(0.2, 2, len(rows))).astype(np.float32)
    if temp == "cold":
        temps = np.full(len(rows), 0.01, np.float32)       # weights down to e^-4000
    # a row's token as the draft would draw it at the row before
    d = draft.double().cpu().numpy()
    tokens = np.zeros(b.T, np.int64)
    for s, n in enumerate(rows):
        t = 1.0 if temps is None else max(0.05, temps[s])
        for r in range(b.rows[s] + 1, b.rows[s + 1]):
            tokens[r] = od.pick(od.chance(d[r - 1], t), rng.random())
    got = _check_verify(b, tokens, target, draft=draft, temps=temps, sample=rng.random(b.T).astype(np.float32),
                        accept=rng.random(b.T).astype(np.float32))
    print("accepted", got[0][:8], flush=True)
    greedy = _check_verify(b, tokens, target, draft=draft)     # no draws: the largest logit
    assert np.array_equal(greedy[2], _check_verify(b, tokens, target)[2])


@pytest.mark.parametrize("temp", ["one", "mixed"])
@pytest.mark.parametrize("i", range(len(VERIFY)))
def test_verify_chosen(i, temp):
    rows, vocab, xt, padded = VERIFY[i]
    print(f"verify chosen {i} {temp}: {VERIFY[i]}", flush=True)
    rng = np.random.default_rng(70 + i)
    b = Batch([(n, n + 5) for n in rows], 1, 64, 16, i)
    target, draft = _inputs(rng, b.T, vocab, xt, 0.3, padded)
    par = np.concatenate([_trees(rng, n, 3) for n in rows if n]).astype(np.int32)
    d = draft.double().cpu().numpy()
    for parents in (par, None):
        tokens = np.zeros(b.T, np.int64)
        for s, n in enumerate(rows):
            taken = np.zeros(max(n, 1), int)
            for r in range(1, n):
                up = r - 1 if parents is None else par[b.rows[s] + r]
                best = np.argsort(-d[b.rows[s] + up], kind="stable")
                tokens[b.rows[s] + r] = best[min(taken[up] // 2, vocab - 1)]   # twins among them
                taken[up] += 1
        temps = None if temp == "one" else np.where(rng.random(len(rows)) < 0.4, 0, rng.uniform(0.1, 1, len(rows))).astype(np.float32)
        got = _check_verify(b, tokens, target, parents=parents, temps=temps, sample=rng.random(b.T).astype(np.float32))
        print("accepted", got[0][:8], flush=True)


LARGE = [
    # rows of each sequence, how far back a row's parent may be, vocab, type, padding: batches whose first rows go before the others
    ([90, 0, 1, 2, 63, 64, 65, 88, 33, 90, 17, 45, 90, 5, 70, 31, 32, 90, 1, 80], 9, 20001, "bf16", 3),
    ([1000, 3, 0, 130], 1, 9000, "f32", 0), ([1024, 1, 40, 700], 30, 9000, "f16", 0),
]


@pytest.mark.parametrize("temp", ["one", "mixed", "none"])
@pytest.mark.parametrize("i", range(len(LARGE)))
def test_verify_large_trees(i, temp):
    """Trees of many rows, whose tokens often are what is drawn, so that the way through them is long; parents that are none, or
    that do not come before their rows."""
    rows, back, vocab, xt, padded = LARGE[i]
    print(f"verify large trees {i} {temp}: {LARGE[i]}", flush=True)
    assert max(rows) * len(rows) * -(-vocab // 1024) >= 32768
    rng = np.random.default_rng(170 + i)
    b = Batch([(n, n + 5) for n in rows], 1, 64, 16, i)
    target, _ = _inputs(rng, b.T, vocab, xt, 0.3, padded)
    target *= 4
    par = np.concatenate([_trees(rng, n, back) for n in rows if n]).astype(np.int32)
    for at, bad in zip(rng.permutation(b.T)[:20], (-1, -2, 5000, 2 ** 31 - 1, -2 ** 31) * 4):
        par[at] = bad
    best = target.argmax(1).cpu().numpy()
    tokens = rng.integers(0, vocab, b.T)
    for s, n in enumerate(rows):
        for r in range(1, n):
            up = par[b.rows[s] + r]
            if 0 <= up < r and rng.random() < (0.98 if back == 1 else 0.5):
                tokens[b.rows[s] + r] = best[b.rows[s] + up]
    kw = {}
    if temp != "none":
        kw["sample"] = rng.random(b.T).astype(np.float32)
    if temp == "mixed":
        kw["temps"] = np.where(rng.random(len(rows)) < 0.4, 0, rng.uniform(0.1, 1, len(rows))).astype(np.float32)
    got = _check_verify(b, tokens, target, parents=par, **kw)
    print("accepted", got[0], flush=True)
    target[b.rows[0]] = float("nan")                           # a first row without a largest: nothing follows it
    got = _check_verify(b, tokens, target, parents=par, **kw)
    assert got[0][0] == 0 and got[1][0] == -1


def test_verify_borders():
    """Draws of 0, of the largest value below 1 and at the edge of a token; ties; tokens that have no probability."""
    inf = float("inf")
    b = Batch([(3, 9)], 1, 64, 16, 1)
    half = torch.tensor([[-inf, 0.0, 0.0, -inf, 0.0, 0.0, -inf]] * 3, device="cuda")
    almost = 1 - 2.0 ** -24
    for u, token in ((0.0, 1), (0.24, 1), (0.26, 2), (0.49, 2), (0.51, 4), (0.76, 5), (almost, 5)):
        got = _check_verify(b, np.array([0, 9, 9]), half, sample=np.full(3, u, np.float32))
        assert got[1][0] == token
    # the draft's and the target's probabilities are the same: every token that was drawn stays
    got = _check_verify(b, np.array([0, 4, 1]), half, draft=half.clone(), sample=np.full(3, 0.0, np.float32),
                        accept=np.full(3, almost, np.float32))
    assert got[0][0] == 2 and got[1][0] == 1
    # tokens outside of the vocabulary, or that the target never gives, go; what follows is the draft's complement
    draft = torch.tensor([[0.0, 0.0, -inf, -inf, -inf, -inf, -inf]] * 3, device="cuda")
    for x in (0, -1, 7, 2 ** 31 - 1, -2 ** 31):
        for a in (0.0, 0.5):
            got = _check_verify(b, np.array([0, x, 1]), half, draft=draft, sample=np.full(3, 0.3, np.float32),
                                accept=np.full(3, a, np.float32))
            assert got[0][0] == 0 and got[1][0] in (2, 4, 5)
    # p <= q wherever the draft has mass only by rounding: a draw of no mass takes p
    same = torch.randn(3, 1000, device="cuda")
    got = _check_verify(b, np.array([0, -1, 1]), same, draft=same.clone(), sample=np.full(3, 0.5, np.float32),
                        accept=np.full(3, 0.5, np.float32))
    assert got[0][0] == 0 and 0 <= got[1][0] < 1000


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
def test_verify_equal_logits_leave_nothing(xt):
    """A target and a draft of the same logits: what is left of one less the other is nothing, whatever their sums and
    temperatures, so a token that goes is followed by a draw from the target."""
    rng = np.random.default_rng(21)
    b = Batch([(3, 9)] * 96, 1, 64, 16, 1)
    target, _ = _inputs(rng, b.T, 1500, xt, 0.0, 1)
    _check_verify(b, np.full(b.T, -1), target, draft=target.clone(), temps=rng.uniform(0.3, 3, 96).astype(np.float32),
                  sample=rng.random(b.T).astype(np.float32), accept=np.full(b.T, 0.5, np.float32))


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_verify_rows_without_probabilities(xt):
    """NaN, infinities and temperatures that are none end a sequence with -1, and reach no other."""
    rng = np.random.default_rng(3)
    b = Batch([(4, 9)] * 9, 1, 64, 16, 1)
    target, draft = _inputs(rng, b.T, 5000, xt, 0.0)
    tokens = np.zeros(b.T, np.int64)
    best = target.argmax(1).cpu().numpy()
    for s in range(9):
        tokens[4 * s + 1:4 * s + 4] = best[4 * s:4 * s + 3]
    inf, nan = float("inf"), float("nan")
    target[1, 4321] = nan            # sequence 0: its second row
    target[4 + 2, :] = -inf          # 1: its third
    target[8 + 0, 7] = inf           # 2: its first
    target[12 + 3, 4999] = nan       # 3: its last
    draft[16 + 1, 17] = nan          # 4: the draft's second: the token goes, the next is the target's
    draft[20 + 3, :] = nan           # 5: the draft's last, which nothing asks
    temps = np.array([1, 1, 1, 1, 1, 1, -1, nan, inf], np.float32)
    u, a = np.full(b.T, 0.4, np.float32), np.zeros(b.T, np.float32)
    got = _check_verify(b, tokens, target, draft=draft, temps=temps, sample=u, accept=a)
    assert got[1].tolist()[:4] == [-1] * 4 and got[1].tolist()[6:] == [-1] * 3 and min(got[1][4:6]) >= 0
    assert got[0].tolist() == [1, 2, 0, 3, 1, 3, 0, 0, 0]
    _check_verify(b, tokens, target, temps=temps, sample=u)
    got = _check_verify(b, tokens, target)                       # an infinity is the largest
    assert got[1][2] >= 0 and got[1][0] == -1


def test_verify_leaves_out_what_contradicts():
    rng = np.random.default_rng(4)
    b = Batch([(3, 9), (3, 9), (3, 9), (3, 9)], 1, 64, 16, 1)
    b.kv_len[1], b.max_kv, b.kv_len[3] = 2, 9, 10
    target, draft = _inputs(rng, b.T, 100, "f32", 0.1)
    got = _check_verify(b, np.zeros(b.T, np.int64), target, sample=rng.random(b.T).astype(np.float32))
    assert got[1][1] == got[1][3] == -1 and got[4].tolist()[1::2] == [2, 10]
    _check_verify(b, np.zeros(b.T, np.int64), target, draft=draft, sample=rng.random(b.T).astype(np.float32),
                  accept=rng.random(b.T).astype(np.float32))


# ---- together ---------------------------------------------------------------------------------------
class Step:
    """A step with drafted tokens as a program runs it: plan, rows into the cache, attention, verification, and the rows that
    stay moved together.  Everything that changes between steps lives in tensors."""

    def __init__(self, b, q_heads, vocab, parents, xt="bf16"):
        rng = b.rng
        self.b, self.q_heads, self.H = b, q_heads, b.H
        T, n = b.T, len(b.kv_len)
        self.kv = _dev(b.kv_len)
        self.rows, self.table = _dev(b.rows), _dev(b.table)
        self.seqs = qg.kv8_seqs(self.table, self.rows, self.kv, T, b.max_new, b.max_kv)
        ints = lambda *m: torch.zeros(*m, dtype=torch.int32, device="cuda")  # noqa: E731
        self.parents, self.mask, self.pos = _dev(parents), ints(T, -(-b.max_new // 32)), ints(T)
        self.outs = [ints(n), ints(n), ints(n + 1), ints(T), ints(n)]
        self.stay = qg.kv8_seqs(self.table, self.outs[2], self.outs[4], T, b.max_new, b.max_kv)
        self.freqs, self.rot = _rotary(b.D, False)
        self.qkv = _values(rng, (T, q_heads + 2 * b.H, b.D), xt).cuda()
        self.q, self.k, self.v = self.qkv.split([q_heads, b.H, b.H], 1)
        self.q_out, self.o = (torch.zeros(T, q_heads, b.D, dtype=TYPES[xt], device="cuda") for _ in "qo")
        self.tokens = torch.from_numpy(rng.integers(0, vocab, T).astype(np.int32)).cuda()
        self.target = torch.randn(T, vocab, device="cuda")
        self.sample = torch.rand(T, device="cuda")
        size = max(16, qg.qg_attn_kv8_workspace(b.cache, self.seqs, q_heads), qg.qg_draft_verify_workspace(self.seqs, vocab))
        self.work = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(self):
        b = self.b
        qg.qg_tree_plan(self.seqs, self.parents, self.mask, self.pos)
        qg.qg_kv8_write_rope(b.cache, self.seqs, self.rot, self.k, self.v, self.q, self.q_out, self.pos)
        qg.qg_attn_kv8_tree(b.cache, self.seqs, self.mask, self.q_out, self.o, self.q_heads, b.D ** -0.5, workspace=self.work)
        qg.qg_draft_verify(self.seqs, self.tokens, self.target, *self.outs, sample=self.sample, parents=self.parents,
                           workspace=self.work)
        qg.qg_kv8_write_rope(b.cache, self.stay, self.rot, self.k, self.v, src=self.outs[3])

    def state(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (*self.b.t, self.o, *self.outs)]

    def reset(self, saved, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for x, y in zip(self.b.t, saved):
            x.copy_(y)
        self.target.normal_(generator=g).mul_(10)
        self.sample.uniform_(generator=g)
        # half of the rows hold the token that is drawn where they follow
        best = self.target.argmax(1).to(torch.int32)
        up = (self.parents.clamp(min=0).long() + self.rows.long()[self.seq])
        other = torch.randint(500, (len(up),), device="cuda", generator=g, dtype=torch.int32)
        self.tokens.copy_(torch.where(torch.rand(len(up), device="cuda", generator=g) < 0.5, best[up], other))
        self.qkv.normal_(generator=g)
        torch.cuda.synchronize()


def _step(seed, lens):
    b = Batch([(n, t + 70) for n, t in lens], 2, 64, 16, seed).upload()
    for s, (n, t) in enumerate(lens):
        b.kv_len[s] = t
    par = np.concatenate([_trees(b.rng, n, 3) for n, _ in lens]).astype(np.int32)
    st = Step(b, 8, 500, par)
    st.seq = torch.from_numpy(np.repeat(np.arange(len(lens)), [n for n, _ in lens])).cuda()
    return st


def test_a_step_and_the_rows_that_stay():
    """After a step the cache holds the accepted rows at the places that follow the history, turned for those places."""
    st = _step(5, [(9, 40), (20, 33), (1, 1), (12, 200)])
    b = st.b
    saved = [x.clone() for x in b.t]
    st.reset(saved, 1)
    st.run()
    torch.cuda.synchronize()
    acc, nxt, rows, path, kv = (x.cpu().numpy() for x in st.outs)
    want = od.verify(b.spans(), b.kv_len, b.T, st.tokens.cpu().numpy(), st.target.double().cpu().numpy(),
                     st.sample.cpu().numpy(), parents=st.parents.cpu().numpy())
    for x, y in zip((acc, nxt, rows, path, kv), want):
        assert np.array_equal(x, y)
    assert acc.max() > 0
    # the plain cache: all rows, then those that stay, K at its positions
    mask, pos = od.plan(st.parents.cpu().numpy(), b.spans(), 1, 0, b.T)
    turn = torch.empty(b.T, 2, 64, device="cuda")
    qg.qg_rope(st.rot, _dev(pos), st.k.float(), turn)
    serve8.kv8_write(b.kc, b.ks, b.table, b.spans(), turn.cpu().numpy())
    serve8.kv8_write(b.vc, b.vs, b.table, b.spans(), st.v.float().cpu().numpy())
    qt = torch.empty_like(st.q_out)
    qg.qg_rope(st.rot, _dev(pos), st.q, qt)
    assert torch.equal(qt, st.q_out)
    _check_attend(b, qt, "bf16", 8, 64 ** -0.5, mask, 0, pos, st.o)
    sp = serve8.spans(rows, kv, b.T, b.max_new, b.max_kv)
    pick = torch.from_numpy(np.maximum(path, 0)).long().cuda()
    place = np.concatenate([np.arange(k - n, k) for (_, n, _), k in zip(sp, kv)] + [np.zeros(b.T - rows[-1])]).astype(np.int32)
    qg.qg_rope(st.rot, _dev(place), st.k[pick].float(), turn)
    serve8.kv8_write(b.kc, b.ks, b.table, sp, turn.cpu().numpy())
    serve8.kv8_write(b.vc, b.vs, b.table, sp, st.v[pick].float().cpu().numpy())
    b.kv_len, b.rows = kv, rows                            # what lies behind is of no sequence
    _check_cache(b, None, None)


@pytest.mark.parametrize("drawn", [False, True])
def test_captured_verification_of_many_rows(drawn):
    """Large trees, and many users' drafts with probabilities, verified in a graph: every replay on other inputs gives the plain
    result, with eager work and another graph on the same workspace between."""
    rows, vocab = ([8, 3, 0, 6] * 8, 9000) if drawn else ([130, 1, 77, 200], 26000)
    print(f"captured verification drawn={drawn}", flush=True)
    b = Batch([(n, n + 5) for n in rows], 1, 64, 16, 3)
    n, T = len(rows), b.T
    seqs = qg.kv8_seqs(_dev(b.table), _dev(b.rows), _dev(b.kv_len), T, b.max_new, b.max_kv)
    work = torch.full((qg.qg_draft_verify_workspace(seqs, vocab),), 255, dtype=torch.uint8, device="cuda")
    target, draft = (torch.zeros(T, vocab, device="cuda") for _ in "td")
    sample, accept = (torch.zeros(T, device="cuda") for _ in "sa")
    tokens, parents = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in "tp")
    kw = dict(draft=draft, accept=accept) if drawn else dict(parents=parents)
    outs = [[torch.full((m,), -9, dtype=torch.int32, device="cuda") for m in (n, n, n + 1, T, n)] for _ in range(2)]
    graphs = []
    for o in outs:
        qg.qg_draft_verify(seqs, tokens, target, *o, sample=sample, workspace=work, **kw)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            qg.qg_draft_verify(seqs, tokens, target, *o, sample=sample, workspace=work, **kw)
    for turn in range(3):
        rng = np.random.default_rng(40 + turn)
        p, q = _inputs(rng, T, vocab, "f32", 0.4)
        target.copy_(p)
        draft.copy_(q)
        sample.copy_(_dev(rng.random(T).astype(np.float32)))
        accept.copy_(_dev(rng.random(T).astype(np.float32)))
        par = np.concatenate([_trees(rng, r, 5) for r in rows if r]).astype(np.int32)
        parents.copy_(_dev(par))
        up = torch.from_numpy(np.repeat(b.rows[:-1], rows) + (np.concatenate([np.arange(r) - 1 for r in rows]) if drawn else par))
        tokens.copy_(torch.where(torch.rand(T, device="cuda") < 0.6, p.argmax(1)[up.clamp(min=0).cuda()].int(), 5))
        torch.cuda.synchronize()
        plain = {k: v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for k, v in kw.items()}
        want = od.verify(b.spans(), b.kv_len, T, tokens.cpu().numpy(), p.double().cpu().numpy(), sample.cpu().numpy(), **plain)
        for g in graphs + graphs[:1]:
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            for x, y in zip(o, want):
                assert np.array_equal(x.cpu().numpy(), y)


def test_captured_steps_replay():
    """Two steps in graphs of their own, replayed in turn with eager work between: every replay gives the eager result."""
    lens = [[(9, 40), (20, 33), (1, 1)], [(30, 64), (5, 700)]]
    steps = [_step(6 + i, l) for i, l in enumerate(lens)]
    saved = [[x.clone() for x in st.b.t] for st in steps]
    for st in steps:
        st.run()
    torch.cuda.synchronize()
    graphs = []
    for st in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.run()
        graphs.append(g)
    for turn in range(4):
        want = []
        for st, sv in zip(steps, saved):
            st.reset(sv, turn)
            st.run()
            want.append(st.state())
            st.reset(sv, turn + 100)                       # other contents in between
        for st, sv, g, w in zip(steps, saved, graphs, want):
            st.reset(sv, turn)
            g.replay()
            for x, y in zip(st.state(), w):
                assert torch.equal(x, y)


def test_two_streams_at_once():
    """Steps of two batches on streams of their own, with a workspace each."""
    steps = [_step(16 + i, l) for i, l in enumerate([[(9, 40), (20, 33)], [(40, 300)]])]
    saved = [[x.clone() for x in st.b.t] for st in steps]
    want = []
    for st, sv in zip(steps, saved):
        st.reset(sv, 3)
        st.run()
        want.append(st.state())
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for st, sv in zip(steps, saved):
            for x, y in zip(st.b.t, sv):
                x.copy_(y)
        torch.cuda.synchronize()
        for st, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                st.run()
        for st, w in zip(steps, want):
            for x, y in zip(st.state(), w):
                assert torch.equal(x, y)


def test_kv_out_over_kv_len():
    """kv_out may be the batch's kv_len."""
    rng = np.random.default_rng(9)
    b = Batch([(6, 30), (0, 4), (3, 8)] * 20, 1, 64, 16, 2)
    target, draft = _inputs(rng, b.T, 9000, "bf16", 0.2)
    tokens = np.zeros(b.T, np.int64)
    tokens[1:] = target.argmax(1).cpu().numpy()[:-1]
    for kw in (dict(), dict(draft=draft, accept=rng.random(b.T).astype(np.float32))):
        u = rng.random(b.T).astype(np.float32)
        want = _verify(b, tokens, target, sample=u, **kw)
        kv = _dev(b.kv_len)
        seqs = qg.kv8_seqs(_dev(b.table), _dev(b.rows), kv, b.T, b.max_new, b.max_kv)
        ints = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")  # noqa: E731
        ws = torch.empty(qg.qg_draft_verify_workspace(seqs, 9000), dtype=torch.uint8, device="cuda")
        outs = [ints(60), ints(60), ints(61), ints(b.T), kv]
        qg.qg_draft_verify(seqs, _dev(tokens.astype(np.int32)), target, *outs, sample=_dev(u), workspace=ws,
                           **{k: _dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()})
        for x, y in zip(outs, want):
            assert np.array_equal(x.cpu().numpy(), y)
