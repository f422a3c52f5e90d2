"""The 8-bit serving operators where their kernels' forms meet: scales that a row must not feel, histories past
the blocks that a tile looks up at a time, every tile and every number of tokens at which another kernel takes
over.  Definitions, tolerances and their derivation: test_gpu_serve8.py."""
import numpy as np
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import serve8
from test_gpu_serve8 import TYPES, Batch, _attend, _check_attend, _dev, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [5, 40, 150])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_a_nan_block_reaches_only_rows_that_see_it(new, which, xt):
    """The block of the last tokens is NaN: rows before it are as if it were not there, rows that see it NaN."""
    print(f"nan block {which} new={new} {xt}", flush=True)
    total = 333                                        # tokens 320..332 lie in the last block
    b = Batch([(new, total)], 1, 128, 32, 21)
    q = _values(b.rng, (b.T, 4, 128), xt).cuda()
    page, off = serve8.place(b.table, 32, b.P, 0, 320)
    (b.ks if which == "k" else b.vs)[page, :, off // 16] = np.nan
    got = _attend(b.upload(), q, 4, 0.09, True, 0)
    before = max(0, new - 13)
    assert torch.all(torch.isnan(got[before:]))
    if before:
        _check_attend(b, q, xt, 4, 0.09, True, 0, got, np.arange(b.T) < before)


@pytest.mark.parametrize("new", [1, 30, 130])
@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
def test_scales_of_any_sign_and_size(new, xt):
    """V scales of 0 and below 0, K scales below 0, a hidden block with a scale of 2^100."""
    print(f"scales new={new} {xt}", flush=True)
    b = Batch([(new, 700)], 2, 64, 48, 22)
    b.vs[:, :, ::3] *= -1
    b.vs[:, 0, 1] = 0
    b.ks[:, :, 2] *= -1
    q = _values(b.rng, (b.T, 8, 64), xt).cuda()
    window = 300
    first = 700 - new - window + 1                     # first token that any row sees
    want = _attend(b.upload(), q, 8, 0.125, True, window)
    _check_attend(b, q, xt, 8, 0.125, True, window, want)
    for j in range(0, first // 16 * 16, 16):
        p, o = serve8.place(b.table, 48, b.P, 0, j)
        b.vs[p, :, o // 16] = np.float32(2.0 ** 100)
    got = _attend(b.upload(), q, 8, 0.125, True, window)
    assert torch.equal(got, want)


@pytest.mark.parametrize("new", [3, 90])
def test_tiny_v_scales(new):
    """All V scales near the smallest f32, and all near the largest: results keep their relative precision (of
    subnormal scales that of their own bits)."""
    for e in (-120, 100):
        print(f"tiny new={new} 2^{e}", flush=True)
        b = Batch([(new, 400)], 1, 64, 16, 23)
        b.vs *= np.float32(2.0 ** e)
        q = _values(b.rng, (b.T, 2, 64), "f32").cuda()
        got = _attend(b.upload(), q, 2, 0.125, True, 0)
        _check_attend(b, q, "f32", 2, 0.125, True, 0, got)


LONG = [
    # more blocks than a tile looks up at a time, in one split and in several, with and without a window
    ([(70, 9000)], 1, 1, 64, 48, 0, "f16"),
    ([(100, 4500), (1, 8000)], 1, 2, 128, 16, 0, "bf16"),
    ([(64, 9100)], 1, 1, 256, 64, 0, "f32"),
    ([(129, 9000)], 2, 2, 96, 32, 5000, "f16"),
    ([(1, 20000), (1, 40), (0, 0)], 1, 3, 192, 128, 0, "bf16"),
]


@pytest.mark.parametrize("i", range(len(LONG)))
def test_long_histories(i):
    lens, heads, q_heads, dim, page, window, xt = LONG[i]
    print(f"long case {i}: {LONG[i]}", flush=True)
    b = Batch(lens, heads, dim, page, 200 + i).upload()
    q = _values(b.rng, (b.T, q_heads, dim), xt).cuda()
    got = _attend(b, q, q_heads, dim ** -0.5, True, window)
    _check_attend(b, q, xt, q_heads, dim ** -0.5, True, window, got)


@pytest.mark.parametrize("dim,xt", [(64, "f16"), (96, "bf16"), (128, "f16"), (128, "f32")])
@pytest.mark.parametrize("seqs", [3, 64])
def test_tiles_of_both_heights(dim, xt, seqs):
    """Few and many tiles for the card: 128 and 256 rows a workgroup; sequences far shorter than the longest."""
    print(f"tiles dim={dim} {xt} seqs={seqs}", flush=True)
    rng = np.random.default_rng(seqs)
    lens = [(64, 190)] + [(int(n), int(n + rng.integers(0, 200))) for n in rng.integers(0, 5, seqs - 1)]
    b = Batch(lens, 4, dim, 32, 24).upload()
    q = _values(b.rng, (b.T, 16, dim), xt).cuda()
    got = _attend(b, q, 16, dim ** -0.5, True, 0)
    _check_attend(b, q, xt, 16, dim ** -0.5, True, 0, got)


# one launch and several splits of few and of many heads, 4 and 8 wavefronts: (sequences, longest)
@pytest.mark.parametrize("seqs,longest", [(33, 2112), (33, 2113), (64, 4096), (64, 4097), (129, 300), (129, 4100),
                                          (1, 40001), (7, 40001), (8, 17000), (12, 9000), (25, 9000), (47, 3000),
                                          (48, 3071), (48, 3073)])
@pytest.mark.parametrize("dim,xt", [(64, "f16"), (96, "f32"), (256, "f32")])
def test_one_token_of_one_long_sequence(seqs, longest, dim, xt):
    """The longest stands among short ones: what the host plans by it holds for all of them."""
    print(f"steps seqs={seqs} longest={longest} dim={dim} {xt}", flush=True)
    rng = np.random.default_rng(seqs + longest)
    lens = [(1, int(n)) for n in rng.integers(1, 40, seqs)]
    lens[seqs // 2] = (1, longest)
    b = Batch(lens, 4, dim, 64, 31).upload()
    q = _values(b.rng, (b.T, 8, dim), xt).cuda()
    got = _attend(b, q, 8, dim ** -0.5, True, 0)
    _check_attend(b, q, xt, 8, dim ** -0.5, True, 0, got)


# T at both sides of every change of kernel; N over one, several and many workgroups; K past a ring's pieces
SIZES = [(t, n, k) for t in (1, 2, 3, 5, 8, 9) for n, k in ((8200, 144), (33, 8208))]
SIZES += [(t, n, k) for t in (16, 17, 32, 33, 48, 49, 64, 65, 96, 97, 128, 129) for n, k in ((100, 2064), (12305, 272))]
SIZES += [(1, 48, 32784), (20, 70, 65536), (129, 65, 32784), (1500, 2001, 400), (3000, 4200, 272)]
# X coded in the product's launch or before it: N at one and two row blocks a workgroup, T K at the limit
SIZES += [(8, 4096, 4080), (8, 4096, 4096), (7, 4097, 2320), (7, 4097, 2352), (1, 8192, 16368), (1, 8193, 16384)]
SIZES += [(1, 4081, 32752), (2, 6000, 8176), (3, 8192, 16)]
# the streaming kernel and the tiles, and the tiles' forms, at both sides of their limits
SIZES += [(65, 12288, 144), (96, 12289, 144), (97, 5120, 272), (128, 5121, 272), (100, 700, 16400)]
SIZES += [(256, 16384, 272), (257, 16400, 272), (640, 13200, 144), (700, 14100, 144)]
SIZES += [(9, 300, 8208), (64, 2048, 8208), (256, 2048, 6160)]       # K in one and in several splits


@pytest.mark.parametrize("i", range(len(SIZES)))
def test_w8a8_sizes(i):
    T, N, K = SIZES[i]
    xt, yt = [("f16", "f32"), ("f32", "bf16"), ("bf16", "f16")][i % 3]
    print(f"w8a8 T={T} N={N} K={K} {xt} -> {yt}", flush=True)
    rng = np.random.default_rng(1000 + i)
    w = rng.integers(-128, 128, (N, K)).astype(np.int8)
    ws = (rng.uniform(0.5, 2, N) / 127 / np.sqrt(K)).astype(np.float32)
    x = _values(rng, (T, K), xt)
    rows = x.float().numpy()
    scales = [serve8.scale_of(r) for r in rows]
    codes = np.stack([serve8.code(r, inv) for r, (_, inv) in zip(rows, scales)])
    acc = codes.astype(np.float64) @ w.astype(np.float64).T          # exact: below 2^53
    d = np.array([s for s, _ in scales], np.float32)
    want = torch.from_numpy((acc.astype(np.float32) * d[:, None]) * ws).to(TYPES[yt])
    y = torch.full((T + 1, N), 5.0, dtype=TYPES[yt], device="cuda")
    size = qg.qgemm_w8a8_workspace(N, K, T)
    work = torch.full((max(16, size) + 64,), 255, dtype=torch.uint8, device="cuda")
    qg.qgemm_w8a8(_dev(w), _dev(ws), x.cuda(), y[:T], N, K, T, work[:max(16, size)])
    assert torch.all(work[max(16, size):] == 255)                     # nothing past the workspace
    assert torch.all(y[T] == 5)
    assert torch.equal(y[:T].cpu(), want)


def test_w8a8_streams_and_refusals():
    """On another stream than the default; what the binding refuses leaves Y untouched."""
    T, N, K = 40, 96, 256
    g = torch.Generator().manual_seed(1)
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    ws = torch.rand(N, generator=g).cuda()
    x = torch.randn(T, K, generator=g).cuda()
    work = torch.empty(qg.qgemm_w8a8_workspace(N, K, T), dtype=torch.uint8, device="cuda")
    want, y = torch.empty(T, N, device="cuda"), torch.zeros(T, N, device="cuda")
    qg.qgemm_w8a8(w, ws, x, want, N, K, T, work)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qg.qgemm_w8a8(w, ws, x, y, N, K, T, work, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    y.fill_(3)
    for bad in (dict(X=x[:, ::2]), dict(X=x[:39]), dict(X=x.double()), dict(w_codes=w.t()), dict(w_codes=w.int()),
                dict(w_scales=ws[:95]), dict(workspace=work[:-1]), dict(workspace=None), dict(Y=y.t()),
                dict(Y=y[:39]), dict(K=K - 8)):
        args = dict(w_codes=w, w_scales=ws, X=x, Y=y, N=N, K=K, T=T, workspace=work)
        args.update(bad)
        with pytest.raises(qg.QGError):
            qg.qgemm_w8a8(**args)
    assert torch.all(y == 3)


def test_pages_past_4_gib():
    """The same tokens in the first pages of a small cache and in the last of one whose codes pass 2^32 bytes: the
    same bits."""
    print("pages past 4 GiB", flush=True)
    heads, dim, page, lens = 8, 128, 256, [(70, 600), (1, 300)]
    pages = 2 ** 32 // (heads * dim * page) + 40
    got = []
    for total, first in ((40, 0), (pages, pages - 5)):
        need = [-(-t // page) for _, t in lens]
        table = torch.full((2, max(need)), -1, dtype=torch.int32)
        at = first
        for s, n in enumerate(need):
            table[s, :n] = torch.arange(at, at + n)
            at += n
        tensors = qg.kv8_pages(total, page, heads, dim)
        cache = qg.kv8_cache(*tensors, page, heads, dim)
        rng = np.random.default_rng(3)
        all_rows = _values(rng, (900, 2, heads, dim), "bf16").cuda()
        ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        seqs = qg.kv8_seqs(table.cuda(), ints(0, 600, 900), ints(600, 300), 900, 600, 600)
        qg.qg_kv8_write(cache, seqs, all_rows[:, 0], all_rows[:, 1])
        k, v = torch.empty(900, heads, dim, device="cuda"), torch.empty(900, heads, dim, device="cuda")
        qg.qg_kv8_read(cache, seqs, k, v)
        seqs = qg.kv8_seqs(table.cuda(), ints(0, 70, 71), ints(600, 300), 71, 70, 600)
        q = _values(rng, (71, 16, dim), "bf16").cuda()
        many = torch.empty_like(q)
        work = torch.empty(max(16, qg.qg_attn_kv8_workspace(cache, seqs, 16)), dtype=torch.uint8, device="cuda")
        qg.qg_attn_kv8(cache, seqs, q, many, 16, 0.09, True, 0, work)
        seqs = qg.kv8_seqs(table.cuda(), ints(0, 1, 2), ints(600, 300), 2, 1, 600)
        single = torch.empty_like(q[:2])
        work = torch.empty(max(16, qg.qg_attn_kv8_workspace(cache, seqs, 16)), dtype=torch.uint8, device="cuda")
        qg.qg_attn_kv8(cache, seqs, q[:2], single, 16, 0.09, True, 0, work)
        torch.cuda.synchronize()
        got.append([x.cpu() for x in (k, v, many, single)])
        del cache, tensors
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.isfinite(got[0][2]).all() and got[0][2].abs().max() > 0
