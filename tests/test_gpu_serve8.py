"""The 8-bit serving operators on the GPU against their plain definitions (oracle/serve8.py).

Cache: codes, scales and values read back are equal bit for bit (the coding is defined in f32).
Product in 8-bit integers: equal bit for bit (exact integer sum, two f32 products, one rounding).
Attention, per element, with u = 2^-24, n tokens and half-steps h (f16 2^-11, bf16 2^-8):
  scores   every product is exact up to q's pieces (f32 q: 2 pieces, 2^-22), D f32 additions, the factor
           scale * k scale (4 roundings), the subtraction of the maximum (u times both, each <= reach) and exp2
           (2^-22): ds <= ((D + 8) u + [f32] 2^-22) reach + 2 u reach + 2^-22; it moves o by <= 2 ds mean
  weights  one f16 rounding (2^-11), for f32 two pieces (2^-22), of the numerator, and for weights under f16's
           range 2^-25 of 2^9 2^ev (ev: the V scales' exponent, <= 2 top / 127 each for a code of 127):
           n 2^-34 * 2 * 127 * vmax
  sums     n + 16 f32 additions in numerator and denominator: 2 (n + 16) u mean
  output   one rounding, h |o| (f32: u |o|)
where mean = sum w |v| / sum w, reach = the largest scale * sum |q k|, vmax the largest V scale seen."""
import numpy as np
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import serve8

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Batch:
    """A cache and a batch on both sides; lens: (rows, tokens) of each sequence."""

    def __init__(self, lens, heads, dim, page, seed, spare=2, max_kv=None):
        rng = self.rng = np.random.default_rng(seed)
        self.H, self.D, self.page = heads, dim, page
        need = [-(-t // page) for _, t in lens]
        self.P = sum(need) + spare
        ids = rng.permutation(self.P)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.rows = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv_len = np.array([t for _, t in lens], np.int32)
        self.T = int(self.rows[-1])
        self.max_new, self.max_kv = max(n for n, _ in lens), max_kv or max(t for _, t in lens)
        self.kc, self.vc = (rng.integers(-127, 128, (self.P, heads, page, dim)).astype(np.int8) for _ in "kv")
        self.ks, self.vs = (rng.uniform(0.004, 0.02, (self.P, heads, page // 16)).astype(np.float32) for _ in "kv")

    def spans(self):
        return serve8.spans(self.rows, self.kv_len, self.T, self.max_new, self.max_kv)

    def upload(self):
        self.t = [_dev(serve8.layout(self.kc, "k")), _dev(self.ks), _dev(serve8.layout(self.vc, "v")), _dev(self.vs)]
        self.cache = qg.kv8_cache(*self.t, self.page, self.H, self.D)
        self.seqs = qg.kv8_seqs(_dev(self.table), _dev(self.rows), _dev(self.kv_len), self.T, self.max_new, self.max_kv)
        return self

    def written(self, which):
        """(place in the codes) of every token there is, as a mask [pages][heads][page]."""
        m = np.zeros((self.P, self.H, self.page), bool)
        for s, (_, n, total) in enumerate(self.spans()):
            for j in range(total):
                at = serve8.place(self.table, self.page, self.P, s, j)
                if at:
                    m[at[0], :, at[1]] = True
        return m


def _values(rng, shape, xt):
    x = rng.normal(size=shape) * np.exp(0.7 * rng.normal(size=shape[:-1] + (1,)))
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[xt])


def _check_cache(b, k, v):
    m = b.written("k")
    for raw, sc, codes, scales, which in ((b.t[0], b.t[1], b.kc, b.ks, "k"), (b.t[2], b.t[3], b.vc, b.vs, "v")):
        got = serve8.meaning(raw.cpu().numpy().reshape(-1), which, b.P, b.H, b.page, b.D)
        nan = np.repeat(np.isnan(scales), 16, -1)      # codes of a NaN block mean nothing
        assert np.array_equal(got[m & ~nan], codes[m & ~nan]), which
        assert np.array_equal(sc.cpu().numpy().reshape(scales.shape), scales, equal_nan=True), which


LENS = {
    "one": [(1, 1)],
    "steps": [(1, 1), (1, 2), (1, 16), (1, 17), (1, 33), (0, 20), (1, 200)],
    "chunks": [(5, 5), (16, 16), (17, 30), (0, 0), (40, 41), (3, 19), (100, 260), (64, 64)],
}


@pytest.mark.parametrize("xt,dim,page,heads", [("bf16", 128, 64, 2), ("f16", 64, 16, 3), ("f32", 96, 48, 1),
                                               ("bf16", 192, 32, 5), ("f32", 256, 256, 2), ("f32", 128, 80, 1)])
@pytest.mark.parametrize("lens", list(LENS))
def test_write_and_read(xt, dim, page, heads, lens):
    print(f"kv8 write/read {xt} dim={dim} page={page} heads={heads} {lens}", flush=True)
    b = Batch(LENS[lens], heads, dim, page, 11).upload()
    kv = _values(b.rng, (b.T, 2, heads, dim), xt)
    if b.T > 3:
        kv[1] = 0                                      # a token of zeros
        kv[2] = kv[2] * 1e-30                          # values near a block's rounding to nothing
    dev = kv.cuda()
    k, v = dev[:, 0], dev[:, 1]                        # side by side, as a fused projection leaves them
    qg.qg_kv8_write(b.cache, b.seqs, k, v)
    ref = kv.float().numpy()
    serve8.kv8_write(b.kc, b.ks, b.table, b.spans(), ref[:, 0])
    serve8.kv8_write(b.vc, b.vs, b.table, b.spans(), ref[:, 1])
    torch.cuda.synchronize()
    _check_cache(b, k, v)
    for yt in ("f32", "f16", "bf16"):
        ko, vo = (torch.full((b.T, heads, dim), 7.0, dtype=TYPES[yt], device="cuda") for _ in "kv")
        qg.qg_kv8_read(b.cache, b.seqs, ko, vo)
        for got, codes, scales in ((ko, b.kc, b.ks), (vo, b.vc, b.vs)):
            want = torch.from_numpy(serve8.kv8_read(codes, scales, b.table, b.spans(), b.T)).to(TYPES[yt])
            assert torch.equal(got.cpu(), want)


def test_write_special_values():
    """Zeros, subnormal scales, NaN and infinities: a block with a non-finite value is NaN, its neighbours whole."""
    b = Batch([(64, 64), (20, 24)], 2, 64, 32, 3).upload()
    x = b.rng.normal(size=(b.T, 2, 64)).astype(np.float32)
    x[0:16] = 0
    x[16:32] *= np.float32(1e-42)                      # a subnormal scale: 1 / d overflows
    x[40, 0, 5] = np.nan
    x[50, 1, 63] = -np.inf
    x[70] = np.float32(3e38)
    dev = torch.from_numpy(x).cuda()
    qg.qg_kv8_write(b.cache, b.seqs, dev, dev)
    serve8.kv8_write(b.kc, b.ks, b.table, b.spans(), x)
    serve8.kv8_write(b.vc, b.vs, b.table, b.spans(), x)
    ko, vo = torch.empty_like(dev), torch.empty_like(dev)
    qg.qg_kv8_read(b.cache, b.seqs, ko, vo)
    got = [ko.cpu().numpy(), vo.cpu().numpy()]
    bad = np.zeros((b.T, 2), bool)
    bad[32:48, 0] = bad[48:64, 1] = True
    for g, codes, scales in zip(got, (b.kc, b.vc), (b.ks, b.vs)):
        want = serve8.kv8_read(codes, scales, b.table, b.spans(), b.T)
        assert np.array_equal(g[~bad], want[~bad])
        assert np.all(np.isnan(g[bad]))


@pytest.mark.parametrize("order", ["token", "head", "apart"])
def test_strides(order):
    """Heads before tokens, and rows with room between them."""
    b = Batch([(7, 9), (30, 31)], 3, 64, 16, 4).upload()
    shape = {"token": (b.T, 3, 64), "head": (3, b.T, 64), "apart": (b.T, 5, 80)}[order]

    def view(t):
        return {"token": t, "head": t.transpose(0, 1) if order == "head" else t, "apart": t[:, 1:4, :64]}[order]

    src = [_values(b.rng, shape, "f16").cuda() for _ in "kv"]
    qg.qg_kv8_write(b.cache, b.seqs, view(src[0]), view(src[1]))
    for x, codes, scales in zip(src, (b.kc, b.vc), (b.ks, b.vs)):
        serve8.kv8_write(codes, scales, b.table, b.spans(), view(x).float().cpu().numpy())
    _check_cache(b, None, None)
    out = [torch.full(shape, 3.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    qg.qg_kv8_read(b.cache, b.seqs, view(out[0]), view(out[1]))
    for x, codes, scales in zip(out, (b.kc, b.vc), (b.ks, b.vs)):
        want = torch.full(shape, 3.0, dtype=torch.float16)
        view(want).copy_(torch.from_numpy(serve8.kv8_read(codes, scales, b.table, b.spans(), b.T)))
        assert torch.equal(x.cpu(), want)


def _attend(b, q, q_heads, scale, causal, window, fill=9.0):
    o = torch.full(q.shape, fill, dtype=q.dtype, device="cuda")
    size = qg.qg_attn_kv8_workspace(b.cache, b.seqs, q_heads)
    ws = torch.full((max(16, size),), 255, dtype=torch.uint8, device="cuda")   # NaN bits: nothing may be read first
    qg.qg_attn_kv8(b.cache, b.seqs, q, o, q_heads, scale, causal, window, ws)
    torch.cuda.synchronize()
    return o


def _check_attend(b, q, xt, q_heads, scale, causal, window, got, rows=None):
    o, mean, reach, top = serve8.attend(b.kc, b.ks, b.vc, b.vs, b.table, b.spans(), q.double().cpu().numpy(), scale,
                                        causal, window)
    u, n, D = 2.0 ** -24, b.max_kv, b.D
    piece = 2.0 ** -22 if xt == "f32" else 0.0
    ds = ((D + 10) * u + piece) * reach + 2.0 ** -22
    tol = 2 * ds * mean + (2.0 ** -22 if xt == "f32" else 2.0 ** -11) * mean + \
        n * 2.0 ** -34 * 254 * np.nanmax(np.abs(b.vs)) + 2 * (n + 16) * u * mean + HALF[xt] * np.abs(o)
    err = np.abs(got.double().cpu().numpy() - o)
    if rows is None:
        rows = ~np.isnan(o).any((1, 2))
    assert rows.any()
    bad = ~(err[rows] <= tol[rows])
    print(f"attend: worst error / tolerance {np.max(err[rows] / np.maximum(tol[rows], 1e-300)):.3f}", flush=True)
    assert not bad.any(), (np.argwhere(bad)[:5], err[rows][bad][:5], tol[rows][bad][:5])


ATTEND = [
    # lens, heads, q_heads, dim, page, causal, window, type
    ([(1, 1)], 1, 1, 64, 16, True, 0, "f16"),
    ([(1, 1), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 300)], 2, 8, 128, 64, True, 0, "bf16"),
    ([(1, 700), (0, 0), (1, 5)], 1, 16, 256, 32, True, 0, "f32"),
    ([(1, 5000), (1, 1023), (1, 1025)], 2, 14, 64, 48, True, 0, "f16"),
    ([(1, 4500), (1, 2049)], 1, 1, 96, 80, True, 1500, "f32"),
    ([(5, 5), (5, 130), (4, 64), (0, 7), (1, 3000)], 2, 16, 128, 32, True, 0, "bf16"),
    ([(9, 200), (9, 9)], 3, 9, 192, 16, True, 0, "f16"),
    ([(37, 37), (20, 90), (64, 128), (1, 1)], 2, 6, 64, 48, True, 0, "f16"),
    ([(70, 300), (33, 33)], 1, 3, 128, 64, True, 40, "bf16"),
    ([(70, 300), (33, 33)], 1, 2, 96, 16, False, 40, "f32"),
    ([(130, 130), (129, 400)], 2, 2, 128, 128, False, 0, "bf16"),
    ([(200, 260)], 1, 5, 256, 256, True, 1, "f32"),
    ([(300, 1500), (17, 1000)], 1, 4, 128, 64, True, 0, "f16"),
    ([(150, 2300)], 1, 7, 192, 32, True, 700, "bf16"),
    ([(257, 257)], 2, 16, 64, 16, True, 0, "f32"),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attend(i):
    lens, heads, q_heads, dim, page, causal, window, xt = ATTEND[i]
    print(f"attend case {i}: {ATTEND[i]}", flush=True)
    b = Batch(lens, heads, dim, page, 100 + i).upload()
    q = _values(b.rng, (b.T, q_heads, dim), xt).cuda()
    scale = dim ** -0.5
    got = _attend(b, q, q_heads, scale, causal, window)
    _check_attend(b, q, xt, q_heads, scale, causal, window, got)
    again = _attend(b, q, q_heads, scale, causal, window)
    assert torch.equal(got, again)


@pytest.mark.parametrize("new,xt", [(1, "f16"), (6, "bf16"), (150, "f16"), (150, "f32")])
def test_attend_ignores_what_is_hidden(new, xt):
    """Scales of NaN past a sequence's end and before every row's window, NaN in other sequences' blocks, codes
    of -128 in unwritten places: nothing of it reaches a result."""
    print(f"attend hidden new={new} {xt}", flush=True)
    window = 100
    b = Batch([(new, 1400), (new, new + 3)], 2, 128, 64, 7)
    hidden = ~b.written("k")
    total, first = 1400, 1400 - new - window + 1       # first token that any row of sequence 0 sees
    for j in range(0, first // 16 * 16):
        p, o = serve8.place(b.table, 64, b.P, 0, j)
        hidden[p, :, o] = True
    b.kc[hidden] = b.vc[hidden] = -128
    block = hidden.reshape(b.P, 2, 4, 16).all(-1)
    clean = [x.copy() for x in (b.ks, b.vs)]
    b.ks[block] = b.vs[block] = np.nan
    b.upload()
    b.ks, b.vs = clean
    q = _values(b.rng, (b.T, 8, 128), xt).cuda()
    got = _attend(b, q, 8, 0.09, True, window)
    _check_attend(b, q, xt, 8, 0.09, True, window, got)


@pytest.mark.parametrize("new", [1, 5, 140])
def test_attend_bad_pages_and_lengths(new):
    """Pages outside the cache hold no tokens (a row that sees nothing gets 0); a sequence whose numbers
    contradict each other is left out, its rows untouched."""
    print(f"attend bad pages new={new}", flush=True)
    b = Batch([(new, 400), (new, 300), (new, 200), (new, 300)], 1, 64, 32, 8, max_kv=400)
    b.table[0, 3], b.table[0, 12], b.table[1, :] = -1, b.P, 2 ** 31 - 1
    b.kv_len[2] = new - 1                              # fewer tokens than rows
    b.kv_len[3] = 401                                  # past the bound
    b.upload()
    q = _values(b.rng, (b.T, 2, 64), "f16").cuda()
    got = _attend(b, q, 2, 0.125, True, 0)
    _check_attend(b, q, "f16", 2, 0.125, True, 0, got, np.arange(b.T) < 2 * new)
    assert torch.all(got[new:2 * new] == 0)
    assert torch.all(got[2 * new:] == 9)
    # and the cache's own kernels
    x = _values(b.rng, (b.T, 1, 64), "f16")
    qg.qg_kv8_write(b.cache, b.seqs, x.cuda(), x.cuda())
    for codes, scales in ((b.kc, b.ks), (b.vc, b.vs)):
        serve8.kv8_write(codes, scales, b.table, b.spans(), x.float().numpy())
    _check_cache(b, None, None)
    out = [torch.full(x.shape, 9.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    qg.qg_kv8_read(b.cache, b.seqs, *out)
    want = serve8.kv8_read(b.kc, b.ks, b.table, b.spans(), b.T)
    want[np.isnan(want)] = 9
    assert np.array_equal(out[0].float().cpu().numpy(), want.astype(np.float16).astype(np.float32))


@pytest.mark.parametrize("new", [1, 100])
def test_attend_extremes(new):
    """Scores far apart, rows of q of very different size, zeros in q, V scales over many powers of two."""
    for xt in ("f16", "bf16", "f32"):
        b = Batch([(new, 500)], 1, 128, 16, 9)
        b.vs *= np.exp2(b.rng.integers(-30, 8, b.vs.shape)).astype(np.float32)
        b.ks[::3] = 0
        b.upload()
        q = _values(b.rng, (b.T, 4, 128), xt) * 8
        q[:, 1] = q[:, 1] * 2.0 ** -12
        q[:, 2] = 0
        q = q.cuda()
        got = _attend(b, q, 4, -0.3, True, 0)
        _check_attend(b, q, xt, 4, -0.3, True, 0, got)
        q[0, 0, 3] = float("nan")                      # a NaN stays in its row and head
        after = _attend(b, q, 4, -0.3, True, 0)
        assert torch.all(torch.isnan(after[0, 0]))
        mask = torch.ones(b.T, 4, dtype=torch.bool)
        mask[0, 0] = False
        assert torch.equal(after.cpu()[mask], got.cpu()[mask])


def test_attend_strides_and_streams():
    """q inside a fused projection, o heads-first, on another stream than the default."""
    b = Batch([(3, 40), (50, 77)], 2, 64, 16, 10).upload()
    fused = _values(b.rng, (b.T, 8, 64), "bf16").cuda()
    q = fused[:, 2:6]
    want = _attend(b, q.contiguous(), 4, 0.125, True, 0)
    o = torch.zeros((4, b.T, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, qg.qg_attn_kv8_workspace(b.cache, b.seqs, 4)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qg.qg_attn_kv8(b.cache, b.seqs, q, o.transpose(0, 1), 4, 0.125, True, 0, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(o.transpose(0, 1), want)


W8A8 = [(1, 64, 16), (1, 257, 4096), (1, 1000, 8208), (2, 130, 128), (3, 33, 400), (7, 96, 2064), (8, 64, 4112),
        (9, 511, 1040), (16, 200, 32), (17, 129, 4112), (33, 1025, 1008), (45, 300, 4112), (64, 128, 256), (65, 384, 528),
        (129, 260, 1040), (200, 513, 400), (256, 256, 128), (300, 1000, 2064), (513, 770, 80), (1030, 511, 336)]


@pytest.mark.parametrize("i", range(len(W8A8)))
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f16", "f16"), ("f32", "bf16")])
def test_w8a8(i, xt, yt):
    T, N, K = W8A8[i]
    print(f"w8a8 T={T} N={N} K={K} {xt} -> {yt}", flush=True)
    rng = np.random.default_rng(i)
    w = rng.integers(-128, 128, (N, K)).astype(np.int8)
    ws = (rng.uniform(0.5, 2, N) / 127 / np.sqrt(K)).astype(np.float32)
    x = _values(rng, (T, K), xt)
    if T > 4:
        x[1] = 0
        x[2] = x[2] * 1e-30
        x[3, K // 2] = float("nan")
        x[4, 0] = float("inf")
    y = torch.full((T + 1, N), 5.0, dtype=TYPES[yt], device="cuda")
    work = torch.full((max(16, qg.qgemm_w8a8_workspace(N, K, T)),), 255, dtype=torch.uint8, device="cuda")
    qg.qgemm_w8a8(_dev(w), _dev(ws), x.cuda(), y[:T], N, K, T, work)
    want = torch.from_numpy(serve8.w8a8(w, ws, x.float().numpy())).to(TYPES[yt])
    got = y.cpu()
    assert torch.all(got[T] == 5)                      # nothing past the last row
    assert torch.equal(torch.isnan(got[:T]), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got[:T].float()), torch.nan_to_num(want.float()))


def test_graph_of_a_decoding_step():
    """Write, attention and products of one step in a captured graph: the tokens' number, their table and their
    values change between replays, and every replay equals the eager calls."""
    print("graph of a decoding step", flush=True)
    heads, q_heads, dim, page = 2, 8, 128, 64
    b = Batch([(1, 1200), (1, 40), (1, 1)], heads, dim, page, 12, max_kv=1400, spare=30)
    b.table = np.concatenate([b.table, np.full((3, 4), -1, np.int32)], 1)
    free = [p for p in range(b.P) if p not in set(b.table.reshape(-1).tolist())]
    for s in range(3):                                  # pages for the tokens to come
        n = int((b.table[s] >= 0).sum())
        b.table[s, n:n + 2] = [free.pop(), free.pop()]
    b.upload()
    hidden = 256
    N = (q_heads + 2 * heads) * dim
    w = _dev(b.rng.integers(-127, 128, (N, hidden)).astype(np.int8))
    ws = torch.full((N,), 1e-3, device="cuda")
    wo = _dev(b.rng.integers(-127, 128, (hidden, q_heads * dim)).astype(np.int8))
    wos = torch.full((hidden,), 1e-3, device="cuda")
    x = torch.zeros(3, hidden, dtype=torch.bfloat16, device="cuda")
    size = max(qg.qgemm_w8a8_workspace(N, hidden, 3), qg.qgemm_w8a8_workspace(hidden, q_heads * dim, 3),
               qg.qg_attn_kv8_workspace(b.cache, b.seqs, q_heads), 16)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step(t):
        qkv, o, y = t
        qg.qgemm_w8a8(w, ws, x, qkv, N, hidden, 3, work)
        h = qkv.view(3, q_heads + 2 * heads, dim)
        qg.qg_kv8_write(b.cache, b.seqs, h[:, q_heads:q_heads + heads], h[:, q_heads + heads:])
        qg.qg_attn_kv8(b.cache, b.seqs, h[:, :q_heads], o, q_heads, dim ** -0.5, True, 0, work)
        qg.qgemm_w8a8(wo, wos, o.view(3, -1), y, hidden, q_heads * dim, 3, work)

    def outs():
        return (torch.empty(3, N, dtype=torch.bfloat16, device="cuda"),
                torch.empty(3, q_heads, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(3, hidden, device="cuda"))

    cap, ref = outs(), outs()
    kv_len = b.seqs.keep[2]
    saved = [t.clone() for t in b.t]
    step(ref)                                           # eager once, before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cap)
    torch.cuda.synchronize()
    for t, s in zip(b.t, saved):
        t.copy_(s)
    for r in range(4):
        x.copy_(_values(b.rng, (3, hidden), "bf16"))
        before = [t.clone() for t in b.t]
        for t in cap:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in b.t]
        for t, s in zip(b.t, before):
            t.copy_(s)
        step(ref)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(cap, ref)), f"replay {r}"
        assert all(torch.equal(p, q) for p, q in zip(after, b.t)), f"replay {r}: cache"
        kv_len.add_(1)
    del g
