"""CPU checks of the 8-bit serving operators: the refusals of their entry points, the cache's index
arithmetic (compiled for the host) against its definition with broken tables and lengths, and hand-worked
pins of the plain definitions that the GPU tests compare with.  Nothing here launches a kernel."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import serve8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # aligned, never dereferenced


def _cache(**kw):
    a = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, pages=8, page=64, heads=2, dim=128)
    a.update(kw)
    return qg.QgKv8Cache(**a)


def _seqs(**kw):
    a = dict(table=A, rows=A, kv_len=A, seqs=3, width=4, T=9, max_new=5, max_kv=200)
    a.update(kw)
    return qg.QgKv8Seqs(**a)


def _write(cache=None, seqs=None, k=A, kr=256, kh=128, v=A, vr=256, vh=128, xt=qg.QG_X_BF16, call="qg_kv8_write"):
    c, s = cache or _cache(), seqs or _seqs()
    return getattr(qg.lib(), call)(C.addressof(c), C.addressof(s), k, kr, kh, v, vr, vh, xt, None)


def _attn(cache=None, seqs=None, q=A, qr=512, qh=128, o=A, orow=512, oh=128, xt=qg.QG_X_BF16, q_heads=4, ws=A,
          size=1 << 40):
    c, s = cache or _cache(), seqs or _seqs()
    return qg.lib().qg_attn_kv8(C.addressof(c), C.addressof(s), q, qr, qh, o, orow, oh, xt, q_heads, 0.1, 1, 0, ws,
                                size, None)


DESCRIPTORS = [
    (dict(cache=_cache(dim=80)), qg.QG_ESHAPE), (dict(cache=_cache(dim=0)), qg.QG_ESHAPE),
    (dict(cache=_cache(page=24)), qg.QG_ESHAPE), (dict(cache=_cache(page=0)), qg.QG_ESHAPE),
    (dict(cache=_cache(page=65552)), qg.QG_ESHAPE), (dict(cache=_cache(heads=0)), qg.QG_ESHAPE),
    (dict(cache=_cache(pages=0)), qg.QG_ESHAPE), (dict(cache=_cache(pages=1 << 29)), qg.QG_ESHAPE),
    (dict(cache=_cache(k_codes=A + 8)), qg.QG_EALIGN), (dict(cache=_cache(v_scales=A + 2)), qg.QG_EALIGN),
    (dict(cache=_cache(k_scales=None)), qg.QG_EINVAL), (dict(cache=_cache(v_codes=None)), qg.QG_EINVAL),
    (dict(seqs=_seqs(seqs=-1)), qg.QG_ESHAPE), (dict(seqs=_seqs(seqs=65536)), qg.QG_ESHAPE),
    (dict(seqs=_seqs(width=0)), qg.QG_ESHAPE), (dict(seqs=_seqs(max_new=10)), qg.QG_ESHAPE),
    (dict(seqs=_seqs(max_kv=4)), qg.QG_ESHAPE), (dict(seqs=_seqs(max_kv=(1 << 24) + 1)), qg.QG_ESHAPE),
    (dict(seqs=_seqs(T=-1)), qg.QG_ESHAPE), (dict(seqs=_seqs(table=None)), qg.QG_EINVAL),
    (dict(seqs=_seqs(rows=A + 2)), qg.QG_EALIGN),
    (dict(seqs=_seqs(seqs=0, table=None)), qg.QG_OK), (dict(seqs=_seqs(T=0, max_new=0, rows=None)), qg.QG_OK),
    (dict(seqs=_seqs(max_new=0), xt=7), qg.QG_EINVAL), (dict(xt=-1), qg.QG_EINVAL),
]


@pytest.mark.parametrize("i", range(len(DESCRIPTORS)))
def test_descriptor_refusals(i):
    kw, want = DESCRIPTORS[i]
    for call in ("qg_kv8_write", "qg_kv8_read"):
        assert _write(call=call, **kw) == want
    assert _attn(**kw) == want


def test_row_refusals():
    assert _write(k=None) == qg.QG_EINVAL
    assert _write(v=A + 8) == qg.QG_EALIGN
    assert _write(kr=260) == qg.QG_EALIGN       # 520 bytes
    assert _write(vh=-128) == qg.QG_ESHAPE
    # outputs whose heads or rows overlap, in either order
    assert _write(call="qg_kv8_read", kh=64) == qg.QG_ESHAPE
    assert _write(call="qg_kv8_read", kr=128) == qg.QG_ESHAPE
    assert _write(call="qg_kv8_read", vr=128, vh=8 * 128) == qg.QG_ESHAPE   # 9 rows a head
    assert _attn(oh=0) == qg.QG_ESHAPE
    assert _attn(q_heads=3) == qg.QG_ESHAPE
    assert _attn(q_heads=0) == qg.QG_ESHAPE
    assert _attn(o=A + 4) == qg.QG_EALIGN
    big = _seqs(T=1 << 21, max_new=1 << 21, max_kv=1 << 22)
    assert _attn(seqs=big, q_heads=1024, qr=1 << 17, orow=1 << 17) == qg.QG_ESHAPE
    c, s = _cache(), _seqs(max_kv=1 << 20, T=3, max_new=1)
    size = qg.lib().qg_attn_kv8_workspace(C.addressof(c), C.addressof(s), 4)
    assert size > 0
    assert _attn(seqs=s, size=0) == qg.QG_EWORKSPACE
    assert _attn(seqs=s, ws=None) == qg.QG_EWORKSPACE
    assert _attn(seqs=s, ws=A + 4) == qg.QG_EALIGN
    assert qg.lib().qg_attn_kv8_workspace(C.addressof(c), C.addressof(s), 3) == 0
    assert qg.lib().qg_attn_kv8_workspace(None, C.addressof(s), 4) == 0


def test_w8a8_refusals():
    L = qg.lib()

    def call(w=A, ws=A, x=A, xt=0, y=A, yt=0, N=64, K=128, T=4, work=A, size=1 << 40):
        return L.qgemm_w8a8(w, ws, x, xt, y, yt, N, K, T, work, size, None)

    assert call(K=24) == qg.QG_ESHAPE
    assert call(K=0) == qg.QG_ESHAPE
    assert call(K=(1 << 17) + 16) == qg.QG_ESHAPE
    assert call(N=0) == qg.QG_ESHAPE
    assert call(T=-1) == qg.QG_ESHAPE
    assert call(xt=3) == qg.QG_EINVAL
    assert call(yt=-1) == qg.QG_EINVAL
    assert call(w=None) == qg.QG_EINVAL
    assert call(y=None) == qg.QG_EINVAL
    assert call(T=0, w=None) == qg.QG_OK
    assert call(w=A + 8) == qg.QG_EALIGN
    assert call(x=A + 4) == qg.QG_EALIGN
    assert call(y=A + 2) == qg.QG_EALIGN
    assert call(T=200, size=qg.qgemm_w8a8_workspace(64, 128, 200) - 1) == qg.QG_EWORKSPACE
    assert call(T=200, work=None) == qg.QG_EWORKSPACE


def test_binding_refusals():
    """The binding checks what the C side cannot see: element types, contiguity, shapes."""
    k, ks, v, vs = qg.kv8_pages(4, 32, 2, 64, device="cpu")
    c = qg.kv8_cache(k, ks, v, vs, 32, 2, 64)
    assert (c.struct.pages, c.struct.page, c.struct.heads, c.struct.dim) == (4, 32, 2, 64)
    with pytest.raises(qg.QGError):
        qg.kv8_cache(k, ks, v[:-1], vs, 32, 2, 64)
    with pytest.raises(qg.QGError):
        qg.kv8_cache(k, ks.double(), v, vs, 32, 2, 64)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    s = qg.kv8_seqs(i(0, 1).view(1, 2), i(0, 3), i(40), 3, 3, 40)
    with pytest.raises(qg.QGError):
        qg.kv8_seqs(i(0, 1).view(1, 2), i(0, 3, 4), i(40), 3, 3, 40)
    with pytest.raises(qg.QGError):
        qg.kv8_seqs(torch.zeros(1, 2, dtype=torch.int64), i(0, 3), i(40), 3, 3, 40)
    x = torch.zeros(3, 2, 64)
    with pytest.raises(qg.QGError):                                   # another shape
        qg.qg_kv8_write(c, s, x[:2], x[:2], stream=0)
    with pytest.raises(qg.QGError):                                   # types that differ
        qg.qg_kv8_write(c, s, x, x.half(), stream=0)
    with pytest.raises(qg.QGError):                                   # dims apart
        qg.qg_kv8_write(c, s, torch.zeros(3, 2, 128)[..., ::2], x, stream=0)
    with pytest.raises(qg.QGError):
        qg.qg_attn_kv8(c, s, x, x.half(), 2, 1.0, stream=0)


@pytest.fixture(scope="module")
def place(tmp_path_factory):
    """qg_kv8.hpp compiled for the host."""
    d = tmp_path_factory.mktemp("kv8")
    src = d / "place.cpp"
    src.write_text('''#include "qg_kv8.hpp"
extern "C" int block(int pages, int page, int heads, const int32_t* table, int seqs, int width, int s, int h, int blk) {
    qg::KvCache c = qg::kv8_cache_of(nullptr, nullptr, nullptr, nullptr, pages, page, heads, 64);
    qg::KvSeqs q{table, nullptr, nullptr, seqs, width, 0, 0, 0};
    return qg::kv8_block(c, q, s, h, blk);
}
extern "C" void span(int r0, int r1, int len, int T, int max_new, int max_kv, int* out) {
    qg::KvSpan v = qg::kv8_span_of(r0, r1, len, T, max_new, max_kv);
    out[0] = v.r0; out[1] = v.n; out[2] = v.len;
}
extern "C" uint32_t quotient(uint32_t blk, int nb) {
    qg::KvCache c = qg::kv8_cache_of(nullptr, nullptr, nullptr, nullptr, 1, 16 * nb, 1, 64);
    return qg::kv8_div(blk, c.nb, c.magic);
}
''')
    so = d / "place.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "block_quantized_weight_affine_amd", "csrc"), str(src), "-o", str(so)], check=True)
    return C.CDLL(str(so))


@pytest.mark.parametrize("page", [16, 48, 64, 4080])
def test_block_index_of_any_table(place, page):
    """Every index that comes out lies inside the cache, whatever the table holds."""
    rng = np.random.default_rng(page)
    pages, heads, seqs, width = 7, 3, 4, 5
    bad = np.array([-1, pages, 2 ** 31 - 1, -2 ** 31, 0, 6, 3], np.int64)
    table = rng.choice(bad, (seqs, width)).astype(np.int32)
    nb = page // 16
    for s in range(seqs):
        for blk in [-5, -1, 0, 1, nb - 1, nb, nb + 1, 3 * nb + nb // 2, 5 * nb - 1, 5 * nb, 5 * nb + 1, 1 << 20]:
            got = place.block(pages, page, heads, table.ctypes.data_as(C.c_void_p), seqs, width, s, 2, blk)
            want = -1
            at = serve8.place(table, page, pages, s, 16 * blk) if blk >= 0 else None
            if at is not None:
                want = (at[0] * heads + 2) * nb + at[1] // 16
            assert got == want
            assert got < pages * heads * nb


def test_division_by_blocks_of_a_page(place):
    rng = np.random.default_rng(5)
    for nb in [1, 2, 3, 5, 7, 255, 1023, 4095, 4096]:
        x = np.concatenate([rng.integers(0, 1 << 20, 400), [0, 1, nb - 1, nb, (1 << 20) - 1, ((1 << 20) // nb) * nb - 1]])
        for b in x.tolist():
            assert place.quotient(b, nb) == b // nb


def test_spans_that_contradict_themselves(place):
    T, max_new, max_kv = 10, 4, 50
    cases = [(0, 4, 50), (0, 5, 50), (3, 2, 9), (-1, 2, 9), (8, 11, 9), (0, 3, 2), (0, 3, 51), (5, 5, 0), (0, 1, 1),
             (-2 ** 31, 2 ** 31 - 1, 5), (2, 4, -1)]
    for r0, r1, n in cases:
        out = (C.c_int * 3)()
        place.span(r0, r1, n, T, max_new, max_kv, out)
        assert list(out) == list(serve8.spans([r0, r1], [n], T, max_new, max_kv)[0])


# ---- pins of the plain definitions ------------------------------------------------------------------
def test_pin_layout():
    c = np.arange(2 * 1 * 32 * 64, dtype=np.int64).astype(np.int8).reshape(2, 1, 32, 64)
    k, v = serve8.layout(c, "k"), serve8.layout(c, "v")
    for p, t, d in [(0, 0, 0), (1, 17, 5), (0, 31, 63), (1, 2, 16)]:
        base = (p * 2 + t // 16) * 16 * 64
        assert k.reshape(-1)[base + (d // 16 * 16 + t % 16) * 16 + d % 16] == c[p, 0, t, d]
        assert v.reshape(-1)[base + d * 16 + t % 16] == c[p, 0, t, d]
    assert np.array_equal(serve8.meaning(k, "k", 2, 1, 32, 64), c)
    assert np.array_equal(serve8.meaning(v, "v", 2, 1, 32, 64), c)


def test_pin_write_by_hand():
    codes, scales = np.zeros((1, 1, 16, 64), np.int8), np.zeros((1, 1, 1), np.float32)
    table = np.zeros((1, 1), np.int32)
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, :3] = [127.0, -63.5, 0.5]        # d = 1 (127 / 127): 127, -64 (tie to even), 0
    x[1, 0, :2] = [254.0, 1.0]
    serve8.kv8_write(codes, scales, table, [(0, 1, 1)], x[:1])
    d1 = np.float32(127) * serve8.PER127
    assert scales[0, 0, 0] == d1 and abs(d1 - 1) < 1e-6
    assert list(codes[0, 0, 0, :3]) == [127, -64, 0]
    serve8.kv8_write(codes, scales, table, [(1, 1, 2)], x)   # the scale doubles: earlier codes are halved
    assert scales[0, 0, 0] == np.float32(254) * serve8.PER127
    assert list(codes[0, 0, 0, :3]) == [64, -32, 0]          # 63.5 to even
    assert list(codes[0, 0, 1, :2]) == [127, 0]              # 0.5 to even


def test_pin_attend_against_brute_force():
    rng = np.random.default_rng(1)
    P, H, page, D, n = 3, 2, 16, 64, 20
    kc, vc = (rng.integers(-127, 128, (P, H, page, D)).astype(np.int8) for _ in "kv")
    ks, vs = (rng.uniform(0.001, 0.01, (P, H, 1)).astype(np.float32) for _ in "kv")
    table = np.array([[2, 0]], np.int32)
    q = rng.normal(size=(2, 4, D))
    o, mean, _, top = serve8.attend(kc, ks, vc, vs, table, [(0, 2, n)], q, 0.125, True, 7)
    for i in range(2):
        for qh in range(4):
            num, den = np.zeros(D), 0.0
            for j in range(n):
                if j <= 18 + i and j > 18 + i - 7:
                    p, t, h = int(table[0, j // 16]), j % 16, qh // 2
                    w = np.exp(0.125 * float(q[i, qh] @ (kc[p, h, t].astype(float) * ks[p, h, 0])))
                    num, den = num + w * vc[p, h, t] * float(vs[p, h, 0]), den + w
            assert np.allclose(o[i, qh], num / den, rtol=1e-12)
    assert np.all(np.abs(o) <= mean + 1e-15) and np.all(mean <= top + 1e-15)
    o, *_ = serve8.attend(kc, ks, vc, vs, np.array([[-1, 9]], np.int32), [(0, 2, n)], q, 0.125, True, 0)
    assert np.all(o == 0)


def test_pin_w8a8_by_hand():
    x = np.zeros((3, 16), np.float32)
    x[0, :2] = [127.0, -2.4]                 # d = 1: codes 127, -2
    x[2, 0] = np.inf
    w = np.zeros((2, 16), np.int8)
    w[0, :2], w[1, 1] = [3, 5], -128
    y = serve8.w8a8(w, np.array([0.5, 2.0], np.float32), x)
    d = np.float32(127) * serve8.PER127
    assert y[0, 0] == np.float32(np.float32(371) * d) * np.float32(0.5)
    assert y[0, 1] == np.float32(np.float32(256) * d) * np.float32(2)
    assert np.all(y[1] == 0) and np.all(np.isnan(y[2]))
