"""CPU checks of the operators for drafted tokens: the refusals of their entry points and binding, the frequencies of
rotary positions, and hand-worked pins of the plain definitions that the GPU tests compare with.  Nothing here launches a
kernel."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import draft as od
from test_serve8_host import A, DESCRIPTORS, _cache, _seqs

BIG = 1 << 40


def _rot(**kw):
    a = dict(freqs=A, rot=64, interleaved=0, mscale=1.0)
    a.update(kw)
    return qg.QgRotary(**a)


def _rope(rot=None, pos=A, x=A, xr=512, xh=128, y=2 * A, yr=512, yh=128, xt=qg.QG_X_BF16, T=5, heads=4, dim=128):
    r = rot or _rot()
    return qg.lib().qg_rope(C.addressof(r), pos, x, xr, xh, y, yr, yh, xt, T, heads, dim, None)


def _write(cache=None, seqs=None, rot=None, pos=None, k=A, kr=256, kh=128, v=A, vr=256, vh=128, src=None, src_rows=9, q=A,
           qr=512, qh=128, qo=A, qor=512, qoh=128, q_heads=4, xt=qg.QG_X_BF16):
    c, s, r = cache or _cache(), seqs or _seqs(), rot or _rot()
    return qg.lib().qg_kv8_write_rope(C.addressof(c), C.addressof(s), C.addressof(r), pos, k, kr, kh, v, vr, vh, src, src_rows,
                                      q, qr, qh, qo, qor, qoh, q_heads, xt, None)


def _tree(cache=None, seqs=None, mask=A, words=1, pos=A, q=A, qr=512, qh=128, o=A, orow=512, oh=128, xt=qg.QG_X_BF16,
          q_heads=4, window=0, ws=A, size=BIG):
    c, s = cache or _cache(), seqs or _seqs()
    return qg.lib().qg_attn_kv8_tree(C.addressof(c), C.addressof(s), mask, words, pos, q, qr, qh, o, orow, oh, xt, q_heads, 0.1,
                                     window, ws, size, None)


def _plan(seqs=None, parents=A, mask=A, words=1, pos=A, window=0):
    s = seqs or _seqs()
    return qg.lib().qg_tree_plan(C.addressof(s), parents, mask, words, pos, window, None)


def _verify(seqs=None, parents=None, tokens=A, target=A, tr=1000, draft=None, dr=1000, xt=qg.QG_X_F32, vocab=1000, temps=None,
            accept=A, sample=A, accepted=A, nxt=A, rows=2 * A, path=A, kv=A, ws=A, size=BIG):
    s = seqs or _seqs()
    return qg.lib().qg_draft_verify(C.addressof(s), parents, tokens, target, tr, draft, dr, xt, vocab, temps, accept, sample,
                                    accepted, nxt, rows, path, kv, ws, size, None)


@pytest.mark.parametrize("i", range(len(DESCRIPTORS)))
def test_descriptor_refusals(i):
    kw, want = DESCRIPTORS[i]
    assert _write(**kw) == want
    assert _tree(**kw) == want
    if "cache" not in kw and "xt" not in kw:
        assert _plan(**kw) == want
        assert _verify(**kw) == want


def test_rope_refusals():
    assert _rope(rot=_rot(rot=63)) == qg.QG_ESHAPE
    assert _rope(rot=_rot(rot=130)) == qg.QG_ESHAPE
    assert _rope(rot=_rot(rot=-2)) == qg.QG_ESHAPE
    assert _rope(rot=_rot(freqs=None)) == qg.QG_EINVAL
    assert _rope(rot=_rot(freqs=A + 4)) == qg.QG_EALIGN
    assert _rope(pos=None) == qg.QG_EINVAL
    assert _rope(pos=A + 2) == qg.QG_EALIGN
    assert _rope(x=None) == qg.QG_EINVAL
    assert _rope(x=A + 8) == qg.QG_EALIGN
    assert _rope(xr=516) == qg.QG_EALIGN
    assert _rope(yh=64) == qg.QG_ESHAPE                     # heads that overlap
    assert _rope(y=A, yr=1024) == qg.QG_ESHAPE              # in place with other strides
    assert _rope(T=-1) == qg.QG_ESHAPE
    assert _rope(T=(1 << 21) + 1) == qg.QG_ESHAPE
    assert _rope(heads=0) == qg.QG_ESHAPE
    assert _rope(dim=100) == qg.QG_ESHAPE
    assert _rope(dim=1032) == qg.QG_ESHAPE
    assert _rope(xt=5) == qg.QG_EINVAL
    assert _rope(T=0, pos=None, x=None) == qg.QG_OK
    assert qg.lib().qg_rope(None, A, A, 512, 128, A, 512, 128, 0, 5, 4, 128, None) == qg.QG_EINVAL


def test_write_rope_refusals():
    assert _write(rot=_rot(rot=130)) == qg.QG_ESHAPE
    assert _write(rot=_rot(freqs=None)) == qg.QG_EINVAL
    assert _write(k=None) == qg.QG_EINVAL
    assert _write(v=A + 8) == qg.QG_EALIGN
    assert _write(kr=260) == qg.QG_EALIGN
    assert _write(vh=-128) == qg.QG_ESHAPE
    assert _write(pos=A + 1) == qg.QG_EALIGN
    assert _write(src=A + 2, q_heads=0) == qg.QG_EALIGN
    assert _write(src=A) == qg.QG_EUNSUPPORTED              # q has the batch's rows, not src's
    assert _write(src_rows=-1) == qg.QG_ESHAPE
    assert _write(q_heads=-1) == qg.QG_ESHAPE
    assert _write(q=None) == qg.QG_EINVAL
    assert _write(qo=None) == qg.QG_EINVAL
    assert _write(qoh=0, qo=2 * A) == qg.QG_ESHAPE
    assert _write(qor=1024) == qg.QG_ESHAPE                 # in place with other strides
    assert _write(seqs=_seqs(T=0, max_new=0), k=None, q=None) == qg.QG_OK
    s, c = _seqs(), _cache()
    assert qg.lib().qg_kv8_write_rope(C.addressof(c), C.addressof(s), None, None, A, 256, 128, A, 256, 128, None, 9, None, 0, 0,
                                      None, 0, 0, 0, 0, None) == qg.QG_EINVAL


def test_tree_refusals():
    wide = _seqs(T=2000, max_new=1025, max_kv=3000)
    assert _plan(seqs=wide, words=33) == qg.QG_ESHAPE
    assert _tree(seqs=wide, words=33) == qg.QG_ESHAPE
    deep = _seqs(T=70, max_new=65)
    for f in (_plan, _tree):
        assert f(seqs=deep, words=2) == qg.QG_ESHAPE
        assert f(words=0) == qg.QG_ESHAPE
        assert f(words=33) == qg.QG_ESHAPE
        assert f(words=1 << 30) == qg.QG_ESHAPE
        assert f(mask=None) == qg.QG_EINVAL
        assert f(mask=A + 2) == qg.QG_EALIGN
        assert f(pos=A + 1) == qg.QG_EALIGN
    assert _plan(parents=None) == qg.QG_EINVAL
    assert _plan(parents=A + 2) == qg.QG_EALIGN
    assert _plan(pos=None) == qg.QG_EINVAL
    assert _plan(seqs=_seqs(T=0, max_new=0), parents=None) == qg.QG_OK
    assert _tree(pos=None, window=5) == qg.QG_EINVAL
    assert _tree(q_heads=3) == qg.QG_ESHAPE
    assert _tree(oh=0) == qg.QG_ESHAPE
    assert _tree(q=None) == qg.QG_EINVAL
    assert _tree(seqs=_seqs(T=0, max_new=0), mask=None) == qg.QG_OK
    long = _seqs(max_kv=1 << 20, T=3, max_new=1)
    assert _tree(seqs=long, size=0) == qg.QG_EWORKSPACE
    assert _tree(seqs=long, ws=A + 4) == qg.QG_EALIGN
    c = _cache()
    L = qg.lib()
    assert L.qg_attn_kv8_tree(C.addressof(c), None, A, 1, A, A, 512, 128, A, 512, 128, 0, 4, 0.1, 0, A, BIG, None) == qg.QG_EINVAL
    assert L.qg_tree_plan(None, A, A, 1, A, 0, None) == qg.QG_EINVAL


def test_verify_refusals():
    assert _verify(xt=4) == qg.QG_EINVAL
    assert _verify(vocab=0, tr=5) == qg.QG_ESHAPE
    assert _verify(vocab=(1 << 24) + 1, tr=1 << 25) == qg.QG_ESHAPE
    assert _verify(tr=999) == qg.QG_ESHAPE
    assert _verify(tr=(1 << 40) + 1) == qg.QG_ESHAPE
    assert _verify(draft=A, dr=999) == qg.QG_ESHAPE
    assert _verify(draft=A, parents=A) == qg.QG_EUNSUPPORTED
    assert _verify(draft=A, accept=None) == qg.QG_EINVAL
    for name in ("tokens", "target", "accepted", "nxt", "rows", "path", "kv"):
        assert _verify(**{name: None}) == qg.QG_EINVAL
        assert _verify(**{name: A + 2}) == qg.QG_EALIGN
    for name in ("parents", "temps", "sample", "accept"):
        assert _verify(**{name: A + 1}) == qg.QG_EALIGN
    assert _verify(xt=qg.QG_X_F16, target=A + 1) == qg.QG_EALIGN
    assert _verify(draft=A + 2) == qg.QG_EALIGN
    assert _verify(rows=A) == qg.QG_EINVAL                  # the batch's own rows
    assert _verify(seqs=_seqs(T=2000, max_new=1025, max_kv=3000)) == qg.QG_ESHAPE
    s = _seqs()
    need = qg.lib().qg_draft_verify_workspace(C.addressof(s), 1000)
    assert need > 0
    assert _verify(size=need - 1) == qg.QG_EWORKSPACE
    assert _verify(ws=None) == qg.QG_EWORKSPACE
    assert _verify(ws=A + 4, size=need) == qg.QG_EALIGN
    assert _verify(seqs=_seqs(T=0, max_new=0), tokens=None, target=None) == qg.QG_OK
    assert qg.lib().qg_draft_verify_workspace(C.addressof(s), 0) == 0
    assert qg.lib().qg_draft_verify_workspace(None, 1000) == 0


def test_binding_refusals():
    """What the C side cannot see: element types, contiguity, shapes."""
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    cache = qg.kv8_cache(*qg.kv8_pages(4, 32, 2, 64, device="cpu"), 32, 2, 64)
    seqs = qg.kv8_seqs(i(1, 2), i(2), i(1), 3, 3, 40)
    rot = qg.rotary(torch.zeros(16, dtype=torch.float64))
    assert (rot.struct.rot, rot.struct.interleaved, rot.struct.mscale) == (32, 0, 1.0)
    none = qg.rotary(None)
    assert none.struct.rot == 0
    x, f = torch.zeros(3, 2, 64), torch.zeros(3)

    def refused(status, call, *a, **kw):
        with pytest.raises(qg.QGError) as e:
            call(*a, stream=0, **kw)
        assert e.value.status == status

    for bad in (torch.zeros(16), torch.zeros(2, 8, dtype=torch.float64), torch.zeros(32, dtype=torch.float64)[::2]):
        with pytest.raises(qg.QGError):
            qg.rotary(bad)
    refused(qg.QG_EINVAL, qg.qg_rope, rot, i(3), x, x.half())
    refused(qg.QG_EINVAL, qg.qg_rope, rot, i(3).long(), x, x)
    refused(qg.QG_ESHAPE, qg.qg_rope, rot, i(2), x, x)
    refused(qg.QG_ESHAPE, qg.qg_rope, rot, i(3), x, x[:2])
    refused(qg.QG_ESHAPE, qg.qg_rope, rot, i(3), x[0], x[0])
    refused(qg.QG_EALIGN, qg.qg_rope, rot, i(6)[::2], x, x)
    refused(qg.QG_EALIGN, qg.qg_rope, rot, i(3), torch.zeros(3, 2, 128)[..., ::2], x)
    w = qg.qg_kv8_write_rope
    refused(qg.QG_EINVAL, w, cache, seqs, rot, x, x.half())
    refused(qg.QG_ESHAPE, w, cache, seqs, rot, x[:2], x[:2])
    refused(qg.QG_ESHAPE, w, cache, seqs, rot, torch.zeros(5, 2, 64), x, src=i(3))
    refused(qg.QG_ESHAPE, w, cache, seqs, rot, x, x, pos=i(2))
    refused(qg.QG_EINVAL, w, cache, seqs, rot, x, x, src=i(3).long())
    refused(qg.QG_EINVAL, w, cache, seqs, rot, x, x, x)
    refused(qg.QG_EINVAL, w, cache, seqs, rot, x, x, x, x.half())
    refused(qg.QG_ESHAPE, w, cache, seqs, rot, x, x, x, torch.zeros(3, 4, 64))
    refused(qg.QG_ESHAPE, w, cache, seqs, rot, x, x, torch.zeros(3, 0, 64), torch.zeros(3, 0, 64))
    refused(qg.QG_EINVAL, qg.qg_tree_plan, seqs, i(3), i(3, 1).long(), i(3))
    refused(qg.QG_EINVAL, qg.qg_tree_plan, seqs, i(3).float(), i(3, 1), i(3))
    refused(qg.QG_ESHAPE, qg.qg_tree_plan, seqs, i(3), i(2, 1), i(3))
    refused(qg.QG_ESHAPE, qg.qg_tree_plan, seqs, i(2), i(3, 1), i(3))
    refused(qg.QG_EALIGN, qg.qg_tree_plan, seqs, i(3), i(3, 2)[:, ::2], i(3))
    refused(qg.QG_EINVAL, qg.qg_attn_kv8_tree, cache, seqs, i(3, 1), x, x.half(), 2, 1.0)
    refused(qg.QG_EINVAL, qg.qg_attn_kv8_tree, cache, seqs, i(3, 1).float(), x, x, 2, 1.0)
    refused(qg.QG_ESHAPE, qg.qg_attn_kv8_tree, cache, seqs, i(3, 1), x, x, 4, 1.0)
    refused(qg.QG_ESHAPE, qg.qg_attn_kv8_tree, cache, seqs, i(3, 1), x, x, 2, 1.0, 5, i(2))
    l, outs = torch.zeros(3, 50), [i(1), i(1), i(2), i(3), i(1)]
    v = qg.qg_draft_verify
    refused(qg.QG_EINVAL, v, seqs, i(3).long(), l, *outs)
    refused(qg.QG_EINVAL, v, seqs, i(3), l, *outs, draft=l.half())
    refused(qg.QG_EINVAL, v, seqs, i(3), l, *outs, sample=f.double())
    refused(qg.QG_EINVAL, v, seqs, i(3), l.double(), *outs)
    refused(qg.QG_ESHAPE, v, seqs, i(3), l[:2], *outs)
    refused(qg.QG_ESHAPE, v, seqs, i(3), l, *outs, draft=torch.zeros(3, 49))
    refused(qg.QG_ESHAPE, v, seqs, i(3), l, *outs, temps=torch.zeros(0))
    refused(qg.QG_ESHAPE, v, seqs, i(3), l, i(1), i(1), i(1), i(3), i(1))
    refused(qg.QG_EALIGN, v, seqs, i(3), torch.zeros(3, 100)[:, ::2], *outs)
    refused(qg.QG_EWORKSPACE, v, seqs, i(3), l, *outs)


# ---- frequencies ------------------------------------------------------------------------------------
def test_frequencies():
    rot, base, s, ctx = 64, 10000.0, 8.0, 4096.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    close = lambda a, b: np.allclose(a, b, rtol=1e-14, atol=0)  # noqa: E731
    got, m = qg.rope_freqs(rot)
    assert close(got, f) and m == 1.0 and got.dtype == np.float64
    got, m = qg.rope_freqs(rot, base, "linear", s)
    assert close(got, f / s) and m == 1.0
    got, m = qg.rope_freqs(rot, base, "ntk", s)
    assert close(got, (base * s ** (64 / 62)) ** (-2.0 * i / rot)) and m == 1.0
    assert close(got[-1], f[-1] / s)                        # the slowest pair is slowed down by the factor
    got, m = qg.rope_freqs(rot, base, "bands", s, ctx, 1.0, 4.0)
    turns = ctx * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    assert close(got, keep * f + (1 - keep) * f / s) and m == 1.0
    assert close(got[turns >= 4], f[turns >= 4]) and close(got[turns <= 1], f[turns <= 1] / s)
    got, m = qg.rope_freqs(rot, base, "yarn", s, ctx, 1.0, 32.0)
    # pairs that make 32 and 1 turns over 4096: 32 ln(4096 / 64 pi) / ln 10000 = 10.5, 32 ln(4096 / 2 pi) / ln 10000 = 22.5
    keep = np.clip(1 - (i - 10) / (23 - 10), 0, 1)
    assert close(got, keep * f + (1 - keep) * f / s)
    assert m == np.float32(0.1 * math.log(8) + 1)
    assert close(qg.rope_freqs(rot, base, "yarn", 1.0, ctx)[0], f)


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), qg.QG_ESHAPE), (dict(rot=63), qg.QG_ESHAPE), (dict(rot=1026), qg.QG_ESHAPE),
    (dict(rot=2, scaling="ntk", factor=2.0), qg.QG_ESHAPE), (dict(rot=64, base=1.0), qg.QG_EINVAL),
    (dict(rot=64, base=math.inf), qg.QG_EINVAL), (dict(rot=64, scaling="linear", factor=0.5), qg.QG_EINVAL),
    (dict(rot=64, scaling="linear", factor=math.nan), qg.QG_EINVAL), (dict(rot=64, scaling="yarn", factor=2.0), qg.QG_EINVAL),
    (dict(rot=64, scaling="bands", factor=2.0, context=4096, low=4.0, high=4.0), qg.QG_EINVAL),
    (dict(rot=64, scaling="bands", factor=2.0, context=4096, low=0.0), qg.QG_EINVAL),
    (dict(rot=64, scaling="other"), qg.QG_EINVAL), (dict(rot=64, scaling=5), qg.QG_EINVAL)])
def test_frequency_refusals(kw, status):
    with pytest.raises(qg.QGError) as e:
        qg.rope_freqs(**kw)
    assert e.value.status == status


# ---- pins of the plain definitions ------------------------------------------------------------------
def test_pin_rope():
    """A quarter of a turn of (3, 4) is (-4, 3), whichever way pairs lie; what is not turned stays."""
    x = np.zeros((2, 1, 8))
    x[:, 0, :] = [3, 30, 4, 40, 5, 6, 7, 8]
    quarter, none = np.pi / 2, 0.0
    y, mag = od.rope(x, [1, 0], np.array([quarter, none]), False, 2.0)
    assert np.allclose(y[0, 0], [-8, 60, 6, 80, 5, 6, 7, 8], atol=1e-14)
    assert np.allclose(y[1, 0], [6, 60, 8, 80, 5, 6, 7, 8])
    assert np.allclose(mag[0, 0], [14, 140, 14, 140, 5, 6, 7, 8])
    y, _ = od.rope(x, [1, -1], np.array([quarter]), True, 1.0)
    assert np.allclose(y[0, 0], [-30, 3, 4, 40, 5, 6, 7, 8], atol=1e-13)
    assert np.allclose(y[1, 0], [30, -3, 4, 40, 5, 6, 7, 8], atol=1e-13)


def test_pin_plan():
    #   0 - 1 - 3        second sequence: 0, and 1 whose parent is no row before it
    #     \ 2
    mask, pos = od.plan([-1, 0, 0, 1, -1, 5], [(0, 4, 14), (4, 2, 2)], 1, 0, 6)
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b1, 0b10]
    assert pos.tolist() == [10, 11, 11, 12, 0, 0]
    mask, _ = od.plan([-1, 0, 0, 1], [(0, 4, 14)], 1, 2, 4)
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1010]


def test_pin_verify():
    p = np.log(np.array([[0.5, 0.25, 0.25], [0.125, 0.375, 0.5], [1.0, 1.0, 2.0]]))
    q = np.log(np.array([[0.25, 0.25, 0.5], [0.5, 0.25, 0.25], [np.nan] * 3]))
    sp, kv = [(0, 3, 20)], [20]

    def run(tokens, accept, sample, **kw):
        return [x.tolist() for x in od.verify(sp, kv, 3, np.array(tokens), p, np.array(sample), draft=q,
                                              accept=np.array(accept), **kw)]

    # token 2 of probability 1/4 under the target, 1/2 under the draft: stays below a half
    assert run([9, 2, 1], [0, 0.49, 0.99], [0, 0, 0.6])[:2] == [[2], [2]]
    assert run([9, 2, 1], [0, 0.51, 0.0], [0.99, 0, 0])[:2] == [[0], [0]]       # p - q is (1/4, 0, -1/4): token 0
    assert run([9, 0, 0], [0, 0.9, 0.26], [0, 0.3, 0])[:2] == [[1], [1]]       # (-3/8, 1/8, 1/4): a third is token 1's
    assert run([9, 0, 0], [0, 0.9, 0.26], [0, 0.34, 0])[:2] == [[1], [2]]
    got = run([9, 0, 0], [0, 0.9, 0.26], [0, 0.34, 0])
    assert got[2:] == [[0, 2], [0, 1, -1], [19]]
    # the largest logit, the first of equal ones
    assert run([9, 0, 2], [0, 0.9, 0.9], [0, 0, 0], temps=[0.0])[:2] == [[2], [2]]
    assert run([9, 1, 2], [0, 0.0, 0.0], [0, 0, 0], temps=[0.0])[:2] == [[0], [0]]
    # chosen tokens in a tree: 0 -> 1, 2 (twins of token 1), 2 -> nothing; row 0 draws token 1 at 0.6
    tree = od.verify(sp, kv, 3, np.array([7, 1, 1]), p, np.array([0.6, 0.2, 0.2]), parents=[-1, 0, 0])
    assert [x.tolist() for x in tree] == [[1], [1], [0, 2], [0, 1, -1], [19]]
    # a temperature of one half squares the odds: (4, 1, 1) / 6
    tree = od.verify(sp, kv, 3, np.array([7, 2, 2]), p, np.array([0.66, 0, 0]), temps=[0.5], parents=[-1, 0, 0])
    assert [tree[0].tolist(), tree[1].tolist()] == [[0], [0]]
    none = od.verify([(0, 0, 0), (0, 1, 5)], [3, 5], 1, np.array([0]), np.full((1, 3), -np.inf), np.array([0.5]))
    assert [x.tolist() for x in none] == [[0, 0], [-1, -1], [0, 0, 1], [0], [3, 5]]


def test_drawn_tokens_follow_the_target():
    """The scheme's point: whatever the draft, what comes out first is distributed as the target's first token."""
    rng = np.random.default_rng(0)
    p, q = np.array([0.5, 0.3, 0.15, 0.05]), np.array([0.1, 0.2, 0.3, 0.4])
    logits, draft = np.log(np.stack([p, p])), np.log(np.stack([q, q]))
    n, hits = 4000, np.zeros(4)
    for _ in range(n):
        x = rng.choice(4, p=q)
        a, nxt, *_ = od.verify([(0, 2, 9)], [9], 2, np.array([0, x]), logits, rng.random(2), draft=draft, accept=rng.random(2))
        hits[x if a[0] else nxt[0]] += 1
    assert np.all(np.abs(hits / n - p) < 5 * np.sqrt(p * (1 - p) / n))   # five standard deviations
