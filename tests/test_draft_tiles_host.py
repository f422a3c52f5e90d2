"""CPU checks of the attention's plans: which kernel the library gives the batches of test_gpu_draft_tiles.py, whose definition is
held against oracle/draft.py's, and that the workspace has room for any call under its bounds and no more than it needs."""
import ctypes as C
import math
import os
import random
import subprocess

import numpy as np
import pytest

import block_quantized_weight_affine_amd as qg
from draft_tiles import CASES, attend
from oracle import draft as od
from test_gpu_serve8 import Batch, _values

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = {"f32": qg.QG_X_F32, "f16": qg.QG_X_F16, "bf16": qg.QG_X_BF16}


@pytest.fixture(scope="session")
def plan(tmp_path_factory):
    """(rows a tile, splits) of a call, by the function that the library itself goes by."""
    qg.lib()
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text('''
#include "qg_internal.hpp"
extern "C" void plan(int seqs, int T, int max_new, int max_kv, int heads, int q_heads, int dim, int window, int xt, int tree, int* out) {
    static const uint32_t some = 0;
    qg::AttnParams a{};
    a.c.heads = heads; a.c.dim = dim;
    a.q.seqs = seqs; a.q.T = T; a.q.max_new = max_new; a.q.max_kv = max_kv;
    a.q_heads = q_heads; a.group = q_heads / heads; a.window = window; a.causal = !tree; a.mask = tree ? &some : nullptr;
    qg::attn8_plan(a, xt);
    out[0] = a.tile_rows; out[1] = a.splits; out[2] = qg::attn8_max_splits(a);
}
''')
    so, lib = d / "plan.so", os.path.join(ROOT, "block_quantized_weight_affine_amd")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(lib, "csrc"), str(d / "plan.cpp"), "-o", str(so), "-L", lib, "-l:libqgemm.so",
                    "-Wl,-rpath," + lib], check=True)
    call = C.CDLL(str(so)).plan

    def of(seqs, T, max_new, max_kv, heads, q_heads, dim, window, xt, tree=True):
        out = (C.c_int * 3)()
        call(seqs, T, max_new, max_kv, heads, q_heads, dim, window, NAMES[xt], int(tree), out)
        assert out[1] <= out[2]                             # what the workspace has room for
        return out[0], out[1]
    return of


@pytest.mark.parametrize("name", list(CASES))
def test_the_batches_take_tiles(plan, name):
    lens, heads, q_heads, dim, _, window, xt, tile = CASES[name]
    news, tokens = [n for n, _ in lens], max(t for _, t in lens)
    for w in {0, window}:
        assert plan(len(lens), sum(news), max(news), tokens, heads, q_heads, dim, window, xt)[0] == tile


def test_the_forms_are_all_there(plan):
    """Every head size by f32's tiles and by 16-bit ones, both 16-bit tiles, several splits and one, windows and none."""
    got = {(c[3], c[6] == "f32", c[7]) for c in CASES.values()}
    assert {(d, f) for d, f, _ in got} == {(d, f) for d in (64, 96, 128, 192, 256) for f in (True, False)}
    assert {(d, t) for d, f, t in got if not f and d <= 128} == {(d, t) for d in (64, 96, 128) for t in (128, 256)}
    splits = []
    for lens, heads, q_heads, dim, _, window, xt, tile in CASES.values():
        news, tokens = [n for n, _ in lens], max(t for _, t in lens)
        splits.append((tile, xt == "f32", plan(len(lens), sum(news), max(news), tokens, heads, q_heads, dim, window, xt)[1] > 1))
    for form in ((128, False), (128, True), (256, False)):
        assert {many for *f, many in splits if tuple(f) == form} == {False, True}


@pytest.mark.parametrize("window", [0, 4])
def test_the_definition_for_all_rows(window):
    b = Batch([(9, 30), (0, 5), (33, 33), (2, 40)], 2, 64, 16, 3)
    b.table[3, 1] = -1
    mask = b.rng.integers(0, 1 << 32, (b.T, 2), dtype=np.uint64).astype(np.uint32)
    mask[::4] = 0
    pos = b.rng.integers(-5, 60, b.T).astype(np.int32)
    q = _values(b.rng, (b.T, 6, 64), "f32")
    o, mean, reach, peak = (x.numpy() for x in attend(b, q, 0.1, mask, window, pos, "cpu"))
    want = od.attend(b.kc, b.ks, b.vc, b.vs, b.table, b.spans(), q.double().numpy(), 0.1, mask, window, pos)
    for x, y in zip((o, mean, reach), want):
        assert np.allclose(x, y, rtol=1e-12, atol=1e-13)
    assert np.all(mean <= 127 * 40 * peak) and np.all(peak <= b.vs.max())


def test_the_workspace_has_room_for_every_plan(plan):
    """Any window, type and kind of call under the same bounds (the fixture compares)."""
    rng = random.Random(3)
    log = lambda lo, hi: max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))  # noqa: E731
    for _ in range(3000):
        seqs, heads, group, new = log(1, 200), log(1, 32), log(1, 64), log(1, 1024)
        tokens = max(new, log(1, 1 << 24))
        for _ in range(4):
            window = rng.choice([0, log(1, tokens)])
            for xt in NAMES:
                for tree in (True, False):
                    plan(seqs, seqs * new, new, tokens, heads, heads * group, rng.choice([64, 96, 128, 192, 256]), window, xt, tree)


def test_the_workspace_of_calls_without_trees():
    """Single tokens and prompts of more than 1024 rows, which no tree has, ask for their own splits alone; what trees of no more than
    1024 rows add is what their largest plan takes.  32 heads of 128 on 8: a split's part is 32 x 130 x 4 bytes a row."""
    def asked(seqs, new, tokens):
        c = qg.QgKv8Cache(0x10000, 0x10000, 0x10000, 0x10000, 8, 64, 8, 128)
        s = qg.QgKv8Seqs(0x10000, 0x10000, 0x10000, seqs, 1 << 17, seqs * new, new, tokens)
        size, part = qg.lib().qg_attn_kv8_workspace(C.addressof(c), C.addressof(s), 32), seqs * new * 32 * 130 * 4
        assert size % part == 0
        return size // part
    assert asked(1, 1, 200000) == 32 and asked(64, 1, 8192) == 6 and asked(16, 1, 32768) == 8
    assert asked(1, 1, 1000) == 0 and asked(1, 2048, 200000) == 0
    assert asked(1, 1024, 200000) == 2                     # 128 tiles of 256 rows, twice for 256 CUs
    assert asked(16, 64, 1 << 15) == 2
