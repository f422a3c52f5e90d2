"""The 8-bit serving operators where a call's bounds ask for more workgroups than one launch may have (a launch counts
its work items in 32 bits): the same results as under tight bounds."""
import pytest
import torch

import block_quantized_weight_affine_amd as qg
from oracle import serve8
from test_gpu_serve8 import TYPES, Batch, _attend, _check_cache, _dev, _values
from test_gpu_serve8_scales import _check

pytestmark = pytest.mark.gpu


def test_attend_tiles_past_one_launch():
    """A bound of 2^17 rows for each of 256 sequences, 8 heads of 8: 2^23 tiles of 256 rows, nearly all of them empty."""
    print("attend: 2^23 tiles", flush=True)
    T = 1 << 17
    b = Batch([(200, 230)] + [(1, 30 + i) for i in range(255)], 8, 64, 64, 61).upload()
    q = torch.zeros(T, 64, 64, dtype=torch.float16, device="cuda")
    q[:b.T] = _values(b.rng, (b.T, 64, 64), "f16").cuda()
    o = torch.full_like(q, 9.0)
    seqs = qg.kv8_seqs(_dev(b.table), _dev(b.rows), _dev(b.kv_len), T, T, T)
    work = torch.empty(max(16, qg.qg_attn_kv8_workspace(b.cache, seqs, 64)), dtype=torch.uint8, device="cuda")
    qg.qg_attn_kv8(b.cache, seqs, q, o, 64, 0.125, True, 0, work)
    torch.cuda.synchronize()
    assert torch.all(o[b.T:] == 9)
    _check(b, q[:b.T], "f16", 0.125, True, 0, o[:b.T])


def test_attend_rows_past_one_launch():
    """65535 sequences of 512 heads, all but a few without rows: 2^25 workgroups of 16 rows."""
    print("attend: 2^25 workgroups of rows", flush=True)
    lens = [(0, 0)] * 65535
    for s, n in ((0, 40), (1, 1), (32768, 250), (65534, 100)):
        lens[s] = (1, n)
    b = Batch(lens, 512, 64, 16, 62).upload()
    q = _values(b.rng, (b.T, 512, 64), "bf16").cuda()
    got = _attend(b, q, 512, 0.125, True, 0)
    _check(b, q, "bf16", 0.125, True, 0, got)


def test_attend_refuses_more_rows_than_it_counts():
    """sequences x max_new x q_heads from 2^37: refused on the host, whatever the type."""
    b = Batch([(1, 20)], 1, 64, 16, 63).upload()
    T = 1 << 16
    table = torch.zeros(1 << 15, 1, dtype=torch.int32, device="cuda")
    rows, kv_len = (torch.zeros((1 << 15) + n, dtype=torch.int32, device="cuda") for n in (1, 0))
    seqs = qg.kv8_seqs(table, rows, kv_len, T, T, T)
    for xt in TYPES.values():
        q = torch.zeros(T, 64, 64, dtype=xt, device="cuda")
        o = torch.full_like(q, 3.0)
        with pytest.raises(qg.QGError) as e:
            qg.qg_attn_kv8(b.cache, seqs, q, o, 64, 0.125, True, 0, None)
        assert e.value.status == qg.QG_ESHAPE
        assert torch.all(o == 3)
    assert qg.qg_attn_kv8_workspace(b.cache, seqs, 64) == 0

def test_write_past_one_launch():
    """A bound of 2^19 new tokens of 1024 heads: 2^24 workgroups.  The rows are one row, repeated by a stride of 0."""
    print("kv8 write: 2^24 workgroups", flush=True)
    b = Batch([(40, 57), (1, 1)], 1024, 64, 16, 64).upload()
    T = 1 << 19
    one = _values(b.rng, (2, 1024, 64), "f16")
    k, v = (x.cuda()[None].expand(T, 1024, 64) for x in one)
    seqs = qg.kv8_seqs(_dev(b.table), _dev(b.rows), _dev(b.kv_len), T, T, T)
    qg.qg_kv8_write(b.cache, seqs, k, v)
    for x, codes, scales in zip(one, (b.kc, b.vc), (b.ks, b.vs)):
        serve8.kv8_write(codes, scales, b.table, b.spans(), x.float().numpy()[None].repeat(b.T, 0))
    torch.cuda.synchronize()
    _check_cache(b, None, None)
