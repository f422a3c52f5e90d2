"""Cases of the 8-bit serving operators: the key/value cache (written and read back), attention over
it, and the product in 8-bit integers.

Where `own` is false, `run` computes an operator in plain torch, 32-bit arithmetic; where it is true,
through the library's entry points.  `exact` gives the same outputs from the definitions in 64 bits.

The cache is paged: a page holds `page` tokens of every head, in blocks of 16 tokens with one f32
scale a block and head for K and one for V.  K codes are [pages][heads][page/16][dim/16][16 tokens]
[16 dims], V codes [pages][heads][page/16][dim][16 tokens], scales [pages][heads][page/16].
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_BLOCK = 16
#: 1/127 and the largest finite value, as f32: a block's scale is d = amax * (1/127), and its values
#: are coded as rint(x * min(1/d, largest)).
_PER_127 = 1.0 / 127.0
_LARGEST = torch.finfo(torch.float32).max


def listed():
    return [
        # one decoding step of a full batch: each sequence's new token into its last block
        dict(name="cache_step", op="cache", seqs=48, new=1, ragged=False, hist=4000, heads=8, dim=128, page=64,
             xt="bf16", yt="bf16", lens=1),
        # whole prompts written into fresh pages, and read back by a kernel that wants 16-bit values
        dict(name="cache_prompt", op="cache", seqs=6, new=4096, ragged=False, hist=0, heads=8, dim=128, page=64,
             xt="bf16", yt="bf16", lens=2),
        # chunks of odd lengths that begin inside a block, f32 from the block-quantised matmuls
        dict(name="cache_chunks", op="cache", seqs=13, new=701, ragged=True, hist=1999, heads=5, dim=96, page=48,
             xt="f32", yt="f16", lens=3),
        # one user's next token: latency
        dict(name="attend_one", op="attend", seqs=1, new=1, ragged=False, hist=1023, spread=False, q_heads=32, heads=8,
             dim=128, page=64, causal=True, window=0, xt="bf16", lens=4),
        # the next token of a batch of users with histories of many lengths
        dict(name="attend_batch", op="attend", seqs=64, new=1, ragged=False, hist=8191, spread=True, q_heads=32,
             heads=8, dim=128, page=64, causal=True, window=0, xt="bf16", lens=5),
        # the next token over very long documents
        dict(name="attend_long", op="attend", seqs=3, new=1, ragged=False, hist=200001, spread=False, q_heads=64,
             heads=8, dim=128, page=128, causal=True, window=0, xt="f16", lens=6),
        # five drafted tokens a sequence, checked in one pass, f32 activations
        dict(name="attend_draft", op="attend", seqs=16, new=5, ragged=False, hist=2990, spread=True, q_heads=16,
             heads=2, dim=256, page=32, causal=True, window=0, xt="f32", lens=7),
        # chunks of prompts on top of a history, a sliding window, an odd number of heads a group
        dict(name="attend_chunks", op="attend", seqs=5, new=517, ragged=True, hist=6000, spread=True, q_heads=24,
             heads=4, dim=64, page=48, causal=True, window=1024, xt="f16", lens=8),
        # two whole prompts
        dict(name="attend_prompt", op="attend", seqs=2, new=4096, ragged=False, hist=0, spread=False, q_heads=32,
             heads=8, dim=128, page=64, causal=True, window=0, xt="bf16", lens=9),
        # a projection of one token
        dict(name="matmul_token", op="matmul", T=1, N=4096, K=4096, xt="bf16", yt="f32"),
        # a projection of a decoding batch, odd sizes
        dict(name="matmul_batch", op="matmul", T=45, N=11009, K=4112, xt="f16", yt="f16"),
        # a projection of long prompts
        dict(name="matmul_prompt", op="matmul", T=8192, N=8192, K=8192, xt="bf16", yt="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "matmul"])
    lens = rng.randrange(1 << 20)
    if op == "matmul":
        T, N = _log(rng, 1, 8192), _log(rng, 64, 16384)
        K = 16 * _log(rng, 8, 1024)
        while T * N * K > 8192 ** 3:
            T = max(1, T // 2)
        return dict(op=op, T=T, N=N, K=K, xt=rng.choice(["f32", "f16", "bf16"]), yt=rng.choice(["f32", "f16", "bf16"]))
    dim, page = rng.choice([64, 96, 128, 128, 192, 256]), 16 * rng.randint(1, 16)
    heads, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "cache":
        seqs, new = _log(rng, 1, 64), _log(rng, 1, 4096)
        while seqs * new * heads * dim > 6 * 4096 * 8 * 128:
            new = max(1, new // 2)
        return dict(op=op, seqs=seqs, new=new, ragged=rng.random() < 0.5, hist=_log(rng, 1, 5000) - 1, heads=heads,
                    dim=dim, page=page, xt=rng.choice(["f32", "f16", "bf16"]), yt=rng.choice(["f16", "bf16"]), lens=lens)
    kind = rng.choice(["step", "draft", "prompt"])
    new = {"step": 1, "draft": rng.randint(2, 9), "prompt": _log(rng, 16, 4096)}[kind]
    seqs = _log(rng, 1, 64 if kind == "step" else 16 if kind == "draft" else 4)
    hist = _log(rng, 1, 65536 if kind == "step" else 8192) - 1
    while seqs * (hist + new) * heads * dim > 2 ** 28 and hist > 1:
        hist //= 2
    while seqs * heads * group * new * (hist + new) > 2 ** 29 and new > 1:
        new //= 2
    window = 0 if rng.random() < 0.7 else _log(rng, 1, 4096)
    return dict(op=op, seqs=seqs, new=new, ragged=rng.random() < 0.5, hist=hist, spread=rng.random() < 0.5,
                q_heads=heads * group, heads=heads, dim=dim, page=page, causal=rng.random() < 0.85, window=window,
                xt=rng.choice(["f32", "f16", "bf16"]), lens=lens)


# ---- lengths and tables ---------------------------------------------------------------------------
def _lengths(c):
    """(new rows, tokens before them) of each sequence."""
    rng = random.Random(c["lens"])
    new = [rng.randint(0, c["new"]) if c["ragged"] else c["new"] for _ in range(c["seqs"])]
    if not any(new):
        new[0] = 1
    spread = c.get("spread", True)
    return new, [rng.randint(0, c["hist"]) if spread else c["hist"] for _ in range(c["seqs"])]


def _offsets(n):
    out = [0]
    for v in n:
        out.append(out[-1] + v)
    return out


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(c, total, g):
    """A block table: shuffled pages, -1 past a sequence's end; the number of pages; one that is in no
    sequence."""
    need = [-(-t // c["page"]) for t in total]
    ids = torch.randperm(sum(need) + 3, generator=g, device="cuda").tolist()
    width, at, rows = max(1, max(need)), 0, []
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    return _ints(rows), sum(need) + 3, ids[at]


def _seq_row(n):
    """(sequence, index in it) of each row, for rows counted by sequence."""
    s = [i for i, k in enumerate(n) for _ in range(k)]
    j = [q for k in n for q in range(k)]
    return torch.tensor(s, device="cuda"), torch.tensor(j, device="cuda")


def _cache(c, pages, g):
    """A cache whose every block holds coded values, as decoding leaves one: K with channels of very
    different size, V about a mean."""
    H, nb, D = c["heads"], c["page"] // _BLOCK, c["dim"]
    gain = torch.exp(0.6 * torch.randn(H, 1, 1, D, device="cuda", generator=g))
    mean = 0.7 * torch.randn(H, 1, 1, D, device="cuda", generator=g)
    out = []
    for which in ("k", "v"):
        codes = torch.empty((pages, H, nb, D * _BLOCK), dtype=torch.int8, device="cuda")
        scales = torch.empty((pages, H, nb), device="cuda")
        step = max(1, (1 << 27) // (H * nb * D * _BLOCK))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = torch.randn(n, H, nb, _BLOCK, D, device="cuda", generator=g)
            x = x * gain if which == "k" else x + mean
            d = x.abs().amax((-1, -2)) * _PER_127
            q = torch.round(x / d[..., None, None]).clamp(-127, 127).to(torch.int8)
            if which == "k":
                q = q.reshape(n, H, nb, _BLOCK, D // 16, 16).transpose(3, 4)
            else:
                q = q.transpose(3, 4)
            codes[p:p + n] = q.reshape(n, H, nb, -1)
            scales[p:p + n] = d
        out += [codes, scales]
    return dict(k_codes=out[0], k_scales=out[1], v_codes=out[2], v_scales=out[3])


# ---- states ---------------------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "matmul":
        # weights as a loader leaves them: coded once, a scale for each output channel
        w = torch.randn(c["N"], c["K"], device="cuda", generator=g)
        w = w * torch.exp(0.3 * torch.randn(c["N"], 1, device="cuda", generator=g)) / math.sqrt(c["K"])
        st["w_scales"] = w.abs().amax(1) * _PER_127
        st["w_codes"] = torch.round(w / st["w_scales"][:, None]).clamp(-127, 127).to(torch.int8)
        x = torch.randn(c["T"], c["K"], device="cuda", generator=g)
        x = x * torch.exp(0.8 * torch.randn(1, c["K"], device="cuda", generator=g))
        st["x"] = x.to(_TYPES[c["xt"]])
        st["y"] = torch.empty(c["T"], c["N"], dtype=_TYPES[c["yt"]], device="cuda")
        return st
    new, hist = _lengths(c)
    total = [a + b for a, b in zip(new, hist)]
    T, H, D = sum(new), c["heads"], c["dim"]
    st["table"], pages, st["spare"] = _table(c, total, g)
    st.update(_cache(c, pages, g), rows=_ints(_offsets(new)), kv_len=_ints(total), T=T, max_new=max(new),
              max_kv=max(total))
    st["row_seq"], st["row_at"] = _seq_row(new)
    xt = _TYPES[c["xt"]]
    if c["op"] == "cache":
        # K and V side by side, as a fused projection leaves them: rows 2 * heads * dim apart
        kv = torch.randn(T, 2, H, D, device="cuda", generator=g)
        kv = kv * torch.exp(0.5 * torch.randn(T, 1, 1, 1, device="cuda", generator=g))
        st["kv"] = kv.to(xt)
        st["k"], st["v"] = st["kv"][:, 0], st["kv"][:, 1]
        # read back from the first token of the first block that the write touches
        back = [n + h % _BLOCK if n else 0 for n, h in zip(new, hist)]
        st["back_rows"], st["back_T"], st["back_max"] = _ints(_offsets(back)), sum(back), max(back)
        st["back_seq"], st["back_at"] = _seq_row(back)
        st["k_out"], st["v_out"] = (torch.empty(sum(back), H, D, dtype=_TYPES[c["yt"]], device="cuda") for _ in "kv")
    else:
        st["q"] = torch.randn(T, c["q_heads"], D, device="cuda", generator=g).to(xt)
        st["o"] = torch.empty_like(st["q"])
    return st


# ---- the plain forms ------------------------------------------------------------------------------
def _positions(st, rows, seq, at):
    """Position in its sequence of each row: the rows are a sequence's last tokens."""
    n = (rows[1:] - rows[:-1]).long()
    return st["kv_len"].long()[seq] - n[seq] + at


def _places(st, seq, pos):
    """(page, block in page, token in block) of each row."""
    page = st["case"]["page"]
    p = st["table"].long()[seq, pos // page]
    return p, pos % page // _BLOCK, pos % _BLOCK


def _plain_cache(st):
    c = st["case"]
    H, D = c["heads"], c["dim"]
    pos = _positions(st, st["rows"], st["row_seq"], st["row_at"])
    p, b, j = _places(st, st["row_seq"], pos)
    old_pos = st["kv_len"].long() - (st["rows"][1:] - st["rows"][:-1]).long()  # a sequence's first new position
    first = pos // _BLOCK == (old_pos // _BLOCK)[st["row_seq"]]
    begun = first & (old_pos % _BLOCK > 0)[st["row_seq"]]                       # its block held tokens before
    # the blocks that held tokens before: one a sequence, where it has rows and begins inside a block
    s_all = torch.arange(c["seqs"], device="cuda")
    op, ob, oj = _places(st, s_all, old_pos.clamp(max=st["table"].shape[1] * c["page"] - 1))
    part = ((oj > 0) & (st["rows"][1:] > st["rows"][:-1]))
    op = torch.where(part, op, torch.full_like(op, st["spare"]))
    rp, rb, rj = _places(st, st["back_seq"], _positions(st, st["back_rows"], st["back_seq"], st["back_at"]))
    outs = []
    for which in ("k", "v"):
        x = st[which].float()
        codes, scales = st[which + "_codes"], st[which + "_scales"]
        nb = scales.shape[2]
        if which == "k":
            tok = codes.view(-1, H, nb, D // 16, _BLOCK, 16)
        else:
            tok = codes.view(-1, H, nb, D, _BLOCK)
        amax = torch.zeros_like(scales)
        flat = (p[:, None] * H + torch.arange(H, device="cuda")) * nb + b[:, None]
        amax.view(-1).scatter_reduce_(0, flat.reshape(-1), x.abs().amax(-1).reshape(-1), "amax")
        d_new = amax.view(-1)[flat] * _PER_127                                    # [T][H]
        d_old = scales.view(-1)[flat]
        d = torch.where(begun[:, None], torch.maximum(d_old, d_new), d_new)
        inv = torch.where(d > 0, (1.0 / d).clamp(max=_LARGEST), torch.zeros_like(d))
        q = torch.round(x * inv[..., None]).clamp(-127, 127).to(torch.int8)
        # earlier tokens of a block that was begun before: coded again under the larger scale
        o_flat = (op[:, None] * H + torch.arange(H, device="cuda")) * nb + ob[:, None]
        o_old = scales.view(-1)[o_flat]
        o_d = torch.maximum(o_old, amax.view(-1)[o_flat] * _PER_127)
        ratio = torch.where(o_d > o_old, o_old / o_d, torch.ones_like(o_d))
        ratio = torch.where(part[:, None], ratio, torch.ones_like(ratio))
        blocks = codes.view(-1, _BLOCK * D)
        again = torch.round(blocks[o_flat].float() * ratio[..., None]).to(torch.int8)
        keep = part[:, None, None]
        blocks.index_copy_(0, o_flat.reshape(-1), torch.where(keep, again, blocks[o_flat]).reshape(-1, _BLOCK * D))
        # the new tokens
        if which == "k":
            tok[p, :, b, :, j] = q.view(-1, H, D // 16, 16)
        else:
            tok[p, :, b, :, j] = q
        scales.view(-1)[flat] = d
        # read back
        val = tok[rp, :, rb, :, rj].reshape(-1, H, D).float() * scales[rp, :, rb][..., None]
        outs.append(val.to(_TYPES[c["yt"]]))
    return outs


def _gathered(st, which):
    """[seqs][heads][tokens][dim] values of the cache, f32, padded to the longest sequence."""
    c = st["case"]
    H, D, P = c["heads"], c["dim"], c["page"]
    n = -(-st["max_kv"] // P)
    t = st["table"][:, :n].clamp(min=0).long()
    codes = st[which + "_codes"][t]                       # [S][n][H][nb][16 D]
    S, nb = t.shape[0], P // _BLOCK
    if which == "k":
        codes = codes.view(S, n, H, nb, D // 16, _BLOCK, 16).permute(0, 2, 1, 3, 5, 4, 6)
    else:
        codes = codes.view(S, n, H, nb, D, _BLOCK).permute(0, 2, 1, 3, 5, 4)
    scales = st[which + "_scales"][t].permute(0, 2, 1, 3)
    x = codes.reshape(S, H, n, nb, _BLOCK, D).float() * scales[..., None, None]
    return x.reshape(S, H, n * P, D)


def _plain_attend(st):
    c = st["case"]
    H, D, G, S, M = c["heads"], c["dim"], c["q_heads"] // c["heads"], c["seqs"], st["max_new"]
    k, v = _gathered(st, "k"), _gathered(st, "v")
    rows = st["rows"].long()
    n = rows[1:] - rows[:-1]
    i = torch.arange(M, device="cuda")
    at = (rows[:-1, None] + i).clamp(max=st["T"] - 1)
    q = st["q"].float()[at].view(S, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * M, D)
    s = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    pos = (st["kv_len"].long() - n)[:, None] + i                       # [S][M]
    j = torch.arange(k.shape[2], device="cuda")
    seen = j < st["kv_len"].long()[:, None, None]
    if c["causal"]:
        seen = seen & (j <= pos[..., None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    seen = seen.expand(S, M, -1)[:, None, None].expand(S, H, G, M, -1).reshape(s.shape)
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    e = torch.exp(s.sub_(top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(S, H, G, M, D).permute(0, 3, 1, 2, 4).reshape(S, M, H * G, D)
    return o[st["row_seq"], st["row_at"]].to(st["q"].dtype)


def _plain_matmul(st):
    c = st["case"]
    x = st["x"].float()
    d = x.abs().amax(1) * _PER_127
    inv = torch.where(d > 0, (1.0 / d).clamp(max=_LARGEST), torch.zeros_like(d))
    q = torch.round(x * inv[:, None]).clamp(-127, 127)
    y = torch.matmul(q, st["w_codes"].float().t())
    return (y * d[:, None] * st["w_scales"]).to(_TYPES[c["yt"]])


# ---- one pass -------------------------------------------------------------------------------------
def _handles(st):
    """What a program makes once: the descriptors of the cache and of the batch, and a workspace."""
    import block_quantized_weight_affine_amd as qg
    if "handles" not in st:
        c = st["case"]
        if c["op"] == "matmul":
            ws = torch.empty(max(16, qg.qgemm_w8a8_workspace(c["N"], c["K"], c["T"])), dtype=torch.uint8, device="cuda")
            st["handles"] = (ws,)
        else:
            cache = qg.kv8_cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], c["page"], c["heads"],
                                 c["dim"])
            seqs = qg.kv8_seqs(st["table"], st["rows"], st["kv_len"], st["T"], st["max_new"], st["max_kv"])
            if c["op"] == "cache":
                back = qg.kv8_seqs(st["table"], st["back_rows"], st["kv_len"], st["back_T"], st["back_max"],
                                   st["max_kv"])
                st["handles"] = (cache, seqs, back)
            else:
                size = qg.qg_attn_kv8_workspace(cache, seqs, c["q_heads"])
                st["handles"] = (cache, seqs, torch.empty(max(16, size), dtype=torch.uint8, device="cuda"))
    return qg, st["handles"]


def _own_run(st):
    c = st["case"]
    qg, h = _handles(st)
    if c["op"] == "matmul":
        qg.qgemm_w8a8(st["w_codes"], st["w_scales"], st["x"], st["y"], c["N"], c["K"], c["T"], h[0])
        return st["y"]
    if c["op"] == "cache":
        qg.qg_kv8_write(h[0], h[1], st["k"], st["v"])
        qg.qg_kv8_read(h[0], h[2], st["k_out"], st["v_out"])
        return [st["k_out"], st["v_out"]]
    qg.qg_attn_kv8(h[0], h[1], st["q"], st["o"], c["q_heads"], 1.0 / math.sqrt(c["dim"]), c["causal"], c["window"], h[2])
    return st["o"]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return _plain_cache(state) if op == "cache" else _plain_attend(state) if op == "attend" else _plain_matmul(state)


# ---- what a pass cannot do without ----------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "matmul":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": N * K + 4 * N + T * K * _BYTES[c["xt"]] + T * N * _BYTES[c["yt"]], "flops": 2 * T * N * K}
    new, hist = _lengths(c)
    row = 2 * c["heads"] * c["dim"]  # values of K and V a token
    if c["op"] == "cache":
        back = sum(n + h % _BLOCK for n, h in zip(new, hist) if n)
        return {"bytes": sum(new) * row * (_BYTES[c["xt"]] + 1) + back * row * (_BYTES[c["yt"]] + 1), "flops": 0}
    pairs = tokens = 0
    for n, h in zip(new, hist):
        if not n:
            continue
        w = c["window"] or n + h
        lo = max(0, h + 1 - w)
        tokens += n + h - lo
        for p in range(h, h + n):
            last = p if c["causal"] else n + h - 1
            pairs += last - max(0, p - w + 1) + 1
    qo = 2 * sum(new) * c["q_heads"] * c["dim"] * _BYTES[c["xt"]]
    return {"bytes": tokens * (row + row // c["dim"] / 4) + qo, "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ---- the definitions in 64 bits -------------------------------------------------------------------
def _tokens64(st, which, s, lo, hi):
    """Codes and scales of tokens lo..hi-1 of sequence s: [tokens][heads][dim] and [tokens][heads], f64."""
    c = st["case"]
    H, D, P = c["heads"], c["dim"], c["page"]
    t = torch.arange(lo, hi, device="cuda")
    page = st["table"][s].long()[t // P]
    blk, j = t % P // _BLOCK, t % _BLOCK
    codes = st[which + "_codes"]
    if which == "k":
        q = codes.view(codes.shape[0], H, P // _BLOCK, D // 16, _BLOCK, 16)[page, :, blk, :, j].reshape(-1, H, D)
    else:
        q = codes.view(codes.shape[0], H, P // _BLOCK, D, _BLOCK)[page, :, blk, :, j]
    return q.double(), st[which + "_scales"][page, :, blk].double()


def _exact_cache(st):
    c = st["case"]
    new, hist = _lengths(c)
    outs = []
    for which in ("k", "v"):
        got, at = [], 0
        for s, (n, h) in enumerate(zip(new, hist)):
            if not n:
                continue
            x = st[which][at:at + n].double()
            at += n
            lo = h - h % _BLOCK
            q_old, d_old = _tokens64(st, which, s, lo, h)
            for b in range(lo, h + n, _BLOCK):
                rows = x[max(b, h) - h:min(b + _BLOCK, h + n) - h]
                d = rows.abs().amax((0, 2)) / 127.0
                if b < h:
                    d = torch.maximum(d, d_old[0])
                    got.append(torch.round(q_old * (d_old / d)[..., None]) * d[:, None])
                got.append(torch.round(rows / d[:, None]).clamp(-127, 127) * d[:, None])
        outs.append(torch.cat(got))
    return outs


def _exact_attend(st):
    c = st["case"]
    new, hist = _lengths(c)
    G, out, at = c["q_heads"] // c["heads"], [], 0
    for s, (n, h) in enumerate(zip(new, hist)):
        q = st["q"][at:at + n].double()
        at += n
        lo = max(0, h + 1 - c["window"]) if c["window"] else 0
        (kq, kd), (vq, vd) = (_tokens64(st, w, s, lo, h + n) for w in "kv")
        j = torch.arange(lo, h + n, device="cuda")[None]
        p = torch.arange(h, h + n, device="cuda")[:, None]
        hidden = (j > p) if c["causal"] else torch.zeros(n, j.shape[1], dtype=torch.bool, device="cuda")
        if c["window"]:
            hidden = hidden | (j <= p - c["window"])
        heads = []
        for head in range(c["q_heads"]):
            kv = head // G
            score = (q[:, head] @ (kq[:, kv] * kd[:, kv, None]).t()) / math.sqrt(c["dim"])
            weight = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            heads.append(weight @ (vq[:, kv] * vd[:, kv, None]))
        out.append(torch.stack(heads, 1))
    return torch.cat(out)


def _exact_matmul(st):
    # which code a value gets is decided in f32, by definition; all that follows is in 64 bits
    x = st["x"].float()
    d = x.abs().amax(1, keepdim=True).mul(torch.tensor(_PER_127, dtype=torch.float32))
    codes = (x * torch.ones_like(d).div(d)).round().double().clamp(-127, 127)
    return (codes * d.double()) @ (st["w_codes"].double() * st["w_scales"].double()[:, None]).t()


def exact(case, seed):
    st = prepare(case, seed)
    return {"cache": _exact_cache, "attend": _exact_attend, "matmul": _exact_matmul}[case["op"]](st)
