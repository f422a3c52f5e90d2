"""Cases of the operators for drafted tokens: rotary positions, rotation on the way into the 8-bit cache, the
plan of a tree of drafted tokens, attention for it over the cache, and the verification of drafted tokens.

Where `own` is false, `run` computes an operator in plain torch; where it is true, through the library's
entry points.  `exact` gives the same outputs from the definitions in 64 bits.

The cache is paged: a page holds `page` tokens of every head, in blocks of 16 tokens with one f32
scale a block and head for K and one for V.  K codes are [pages][heads][page/16][dim/16][16 tokens]
[16 dims], V codes [pages][heads][page/16][dim][16 tokens], scales [pages][heads][page/16].

A batch's rows are its sequences' last tokens: row r of sequence s is row rows[s] + r of the operands.  In a
tree, parents[r] is the row that row r follows (before it, in its own sequence), -1 where it follows the cache.
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
        # q and K of one decoding step, positions far into long contexts, frequencies scaled for them
        dict(name="rope_step", op="rope", T=48, heads=40, dim=128, rot=128, inter=False, far=1000000, scaled=True,
             fused=8, xt="bf16", lens=1),
        # q and K of long prompts, pairs side by side, half of the head turned, f32 from the block-quantised matmuls
        dict(name="rope_prompt", op="rope", T=8191, heads=40, dim=128, rot=64, inter=True, far=8191, scaled=False,
             fused=0, xt="f32", lens=2),
        # one decoding step of a full batch: q, K turned, K and V into their last blocks
        dict(name="append_step", op="append", seqs=48, new=1, ragged=False, hist=4000, q_heads=32, heads=8, dim=128,
             page=64, rot=128, inter=False, scaled=False, tree=False, picked=False, xt="bf16", yt="bf16", lens=3),
        # prompts of odd lengths on top of histories, part of the head turned
        dict(name="append_prompt", op="append", seqs=7, new=4096, ragged=True, hist=1999, q_heads=32, heads=8, dim=128,
             page=64, rot=64, inter=True, scaled=True, tree=False, picked=False, xt="f16", yt="f16", lens=4),
        # masks and positions of one user's drafts
        dict(name="plan_one", op="plan", seqs=1, nodes=25, ragged=False, hist=1000, wide=4, window=0, lens=5),
        # of a batch of users with larger trees and a sliding window
        dict(name="plan_batch", op="plan", seqs=64, nodes=255, ragged=True, hist=9000, wide=2, window=7, lens=6),
        # one user's tree: latency
        dict(name="tree_one", op="tree", seqs=1, nodes=25, ragged=False, hist=1023, spread=False, q_heads=32, heads=8,
             dim=128, page=64, wide=4, window=0, xt="bf16", lens=7),
        # trees of a batch of users with histories of many lengths
        dict(name="tree_batch", op="tree", seqs=16, nodes=61, ragged=False, hist=8191, spread=True, q_heads=32, heads=8,
             dim=128, page=64, wide=3, window=0, xt="bf16", lens=8),
        # small trees over long documents, f32 activations, a sliding window
        dict(name="tree_long", op="tree", seqs=5, nodes=9, ragged=True, hist=120001, spread=True, q_heads=20, heads=4,
             dim=96, page=48, wide=2, window=90000, xt="f32", lens=9),
        # one user's five drafted tokens against the target's and the draft's probabilities
        dict(name="verify_one", op="verify", seqs=1, nodes=6, ragged=False, vocab=32000, tree=False, sampled=True,
             greedy=0.0, wide=1, xt="f32", lens=10),
        # seven drafted tokens each of a batch of users, some of whom decode greedily
        dict(name="verify_batch", op="verify", seqs=32, nodes=8, ragged=True, vocab=128000, tree=False, sampled=True,
             greedy=0.2, wide=1, xt="bf16", lens=11),
        # trees of chosen tokens, an odd vocabulary
        dict(name="verify_tree", op="verify", seqs=16, nodes=45, ragged=False, vocab=100003, tree=True, sampled=False,
             greedy=0.2, wide=4, xt="f16", lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "plan", "tree", "tree", "verify", "verify"])
    lens = rng.randrange(1 << 20)
    xt = rng.choice(["f32", "f16", "bf16"])
    if op == "plan":
        return dict(op=op, seqs=_log(rng, 1, 64), nodes=_log(rng, 2, 256), ragged=rng.random() < 0.5,
                    hist=_log(rng, 1000, 100000), wide=rng.randint(1, 8), window=0 if rng.random() < 0.6 else _log(rng, 1, 64),
                    lens=lens)
    if op == "verify":
        tree = rng.random() < 0.5
        c = dict(op=op, seqs=_log(rng, 1, 32), nodes=_log(rng, 4, 64) if tree else rng.randint(1, 9),
                 ragged=rng.random() < 0.5, vocab=_log(rng, 500, 160000), tree=tree,
                 sampled=not tree and rng.random() < 0.7, greedy=rng.choice([0.0, 0.2, 1.0]), wide=rng.randint(2, 6), xt=xt,
                 lens=lens)
        while c["seqs"] * c["nodes"] * c["vocab"] > 32 * 8 * 128000:
            c["vocab"] = max(500, c["vocab"] // 2)
        return c
    heads, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        c = dict(op=op, T=_log(rng, 1, 16384), heads=heads * (group + 1), dim=dim, rot=_rot(rng, dim),
                 inter=rng.random() < 0.5, far=_log(rng, 1, 4000000), scaled=rng.random() < 0.5,
                 fused=rng.choice([0, heads]), xt=xt, lens=lens)
        while c["T"] * c["heads"] * dim > 8192 * 40 * 128:
            c["T"] //= 2
        return c
    dim, page = rng.choice([64, 96, 128, 128, 192, 256]), 16 * rng.randint(1, 16)
    if op == "append":
        tree, picked = rng.choice([(False, False), (False, False), (True, False), (False, True)])
        seqs, new = _log(rng, 1, 64), _log(rng, 2, 64) if tree or picked else _log(rng, 1, 4096)
        while seqs * new * heads * (group + 2) * dim > 4 * 4096 * 48 * 128:
            new = max(1, new // 2)
        return dict(op=op, seqs=seqs, new=new, ragged=rng.random() < 0.5, hist=_log(rng, 1, 5000) - 1,
                    q_heads=0 if picked else heads * rng.choice([0, group]), heads=heads, dim=dim, page=page,
                    rot=_rot(rng, dim), inter=rng.random() < 0.5, scaled=rng.random() < 0.5, tree=tree, picked=picked,
                    xt=xt, yt=rng.choice(["f16", "bf16"]), lens=lens)
    nodes, seqs = _log(rng, 2, 160), _log(rng, 1, 16)
    hist = _log(rng, 1, 65536) - 1
    while seqs * (hist + nodes) * heads * dim > 2 ** 28 and hist > 1:
        hist //= 2
    while seqs * heads * group * nodes * (hist + nodes) > 2 ** 29 and nodes > 2:
        nodes //= 2
    return dict(op=op, seqs=seqs, nodes=nodes, ragged=rng.random() < 0.5, hist=hist, spread=rng.random() < 0.5,
                q_heads=heads * group, heads=heads, dim=dim, page=page, wide=rng.randint(1, 6),
                window=0 if rng.random() < 0.7 else _log(rng, 1, 4096), xt=xt, lens=lens)


def _rot(rng, dim):
    """All of the head, half, a quarter, or any even number."""
    return rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])


# ---- lengths, tables, trees -----------------------------------------------------------------------
def _lengths(c):
    """(new rows, tokens before them) of each sequence."""
    rng = random.Random(c["lens"])
    most = c["new"] if "new" in c else c["nodes"]
    new = [rng.randint(0, most) if c["ragged"] else most for _ in range(c["seqs"])]
    if not any(new):
        new[0] = 1
    spread = c.get("spread", True)
    return new, [rng.randint(0, c["hist"]) if spread else c["hist"] for _ in range(c["seqs"])]


def _parents(c, new, seed=0):
    """A tree of each sequence's rows: chains where `wide` is 1, else up to `wide` rows that follow the same one."""
    rng = random.Random(c["lens"] + 1 + seed)
    out = []
    for n in new:
        kids, par = [0] * n, []
        for r in range(n):
            free = [p for p in range(max(0, r - 4 * c["wide"]), r) if kids[p] < c["wide"]]
            par.append(-1 if r == 0 else r - 1 if c["wide"] == 1 else rng.choice(free))
            if r:
                kids[par[-1]] += 1
        out.append(par)
    return out


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
            q = q.reshape(n, H, nb, _BLOCK, D // 16, 16).transpose(3, 4) if which == "k" else q.transpose(3, 4)
            codes[p:p + n] = q.reshape(n, H, nb, -1)
            scales[p:p + n] = d
        out += [codes, scales]
    return dict(k_codes=out[0], k_scales=out[1], v_codes=out[2], v_scales=out[3])


def _freqs(c):
    """Radians a position, f64 [rot / 2], and the factor of the turned values: where scaled, turns that are long against
    a context of 8192 are slowed down by 16, short ones are kept, those between ramped."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / c["rot"])
    if not c["scaled"]:
        return f.cuda(), 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (f * keep + f / 16 * (1 - keep)).cuda(), 0.1 * math.log(16) + 1


# ---- states ---------------------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "rope":
        st["freqs"], st["mscale"] = _freqs(c)
        # heads side by side in a fused projection's rows, V's `fused` heads after them
        x = torch.randn(c["T"], c["heads"] + c["fused"], c["dim"], device="cuda", generator=g)
        st["qkv"] = x.to(_TYPES[c["xt"]])
        st["x"] = st["qkv"][:, :c["heads"]]
        st["pos"] = torch.randint(0, c["far"] + 1, (c["T"],), device="cuda", generator=g, dtype=torch.int32)
        st["y"] = torch.empty(st["x"].shape, dtype=st["x"].dtype, device="cuda")
        return st
    new, hist = _lengths(dict(c, hist=c.get("hist", 3000)))
    if c["op"] == "plan":
        lens = random.Random(seed)
        st["hist"] = hist = [lens.randint(0, c["hist"]) for _ in hist]
    total = [a + b for a, b in zip(new, hist)]
    T = sum(new)
    st.update(rows=_ints(_offsets(new)), kv_len=_ints(total), T=T, max_new=max(new), max_kv=max(total))
    st["row_seq"], st["row_at"] = _seq_row(new)
    if c["op"] == "plan" or c.get("tree") or c["op"] == "tree":
        # work() has to know what a tree's rows see, so only the plan's trees go by the seed
        st["trees"] = _parents(dict(c, wide=c.get("wide", 3)), new, seed if c["op"] == "plan" else 0)
        st["parents"] = _ints([p for par in st["trees"] for p in par])
    words = -(-st["max_new"] // 32)
    if c["op"] == "plan":
        st["table"] = torch.zeros(c["seqs"], 1, dtype=torch.int32, device="cuda")
        st["mask"] = torch.empty(T, words, dtype=torch.int32, device="cuda")
        st["pos"] = torch.empty(T, dtype=torch.int32, device="cuda")
        return st
    if c["op"] == "verify":
        return _prepare_verify(st, g)
    H, D = c["heads"], c["dim"]
    st["table"], pages, st["spare"] = _table(c, total, g)
    st.update(_cache(c, pages, g))
    xt = _TYPES[c["xt"]]
    if c["op"] == "tree":
        seen = _ancestors(st)
        st["mask"], st["pos"] = _bits(seen[st["row_seq"], st["row_at"]], words), _tree_positions(st, seen)
        st["q"] = torch.randn(T, c["q_heads"], D, device="cuda", generator=g).to(xt)
        st["o"] = torch.empty_like(st["q"])
        return st
    st["freqs"], st["mscale"] = _freqs(c)
    # q, K and V side by side, as a fused projection leaves them; of drafted rows those that were taken are picked
    R = 3 * T + 5 if c["picked"] else T
    x = torch.randn(R, c["q_heads"] + 2 * H, D, device="cuda", generator=g)
    x = x * torch.exp(0.5 * torch.randn(R, 1, 1, device="cuda", generator=g))
    st["qkv"] = x.to(xt)
    st["q"], st["k"], st["v"] = st["qkv"].split([c["q_heads"], H, H], 1)
    st["src"] = torch.randperm(R, device="cuda", generator=g)[:T].to(torch.int32) if c["picked"] else None
    st["pos"] = _tree_positions(st, _ancestors(st)) if c["tree"] else None
    st["q_out"] = torch.empty(T, c["q_heads"], D, dtype=xt, device="cuda")
    st["k_out"], st["v_out"] = (torch.empty(T, H, D, dtype=_TYPES[c["yt"]], device="cuda") for _ in "kv")
    return st


def _prepare_verify(st, g):
    """Logits of a target and a draft that agree mostly, drafted tokens as the draft would draw or choose them."""
    c, T, V = st["case"], st["T"], st["case"]["vocab"]
    xt = _TYPES[c["xt"]]
    st["table"] = torch.zeros(c["seqs"], 1, dtype=torch.int32, device="cuda")
    skew = 3.0 * torch.randn(V, device="cuda", generator=g)
    target = 4.0 * torch.randn(T, V, device="cuda", generator=g) + skew
    draft = (target + 0.7 * torch.randn(T, V, device="cuda", generator=g)).to(xt)
    st["target"] = target.to(xt)
    temps = 0.6 + 0.6 * torch.rand(c["seqs"], device="cuda", generator=g)
    pick = torch.rand(c["seqs"], device="cuda", generator=g)
    st["temps"] = torch.where(pick < c["greedy"], torch.zeros_like(temps), temps)
    st["accept"] = torch.rand(T, device="cuda", generator=g)
    st["sample"] = torch.rand(T, device="cuda", generator=g)
    first = st["rows"].long()[:-1][st["row_seq"]]
    if c["tree"]:
        # the rows that follow row p hold the draft's likeliest tokens there, one each
        par = st["parents"].long()
        up = first + par.clamp(min=0)
        same = (up[:, None] == up[None]) & (par >= 0)[None] & (par >= 0)[:, None]
        rank = (same & (torch.arange(T, device="cuda")[:, None] > torch.arange(T, device="cuda")[None])).sum(1)
        best = draft.float().topk(c["wide"], 1).indices
        st["tokens"] = best[up, rank.clamp(max=c["wide"] - 1)].to(torch.int32)
    else:
        st["parents"] = None
        before = (torch.arange(T, device="cuda") - 1).clamp(min=0)
        tau = st["temps"].clamp(min=0.05)[st["row_seq"]][:, None]
        st["tokens"] = torch.multinomial(torch.softmax(draft.float() / tau, 1), 1, generator=g)[:, 0][before].to(torch.int32)
    if c["sampled"]:
        st["draft"] = draft
    n = c["seqs"]
    st["accepted"], st["next"], st["kv_out"] = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3))
    st["rows_out"] = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    st["path"] = torch.empty(T, dtype=torch.int32, device="cuda")
    return st


# ---- the plain forms ------------------------------------------------------------------------------
def _turned(x, pos, freqs, rot, inter, mscale):
    """x [T][heads][dim] turned by the angles pos * freqs, in 64 bits: far positions, and values next to a code's
    border."""
    t = pos.double()[:, None, None] * freqs
    cos, sin = torch.cos(t) * mscale, torch.sin(t) * mscale
    y = x.double().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a].double() * cos - x[..., b].double() * sin
    y[..., b] = x[..., b].double() * cos + x[..., a].double() * sin
    return y


def _plain_rope(st):
    c = st["case"]
    return _turned(st["x"], st["pos"], st["freqs"], c["rot"], c["inter"], st["mscale"]).to(st["x"].dtype)


def _positions(st):
    """Position in its sequence of each row: the rows are a sequence's last tokens."""
    rows = st["rows"].long()
    return (st["kv_len"].long() - (rows[1:] - rows[:-1]))[st["row_seq"]] + st["row_at"]


def _places(st, seq, pos):
    """(page, block in page, token in block) of each row."""
    page = st["case"]["page"]
    p = st["table"].long()[seq, pos // page]
    return p, pos % page // _BLOCK, pos % _BLOCK


def _plain_append(st):
    c = st["case"]
    H, D = c["heads"], c["dim"]
    at = _positions(st)
    turn = (at if st["pos"] is None else st["pos"], st["freqs"], c["rot"], c["inter"], st["mscale"])
    k, v = (st["k"], st["v"]) if st["src"] is None else (st["k"][st["src"].long()], st["v"][st["src"].long()])
    new = {"k": _turned(k, *turn).float(), "v": v.float()}
    outs = [_turned(st["q"], *turn).to(st["q"].dtype)] if c["q_heads"] else []
    p, b, j = _places(st, st["row_seq"], at)
    old_at = st["kv_len"].long() - (st["rows"][1:] - st["rows"][:-1]).long()  # a sequence's first new position
    first = at // _BLOCK == (old_at // _BLOCK)[st["row_seq"]]
    begun = first & (old_at % _BLOCK > 0)[st["row_seq"]]                       # its block held tokens before
    # the blocks that held tokens before: one a sequence, where it has rows and begins inside a block
    s_all = torch.arange(c["seqs"], device="cuda")
    op, ob, oj = _places(st, s_all, old_at.clamp(max=st["table"].shape[1] * c["page"] - 1))
    part = ((oj > 0) & (st["rows"][1:] > st["rows"][:-1]))
    op = torch.where(part, op, torch.full_like(op, st["spare"]))
    heads = torch.arange(H, device="cuda")
    for which in ("k", "v"):
        x = new[which]
        codes, scales = st[which + "_codes"], st[which + "_scales"]
        nb = scales.shape[2]
        tok = codes.view(-1, H, nb, D // 16, _BLOCK, 16) if which == "k" else codes.view(-1, H, nb, D, _BLOCK)
        amax = torch.zeros_like(scales)
        flat = (p[:, None] * H + heads) * nb + b[:, None]
        amax.view(-1).scatter_reduce_(0, flat.reshape(-1), x.abs().amax(-1).reshape(-1), "amax")
        d_new = amax.view(-1)[flat] * _PER_127                                    # [T][H]
        d_old = scales.view(-1)[flat]
        d = torch.where(begun[:, None], torch.maximum(d_old, d_new), d_new)
        inv = torch.where(d > 0, (1.0 / d).clamp(max=_LARGEST), torch.zeros_like(d))
        q = torch.round(x * inv[..., None]).clamp(-127, 127).to(torch.int8)
        # earlier tokens of a block that was begun before: coded again under the larger scale
        o_flat = (op[:, None] * H + heads) * nb + ob[:, None]
        o_old = scales.view(-1)[o_flat]
        o_d = torch.maximum(o_old, amax.view(-1)[o_flat] * _PER_127)
        ratio = torch.where(o_d > o_old, o_old / o_d, torch.ones_like(o_d))
        ratio = torch.where(part[:, None], ratio, torch.ones_like(ratio))
        blocks = codes.view(-1, _BLOCK * D)
        again = torch.round(blocks[o_flat].float() * ratio[..., None]).to(torch.int8)
        keep = part[:, None, None]
        blocks.index_copy_(0, o_flat.reshape(-1), torch.where(keep, again, blocks[o_flat]).reshape(-1, _BLOCK * D))
        # the new tokens
        tok[p, :, b, :, j] = q.view(-1, H, D // 16, 16) if which == "k" else q
        scales.view(-1)[flat] = d
        val = tok[p, :, b, :, j].reshape(-1, H, D).float() * scales[p, :, b][..., None]
        outs.append(val.to(_TYPES[c["yt"]]))
    return outs


def _padded(st, v, fill):
    """Values of rows as [seqs][max_new]."""
    out = torch.full((len(st["kv_len"]), st["max_new"]), fill, dtype=v.dtype, device="cuda")
    out[st["row_seq"], st["row_at"]] = v
    return out


def _ancestors(st):
    """[seqs][max_new][max_new] bool: row r descends from row a, or is it.  The relation's powers, squared."""
    M = st["max_new"]
    par = _padded(st, st["parents"].long(), -1)
    up = torch.zeros(len(par), M, M, device="cuda")
    up.scatter_(2, par.clamp(min=0)[..., None], (par >= 0).float()[..., None])
    up = (up + torch.eye(M, device="cuda")).clamp(max=1)
    for _ in range(max(1, (M - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _tree_positions(st, seen):
    """Position of each row: the tokens before the batch's rows, and the rows that it descends from."""
    rows = st["rows"].long()
    before = (st["kv_len"].long() - (rows[1:] - rows[:-1]))[st["row_seq"]]
    return (before + seen.sum(2)[st["row_seq"], st["row_at"]] - 1).to(torch.int32)


def _bits(seen, words):
    """bool [T][max_new] -> int32 [T][words], bit j % 32 of word j / 32 for row j."""
    x = torch.zeros(seen.shape[0], 32 * words, dtype=torch.int64, device="cuda")
    x[:, :seen.shape[1]] = seen.long()
    x = (x.view(-1, words, 32) << torch.arange(32, device="cuda")).sum(2)
    return torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)


def _plain_plan(st):
    seen = _ancestors(st)
    depth, pos = seen.sum(2), _tree_positions(st, seen)
    if st["case"]["window"]:
        seen = seen & (depth[:, :, None] - depth[:, None, :] < st["case"]["window"])
    words = -(-st["max_new"] // 32)
    return [_bits(seen[st["row_seq"], st["row_at"]], words), pos]


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


def _unpacked(st):
    """The masks as bool [seqs][max_new][max_new]."""
    x = st["mask"].long()[..., None] >> torch.arange(32, device="cuda") & 1
    x = x.reshape(st["T"], -1)[:, :st["max_new"]].bool()
    out = torch.zeros(len(st["kv_len"]), st["max_new"], st["max_new"], dtype=torch.bool, device="cuda")
    out[st["row_seq"], st["row_at"]] = x
    return out


def _plain_tree(st):
    c = st["case"]
    H, D, G, S, M = c["heads"], c["dim"], c["q_heads"] // c["heads"], c["seqs"], st["max_new"]
    k, v = _gathered(st, "k"), _gathered(st, "v")
    rows = st["rows"].long()
    n = rows[1:] - rows[:-1]
    at = (rows[:-1, None] + torch.arange(M, device="cuda")).clamp(max=st["T"] - 1)
    q = st["q"].float()[at].view(S, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * M, D)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()) * (1.0 / math.sqrt(D))
    hist = (st["kv_len"].long() - n)[:, None, None]
    j = torch.arange(k.shape[2], device="cuda")
    seen = (j < hist).expand(S, M, -1)
    if c["window"]:
        seen = seen & (j > _padded(st, st["pos"].long(), 0)[..., None] - c["window"])
    own_row = (j - hist).clamp(min=0, max=M - 1).expand(S, M, -1)
    drafted = (j >= hist) & (j < st["kv_len"].long()[:, None, None])
    seen = seen | (drafted & torch.gather(_unpacked(st), 2, own_row))
    seen = seen[:, None, None].expand(S, H, G, M, -1).reshape(s.shape)
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    e = torch.exp(s.sub_(top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(S, H, G, M, D).permute(0, 3, 1, 2, 4).reshape(S, M, H * G, D)
    return o[st["row_seq"], st["row_at"]].to(st["q"].dtype)


def _weights(logits, tau):
    """exp((l - max) / tau) in 64 bits: sums of many values, and draws next to a border."""
    l = logits.double()
    return torch.exp((l - l.amax(1, keepdim=True)) / tau[:, None])


def _drawn(w, u):
    """The first index whose running sum of w exceeds u times the whole."""
    run = torch.cumsum(w, 1)
    v = torch.searchsorted(run, (u.double() * run[:, -1])[:, None], right=True)[:, 0]
    last = (w.shape[1] - 1) - (w > 0).flip(1).to(torch.uint8).argmax(1)
    return torch.minimum(v, last)


def _plain_verify(st):
    c, T = st["case"], st["T"]
    rows, tokens = st["rows"].long(), st["tokens"].long()
    S, M = c["seqs"], st["max_new"]
    n = rows[1:] - rows[:-1]
    tau = st["temps"].double()[st["row_seq"]]
    greedy = tau == 0
    w = _weights(st["target"], torch.where(greedy, torch.ones_like(tau), tau))
    best = st["target"].float().argmax(1)                    # the first of the largest
    if c["sampled"]:
        # row r + 1's token against the probabilities at row r
        wq = _weights(st["draft"], torch.where(greedy, torch.ones_like(tau), tau))
        p, q = w / w.sum(1, keepdim=True), wq / wq.sum(1, keepdim=True)
        r = torch.arange(T, device="cuda")
        up = (r - 1).clamp(min=0)
        pt, qt = p[up, tokens], q[up, tokens]
        ok = torch.where(greedy, best[up] == tokens, st["accept"].double() * qt < pt)
        ok = _padded(st, ok, False)
        ok[:, 0] = True
        taken = torch.cumprod(ok.long(), 1).sum(1) * (n > 0) - 1      # rows taken after the first
        end = (rows[:-1] + taken.clamp(min=0)).clamp(max=T - 1)
        rest = torch.where((taken + 1 < n)[:, None], (p[end] - q[end]).clamp(min=0), p[end])
        rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p[end])
        nxt = torch.where(greedy[end], best[end], _drawn(rest, st["sample"][end]))
        on_path = torch.arange(M, device="cuda") <= taken[:, None]
    else:
        got = torch.where(greedy, best, _drawn(w, st["sample"]))
        if c["tree"]:
            seen, par = _ancestors(st), _padded(st, st["parents"].long(), -1)
        else:
            i = torch.arange(M, device="cuda")
            seen, par = (i[:, None] >= i).expand(S, M, M), (i - 1).expand(S, M)
        tok, hit = _padded(st, tokens, -1), _padded(st, got, -2)
        match = torch.gather(hit, 1, par.clamp(min=0)) == tok
        # of rows that follow the same one with the same token the first counts
        twin = (par[:, :, None] == par[:, None]) & (tok[:, :, None] == tok[:, None])
        twin = twin & (torch.arange(M, device="cuda")[:, None] > torch.arange(M, device="cuda"))
        match = match & (par >= 0) & ~twin.any(2)
        match[:, 0] = True
        on_path = (match[:, None] | ~seen).all(2) & seen[:, :, 0] & (torch.arange(M, device="cuda") < n[:, None])
        taken = on_path.sum(1) - 1
        end = (rows[:-1] + (M - 1 - on_path.flip(1).to(torch.uint8).argmax(1))).clamp(max=T - 1)
        nxt = got[end]
    some = n > 0
    on_path = on_path & some[:, None]
    taken = torch.where(some, taken, torch.zeros_like(taken))
    count = on_path.sum(1)
    rows_out = torch.cat([torch.zeros_like(rows[:1]), torch.cumsum(count, 0)])
    path = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    flat = on_path[st["row_seq"], st["row_at"]]
    place = (rows_out[:-1])[st["row_seq"]] + (torch.cumsum(on_path.long(), 1) - 1)[st["row_seq"], st["row_at"]]
    # rows off the path go to a place behind the last
    spot = torch.where(flat, place, torch.full_like(place, T))
    path = torch.cat([path, path[:1]]).scatter_(0, spot, torch.arange(T, device="cuda", dtype=torch.int32))[:T]
    kv = st["kv_len"].long() - n + count
    return [v.to(torch.int32) for v in (taken, torch.where(some, nxt, torch.full_like(nxt, -1)), rows_out, path, kv)]


# ---- one pass -------------------------------------------------------------------------------------
def _handles(st):
    """What a program makes once: the descriptors of the cache, the batch and the rotation, and a workspace."""
    import block_quantized_weight_affine_amd as qg
    if "handles" not in st:
        c, h = st["case"], {}
        if "freqs" in st:
            h["rot"] = qg.rotary(st["freqs"], c["inter"], st["mscale"])
        if "k_codes" in st:
            h["cache"] = qg.kv8_cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], c["page"],
                                      c["heads"], c["dim"])
        if "rows" in st:
            h["seqs"] = qg.kv8_seqs(st["table"], st["rows"], st["kv_len"], st["T"], st["max_new"], st["max_kv"])
        size = 0
        if c["op"] == "tree":
            size = qg.qg_attn_kv8_workspace(h["cache"], h["seqs"], c["q_heads"])
        if c["op"] == "verify":
            size = qg.qg_draft_verify_workspace(h["seqs"], c["vocab"])
        h["work"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
        st["handles"] = h
    return qg, st["handles"]


def _own_run(st):
    c = st["case"]
    qg, h = _handles(st)
    if c["op"] == "rope":
        qg.qg_rope(h["rot"], st["pos"], st["x"], st["y"])
        return st["y"]
    if c["op"] == "append":
        q, q_out = (st["q"], st["q_out"]) if c["q_heads"] else (None, None)
        qg.qg_kv8_write_rope(h["cache"], h["seqs"], h["rot"], st["k"], st["v"], q, q_out, st["pos"], st["src"])
        qg.qg_kv8_read(h["cache"], h["seqs"], st["k_out"], st["v_out"])
        return ([q_out] if c["q_heads"] else []) + [st["k_out"], st["v_out"]]
    if c["op"] == "plan":
        qg.qg_tree_plan(h["seqs"], st["parents"], st["mask"], st["pos"], c["window"])
        return [st["mask"], st["pos"]]
    if c["op"] == "tree":
        qg.qg_attn_kv8_tree(h["cache"], h["seqs"], st["mask"], st["q"], st["o"], c["q_heads"], 1.0 / math.sqrt(c["dim"]),
                            c["window"], st["pos"], h["work"])
        return st["o"]
    outs = [st["accepted"], st["next"], st["rows_out"], st["path"], st["kv_out"]]
    qg.qg_draft_verify(h["seqs"], st["tokens"], st["target"], *outs, sample=st["sample"], temps=st["temps"],
                       parents=st["parents"], draft=st.get("draft"), accept=st["accept"], workspace=h["work"])
    return outs


def run(state):
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "append": _plain_append, "plan": _plain_plan, "tree": _plain_tree,
            "verify": _plain_verify}[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["heads"] * c["dim"]
        return {"bytes": 2 * n * _BYTES[c["xt"]] + 4 * c["T"], "flops": 3 * c["T"] * c["heads"] * c["rot"]}
    new, hist = _lengths(dict(c, hist=c.get("hist", 3000)))
    T = sum(new)
    if c["op"] == "plan":
        return {"bytes": T * (4 + 4 + 4 * -(-max(new) // 32)) + 8 * len(new), "flops": 0}
    if c["op"] == "verify":
        # which rows the walk reaches is known when it ends: each row's probabilities once, the draft's but at a last row
        rows = T + (T - sum(n > 0 for n in new) if c["sampled"] else 0)
        return {"bytes": rows * c["vocab"] * _BYTES[c["xt"]] + 20 * T, "flops": 2 * rows * c["vocab"]}
    row = 2 * c["heads"] * c["dim"]  # values of K and V a token
    if c["op"] == "append":
        turned = T * (c["q_heads"] + c["heads"]) * c["rot"]
        return {"bytes": T * row * (_BYTES[c["xt"]] + 1 + 1 + _BYTES[c["yt"]])
                + 2 * T * c["q_heads"] * c["dim"] * _BYTES[c["xt"]], "flops": 3 * turned}
    pairs = tokens = 0
    for n, h, par in zip(new, hist, _parents(c, new)):
        depth = []
        for p in par:
            depth.append(0 if p < 0 else depth[p] + 1)
        lo = [max(0, h + d - c["window"] + 1) if c["window"] else 0 for d in depth]
        pairs += sum(max(0, h - v) + d + 1 for v, d in zip(lo, depth))
        tokens += h - min(min(lo), h) + n if n else 0
    qo = 2 * T * c["q_heads"] * c["dim"] * _BYTES[c["xt"]]
    return {"bytes": tokens * (row + row // c["dim"] / 4) + qo, "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ---- the definitions in 64 bits -------------------------------------------------------------------
def _turn64(st, x, pos):
    """Each pair as a complex number times exp(i angle)."""
    c = st["case"]
    f = x.double()
    pairs = f[..., :c["rot"]].unflatten(-1, (-1, 2) if c["inter"] else (2, -1))
    pairs = pairs if c["inter"] else pairs.transpose(-1, -2)
    angle = torch.outer(pos.double(), st["freqs"])[:, None]
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, st["mscale"]), angle)
    z = torch.view_as_real(z)
    return torch.cat([(z if c["inter"] else z.transpose(-1, -2)).flatten(-2), f[..., c["rot"]:]], -1)


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


def _exact_append(st):
    c = st["case"]
    new, hist = _lengths(c)
    pos = st["pos"]
    if pos is None:
        pos = torch.cat([torch.arange(h, h + n, device="cuda") for n, h in zip(new, hist)])
    pick = torch.arange(st["T"], device="cuda") if st["src"] is None else st["src"].long()
    vals = {"k": _turn64(st, st["k"][pick], pos), "v": st["v"][pick].double()}
    outs = [_turn64(st, st["q"], pos)] if c["q_heads"] else []
    for which in ("k", "v"):
        got, at = [], 0
        for s, (n, h) in enumerate(zip(new, hist)):
            if not n:
                continue
            x = vals[which][at:at + n]
            at += n
            lo = h - h % _BLOCK
            _, d_old = _tokens64(st, which, s, lo, h)
            # the rows by blocks, the first and last of them padded with zeros
            padded = torch.zeros(-(-(h + n - lo) // _BLOCK) * _BLOCK, *x.shape[1:], dtype=torch.float64, device="cuda")
            padded[h - lo:h - lo + n] = x
            blocks = padded.unflatten(0, (-1, _BLOCK))
            d = blocks.abs().amax((1, 3), keepdim=True) / 127.0
            if lo < h:
                d[0] = torch.maximum(d[0], d_old[0][None, :, None])
            q = torch.round(blocks / torch.where(d > 0, d, torch.ones_like(d))).clamp(-127, 127)
            got.append((q * d).flatten(0, 1)[h - lo:h - lo + n])
        outs.append(torch.cat(got))
    return outs


def _exact_tree(st):
    c = st["case"]
    new, hist = _lengths(c)
    G, out, at = c["q_heads"] // c["heads"], [], 0
    for s, (n, h, par) in enumerate(zip(new, hist, st["trees"])):
        if not n:
            continue
        lines = []
        for r, p in enumerate(par):
            lines.append({r} if p < 0 else lines[p] | {r})
        q = st["q"][at:at + n].double()
        at += n
        lo = max(0, h - c["window"]) if c["window"] else 0
        (kq, kd), (vq, vd) = (_tokens64(st, w, s, lo, h + n) for w in "kv")
        hidden = torch.ones(n, h + n - lo, dtype=torch.bool)
        for r, line in enumerate(lines):
            since = max(lo, h + len(line) - 1 - c["window"] + 1) if c["window"] else lo
            hidden[r, since - lo:h - lo] = False
            hidden[r, [h - lo + a for a in line]] = False
        hidden = hidden.cuda()
        heads = []
        for head in range(c["q_heads"]):
            kv = head // G
            score = (q[:, head] @ (kq[:, kv] * kd[:, kv, None]).t()) / math.sqrt(c["dim"])
            weight = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            heads.append(weight @ (vq[:, kv] * vd[:, kv, None]))
        out.append(torch.stack(heads, 1))
    return torch.cat(out)


def _exact_plan(st):
    c = st["case"]
    new, _ = _lengths(c)
    words = -(-max(new) // 32)
    masks, pos = [], []
    for n, h, par in zip(new, st["hist"], st["trees"]):
        lines = []
        for r, p in enumerate(par):
            lines.append(([] if p < 0 else lines[p]) + [r])
            pos.append(h + len(lines[-1]) - 1)
            bits = sum(1 << a for a in (lines[-1][-c["window"]:] if c["window"] else lines[-1]))
            w = [bits >> 32 * i & 0xffffffff for i in range(words)]
            masks.append([v - (1 << 32) if v >= 1 << 31 else v for v in w])
    return [_ints(masks), _ints(pos)]


def _exact_verify(st):
    """Row by row, as a program for one user would go."""
    c = st["case"]
    new, hist = _lengths(dict(c, hist=c.get("hist", 3000)))
    parents = st["trees"] if c["tree"] else [[r - 1 for r in range(n)] for n in new]
    tokens, temps = st["tokens"].tolist(), st["temps"].tolist()
    accept, sample = st["accept"].tolist(), st["sample"].tolist()
    taken, nxt, offs, path, kv = [], [], [0], [], []
    base = 0
    for n, h, par, tau in zip(new, hist, parents, temps):
        line, then = [], -1
        row = 0
        while n:
            line.append(base + row)
            here = st["target"][base + row].double()
            kids = [r for r in range(row + 1, n) if par[r] == row]
            if tau == 0:
                then = int(here.argmax())
            else:
                w = torch.softmax(here / tau, 0)
                if c["sampled"] and kids:
                    q = torch.softmax(st["draft"][base + row].double() / tau, 0)
                    x = tokens[base + kids[0]]
                    if accept[base + kids[0]] * float(q[x]) < float(w[x]):
                        row = kids[0]
                        continue
                    w, kids = (w - q).clamp(min=0), []
                run = torch.cumsum(w, 0)
                then = int((run <= sample[base + row] * run[-1]).sum())
            kids = [r for r in kids if tokens[base + r] == then]
            if not kids:
                break
            row = kids[0]
        taken.append(max(0, len(line) - 1))
        nxt.append(then)
        path += line
        offs.append(len(path))
        kv.append(h + len(line))
        base += n
    return [_ints(v) for v in (taken, nxt, offs, path + [-1] * (base - len(path)), kv)]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turn64(st, st["x"], st["pos"])
    return {"append": _exact_append, "plan": _exact_plan, "tree": _exact_tree, "verify": _exact_verify}[op](st)
