#!/usr/bin/env python3
"""Serving in 8 bits with drafted tokens, end to end: every step checks a small tree of tokens a user at once.

    python examples/serve_draft.py [--users 16] [--prompt 512] [--tokens 128] [--layers 4] [--temperature 0] [--eager]

The model of serve_int8.py with rotary positions.  What followed a token before, lately and before that, is drafted as what
follows it now, in a tree of 8 rows; a step is one captured graph: the plan (qg_tree_plan), in every layer the rows into the
cache (qg_kv8_write_rope) and their attention (qg_attn_kv8_tree), the verification (qg_draft_verify), and the rows that stay
moved together (qg_kv8_write_rope).  Lengths, tokens and drafts stay on the GPU.  Prints tokens a step and
tokens/s (a random model seldom says what it said before, so here few drafts come true).
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from serve_int8 import Model, norm, qg  # noqa: E402

PARENTS = [-1, 0, 0, 1, 1, 2, 3, 6]         # a row's parent, and what it drafts: what followed last (0), or before that (1)
WHICH = [0, 0, 1, 0, 1, 0, 0, 0]
DEEPEST = 5                                  # rows from the first to the last of the longest line
ROWS = len(PARENTS)


class DraftModel(Model):
    def __init__(self, *a, **k):
        super().__init__(*a, **k)
        freqs, mscale = qg.rope_freqs(self.dim)
        self.rot = qg.rotary(torch.from_numpy(freqs).cuda(), mscale=mscale)

    def logits(self, tokens, seqs, work, rows=slice(None), mask=None, pos=None):
        """Logits of `rows`, and what every layer wrote (to be moved): tokens [T] of all users' rows, causal or by mask."""
        x, wrote = self.embed[tokens], []
        for cache, qkv, out, up, down in self.layers:
            h = qkv(norm(x), work).view(-1, self.q_heads + 2 * self.heads, self.dim)
            q, k, v = h.split([self.q_heads, self.heads, self.heads], 1)
            wrote.append((k, v))
            qg.qg_kv8_write_rope(cache, seqs, self.rot, k, v, q, q, pos)
            o = torch.empty(q.shape, dtype=q.dtype, device="cuda")
            if mask is None:
                qg.qg_attn_kv8(cache, seqs, q, o, self.q_heads, self.dim ** -0.5, True, 0, work)
            else:
                qg.qg_attn_kv8_tree(cache, seqs, mask, q, o, self.q_heads, self.dim ** -0.5, workspace=work)
            x = x + out(o.view(o.shape[0], -1), work)
            gate, value = up(norm(x), work).chunk(2, -1)
            x = x + down((torch.nn.functional.silu(gate) * value).contiguous(), work)
        return self.head(norm(x[rows]), work), wrote


class Drafts:
    """What followed each token of each user: last, and before that (-1: nothing yet)."""

    def __init__(self, users, vocab):
        self.users = torch.arange(users, device="cuda")
        self.after = torch.full((2, users, vocab), -1, dtype=torch.int64, device="cuda")

    def learn(self, token, follows, valid):
        """follows [users] came after token [users], where valid."""
        last, before = self.after[0, self.users, token], self.after[1, self.users, token]
        new = valid & (follows != last)
        self.after[0, self.users, token] = torch.where(new, follows, last)
        self.after[1, self.users, token] = torch.where(new, last, before)

    def tree(self, first):
        """Tokens [users][ROWS] that begin with first [users]; a row without a draft holds -1, which never stays."""
        rows = [first]
        for up, which in zip(PARENTS[1:], WHICH[1:]):
            draft = self.after[which, self.users, rows[up].clamp(min=0)]
            rows.append(torch.where(rows[up] >= 0, draft, rows[up]))
        return torch.stack(rows, 1)


def serve(model, lengths, tokens, temperature=0.0, graph=True, seed=1):
    """Prompts of these lengths, then steps until every user has `tokens` more, or one has ROWS beyond them: each user's tokens
    (lists), the steps and the seconds that they took.  The cache holds a step's rows past those that stay."""
    users, T, vocab = model.users, sum(lengths), len(model.embed)
    assert max(lengths) + tokens + 2 * ROWS <= model.tokens
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    prompt = torch.randint(vocab, (T,), device="cuda", generator=gen)
    rows = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    kv_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    seqs = qg.kv8_seqs(model.table, rows, kv_len, T, max(lengths), model.tokens)
    first = model.logits(prompt, seqs, model.workspace(seqs), rows[1:].long() - 1)[0].argmax(-1)
    drafts = Drafts(users, vocab)
    for u in range(users):
        part = prompt[int(rows[u]):int(rows[u + 1])]
        drafts.after[0, u, part[:-1]] = part[1:]

    T = users * ROWS
    ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = torch.arange(users + 1, dtype=torch.int32, device="cuda") * ROWS
    parents = torch.tensor(PARENTS, dtype=torch.int32, device="cuda").repeat(users)
    tree, mask, pos = ints(T), ints(T, 1), ints(T)
    accepted, following, rows_out, path = ints(users), ints(users), ints(users + 1), ints(T)
    seqs = qg.kv8_seqs(model.table, rows, kv_len, T, ROWS, model.tokens)
    stay = qg.kv8_seqs(model.table, rows_out, kv_len, T, ROWS, model.tokens)
    sample = torch.zeros(T, device="cuda")
    temps = torch.full((users,), float(temperature), device="cuda")
    size = max(qg.qg_draft_verify_workspace(seqs, vocab), qg.qgemm_w8a8_workspace(model.head.N, model.head.K, T))
    work = max(model.workspace(seqs), torch.empty(size, dtype=torch.uint8, device="cuda"), key=len)
    made = torch.full((users, DEEPEST), -1, dtype=torch.int64, device="cuda")

    def step():
        qg.qg_tree_plan(seqs, parents, mask, pos)
        # a row without a draft is computed as token 0
        logits, wrote = model.logits(tree.clamp(min=0).long(), seqs, work, mask=mask, pos=pos)
        qg.qg_draft_verify(seqs, tree, logits, accepted, following, rows_out, path, kv_len, sample=sample, temps=temps,
                           parents=parents, workspace=work)
        for (cache, *_), (k, v) in zip(model.layers, wrote):
            qg.qg_kv8_write_rope(cache, stay, model.rot, k, v, src=path)
        at = rows_out[:-1].long()
        for d in range(DEEPEST):                # along each user's line: the token of a row, and what came after it
            here, after = (tree[path[(at + d + i).clamp(max=T - 1)].clamp(min=0).long()] for i in (0, 1))
            follows = torch.where(accepted > d, after, following).long()
            drafts.learn(here.long(), follows, accepted >= d)
            made[:, d] = torch.where(accepted >= d, follows, -1)
        tree.copy_(drafts.tree(following.long()).view(-1))
        kv_len.add_(ROWS)

    tree.copy_(drafts.tree(first).view(-1))
    kv_len.add_(ROWS)
    replay = step
    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        replay = captured.replay
    out = [[int(t)] for t in first]
    torch.cuda.synchronize()
    start, steps = time.perf_counter(), 0
    while min(map(len, out)) <= tokens and max(map(len, out)) <= tokens + ROWS:
        sample.uniform_(generator=gen).clamp_(max=1 - 2 ** -24)
        replay()
        steps += 1
        for line, new in zip(out, made.tolist()):
            line += [t for t in new if t >= 0]
    torch.cuda.synchronize()
    return out, steps, time.perf_counter() - start


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--users", type=int, default=16)
    p.add_argument("--prompt", type=int, default=512, help="longest prompt; the others spread below it")
    p.add_argument("--tokens", type=int, default=128)
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--temperature", type=float, default=0.0)
    p.add_argument("--eager", action="store_true", help="no captured graph")
    a = p.parse_args()
    dim = 128
    model = DraftModel(a.layers, a.hidden, a.hidden // dim, max(1, a.hidden // dim // 4), dim, 32000, a.users,
                       a.prompt + a.tokens + 3 * ROWS)
    lengths = [max(1, a.prompt * (u + 1) // a.users) for u in range(a.users)]
    serve(model, lengths, 1, a.temperature, not a.eager)      # loads the kernels
    out, steps, spent = serve(model, lengths, a.tokens, a.temperature, not a.eager)
    made = sum(len(line) - 1 for line in out)
    print(f"{steps} steps of {a.users} x {ROWS} rows, {made} tokens ({made / max(steps * a.users, 1):.2f} a user and step), "
          f"{spent / max(steps, 1) * 1e3:.3f} ms a step ({made / spent:.0f} tokens/s)")


if __name__ == "__main__":
    main()
