#!/usr/bin/env python3
"""Serving in 8 bits, end to end: weights as int8 with a scale an output channel, activations coded a token at
a time, keys and values in the paged 8-bit cache.

    python examples/serve_int8.py [--users 16] [--prompt 512] [--steps 64] [--layers 4] [--eager]

A random model of the given sizes reads prompts of different lengths in one batch (qgemm_w8a8, qg_kv8_write,
qg_attn_kv8), then makes one token a user and step from a captured graph: lengths and tokens live on the GPU and
change between replays, the descriptors hold the bounds.  Prints tokens/s of both phases.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_affine_amd as qg  # noqa: E402

PAGE = 64


class Linear:
    """int8 weights [N][K] with a scale an output channel."""

    def __init__(self, N, K, gen):
        w = torch.randn(N, K, device="cuda", generator=gen) / K ** 0.5
        self.scales = w.abs().amax(1) / 127
        self.codes = torch.round(w / self.scales[:, None]).to(torch.int8)
        self.N, self.K = N, K

    def __call__(self, x, work):
        y = torch.empty(x.shape[0], self.N, dtype=x.dtype, device="cuda")
        qg.qgemm_w8a8(self.codes, self.scales, x, y, self.N, self.K, x.shape[0], work)
        return y


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Model:
    def __init__(self, layers, hidden, q_heads, heads, dim, vocab, users, tokens, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.q_heads, self.heads, self.dim, self.users, self.tokens = q_heads, heads, dim, users, tokens
        self.embed = torch.randn(vocab, hidden, device="cuda", generator=gen).to(torch.bfloat16)
        per_user = -(-tokens // PAGE)
        order = torch.randperm(users * per_user, device="cuda", generator=gen, dtype=torch.int32)
        self.table = order.view(users, per_user)
        self.layers = []
        for _ in range(layers):
            cache = qg.kv8_cache(*qg.kv8_pages(users * per_user, PAGE, heads, dim), PAGE, heads, dim)
            self.layers.append((cache, Linear((q_heads + 2 * heads) * dim, hidden, gen),
                                Linear(hidden, q_heads * dim, gen), Linear(2 * 4 * hidden, hidden, gen),
                                Linear(hidden, 4 * hidden, gen)))
        self.head = Linear(vocab, hidden, gen)

    def workspace(self, seqs):
        """A buffer of the bytes that one call needs at most; they follow each other on one stream and share it.  Each
        call's own number of rows counts: fewer of them can need more."""
        sizes = [qg.qg_attn_kv8_workspace(self.layers[0][0], seqs, self.q_heads)]
        for m, rows in [(m, seqs.T) for m in self.layers[0][1:]] + [(self.head, self.users)]:
            sizes.append(qg.qgemm_w8a8_workspace(m.N, m.K, rows))
        return torch.empty(max(sizes + [16]), dtype=torch.uint8, device="cuda")

    def __call__(self, tokens, seqs, last, work):
        """The next token of every user: tokens [T] of all users' rows, last [users] each user's last row."""
        x = self.embed[tokens]
        for cache, qkv, out, up, down in self.layers:
            h = qkv(norm(x), work).view(-1, self.q_heads + 2 * self.heads, self.dim)
            q, k, v = h.split([self.q_heads, self.heads, self.heads], 1)
            qg.qg_kv8_write(cache, seqs, k, v)
            o = torch.empty(q.shape, dtype=q.dtype, device="cuda")
            qg.qg_attn_kv8(cache, seqs, q, o, self.q_heads, self.dim ** -0.5, True, 0, work)
            x = x + out(o.view(o.shape[0], -1), work)
            gate, value = up(norm(x), work).chunk(2, -1)
            x = x + down((torch.nn.functional.silu(gate) * value).contiguous(), work)
        return self.head(norm(x[last]), work).argmax(-1)


def serve(model, lengths, steps, graph=True, seed=1):
    """Prompts of these lengths, then `steps` tokens a user: the tokens [steps + 1][users] and the two phases' s."""
    users, T = model.users, sum(lengths)
    assert max(lengths) + steps <= model.tokens
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    prompt = torch.randint(len(model.embed), (T,), device="cuda", generator=gen)
    rows = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    kv_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    seqs = qg.kv8_seqs(model.table, rows, kv_len, T, max(lengths), model.tokens)
    work = model.workspace(seqs)
    torch.cuda.synchronize()
    start = time.perf_counter()
    token = model(prompt, seqs, rows[1:].long() - 1, work)
    torch.cuda.synchronize()
    read = time.perf_counter() - start

    one = torch.arange(users + 1, dtype=torch.int32, device="cuda")
    seqs = qg.kv8_seqs(model.table, one, kv_len, users, 1, model.tokens)
    work, last = model.workspace(seqs), one[:-1].long()
    out = [token.clone()]

    def step():
        kv_len.add_(1)
        token.copy_(model(token, seqs, last, work))

    replay = step
    if graph and steps:
        saved = [kv_len.clone(), token.clone()]
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        kv_len.copy_(saved[0])
        token.copy_(saved[1])
        replay = captured.replay
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(steps):
        replay()
        out.append(token.clone())
    torch.cuda.synchronize()
    return torch.stack(out), read, time.perf_counter() - start


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--users", type=int, default=16)
    p.add_argument("--prompt", type=int, default=512, help="longest prompt; the others spread below it")
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--eager", action="store_true", help="no captured graph")
    a = p.parse_args()
    dim = 128
    model = Model(a.layers, a.hidden, a.hidden // dim, max(1, a.hidden // dim // 4), dim, 32000, a.users, a.prompt + a.steps)
    lengths = [max(1, a.prompt * (u + 1) // a.users) for u in range(a.users)]
    serve(model, lengths, min(a.steps, 2), not a.eager)      # loads the kernels
    _, read, made = serve(model, lengths, a.steps, not a.eager)
    print(f"prompts: {sum(lengths)} tokens in {read * 1e3:.2f} ms ({sum(lengths) / read:.0f} tokens/s); "
          f"steps: {a.steps} x {a.users} tokens, {made / max(a.steps, 1) * 1e3:.3f} ms a step "
          f"({a.steps * a.users / made if made else 0:.0f} tokens/s)")


if __name__ == "__main__":
    main()
