"""Batches whose trees of drafted tokens the attention's tiles of 128 or 256 rows take, and the definition of that attention for
all rows of a head at once (oracle/draft.py has it row by row)."""
import numpy as np
import torch

from oracle import serve8

CASES = {
    # lens, heads, q_heads, dim, page, window, type, rows a tile
    "pairs": ([(100, 2100), (128, 2228), (77, 900), (1, 1500), (0, 5)], 4, 32, 64, 64, 0, "bf16", 128),
    "pairs, history inside a stage": ([(127, 127), (128, 1600), (65, 1601), (128, 1663), (9, 1472), (31, 1505)], 4, 32, 128, 16, 0, "f16", 128),
    "pairs, window": ([(n, 128 + 7 * n) for n in range(1, 35)] + [(128, 128), (128, 300)], 4, 32, 96, 48, 3, "bf16", 128),
    "pairs, long window": ([(90, 2090), (128, 2400), (17, 1300), (64, 64), (128, 1400)], 4, 32, 128, 128, 1100, "f16", 128),
    "one tile a head": ([(16, n) for n in range(500, 548)], 8, 64, 64, 32, 0, "f16", 128),
    "wide": ([(160, 1100), (129, 1000), (1, 999), (160, 160)], 4, 32, 128, 64, 0, "bf16", 256),
    "wide, window": ([(160, 160 + 33 * n) for n in range(7)] + [(131, 900), (129, 129), (3, 160), (0, 0), (64, 777)], 8, 64, 64, 48, 3, "f16", 256),
    "wide, all rows": ([(1024, 1500), (1000, 1000)], 2, 16, 64, 64, 0, "f16", 256),
    "wide, odd group": ([(517, 1303), (300, 811)], 3, 21, 96, 80, 700, "bf16", 256),
    "f32": ([(64, 1064), (33, 1900), (64, 64), (1, 300)], 4, 64, 128, 64, 0, "f32", 128),
    "f32, window": ([(128, 128 + 40 * n) for n in range(13)] + [(100, 100), (70, 1111), (1, 1)], 4, 64, 64, 16, 5, "f32", 128),
    "f32, all rows": ([(1024, 1024), (600, 1300)], 2, 16, 96, 48, 0, "f32", 128),
    "f32, heads of 192": ([(200, 1240), (90, 1001)], 4, 64, 192, 32, 0, "f32", 128),
    "f32, heads of 256": ([(80, 1580), (129, 700), (129, 129), (77, 850)], 4, 64, 256, 64, 600, "f32", 128),
    "heads of 192": ([(300, 1200), (150, 1100)], 4, 48, 192, 64, 0, "bf16", 128),
    "heads of 256": ([(130, 1230), (260, 990), (7, 400), (260, 260)], 4, 64, 256, 256, 50, "f16", 128),
}


def sights(b, mask, window, pos):
    """Which tokens each row sees by its mask and window: (sequence, first row, [rows][tokens]) of each sequence with rows."""
    out = []
    for s, (r0, n, total) in enumerate(b.spans()):
        if not n:
            continue
        hist = total - n
        bits = np.unpackbits(np.ascontiguousarray(mask[r0:r0 + n]).view(np.uint8), axis=1, bitorder="little")[:, :n].astype(bool)
        seen = np.zeros((n, total), bool)
        for i in range(n):
            since = min(max(int(pos[r0 + i]), hist), total - 1) - window + 1 if window > 0 else 0
            seen[i, max(since, 0):hist] = True
        seen[:, hist:] = bits
        out.append((s, r0, seen))
    return out


def attend(b, q, scale, mask, window, pos, device):
    """Of every row and head, f64: o, the weighted means of |v|, the largest scale * sum |q k| and the largest (weight / sum of
    weights) * |V scale|; rows of no sequence are 0."""
    T, QH, D = q.shape
    G = QH // b.H
    q = q.double().to(device)
    o, mean = torch.zeros_like(q), torch.zeros_like(q)
    reach, peak = (torch.zeros(T, QH, 1, dtype=torch.float64, device=device) for _ in "rp")
    for s, r0, seen in sights(b, mask, window, pos):
        n, total = seen.shape
        j = np.arange(total)
        page, off = b.table[s][j // b.page], j % b.page // 16
        page = np.where((page >= 0) & (page < b.P), page, 0)
        for h in range(b.H):
            k, there = serve8.tokens(b.kc, b.ks, b.table, s, h, total)
            v, _ = serve8.tokens(b.vc, b.vs, b.table, s, h, total)
            k, v, vd = (torch.from_numpy(x).to(device) for x in (k, v, np.abs(b.vs[page, h, off].astype(np.float64))))
            see = torch.from_numpy(seen & there).to(device).repeat_interleave(G, 0)
            x = q[r0:r0 + n, h * G:(h + 1) * G].reshape(n * G, D)
            sc = (x @ k.t().contiguous() * scale).masked_fill(~see, -torch.inf)
            top = sc.amax(1, keepdim=True)
            w = torch.exp(sc - torch.where(top > -torch.inf, top, 0.0))
            w /= torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), 1.0)
            far = (x.abs() @ k.abs().t().contiguous()).masked_fill(~see, 0.0).amax(1)
            at = slice(r0, r0 + n), slice(h * G, (h + 1) * G)
            o[at] = (w @ v).view(n, G, D)
            mean[at] = (w @ v.abs()).view(n, G, D)
            reach[at] = abs(scale) * far.view(n, G, 1)
            peak[at] = (w * vd).amax(1).view(n, G, 1)
    return o, mean, reach, peak
