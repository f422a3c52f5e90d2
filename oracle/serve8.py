"""Plain definitions of the 8-bit serving operators (numpy, sums in f64): the key/value cache, attention
over it and the product in 8-bit integers.  Test infrastructure; shares no code with the library.

A cache is held as its meaning, not its layout: codes [pages][heads][page][dim] and scales
[pages][heads][page / 16] for K and V; `layout` and `meaning` convert to and from the bytes of the
documented layout.
"""
import numpy as np

BLOCK = 16
PER127 = np.float32(1.0 / 127.0)
FLT_MAX = np.finfo(np.float32).max


def layout(codes, which):
    """codes int8 [pages][heads][page][dim] -> the cache's bytes."""
    P, H, page, D = codes.shape
    b = codes.reshape(P, H, page // BLOCK, BLOCK, D)
    if which == "k":  # [dim/16][16 tokens][16 dims]
        return np.ascontiguousarray(b.reshape(P, H, page // BLOCK, BLOCK, D // 16, 16).swapaxes(3, 4))
    return np.ascontiguousarray(b.swapaxes(3, 4))  # [dim][16 tokens]


def meaning(raw, which, P, H, page, D):
    """The cache's bytes -> codes int8 [pages][heads][page][dim]."""
    if which == "k":
        b = raw.reshape(P, H, page // BLOCK, D // 16, BLOCK, 16).swapaxes(3, 4)
    else:
        b = raw.reshape(P, H, page // BLOCK, D, BLOCK).swapaxes(3, 4)
    return b.reshape(P, H, page, D).copy()


def scale_of(x):
    """(scale, factor) of values that share a scale, in f32."""
    with np.errstate(all="ignore"):
        top = np.float32(np.max(np.abs(x), initial=np.float32(0.0)))
        d = top * PER127 if np.isfinite(top) else np.float32(np.nan)
        inv = np.minimum(np.float32(1.0) / d, FLT_MAX) if d > 0 else np.float32(0.0)
    return d, np.float32(inv)


def code(x, inv):
    with np.errstate(all="ignore"):
        r = np.rint((x * inv).astype(np.float32))
    return np.clip(np.nan_to_num(r), -127, 127).astype(np.int8)


def place(table, page, pages, s, j):
    """Page and offset of token j of sequence s, or None where there is none."""
    if j // page >= table.shape[1]:
        return None
    p = int(table[s, j // page])
    return (p, j % page) if 0 <= p < pages else None


def spans(rows, kv_len, T, max_new, max_kv):
    """(first row, rows, tokens) of each sequence; (0, 0, 0) where the numbers contradict each other."""
    out = []
    for r0, r1, n in zip(rows[:-1], rows[1:], kv_len):
        ok = 0 <= r0 <= r1 <= T and r1 - r0 <= max_new and r1 - r0 <= n <= max_kv
        out.append((int(r0), int(r1 - r0), int(n)) if ok else (0, 0, 0))
    return out


def kv8_write(codes, scales, table, sp, x):
    """x f32 [T][heads][dim] into codes / scales (in place)."""
    pages, H, page, D = codes.shape
    for s, (r0, n, total) in enumerate(sp):
        first = total - n
        for blk in range(first // BLOCK, -(-total // BLOCK) if n else 0):
            at = place(table, page, pages, s, blk * BLOCK)
            if at is None:
                continue
            p, o = at
            lo, hi = max(first, blk * BLOCK), min(total, (blk + 1) * BLOCK)
            for h in range(H):
                new = x[r0 + lo - first:r0 + hi - first, h]
                d, inv = scale_of(new)
                old = scales[p, h, o // BLOCK]
                if lo > blk * BLOCK:
                    if old > d:
                        d = old
                        inv = np.minimum(np.float32(1.0) / d, FLT_MAX)
                    elif d > old:
                        with np.errstate(all="ignore"):
                            ratio = np.float32(old / d)
                        codes[p, h, o:o + lo - blk * BLOCK] = code(
                            codes[p, h, o:o + lo - blk * BLOCK].astype(np.float32), ratio)
                scales[p, h, o // BLOCK] = d
                a = o + lo - blk * BLOCK
                codes[p, h, a:a + hi - lo] = code(new, inv)


def tokens(codes, scales, table, s, h, n):
    """Values of tokens 0..n-1 of a sequence and head in f64 [n][dim], and which of them there are."""
    pages, _, page, D = codes.shape
    out, there = np.zeros((n, D)), np.zeros(n, bool)
    for j in range(n):
        at = place(table, page, pages, s, j)
        if at is not None:
            p, o = at
            out[j] = codes[p, h, o].astype(np.float64) * np.float64(scales[p, h, o // BLOCK])
            there[j] = True
    return out, there


def kv8_read(codes, scales, table, sp, T):
    """f32 values of every sequence's last rows, [T][heads][dim] (NaN where no sequence has the row)."""
    H, D = codes.shape[1], codes.shape[3]
    out = np.full((T, H, D), np.nan, np.float32)
    for s, (r0, n, total) in enumerate(sp):
        for i in range(n):
            at = place(table, codes.shape[2], codes.shape[0], s, total - n + i)
            for h in range(H):
                with np.errstate(invalid="ignore"):
                    out[r0 + i, h] = 0 if at is None else \
                        codes[at[0], h, at[1]].astype(np.float32) * scales[at[0], h, at[1] // BLOCK]
    return out


def attend(kc, ks, vc, vs, table, sp, q, scale, causal, window):
    """Attention in f64: q f64 [T][q_heads][dim] -> o, and three magnitudes for error bounds: the weighted mean
    of |v|, the largest scale * sum |q k| and the largest |v| a row sees."""
    T, QH, D = q.shape
    H = kc.shape[1]
    o, mean, reach, top = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros((T, QH, 1)), np.zeros((T, QH, 1))
    for s, (r0, n, total) in enumerate(sp):
        if not n:
            continue
        for h in range(H):
            k, there = tokens(kc, ks, table, s, h, total)
            v, _ = tokens(vc, vs, table, s, h, total)
            for i in range(n):
                pos, j = total - n + i, np.arange(total)
                seen = there.copy()
                if causal:
                    seen &= j <= pos
                if window > 0:
                    seen &= j > pos - window
                for qh in range(h * (QH // H), (h + 1) * (QH // H)):
                    if not seen.any():
                        o[r0 + i, qh] = 0
                        continue
                    x = q[r0 + i, qh]
                    sc = (k[seen] @ x) * scale
                    w = np.exp(sc - sc.max())
                    w /= w.sum()
                    o[r0 + i, qh] = w @ v[seen]
                    mean[r0 + i, qh] = w @ np.abs(v[seen])
                    reach[r0 + i, qh] = abs(scale) * (np.abs(k[seen]) @ np.abs(x)).max()
                    top[r0 + i, qh] = np.abs(v[seen]).max()
    return o, mean, reach, top


def w8a8(w, ws, x):
    """f32 results before the last rounding, from the definition: x f32 [T][K], w int8 [N][K], ws f32 [N]."""
    out = np.empty((x.shape[0], w.shape[0]), np.float32)
    w64 = w.astype(np.int64)
    for t, row in enumerate(x):
        d, inv = scale_of(row)
        acc = w64 @ code(row, inv).astype(np.int64)
        with np.errstate(all="ignore"):
            out[t] = (acc.astype(np.float32) * d) * ws
    return out
