"""Plain definitions of the operators for drafted tokens (numpy, f64): rotary positions, the plan of a tree, attention
among a tree's rows over the 8-bit cache, and the verification of drafted tokens.  Test infrastructure; shares no code
with the library."""
import numpy as np

from oracle import serve8


def rope(x, pos, freqs, interleaved, mscale):
    """x [T][heads][dim] turned, in f64, and the sum of the magnitudes that each result is made of."""
    x = np.asarray(x, np.float64)
    out, mag = x.copy(), np.abs(x)
    n = len(freqs)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        t = np.asarray(pos, np.float64)[:, None] * freqs[i]
        c, s = np.cos(t), np.sin(t)
        out[..., a] = mscale * (x[..., a] * c - x[..., b] * s)
        out[..., b] = mscale * (x[..., b] * c + x[..., a] * s)
        mag[..., a] = mag[..., b] = abs(mscale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, mag


def lines(parents):
    """The rows that each row descends from, itself last."""
    out = []
    for r, p in enumerate(parents):
        out.append((out[p] if 0 <= p < r else []) + [r])
    return out


def plan(parents, sp, words, window, T):
    """Masks uint32 [T][words] and positions [T]; rows of no sequence keep 0x55555555 and -7."""
    mask, pos = np.full((T, words), 0x55555555, np.uint32), np.full(T, -7, np.int32)
    for r0, n, total in sp:
        for r, line in enumerate(lines(parents[r0:r0 + n])):
            pos[r0 + r] = total - n + len(line) - 1
            mask[r0 + r] = 0
            for a in line[-window:] if window > 0 else line:
                mask[r0 + r, a // 32] |= np.uint32(1 << (a % 32))
    return mask, pos


def attend(kc, ks, vc, vs, table, sp, q, scale, mask, window, pos):
    """As serve8.attend, with the batch's rows seeing each other by mask."""
    T, QH, D = q.shape
    H = kc.shape[1]
    o, mean, reach, top = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros((T, QH, 1)), np.zeros((T, QH, 1))
    for s, (r0, n, total) in enumerate(sp):
        hist = total - n
        for h in range(H if n else 0):
            k, there = serve8.tokens(kc, ks, table, s, h, total)
            v, _ = serve8.tokens(vc, vs, table, s, h, total)
            for i in range(n):
                j = np.arange(total)
                seen = there & (j < hist)
                if window > 0:
                    seen &= j > min(max(int(pos[r0 + i]), hist), total - 1) - window
                for a in range(n):
                    if mask[r0 + i, a // 32] >> np.uint32(a % 32) & 1:
                        seen[hist + a] = there[hist + a]
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


def chance(logits, tau):
    """Probabilities of a row in f64, or None where it has none."""
    l = np.asarray(logits, np.float64)
    if np.isnan(l).any() or l.max() in (np.inf, -np.inf):
        return None
    w = np.exp((l - l.max()) / tau)
    return w / w.sum()


def pick(w, u):
    """The first index at which the running sum of w exceeds u times the whole."""
    run = np.cumsum(w)
    at = int(np.searchsorted(run, np.float64(u) * run[-1], side="right"))
    return min(at, int(np.flatnonzero(w > 0)[-1]))


def verify(sp, kv_len, T, tokens, target, sample=None, temps=None, parents=None, draft=None, accept=None):
    """accepted, next, rows_out, path, kv_out as int32 arrays; target and draft f64 [T][vocab]."""
    accepted, nxt, rows, path, kv = [], [], [0], [], []
    for s, (r0, n, _) in enumerate(sp):
        tau = 0.0 if sample is None else 1.0 if temps is None else float(temps[s])
        line, token, r = [], -1, 0
        while n:
            line.append(r0 + r)
            up = [c - 1 if parents is None else parents[r0 + c] if 0 <= parents[r0 + c] < c else -1 for c in range(n)]
            kids = [c for c in range(r + 1, n) if up[c] == r]
            here = target[r0 + r]
            token = -1
            if tau == 0:
                if np.isnan(here).any() or here.max() == -np.inf:
                    break
                token = int(np.argmax(here))
            else:
                p = chance(here, tau) if 0 < tau < np.inf else None
                if p is None:
                    break
                if draft is not None and kids:
                    q, x = chance(draft[r0 + r], tau), int(tokens[r0 + kids[0]])
                    if q is not None and 0 <= x < len(p) and float(accept[r0 + kids[0]]) * q[x] < p[x]:
                        r = kids[0]
                        continue
                    rest = p if q is None else np.maximum(p - q, 0)
                    token = pick(rest if rest.sum() > 0 else p, sample[r0 + r])
                    break
                token = pick(p, sample[r0 + r])
            kids = [c for c in kids if tokens[r0 + c] == token]
            if not kids:
                break
            r = kids[0]
        accepted.append(max(0, len(line) - 1))
        nxt.append(token)
        path += line
        rows.append(len(path))
        kv.append(int(kv_len[s]) - n + len(line))
    path += [-1] * (T - len(path))
    return [np.array(x, np.int32) for x in (accepted, nxt, rows, path, kv)]
