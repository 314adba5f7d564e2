"""Plain float64 forms of the paged operators, for the tests: written from the
definitions in include/moe_paged.h with numpy on the CPU, sharing nothing with the
library.  A sequence is (q0, lq, lk): its first row, its rows, its tokens."""
import numpy as np


def page_of(table, b, p, page, n_pages):
    """The page of position p of sequence b, or None."""
    if p < 0 or p // page >= table.shape[1]:
        return None
    t = int(table[b, p // page])
    return t if 0 <= t < n_pages else None


def turn(x, weight, norm, eps, pos, cos_sin, off, interleaved):
    """Heads [H, D] of one token, normed and rotated -> (result, magnitude of what was summed)."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) if norm else x.copy()
        if weight is not None:
            n = n * weight
        y, mag = n.copy(), np.abs(n)
        if cos_sin is not None:
            R = cos_sin.shape[1]
            ok = 0 <= pos < cos_sin.shape[0]
            for j in range(R // 2):
                a, b = (off + 2 * j, off + 2 * j + 1) if interleaved else (off + j, off + R // 2 + j)
                c, s = (cos_sin[pos, j], cos_sin[pos, R // 2 + j]) if ok else (np.nan, np.nan)
                u, v = n[:, a], n[:, b]
                y[:, a], y[:, b] = u * c - v * s, v * c + u * s
                mag[:, a], mag[:, b] = abs(u * c) + abs(v * s), abs(v * c) + abs(u * s)
    return y, mag


def visible(seqs, table, page, n_pages, kv_heads, blocks=None, prefix=None, max_q=None, max_prefix=0, max_kv=None):
    """Per sequence a truth array [lq, kv_heads, lk], or None beside the row's output: which keys each row sees.
    prefix: the prefix length that each sequence's group names."""
    out = []
    for b, (q0, lq, lk) in enumerate(seqs):
        i, j = np.arange(lq)[:, None], np.arange(lk)[None]
        see = j <= i + lk - lq
        if max_kv is not None:
            see = see & (j < min(max(0 if prefix is None else prefix[b], 0), max_prefix) + max_kv)
        there = np.array([page_of(table, b, p, page, n_pages) is not None for p in range(lk)], bool)
        see = np.repeat((see & there[None])[:, None], kv_heads, 1)
        if blocks is not None:
            for r in range(lq):
                for h in range(kv_heads):
                    see[r, h] &= np.isin(np.arange(lk) // page, blocks[q0 + r, h])
        out.append(see)
    return out


def attention(q, k_pages, v_pages, table, seqs, see, scale):
    """q [T, Hq, D], k_pages and v_pages [n_pages, page, Hkv, D], float64; see: of `visible` -> out, lse, sum p |v|, the largest
    sum |q||k| of a row's scores, and the number of keys a row sees; rows of no sequence are NaN."""
    T, Hq, D = q.shape
    n_pages, page, Hkv, _ = k_pages.shape
    G = Hq // Hkv
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    mag, dot, count = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq))
    with np.errstate(all="ignore"):
        for b, (q0, lq, lk) in enumerate(seqs):
            p = np.arange(lk)
            col = np.minimum(p // page, max(table.shape[1] - 1, 0))
            at = np.where(np.isin(table[b, col], np.arange(n_pages)), table[b, col], 0) if lk else p
            k, v = (t[at, p % page] if lk else np.zeros((0, Hkv, D)) for t in (k_pages, v_pages))
            for h in range(Hq):
                for i in range(lq):
                    m = see[b][i, h // G]
                    kk, vv = k[m, h // G], v[m, h // G]
                    count[q0 + i, h] = m.sum()
                    if not m.any():
                        out[q0 + i, h], lse[q0 + i, h] = 0, -np.inf
                        continue
                    z = kk @ q[q0 + i, h] * scale
                    top = z.max()
                    w = np.exp(z - top)
                    l = w.sum()
                    out[q0 + i, h] = (w @ vv) / l
                    lse[q0 + i, h] = top + np.log(l)
                    mag[q0 + i, h] = (w @ np.abs(vv)) / l
                    dot[q0 + i, h] = (np.abs(kk) @ np.abs(q[q0 + i, h])).max() * scale
    return out, lse, mag, dot, count


def select(q, bounds, table, seqs, page, n_blocks, first, last, max_kv=None):
    """blocks [T, Hkv, n_blocks], -2 in rows of no sequence."""
    T, Hq, D = q.shape
    n_pages, _, Hkv, _ = bounds.shape
    G = Hq // Hkv
    out = np.full((T, Hkv, n_blocks), -2)
    with np.errstate(all="ignore"):
        for b, (q0, lq, lk) in enumerate(seqs):
            for i in range(lq):
                end = min(i + lk - lq, min(lk if max_kv is None else max_kv, table.shape[1] * page) - 1)
                n = end // page + 1 if end >= 0 else 0
                for h in range(Hkv):
                    qq = q[q0 + i, h * G:(h + 1) * G]
                    up, down = np.maximum(qq, 0).sum(0), np.minimum(qq, 0).sum(0)
                    rank = []
                    for c in range(n):
                        t = int(table[b, c])
                        if c < first or c >= n - last:
                            key = (4, 0.0)
                        elif not 0 <= t < n_pages:
                            key = (0, 0.0)
                        else:
                            s = float(up @ bounds[t, 1, h] + down @ bounds[t, 0, h])
                            key = (1, s) if np.isfinite(s) else (3, 0.0)
                        rank.append((-key[0], -key[1], c))
                    pick = sorted(c for _, _, c in sorted(rank)[:n_blocks])
                    out[q0 + i, h] = pick + [-1] * (n_blocks - len(pick))
    return out
