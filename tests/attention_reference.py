"""Plain float64 forms of the attention-side operators, for the tests: written
from the definitions in include/moe_attention.h with numpy on the CPU, sharing
nothing with the library.  Each returns the result together with what its
error bound needs."""
import numpy as np


def bf16(a):
    """float array -> the nearest bf16 values (ties to even), as float64."""
    b = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7fff + ((b >> 16) & 1)) >> 16) << 16
    out = r.astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(np.isnan(a), np.nan, out)


def e4m3_values():
    """The 256 E4M3 values: bias 7, no infinities, 0x7f and 0xff NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return v


E4M3 = e4m3_values()


def round_e4m3(a):
    """float64 -> the nearest E4M3 value, ties to even; |a| <= 464 or NaN, infinity (-> NaN)."""
    a = np.asarray(a, np.float64)
    mag = np.abs(a)
    with np.errstate(all="ignore"):
        e = np.floor(np.log2(np.where((mag > 0) & np.isfinite(mag), mag, 1.0)))
        step = np.exp2(np.maximum(e, -6) - 3)
        r = np.round(mag / step) * step  # numpy rounds halves to even
    r = np.where(np.isfinite(mag), r, np.nan)
    return np.copysign(r, a)


def quantise(x, kind):
    """bf16 values [T, K] -> (E4M3 values [T, K], scales [T, blocks])."""
    T, K = x.shape
    kb = -(-K // 128)
    q, s = np.empty((T, K)), np.empty((T, kb))
    for b in range(kb):
        xb = x[:, 128 * b:128 * (b + 1)]
        with np.errstate(all="ignore"):
            a = np.maximum(np.nanmax(np.where(np.isnan(xb), 0, np.abs(xb)), 1), 2.0 ** -100)
            if kind == "e8m0":
                s[:, b] = [2.0 ** next(e for e in range(-127, 128) if 448 * 2.0 ** e >= v) if np.isfinite(v) else 2.0 ** 120
                           for v in a]
                q[:, 128 * b:128 * (b + 1)] = round_e4m3(xb / s[:, b:b + 1])
            else:
                f = np.float32(a)
                s[:, b] = f / np.float32(448)
                inv = np.float32(448) / f
                q[:, 128 * b:128 * (b + 1)] = round_e4m3(np.float32(xb) * inv[:, None])
    return q, s


def fp8_linear(x, w_codes, w_scale, kind):
    """x [T, K] (bf16 values), w_codes uint8 [N, K], w_scale [nb, kb] as values
    -> (y, sum of magnitudes, sum over the groups of 8 columns of the group's
    largest product), float64 [T, N]."""
    q, s = quantise(x, kind)
    w = E4M3[w_codes]
    N, K = w.shape
    y, mag, top = (np.zeros((x.shape[0], N)) for _ in range(3))
    for b in range(s.shape[1]):
        cut = slice(128 * b, 128 * (b + 1))
        sw = np.repeat(w_scale[:, b], 128)[:N]
        with np.errstate(all="ignore"):
            y += s[:, b:b + 1] * (q[:, cut] @ w[:, cut].T) * sw
            mag += s[:, b:b + 1] * (np.abs(q[:, cut]) @ np.abs(w[:, cut]).T) * np.abs(sw)
            for k0 in range(128 * b, min(128 * b + 128, K), 8):
                m = np.zeros_like(y)
                for k in range(k0, min(k0 + 8, K)):
                    m = np.fmax(m, np.abs(q[:, k])[:, None] * np.abs(w[:, k]))
                top += s[:, b:b + 1] * m * np.abs(sw)
    return y, mag, top


def norm_rope(x, weight, pos, cos_sin, off, interleaved, eps):
    """x [T, H, D] -> (result, magnitude of what was summed), float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    if weight is not None:
        n = n * weight
    y, mag = n.copy(), np.abs(n)
    if cos_sin is not None:
        R = cos_sin.shape[1]
        for t in range(x.shape[0]):
            for j in range(R // 2):
                a, b = (off + 2 * j, off + 2 * j + 1) if interleaved else (off + j, off + R // 2 + j)
                ok = 0 <= pos[t] < cos_sin.shape[0]
                c, s = (cos_sin[pos[t], j], cos_sin[pos[t], R // 2 + j]) if ok else (np.nan, np.nan)
                u, v = n[t, :, a], n[t, :, b]
                y[t, :, a], y[t, :, b] = u * c - v * s, v * c + u * s
                mag[t, :, a], mag[t, :, b] = abs(u * c) + abs(v * s), abs(v * c) + abs(u * s)
    return y, mag


def attention(q, k, v, seqs, scale, causal):
    """q [Tq, Hq, D], k, v [Tk, Hkv, D] float64; seqs: (q0, lq, k0, lk) each ->
    out [Tq, Hq, D], lse [Tq, Hq], sum p |v|, and the largest sum |q||k| of a row's scores;
    rows of no sequence are NaN."""
    Tq, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.full((Tq, Hq, D), np.nan), np.full((Tq, Hq), np.nan)
    mag, dot = np.zeros((Tq, Hq, D)), np.zeros((Tq, Hq))
    with np.errstate(all="ignore"):
        for q0, lq, k0, lk in seqs:
            for h in range(Hq):
                kk, vv = k[k0:k0 + lk, h // G], v[k0:k0 + lk, h // G]
                for i in range(lq):
                    n = min(max(i + lk - lq + 1, 0), lk) if causal else lk
                    if n == 0:
                        out[q0 + i, h], lse[q0 + i, h] = 0, -np.inf
                        continue
                    z = kk[:n] @ q[q0 + i, h] * scale
                    m = z.max()
                    p = np.exp(z - m)
                    l = p.sum()
                    out[q0 + i, h] = (p @ vv[:n]) / l
                    lse[q0 + i, h] = m + np.log(l)
                    mag[q0 + i, h] = (p @ np.abs(vv[:n])) / l
                    dot[q0 + i, h] = (np.abs(kk[:n]) @ np.abs(q[q0 + i, h])).max() * scale
    return out, lse, mag, dot
