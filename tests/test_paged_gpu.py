"""The paged operators on the GPU against float64 references, at the lengths, page
sizes, masks, tables and values where they can go wrong.

Bounds (u = 2^-8, half a step of bf16).
 paged_append: u |y| plus a relative 2^-17 of the magnitudes summed, as qk_norm_rope (the
  same sums of D squares and two products); values are copied, and the bounds of a
  page are compared with the keys that the call stored: exact.
 paged_attention: as the contiguous attention: with A = sum p |v|, u |o| for the result,
  2 u A for the weights rounded to bf16 (once in the product, once in their sum); the scores are
  off by d = (D + 4) 2^-23 (scale max |q| |k|), which changes the result by at most 2 (e^d - 1)
  A; and the sums over n keys by (n + 64) 2^-23 A.  A join of shares is part of these sums.
 select_blocks: exact.  Scores of the drawn values are sums of products with at most 16 bits each,
  spread over far less than 37 binary orders but for rare tiny terms: float64 sums in any
  order agree to 2^-50, and no two scores are that close unless they are equal.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from mxfp4_routed_expert_moe_amd import paged as P  # noqa: E402
from tests import attention_reference as AR  # noqa: E402
from tests import paged_reference as PR  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
BF = torch.bfloat16


def _say(*a):
    print("[paged]", *a, flush=True)


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(BF).cuda()


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _seqs(lq, lk, lead=0):
    out, a = [], lead
    for n, m in zip(lq, lk):
        out.append((a, n, m))
        a += n
    return out


def _table(g, lens, page, spare=3, n_pages=None):
    """A table with every sequence's pages anywhere in a pool; -> table, pages of the pool."""
    need = [-(-n // page) for n in lens]
    n = n_pages or sum(need) + spare
    perm = g.permutation(n)
    table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, n


def _pool(g, n_pages, page, Hkv, D, std=1.0, layout="pshd"):
    """bf16 keys and values [n_pages, page, Hkv, D] as float64, and as tensors in the given order of dimensions."""
    k, v = (AR.bf16(g.normal(0, std, (n_pages, page, Hkv, D))) for _ in range(2))
    if layout == "pshd":
        return k, v, _bf16(k), _bf16(v)
    if layout == "phsd":
        put = lambda t: _bf16(t.transpose(0, 2, 1, 3)).transpose(1, 2)  # noqa: E731
        return k, v, put(k), put(v)
    both = _bf16(np.concatenate([k, v], 2))  # keys and values of a token side by side
    return k, v, both[:, :, :Hkv], both[:, :, Hkv:]


def _angles(n, Rd):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, Rd, 2) / Rd)
    return np.float32(np.concatenate([np.cos(ang), np.sin(ang)], 1))


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,page,Rd,off,norm", [
    ([1], [1], 1, 1, 64, 16, 64, 0, True), ([1, 1, 1], [16, 17, 300], 8, 2, 128, 64, 128, 0, True),
    ([5, 0, 40, 1], [5, 9, 57, 33], 4, 4, 64, 16, 32, 32, False), ([100], [163], 6, 2, 256, 32, 256, 0, True),
    ([33, 130], [33, 500], 4, 1, 128, 128, 64, 64, True), ([70, 3], [200, 3], 0, 2, 128, 64, 0, 0, False),
    ([260, 1, 17], [260, 65, 30], 12, 4, 64, 32, 48, 8, True), ([7], [900], 5, 5, 256, 16, 128, 128, False)])
def test_append(lq, lk, Hq, Hkv, D, page, Rd, off, norm, interleaved):
    """Keys, values, queries and bounds; slots, rows and bounds that the call does not name keep what they hold."""
    _say("append", lq, lk, Hq, Hkv, D, page, Rd, off, norm, interleaved)
    g = np.random.default_rng(sum(lk) + D + page)
    lead, tail = 2, 3
    T = lead + sum(lq) + tail
    table, n_pages = _table(g, lk, page)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D, layout="pshd" if D == 64 else "phsd" if D == 128 else "both")
    buf = AR.bf16(g.normal(0, 2, (T, Hq + 2 * Hkv, D)))
    bt = _bf16(buf)
    q, k, v = bt[:, :Hq], bt[:, Hq:Hq + Hkv], bt[:, Hq + Hkv:]
    qw, kw = np.float32(g.normal(1, 0.2, D)), np.float32(g.normal(1, 0.2, D))
    cs = _angles(max(lk) + 1, Rd) if Rd else None
    old = AR.bf16(g.normal(0, 0.3, (n_pages, 2, Hkv, D)))
    bounds = _bf16(old)
    q_out = torch.full((T, max(Hq, 1), D), 9.0, dtype=BF, device="cuda")[:, :Hq]
    seqs = _seqs(lq, lk, lead)
    P.paged_append(k, v, kt, vt, _i32([lead] + [s[0] + s[1] for s in seqs]), _i32(lk), _i32(table),
                   q=q if Hq else None, q_out=q_out if Hq else None, bounds=bounds,
                   q_weight=_gpu(qw) if norm and Hq else None, k_weight=_gpu(kw) if norm else None, norm=norm,
                   cos_sin=None if cs is None else _gpu(cs), rot_offset=off, interleaved=interleaved)
    want_k, want_v, tol = kp.copy(), vp.copy(), np.zeros_like(kp)
    qo, got_k, got_v = _np(q_out), _np(kt), _np(vt)
    touched = {}
    for b, (q0, n, m) in enumerate(seqs):
        for i in range(n):
            p = i + m - n
            at = table[b, p // page], p % page
            want_k[at], mag = PR.turn(buf[q0 + i, Hq:Hq + Hkv], kw if norm else None, norm, 1e-6, p, cs, off, interleaved)
            tol[at] = U * np.abs(want_k[at]) + 2.0 ** -17 * mag
            want_v[at] = buf[q0 + i, Hq + Hkv:]
            touched.setdefault(at[0], []).append(at[1])
            if Hq:
                r, mag = PR.turn(buf[q0 + i, :Hq], qw if norm else None, norm, 1e-6, p, cs, off, interleaved)
                assert np.all(np.abs(qo[q0 + i] - r) <= U * np.abs(r) + 2.0 ** -17 * mag)
    assert np.all(np.abs(got_k - want_k) <= tol) and np.array_equal(got_v, want_v)
    assert np.all(qo[:lead] == 9) and np.all(qo[T - tail:] == 9)
    got = _np(bounds)
    for page_, slots in touched.items():
        low, high = got_k[page_, slots].min(0), got_k[page_, slots].max(0)
        if 0 not in slots:
            low, high = np.minimum(low, old[page_, 0]), np.maximum(high, old[page_, 1])
        assert np.array_equal(got[page_, 0], low) and np.array_equal(got[page_, 1], high)
    rest = [i for i in range(n_pages) if i not in touched]
    assert np.array_equal(got[rest], old[rest])


def test_append_positions_and_pages_that_are_none():
    """Entries outside the pool, positions past the table and below 0 store nothing; the queries of those rows are done all the
    same; positions of the caller's own turn, those outside the angles give NaN in the rotated part alone."""
    _say("append bad pages")
    g = np.random.default_rng(5)
    lq, lk, page, Hq, Hkv, D, Rd, off = [20, 30, 8, 3], [20, 70, 3, 1 << 30], 16, 4, 2, 64, 32, 16
    table, n_pages = _table(g, [20, 64, 3, 0], page, spare=2)
    table = table[:, :4].copy()
    table[0, 1], table[1, 3] = n_pages, -7
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D)
    T = sum(lq)
    buf = AR.bf16(g.normal(0, 1, (T, Hq + 2 * Hkv, D)))
    bt = _bf16(buf)
    pos = g.integers(0, 50, T).astype(np.int32)
    pos[3], pos[25] = -1, 50
    cs = _angles(50, Rd)
    bounds = torch.zeros(n_pages, 2, Hkv, D, dtype=BF, device="cuda")
    seqs = _seqs(lq, lk)
    q_out = P.paged_append(bt[:, Hq:Hq + Hkv], bt[:, Hq + Hkv:], kt, vt, _i32(np.r_[0, np.cumsum(lq)]), _i32(lk), _i32(table),
                           q=bt[:, :Hq], bounds=bounds, norm=False, positions=_gpu(pos), cos_sin=_gpu(cs), rot_offset=off)
    got_k, got_v, qo = _np(kt), _np(vt), _np(q_out)
    want_k, want_v = kp.copy(), vp.copy()
    stored = 0
    for b, (q0, n, m) in enumerate(seqs):
        for i in range(n):
            r, mag = PR.turn(buf[q0 + i, :Hq], None, False, 0, pos[q0 + i], cs, off, False)
            assert np.array_equal(np.isnan(qo[q0 + i]), np.isnan(r))
            ok = ~np.isnan(r)
            assert np.all(np.abs(qo[q0 + i] - r)[ok] <= (U * np.abs(r) + 2.0 ** -17 * mag)[ok])
            p = i + m - n
            t = PR.page_of(table, b, p, page, n_pages)
            if t is None:
                continue
            stored += 1
            want_k[t, p % page] = PR.turn(buf[q0 + i, Hq:Hq + Hkv], None, False, 0, pos[q0 + i], cs, off, False)[0]
            want_v[t, p % page] = buf[q0 + i, Hq + Hkv:]
    assert stored == 16 + 8 + 3  # of the second sequence, positions 40 to 47 have a page, 48 to 69 none
    assert np.array_equal(np.isnan(got_k), np.isnan(want_k)) and np.array_equal(got_v, want_v)
    ok = ~np.isnan(want_k)
    assert np.all(np.abs(got_k - want_k)[ok] <= (2 * U * np.abs(want_k) + 1e-6)[ok])
    assert not np.isnan(_np(bounds)).any()


def test_append_values():
    """Keys that are NaN, infinite or zero: NaN does not count in the bounds, a column of NaN alone is left open."""
    _say("append values")
    page, Hkv, D = 16, 1, 64
    k = torch.zeros(6, Hkv, D, dtype=BF, device="cuda")
    k[0, 0, 0], k[1, 0, 0], k[2, 0, 1], k[:, 0, 2] = float("inf"), -3, float("nan"), float("nan")
    k[3, 0, 1] = -2
    kt, vt = (torch.zeros(2, page, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    bounds = torch.full((2, 2, Hkv, D), 7.0, dtype=BF, device="cuda")
    for lens in ([6], [1]):  # a run of several rows, then one row that begins the page anew
        n = lens[0]
        P.paged_append(k[:n], k[:n], kt, vt, _i32([0, n]), _i32(lens), _i32([[1]]), bounds=bounds, norm=False)
        assert torch.equal(kt[1, :n].isnan(), k[:n].isnan()) and torch.equal(kt[1, :n].nan_to_num(), k[:n].nan_to_num())
        low, high = _np(bounds)[1, :, 0]
        assert (low[2], high[2]) == (np.inf, -np.inf)
        assert (low[0], high[0]) == ((-3, np.inf) if n == 6 else (np.inf, np.inf))
        assert (low[1], high[1]) == ((-2, 0) if n == 6 else (0, 0))
    # one row behind what is there
    P.paged_append(k[1:2], k[1:2], kt, vt, _i32([0, 1]), _i32([2]), _i32([[1]]), bounds=bounds, norm=False)
    assert _np(bounds)[1, 0, 0, 0] == -3 and _np(bounds)[1, 1, 0, 0] == np.inf
    assert torch.all(bounds[0] == 7)


# ---------------------------------------------------------------- attention
def _check(out, lse, q, kp, vp, table, seqs, see, scale):
    D = q.shape[2]
    ref, rl, mag, dot, count = PR.attention(q, kp, vp, table, seqs, see, scale)
    y, l = _np(out), None if lse is None else _np(lse)
    for q0, n, _ in seqs:
        r, o, m = ref[q0:q0 + n], y[q0:q0 + n], mag[q0:q0 + n]
        assert np.array_equal(np.isnan(o), np.isnan(r)) and np.array_equal(np.isinf(o), np.isinf(r))
        fin = np.isfinite(r) & np.isfinite(m)
        d = (D + 4) * 2.0 ** -23 * dot[q0:q0 + n]
        sums = (count[q0:q0 + n] + 64) * 2.0 ** -23
        tol = U * np.abs(r) + (2 * U + 2 * np.expm1(d) + sums)[..., None] * m + 1e-38
        with np.errstate(all="ignore"):
            assert np.all(np.abs(o - r)[fin] <= tol[fin]), f"worst {np.max(np.abs(o - r)[fin] / tol[fin]):.3f} of its bound"
        assert np.all(o[np.isinf(r)] == r[np.isinf(r)])
        if l is not None:
            a, b = l[q0:q0 + n], rl[q0:q0 + n]
            assert np.array_equal(a == -np.inf, b == -np.inf)
            ok = np.isfinite(b)
            assert np.all(np.abs(a - b)[ok] <= (2 * U + d + sums + 2.0 ** -21 * (1 + np.abs(b)))[ok])


def _run(q, kt, vt, table, seqs, lead=0, **kw):
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    kw.setdefault("max_q", max([s[1] for s in seqs] + [0]))
    kw.setdefault("max_kv", max([s[2] for s in seqs] + [0]))
    mq, mk = kw.pop("max_q"), kw.pop("max_kv")
    cu = _i32([lead] + [s[0] + s[1] for s in seqs])
    return P.paged_attention(q, kt, vt, cu, _i32([s[2] for s in seqs]), _i32(table), mq, mk, lse=lse, **kw), lse


DENSE = [
    # lq, lk, Hq, Hkv, D, page
    ([1], [1], 1, 1, 64, 16), ([1, 1, 1, 1, 1], [1, 31, 0, 65, 300], 4, 1, 128, 16), ([1, 1, 1], [700, 33, 128], 8, 8, 64, 32),
    ([1, 1], [513, 64], 16, 2, 256, 64), ([1], [2600], 4, 1, 128, 128), ([1, 0, 1], [100, 50, 1], 32, 2, 128, 64),
    ([1, 1], [200, 129], 40, 1, 64, 16), ([1], [97], 20, 2, 256, 32), ([7, 40], [70, 300], 4, 2, 128, 16),
    ([100, 3], [160, 3], 2, 1, 64, 64), ([20, 60], [5, 0], 4, 2, 128, 32), ([2, 4], [300, 1], 4, 2, 128, 128),
    ([40], [1500], 2, 2, 128, 16), ([3], [900], 10, 2, 256, 16), ([130], [64], 2, 1, 64, 16), ([5, 5], [600, 2], 6, 2, 64, 64),
    ([150, 1, 90], [150, 1, 90], 6, 2, 128, 32), ([200], [333], 2, 1, 256, 16), ([300], [300], 2, 1, 64, 128)]


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,page", DENSE)
def test_attention(lq, lk, Hq, Hkv, D, page):
    _say("attention", lq, lk, Hq, Hkv, D, page)
    g = np.random.default_rng(sum(lq) * 31 + D + Hq + page)
    table, n_pages = _table(g, lk, page)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D, layout=("pshd", "phsd", "both")[(Hq + page // 16) % 3])
    lead, tail = 2, 3
    q = AR.bf16(g.normal(0, 2, (lead + sum(lq) + tail, Hq, D)))
    out = torch.full((len(q), Hq, 2 * D), 9.0, dtype=BF, device="cuda")
    seqs = _seqs(lq, lk, lead)
    _, lse = _run(_bf16(q), kt, vt, table, seqs, lead, out=out[..., :D])
    _check(out[..., :D], lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv), D ** -0.5)
    assert torch.all(out[..., D:] == 9) and torch.all(out[:lead] == 9) and torch.all(out[lead + sum(lq):] == 9)
    assert torch.all(lse[:lead] == 3) and torch.all(lse[lead + sum(lq):] == 3)


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,page", [
    ([1], [40000], 4, 1, 128, 64), ([1, 1, 1], [20000, 0, 129], 8, 2, 64, 16), ([1, 1], [300, 9000], 16, 2, 256, 32),
    ([6, 1], [9000, 1], 4, 1, 128, 128), ([50, 3], [9000, 600], 2, 1, 64, 16), ([40], [6000], 2, 1, 256, 64)])
def test_attention_many_splits(lq, lk, Hq, Hkv, D, page):
    _say("attention many splits", lq, lk, Hq, Hkv, D, page)
    g = np.random.default_rng(sum(lk) + D)
    table, n_pages = _table(g, lk, page)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D)
    q = AR.bf16(g.normal(0, 2, (sum(lq), Hq, D)))
    seqs = _seqs(lq, lk)
    out, lse = _run(_bf16(q), kt, vt, table, seqs)
    _check(out, lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv), D ** -0.5)


def _group_table(g, lk, page, cu, prefix):
    """A table where the sequences of a group share the pages that their prefix fills; one that is shorter than the prefix
    shares all of its pages."""
    table, n_pages = _table(g, lk, page)
    for i, j, p in zip(cu, cu[1:], prefix):
        for b in range(i, j):
            n = min(max(p, 0), lk[b], lk[i]) // page if lk[b] >= p else -(-lk[b] // page)
            table[b, :n] = table[i, :n]
    return table, n_pages


GROUPS = [
    # lq, lk, cu_group, prefix, Hq, Hkv, D, page
    ([1, 1, 1], [100, 90, 70], [0, 3], [64], 4, 2, 128, 16), ([1, 1], [200, 64], [0, 2], [64], 8, 1, 64, 64),
    ([1] * 5, [300, 280, 33, 500, 70], [0, 2, 3, 5], [257, 33, 66], 4, 4, 64, 32),
    ([1] * 9, [1000 + i for i in range(9)], [0, 9], [1000], 16, 2, 128, 64), ([1] * 3, [700, 650, 641], [0, 3], [640], 8, 2, 256, 128),
    ([20, 7, 33], [150, 130, 128], [0, 3], [100], 4, 2, 128, 16), ([40, 1, 0, 12], [400, 390, 380, 395], [0, 4], [384], 2, 1, 256, 32),
    # sequences outside every group; groups without sequences, without a prefix, with one shorter than a page
    ([1] * 6, [90] * 6, [1, 1, 3, 4, 5], [80, 64, 0, 15], 4, 2, 128, 16),
    # a prefix that rows see part of (they are rows of it), or that is longer than the sequence
    ([60, 60], [100, 100], [0, 2], [96], 4, 2, 64, 16), ([3, 1], [50, 20], [0, 2], [48], 2, 2, 128, 16),
    ([1] * 40, [600 + 7 * i for i in range(40)], [0, 40], [576], 8, 2, 64, 64),
    # own keys that begin inside a tile of 64, and end in its first, second and last 16
    ([1, 1, 1], [230, 195, 300], [0, 3], [106], 2, 1, 64, 16), ([9, 40], [300, 470], [0, 2], [250], 4, 2, 128, 16),
    ([2, 70], [330, 305], [0, 2], [165], 2, 1, 256, 32), ([0, 3], [190, 230], [0, 2], [106], 2, 1, 256, 16),
    # many tiles whose own keys fill a piece but for what is left of the prefix's page; chunks of wide heads behind many pieces
    ([1] * 40, [2024 - 3 * i for i in range(40)], [0, 40], [1000], 8, 8, 64, 64),
    ([30, 20, 40], [2300, 2250, 2292], [0, 3], [2048], 16, 4, 256, 64)]


@pytest.mark.parametrize("lq,lk,cu,prefix,Hq,Hkv,D,page", GROUPS)
def test_shared_prefix(lq, lk, cu, prefix, Hq, Hkv, D, page):
    """Against the reference, which knows nothing of groups; rows behind the last sequence keep what they hold."""
    _say("shared prefix", lq, lk, cu, prefix, Hq, Hkv, D, page)
    g = np.random.default_rng(sum(lk) + D + page)
    table, n_pages = _group_table(g, lk, page, cu, prefix)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D, layout="both" if page == 16 else "phsd")
    tail = 2
    q = AR.bf16(g.normal(0, 2, (sum(lq) + tail, Hq, D)))
    seqs = _seqs(lq, lk)
    out = torch.full(q.shape, 9.0, dtype=BF, device="cuda")
    of = [0] * len(lk)
    for i, j, p in zip(cu, cu[1:], prefix):
        of[i:j] = [p] * (j - i)
    _, lse = _run(_bf16(q), kt, vt, table, seqs, cu_group=_i32(cu), prefix_len=_i32(prefix), max_prefix=max(prefix),
                  max_kv=max(max(m - p, 0) for m, p in zip(lk, of)), out=out)
    _check(out, lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv), D ** -0.5)
    assert torch.all(out[sum(lq):] == 9) and torch.all(lse[sum(lq):] == 3)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 64), (2, 2, 64, 16), (4, 1, 256, 32), (4, 4, 128, 128)])
@pytest.mark.parametrize("lq,lk,cu,prefix,max_kv", [
    ([1], [0], [0, 1], [0], 8), ([1, 1, 1, 1], [0, 5, 0, 1], [0, 2, 4], [0, 0], 9), ([200], [50], [0, 1], [0], 50),
    ([1, 40, 0, 1], [3, 30, 0, 0], [1, 4], [15], 20), ([130, 2], [1, 0], [0, 1, 2], [0, 0], 1), ([3], [2], [0, 1], [9], 0)])
def test_groups_that_share_nothing_in_one_piece(lq, lk, cu, prefix, max_kv, Hq, Hkv, D, page):
    """Groups without a whole page, over so few keys that a row has one share and the call needs no workspace: rows
    that see no key get their zeros."""
    _say("groups in one piece", lq, lk, cu, prefix, max_kv, Hq, Hkv, D, page)
    g = np.random.default_rng(sum(lq) + D)
    table, n_pages = _table(g, lk, page)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D)
    q = AR.bf16(g.normal(0, 2, (sum(lq) + 2, Hq, D)))
    seqs = _seqs(lq, lk)
    of = [0] * len(lk)
    for i, j, p in zip(cu, cu[1:], prefix):
        of[i:j] = [p] * (j - i)
    out = torch.full(q.shape, 9.0, dtype=BF, device="cuda")
    assert P.paged_attention_workspace_size(_bf16(q), kt, len(lq), max(lq), max_kv, n_groups=len(prefix), max_prefix=max(prefix)) == 0
    _, lse = _run(_bf16(q), kt, vt, table, seqs, cu_group=_i32(cu), prefix_len=_i32(prefix), max_prefix=max(prefix), max_kv=max_kv,
                  out=out)
    see = PR.visible(seqs, table, page, n_pages, Hkv, prefix=of, max_prefix=max(prefix), max_kv=max_kv)
    _check(out, lse, q, kp, vp, table, seqs, see, D ** -0.5)
    assert torch.all(out[sum(lq):] == 9) and torch.all(lse[sum(lq):] == 3)


@pytest.mark.parametrize("pages,width,max_kv", [(0, 2, 100), (5, 0, 0)])
def test_groups_over_an_empty_cache(pages, width, max_kv):
    """A pool without pages, and a table without entries: every row sees nothing."""
    _say("groups, empty cache", pages, width)
    pool = torch.zeros(pages, 64, 2, 128, dtype=BF, device="cuda")
    q = torch.ones(3, 8, 128, dtype=BF, device="cuda")
    lse = torch.full((3, 8), 3.0, device="cuda")
    args = q, pool, pool, _i32([0, 1, 3]), _i32([50, 2]), torch.zeros(2, width, dtype=torch.int32, device="cuda"), 2, max_kv
    assert P.paged_attention_workspace_size(q, pool, 2, 2, max_kv, n_groups=1) == 0
    out = P.paged_attention(*args, cu_group=_i32([0, 2]), prefix_len=_i32([0]), lse=lse)
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


def _blocks(g, seqs, T, Hkv, page, n, junk=True):
    """Lists of blocks: distinct ones, and now and then one twice, out of order, past the row's end, below 0, or none at all."""
    out = np.full((T, Hkv, n), -1)
    for q0, lq, lk in seqs:
        for i in range(lq):
            for h in range(Hkv):
                c = max((i + lk - lq) // page + 1, 0)
                pick = g.permutation(c)[:n]
                out[q0 + i, h, :len(pick)] = np.sort(pick)
                if junk and n > 2 and g.random() < 0.3:
                    out[q0 + i, h, g.integers(n)] = g.choice([-1, -(1 << 31), c, c + 7, (1 << 31) - 1, 0])
                    g.shuffle(out[q0 + i, h])
                if junk and g.random() < 0.05:
                    out[q0 + i, h] = -1
    return out


SPARSE = [
    # lq, lk, Hq, Hkv, D, page, n_blocks
    ([1], [1], 1, 1, 64, 16, 1), ([1, 1, 1], [300, 40, 0], 8, 2, 128, 16, 5), ([1, 1], [900, 1000], 4, 4, 64, 32, 7),
    ([1], [5000], 16, 2, 128, 64, 20), ([1, 1], [800, 129], 8, 1, 256, 128, 3), ([9, 30], [200, 300], 4, 2, 128, 16, 6),
    ([70], [600], 2, 2, 64, 64, 4), ([33, 1, 0, 5], [333, 64, 10, 700], 10, 2, 128, 32, 9), ([20], [400], 6, 1, 256, 16, 8),
    ([3, 2], [2000, 1500], 40, 1, 64, 16, 60), ([40], [3000], 3, 3, 128, 16, 100), ([2], [16000], 32, 1, 128, 16, 1000)]


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,page,n", SPARSE)
def test_listed_blocks(lq, lk, Hq, Hkv, D, page, n):
    _say("listed blocks", lq, lk, Hq, Hkv, D, page, n)
    g = np.random.default_rng(sum(lk) + D + n)
    table, n_pages = _table(g, lk, page)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D, layout="phsd" if page == 16 else "pshd")
    lead = 1
    q = AR.bf16(g.normal(0, 2, (lead + sum(lq) + 2, Hq, D)))
    seqs = _seqs(lq, lk, lead)
    blocks = _blocks(g, seqs, len(q), Hkv, page, n)
    out = torch.full(q.shape, 9.0, dtype=BF, device="cuda")
    _, lse = _run(_bf16(q), kt, vt, table, seqs, lead, blocks=_i32(blocks), out=out)
    _check(out, lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv, blocks), D ** -0.5)
    assert torch.all(out[:lead] == 9) and torch.all(out[lead + sum(lq):] == 9)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lq,lk,G,D,page,mode", [
    ([1, 1], [70, 33], 4, 128, 16, "dense"), ([3], [100], 2, 128, 64, "dense"), ([60, 60], [700, 61], 1, 128, 32, "dense"),
    ([2], [600], 4, 256, 16, "dense"), ([1, 1, 1], [200, 150, 131], 4, 64, 16, "groups"), ([40, 9], [300, 290], 2, 128, 64, "groups"),
    ([1, 1], [500, 300], 4, 128, 64, "blocks"), ([12], [400], 4, 64, 16, "blocks"), ([5], [500], 8, 256, 32, "blocks")])
def test_hidden_values(lq, lk, G, D, page, mode, bad):
    """What a row must not see does not reach it, whatever it holds: slots past a sequence's end, pages of nobody, later keys of a
    chunk, blocks that other tokens list; rows that do see it show it as the formula does."""
    _say("hidden values", lq, lk, G, D, page, mode, bad)
    g = np.random.default_rng(11)
    Hkv = 2
    cu, prefix = [0, len(lk)], [min(lk) - max(lq)]
    table, n_pages = _group_table(g, lk, page, cu, prefix) if mode == "groups" else _table(g, lk, page)
    kp, vp, _, _ = _pool(g, n_pages, page, Hkv, D)
    q = AR.bf16(g.normal(0, 1, (sum(lq), 2 * G, D)))
    held = np.zeros((n_pages, page), bool)
    seqs = _seqs(lq, lk)
    for b, (_, n, m) in enumerate(seqs):
        for p in range(m):
            held[table[b, p // page], p % page] = True
        if n > 2:  # a value that only the last two rows see
            at = table[b, (m - 2) // page], (m - 2) % page
            vp[at][1, 5], vp[at][0, 6] = bad, -bad
    kp[~held], vp[~held] = bad, bad
    kw, blocks = {}, None
    if mode == "blocks":
        blocks = _blocks(g, seqs, len(q), Hkv, page, 3, junk=False)
        blocks[0, 0, 0] = 0
        blocks[-1, 1] = [1, -1, -1]
        t = table[0, 1]
        vp[t, 3, 1, 7] = bad  # block 1 of the first sequence: not every row lists it
        kw["blocks"] = _i32(blocks)
    elif mode == "groups":
        kw = dict(cu_group=_i32(cu), prefix_len=_i32(prefix), max_prefix=prefix[0], max_kv=max(lk) - prefix[0])
    out, lse = _run(_bf16(q), _bf16(kp), _bf16(vp), table, seqs, **kw)
    _check(out, lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv, blocks), D ** -0.5)


@pytest.mark.parametrize("lq,lk,Hq,D,page,mode", [
    ([1, 1], [300, 100], 4, 128, 16, "dense"), ([50], [400], 2, 64, 32, "dense"), ([30], [300], 8, 256, 16, "dense"),
    ([1, 1], [400, 380], 4, 128, 64, "groups"), ([20, 20], [300, 290], 4, 64, 16, "groups"),
    ([1, 1], [400, 300], 4, 128, 16, "blocks"), ([10], [300], 4, 64, 64, "blocks")])
def test_pages_that_are_none(lq, lk, Hq, D, page, mode):
    """Entries of the table outside the pool: their keys are not seen, and nothing is read through them."""
    _say("pages that are none", lq, lk, Hq, D, page, mode)
    g = np.random.default_rng(21)
    cu, prefix = [0, len(lk)], [min(lk) - max(lq)]
    table, n_pages = _group_table(g, lk, page, cu, prefix) if mode == "groups" else _table(g, lk, page)
    kp, vp, kt, vt = _pool(g, n_pages, page, 1, D)
    bad = [-1, n_pages, -(1 << 31), (1 << 31) - 1]
    for i, c in enumerate((0, 2, 3, 5)):
        if c < table.shape[1]:
            table[:, c] = bad[i]
    table[-1, (lk[-1] - 1) // page] = -3  # the last row's own page
    q = AR.bf16(g.normal(0, 1, (sum(lq), Hq, D)))
    seqs, kw, blocks = _seqs(lq, lk), {}, None
    if mode == "blocks":
        blocks = _blocks(g, seqs, len(q), 1, page, 4, junk=False)
        kw["blocks"] = _i32(blocks)
    elif mode == "groups":
        kw = dict(cu_group=_i32(cu), prefix_len=_i32(prefix), max_prefix=prefix[0], max_kv=max(lk) - prefix[0])
    out, lse = _run(_bf16(q), kt, vt, table, seqs, **kw)
    _check(out, lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, 1, blocks), D ** -0.5)


@pytest.mark.parametrize("lq,lk,prefix,max_q,max_prefix,max_kv,Hq,D,page", [
    ([40], [100], None, 25, 0, 60, 4, 128, 16), ([1, 1], [300, 90], None, 1, 0, 77, 4, 64, 32), ([200], [300], None, 130, 0, 280, 2, 256, 16),
    ([1, 1], [300, 200], 160, 1, 90, 100, 4, 128, 16), ([20, 9], [300, 200], 150, 12, 64, 120, 4, 64, 64),
    ([1, 1], [300, 200], 160, 1, 160, 0, 4, 128, 16), ([1], [300], 200, 1, 10, 50, 4, 128, 64)])
def test_cuts_leave_the_diagonal(lq, lk, prefix, max_q, max_prefix, max_kv, Hq, D, page):
    """Rows past max_q get no output; a prefix is cut to max_prefix, keys from there + max_kv on are not seen."""
    _say("cuts", lq, lk, prefix, max_q, max_prefix, max_kv)
    g = np.random.default_rng(31)
    cu, pre = [0, len(lk)], [prefix or 0]
    table, n_pages = _group_table(g, lk, page, cu, pre)
    kp, vp, kt, vt = _pool(g, n_pages, page, 2, D)
    q = AR.bf16(g.normal(0, 2, (sum(lq), Hq, D)))
    seqs = _seqs(lq, lk)
    kw = dict(cu_group=_i32(cu), prefix_len=_i32(pre), max_prefix=max_prefix) if prefix else {}
    out = torch.full(q.shape, 9.0, dtype=BF, device="cuda")
    _, lse = _run(_bf16(q), kt, vt, table, seqs, max_q=max_q, max_kv=max_kv, out=out, **kw)
    see = PR.visible(seqs, table, page, n_pages, 2, prefix=[prefix] * len(lk) if prefix else None, max_prefix=max_prefix,
                     max_kv=max_kv)
    for b, (q0, n, m) in enumerate(seqs):
        k = min(n, max_q)
        one, which = [(0, 0, 0)] * len(seqs), list(see)
        one[b], which[b] = (q0, k, m), see[b][:k]
        _check(out, lse, q, kp, vp, table, one, which, D ** -0.5)
        assert torch.all(out[q0 + k:q0 + n] == 9) and torch.all(lse[q0 + k:q0 + n] == 3)


@pytest.mark.parametrize("mode", ["dense", "groups", "blocks"])
def test_arrays_are_cut_to_the_tensors(mode):
    """cu_q, kv_len, cu_group and prefix_len that point anywhere read and write nothing outside; a sequence that is whole beside
    them is right."""
    _say("arrays", mode)
    g = np.random.default_rng(14)
    low, high = -(1 << 31), (1 << 31) - 1
    page, D = 16, 64
    table, n_pages = _table(g, [60, 100, 30, 30, 30, 30], page)
    kp, vp, kt, vt = _pool(g, n_pages, page, 1, D)
    q = AR.bf16(g.normal(0, 1, (40, 2, D)))
    lead = 8
    out = torch.full((lead + 40 + lead, 2, D), 9.0, dtype=BF, device="cuda")
    kw = {}
    if mode == "groups":
        kw = dict(cu_group=_i32([low, -5, 1, 2, 3, high, 7]), prefix_len=_i32([50, 50, 48, low, high, 9]), max_prefix=64)
    elif mode == "blocks":
        kw = dict(blocks=_i32(np.tile([0, 3, 5, high, low], (40, 1, 1))))
    cu, lens = [5, low, 10, 30, high, 30, low + 3], [60, 100, 61, high, low, 0]
    P.paged_attention(_bf16(q), kt, vt, _i32(cu), _i32(lens), _i32(table), 40, 112, out=out[lead:lead + 40], **kw)
    torch.cuda.synchronize()
    assert torch.all(out[:lead] == 9) and torch.all(out[lead + 40:] == 9)
    if mode == "dense":  # rows 10 to 29 are the third sequence's
        seqs = [(0, 0, 0)] * 2 + [(10, 20, 61)]
        _check(out[lead:lead + 40], None, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, 1), D ** -0.5)


@pytest.mark.parametrize("mode", ["token", "rows", "groups", "blocks"])
def test_cache_past_32_bits(mode):
    """A pool of more than 2^31 elements, with pages at its ends and on both sides of element 2^31."""
    page, Hkv, D = 64, 8, 128
    n_pages = (1 << 15) + 100
    _say("long cache", mode)
    kt, vt = (torch.empty(n_pages, page, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    g = np.random.default_rng(3)
    use = np.r_[0:8, (1 << 15) - 8:(1 << 15) + 8, n_pages - 8:n_pages]
    lk = [500, 400, 300]
    table = np.full((3, 9), -1, np.int32)
    pick = g.permutation(use)
    at = 0
    for b, m in enumerate(lk):
        n = -(-m // page)
        table[b, :n] = pick[at:at + n]
        at += n
    lq = [100, 1, 30] if mode == "rows" else [1, 1, 1]
    seqs = _seqs(lq, lk)
    T = sum(lq)
    k, v = (torch.randn(T, Hkv, D, device="cuda").to(BF) for _ in range(2))
    sel = torch.from_numpy(use).cuda()
    kt[sel], vt[sel] = (torch.randn(len(use), page, Hkv, D, device="cuda").to(BF) for _ in range(2))
    P.paged_append(k, v, kt, vt, _i32(np.r_[0, np.cumsum(lq)]), _i32(lk), _i32(table), norm=False)
    q = torch.randn(T, 8, D, device="cuda").to(BF)
    kw, blocks = {}, None
    if mode == "groups":
        table[1, :4], table[2, :4] = table[0, :4], table[0, :4]
        kw = dict(cu_group=_i32([0, 3]), prefix_len=_i32([256]), max_prefix=256, max_kv=300)
    elif mode == "blocks":
        blocks = _blocks(g, seqs, T, Hkv, page, 4, junk=False)
        kw["blocks"] = _i32(blocks)
    out, lse = _run(q, kt, vt, table, seqs, **kw)
    place = {int(p): i for i, p in enumerate(use)}
    small = np.vectorize(lambda p: place.get(int(p), -1))(table)
    kp, vp = _np(kt[sel]), _np(vt[sel])
    for b, (q0, n, m) in enumerate(seqs):  # what append stored
        for i in range(n):
            p = i + m - n
            if mode != "groups":
                assert np.array_equal(kp[small[b, p // page], p % page], _np(k[q0 + i]))
    _check(out, lse, _np(q), kp, vp, small, seqs, PR.visible(seqs, small, page, len(use), Hkv, blocks), D ** -0.5)


# ---------------------------------------------------------------- selection
SELECT = [
    # lq, lk, Hq, Hkv, D, page, n_blocks, first, last
    ([1], [1], 1, 1, 64, 16, 1, 0, 1), ([1, 1, 1], [300, 16, 0], 8, 2, 128, 16, 5, 1, 1), ([1], [8192], 4, 1, 64, 16, 30, 1, 2),
    ([1, 1], [9000, 700], 16, 2, 256, 32, 17, 0, 1), ([40, 0, 3], [900, 5, 33], 6, 2, 128, 16, 8, 2, 3),
    ([20], [5], 4, 2, 64, 16, 3, 1, 1), ([130], [4000], 5, 1, 128, 64, 12, 1, 2), ([7], [70000], 8, 4, 64, 16, 64, 1, 1),
    ([2], [150000], 2, 1, 64, 16, 200, 3, 4), ([1], [524288], 2, 2, 64, 16, 1024, 1, 1), ([3], [600], 4, 4, 128, 16, 38, 1, 1),
    ([17, 16, 15, 1], [1700, 1600, 1500, 1400], 32, 4, 128, 16, 9, 1, 2), ([65], [40000], 4, 2, 256, 128, 20, 0, 1),
    # tiles of 16 rows: with ends of sequences and empty ones inside, rows that see fewer blocks than are wanted, every head size
    ([300, 0, 5, 211], [700, 0, 5, 1900], 4, 2, 128, 16, 9, 1, 2), ([600], [600], 2, 1, 64, 16, 7, 0, 1), ([100, 90, 110], [900, 90, 4000], 9, 3, 256, 32, 12, 2, 3),
    ([260], [9000], 4, 2, 64, 16, 30, 1, 1)]


@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,page,n,first,last", SELECT)
def test_select(lq, lk, Hq, Hkv, D, page, n, first, last):
    _say("select", lq, lk, Hq, Hkv, D, page, n, first, last)
    g = np.random.default_rng(sum(lk) + n)
    table, n_pages = _table(g, lk, page)
    mid, spread = g.normal(0, 1, (n_pages, 1, Hkv, D)), np.abs(g.normal(0, 0.5, (n_pages, 1, Hkv, D)))
    bounds = AR.bf16(np.concatenate([mid - spread, mid + spread], 1))
    lead = 1
    q = AR.bf16(g.normal(0, 2, (lead + sum(lq) + 2, Hq, D)))
    seqs = _seqs(lq, lk, lead)
    out = torch.full((len(q), Hkv, n), -2, dtype=torch.int32, device="cuda")
    P.select_blocks(_bf16(q), _bf16(bounds), _i32([lead] + [s[0] + s[1] for s in seqs]), _i32(lk), _i32(table), max(lq), max(lk), page,
                    n, first=first, last=last, blocks=out)
    assert np.array_equal(out.cpu().numpy(), PR.select(q, bounds, table, seqs, page, n, first, last))


def test_select_ties_and_values():
    """Equal scores go to the lower block, also far apart; scores that are not finite come first, pages that are none last; a query
    of zeros or NaN; keys past max_kv and rows past max_q."""
    _say("select ties")
    g = np.random.default_rng(8)
    page, D, Hkv = 16, 64, 2
    for L in (400 * page, 3000 * page, 9000 * page):
        lq = 6
        table, n_pages = _table(g, [L], page)
        some = AR.bf16(g.normal(0, 1, (5, 2, Hkv, D)))
        some.sort(1)
        bounds = some[g.integers(0, 5, n_pages)]  # five kinds of pages: ties everywhere
        bounds[table[0, 7], 1, 0, 3], bounds[table[0, 300], 0, 1, 9] = np.inf, np.nan
        table[0, 11] = -1
        q = AR.bf16(g.normal(0, 1, (lq, 4, D)))
        q[2] = 0
        q[3, 0, 0] = np.nan
        q[4] = -q[4]
        for n, first, last in ((20, 1, 2), (150, 0, 1)):
            args = (_bf16(q), _bf16(bounds), _i32([0, lq]), _i32([L]), _i32(table), lq, L, page, n)
            got = P.select_blocks(*args, first=first, last=last).cpu().numpy()
            assert np.array_equal(got, PR.select(q, bounds, table, [(0, lq, L)], page, n, first, last))
    out = torch.full((lq, Hkv, 20), -2, dtype=torch.int32, device="cuda")
    P.select_blocks(*args[:5], 4, L - 5000, page, 20, blocks=out)
    want = PR.select(q, bounds, table, [(0, lq, L)], page, 20, 1, 1, max_kv=L - 5000)
    assert np.array_equal(out.cpu().numpy()[:4], want[:4]) and torch.all(out[4:] == -2)


def test_select_in_batches():
    """More rows than the scores of one launch have room for."""
    T, L, page, Hkv, D = 3000, 1 << 18, 16, 2, 64
    _say("select batches")
    g = np.random.default_rng(9)
    table, n_pages = _table(g, [L], page)
    bounds = AR.bf16(np.sort(g.normal(0, 1, (n_pages, 2, Hkv, D)), 1))
    q = AR.bf16(g.normal(0, 1, (T, 2, D)))
    got = P.select_blocks(_bf16(q), _bf16(bounds), _i32([0, T]), _i32([L]), _i32(table), T, L, page, 10).cpu().numpy()
    rows = np.unique(np.r_[0, T - 1, g.integers(0, T, 12), 1023, 1024])
    for r in rows:
        want = PR.select(q[r:r + 1], bounds, table, [(0, 1, L - T + 1 + r)], page, 10, 1, 1)
        assert np.array_equal(got[r], want[0]), r


def test_select_single_tokens_in_batches():
    """The same for single tokens of many sequences over very long tables."""
    B, page, Hkv, D, n_pages = 600, 16, 2, 64, 900
    width = 32768
    _say("select batches of tokens")
    g = np.random.default_rng(10)
    table = torch.randint(0, n_pages, (B, width), dtype=torch.int32, device="cuda")
    lk = g.integers(1, width * page + 1, B)
    lk[0], lk[599] = width * page, width * page - 3
    bounds = AR.bf16(np.sort(g.normal(0, 1, (n_pages, 2, Hkv, D)), 1))
    q = AR.bf16(g.normal(0, 1, (B, 2, D)))
    got = P.select_blocks(_bf16(q), _bf16(bounds), _i32(np.arange(B + 1)), _i32(lk), table, 1, width * page, page, 40,
                          first=2).cpu().numpy()
    for r in (0, 255, 511, 512, 598, 599):  # a table of 900 pages: equal scores everywhere
        assert np.array_equal(got[r], PR.select(q[r:r + 1], bounds, table[r:r + 1].cpu().numpy(), [(0, 1, int(lk[r]))], page, 40, 2, 1)[0]), r


# ---------------------------------------------------------------- together
def _state(seed=0, B=5, Hq=8, Hkv=2, D=128, page=16):
    g = np.random.default_rng(seed)
    lens = [int(n) for n in g.integers(100, 900, B)]
    table, n_pages = _table(g, [n + 8 for n in lens], page)
    table = np.pad(table, ((0, 0), (0, 63 - table.shape[1])), constant_values=-1)
    _, _, kt, vt = _pool(g, n_pages, page, Hkv, D)
    bounds = torch.stack([kt.amin(1), kt.amax(1)], 1).contiguous()
    qkv = _bf16(g.normal(0, 1, (B, Hq + 2 * Hkv, D)))
    st = dict(qkv=qkv, kt=kt, vt=vt, bounds=bounds, table=_i32(table), len=_i32(lens), cu=_i32(np.arange(B + 1)),
              cs=_gpu(_angles(1000, D)), q=torch.empty(B, Hq, D, dtype=BF, device="cuda"),
              blocks=torch.empty(B, Hkv, 12, dtype=torch.int32, device="cuda"), out=torch.empty(B, Hq, D, dtype=BF, device="cuda"),
              dense=torch.empty(B, Hq, D, dtype=BF, device="cuda"), start=lens, Hq=Hq, Hkv=Hkv)
    st["group"], st["prefix"] = _i32([0, 3, B]), _i32([64, 0])
    table[1:3, :4] = table[0, :4]
    st["table"] = _i32(table)
    st["ws"] = [P.select_blocks_workspace(st["q"], bounds, B, 1, 1000, page),
                P.paged_attention_workspace(st["q"], kt, B, 1, 1000, n_blocks=12),
                P.paged_attention_workspace(st["q"], kt, B, 1, 1000, n_groups=2, max_prefix=64)]
    return st


def _step(st):
    """A single-token step: append, select, attention over the selected blocks and over everything behind a shared prefix."""
    Hq, Hkv = st["Hq"], st["Hkv"]
    at = st["cu"], st["len"], st["table"]
    P.paged_append(st["qkv"][:, Hq:Hq + Hkv], st["qkv"][:, Hq + Hkv:], st["kt"], st["vt"], *at, q=st["qkv"][:, :Hq], q_out=st["q"],
                   bounds=st["bounds"], cos_sin=st["cs"])
    P.select_blocks(st["q"], st["bounds"], *at, 1, 1000, st["kt"].shape[1], 12, last=2, blocks=st["blocks"], ws=st["ws"][0])
    P.paged_attention(st["q"], st["kt"], st["vt"], *at, 1, 1000, blocks=st["blocks"], out=st["out"], ws=st["ws"][1])
    P.paged_attention(st["q"], st["kt"], st["vt"], *at, 1, 1000, cu_group=st["group"], prefix_len=st["prefix"], max_prefix=64,
                      out=st["dense"], ws=st["ws"][2])


def _same(a, b):
    return all(torch.equal(a[k], b[k]) for k in ("q", "blocks", "out", "dense", "kt", "vt", "bounds"))


def test_steps_together():
    """Steps of one token against the references over what the cache then holds."""
    _say("together")
    st = _state()
    page, B = 16, 5
    for step in range(6):
        _step(st)
        lens = [n + step for n in st["start"]]
        assert st["len"].tolist() == lens
        seqs, table = [(b, 1, lens[b]) for b in range(B)], st["table"].cpu().numpy()
        kp, vp, q = _np(st["kt"]), _np(st["vt"]), _np(st["q"])
        blocks = st["blocks"].cpu().numpy()
        assert np.array_equal(blocks, PR.select(q, _np(st["bounds"]), table, seqs, page, 12, 1, 2))
        for out, b in ((st["out"], blocks), (st["dense"], None)):
            _check(out, None, q, kp, vp, table, seqs, PR.visible(seqs, table, page, len(kp), 2, b), 128 ** -0.5)
        for b in range(B):  # the bounds hold for every key of a page
            t, n = table[b, (lens[b] - 1) // page], (lens[b] - 1) % page + 1
            assert np.all(kp[t, :n] >= _np(st["bounds"])[t, 0]) and np.all(kp[t, :n] <= _np(st["bounds"])[t, 1])
        st["len"].add_(1)
        st["qkv"].mul_(-0.75)


def test_graph_replays_match_eager():
    """A captured step that moves on by itself, replayed with eager work between, against an eager twin."""
    _say("graph")
    a, b = _state(1), _state(1)

    def step(st):
        _step(st)
        st["len"].add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    torch.cuda.current_stream().wait_stream(side)
    step(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for i in range(5):
        for st in (a, b):
            st["qkv"].mul_(-0.75)
            st["out"].zero_()
        for w in a["ws"]:
            w.fill_(255)
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert _same(a, b), i


def test_other_stream_and_repeats():
    """The calls go to the current stream; the same inputs give the same bits."""
    _say("stream")
    a, b = _state(2), _state(2)
    _step(a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b["qkv"].mul_(2.0)
        b["qkv"].mul_(0.5)
        _step(b)
    s.synchronize()
    assert _same(a, b)
    _step(a)
    assert _same(a, b)


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own."""
    _say("two streams")
    want, got = [_state(3), _state(4)], [_state(3), _state(4)]
    for st in want:
        _step(st)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, s in zip(got, streams):
        with torch.cuda.stream(s):
            _step(st)
    torch.cuda.synchronize()
    assert all(_same(a, b) for a, b in zip(want, got))


# ---------------------------------------------------------------- the binding
def test_binding_refusals():
    _say("refusals")
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    q, k, pool, cu, n = z(4, 2, 64), z(4, 1, 64), z(3, 16, 1, 64), _i32([0, 4]), _i32([4])
    table, bounds = _i32([[0, 1]]), z(3, 2, 1, 64)
    for args, kw in [((k.float(), k, pool, pool, cu, n, table), {}), ((k, k[:3], pool, pool, cu, n, table), {}),
                     ((k, k, pool[:2], pool, cu, n, table), {}), ((k, k, pool, pool[:2], cu, n, table), {}),
                     ((k, k, pool, pool, cu.long(), n, table), {}), ((k, k, pool, pool, cu, _i32([4, 4]), table), {}),
                     ((k, k, pool, pool, cu, n, table[0]), {}), ((k, k, pool, pool, cu, n, table.cpu()), {}),
                     ((k, k, pool, pool, cu, n, table), dict(q=q[:3])), ((k, k, pool, pool, cu, n, table), dict(q_out=q)),
                     ((k, k, pool, pool, cu, n, table), dict(bounds=bounds[:2])),
                     ((k, k, pool, pool, cu, n, table), dict(cos_sin=torch.zeros(64, device="cuda"))),
                     ((k, k, pool.cpu(), pool, cu, n, table), {}), ((k, k, pool[..., :32], pool[..., :32], cu, n, table), {})]:
        with pytest.raises(ValueError):
            P.paged_append(*args, **kw)
    for kw in (dict(norm=False, k_weight=torch.ones(64, device="cuda")), dict(eps=-1.0)):
        with pytest.raises(P.MoeError):
            P.paged_append(k, k, pool, pool, cu, n, table, **kw)
    with pytest.raises(P.MoeError):
        P.paged_append(k, k, z(3, 24, 1, 64), z(3, 24, 1, 64), cu, n, table)
    for args, kw in [((q.float(), pool, pool, cu, n, table, 4, 4), {}), ((q, pool, pool[:2], cu, n, table, 4, 4), {}),
                     ((z(4, 2, 128), pool, pool, cu, n, table, 4, 4), {}), ((q, pool, pool, cu, n, table, 4, 4), dict(cu_group=cu)),
                     ((q, pool, pool, cu, n, table, 4, 4), dict(cu_group=cu, prefix_len=_i32([1, 1]))),
                     ((q, pool, pool, cu, n, table, 4, 4), dict(blocks=_i32(np.zeros((4, 2, 3))))),
                     ((q, pool, pool, cu, n, table, 4, 4), dict(blocks=_i32(np.zeros((4, 1, 0))))),
                     ((q, pool, pool, cu, n, table, 4, 4), dict(out=q[:3])),
                     ((q, pool, pool, cu, n, table, 4, 4), dict(lse=torch.zeros(4, 3, device="cuda")))]:
        with pytest.raises(ValueError):
            P.paged_attention(*args, **kw)
    for mq, mk in ((5, 4), (-1, 4), (4, 33), (4, -1)):
        with pytest.raises(P.MoeError):
            P.paged_attention(q, pool, pool, cu, n, table, mq, mk)
    for args, kw in [((q.float(), bounds, cu, n, table, 4, 4, 16, 2), {}), ((q, bounds[0], cu, n, table, 4, 4, 16, 2), {}),
                     ((q, bounds, cu, n, table, 4, 4, 16, 2), dict(blocks=_i32(np.zeros((4, 1, 3)))))]:
        with pytest.raises(ValueError):
            P.select_blocks(*args, **kw)
    for kw in (dict(first=2), dict(last=0)):
        with pytest.raises(P.MoeError):
            P.select_blocks(q, bounds, cu, n, table, 4, 4, 16, 2, **kw)
    # 4 rows over 512 pages: the scores go through a workspace
    long, ws = _i32(np.zeros((1, 512))), torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert P.select_blocks_workspace(q, bounds, 1, 4, 8192, 16).numel() > 256
    with pytest.raises(P.MoeError):
        P.select_blocks(q, bounds, cu, n, long, 4, 8192, 16, 2, ws=ws)


def test_no_tokens():
    """Empty batches, empty caches and empty tables."""
    _say("nothing")
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert P.paged_append(z(0, 1, 64), z(0, 1, 64), z(3, 16, 1, 64), z(3, 16, 1, 64), _i32([0]), none, none.view(0, 0),
                          q=z(0, 2, 64)).shape == (0, 2, 64)
    assert P.paged_attention(z(0, 2, 64), z(3, 16, 1, 64), z(3, 16, 1, 64), _i32([0]), none, none.view(0, 0), 0, 0).shape == (0, 2, 64)
    # rows, but no pages
    q, cu, n = z(3, 2, 64) + 1, _i32([0, 3]), _i32([3])
    for pool, table in ((z(0, 16, 1, 64), _i32([[0]])), (z(2, 16, 1, 64), none.view(1, 0))):
        width = table.shape[1] * 16
        out, lse = P.paged_attention(q, pool, pool, cu, n, table, 3, min(3, width)), None
        assert torch.all(out == 0)
        P.paged_append(q[:, :1], q[:, :1], pool, pool, cu, n, table)
        assert torch.all(pool == 0)
        blocks = P.select_blocks(q, z(pool.shape[0], 2, 1, 64), cu, n, table, 3, min(3, width), 16, 2)
        assert torch.all(blocks == -1)


# ---------------------------------------------------------------- many, odd, strided
def test_many_sequences_and_groups():
    """More sequences and groups than a wave looks up at once, in a table whose rows are parts of wider ones; sequences of no rows
    and of no tokens among them."""
    _say("many sequences")
    g = np.random.default_rng(15)
    B, page, Hq, Hkv, D = 200, 16, 4, 2, 64
    lq = [int(n) for n in g.integers(0, 4, B)]
    lq[7], lq[150] = 45, 70
    lk = [n + int(g.integers(0, 90)) for n in lq]
    lk[3], lk[20], lk[199] = 0, 0, 300
    cu = np.unique(np.r_[0, g.integers(0, B, 90), B])
    prefix = [int(min(lk[b] for b in range(i, j))) - 5 for i, j in zip(cu, cu[1:])]
    table, n_pages = _group_table(g, lk, page, cu, prefix)
    wide = torch.full((B, table.shape[1] + 9), 77777, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + table.shape[1]] = _i32(table)
    strided = wide[:, 4:4 + table.shape[1]]
    seqs, T = _seqs(lq, lk), sum(lq)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D)
    q = AR.bf16(g.normal(0, 1, (T, Hq, D)))
    see = PR.visible(seqs, table, page, n_pages, Hkv)
    at = _i32(np.r_[0, np.cumsum(lq)]), _i32(lk), strided
    out = P.paged_attention(_bf16(q), kt, vt, *at, max(lq), max(lk))
    _check(out, None, q, kp, vp, table, seqs, see, D ** -0.5)
    out = P.paged_attention(_bf16(q), kt, vt, *at, max(lq), max(lk), cu_group=_i32(cu), prefix_len=_i32(prefix), max_prefix=max(prefix))
    _check(out, None, q, kp, vp, table, seqs, see, D ** -0.5)
    bounds = torch.stack([kt.amin(1), kt.amax(1)], 1).contiguous()
    blocks = P.select_blocks(_bf16(q), bounds, *at, max(lq), max(lk), page, 3, first=0)
    want = PR.select(q, _np(bounds), table, seqs, page, 3, 0, 1)
    assert np.array_equal(blocks.cpu().numpy(), want)
    out = P.paged_attention(_bf16(q), kt, vt, *at, max(lq), max(lk), blocks=blocks)
    _check(out, None, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv, want), D ** -0.5)
    k, v = (AR.bf16(g.normal(0, 1, (T, Hkv, D))) for _ in range(2))
    own, n_own = _table(g, lk, page)  # every sequence writes to pages of its own
    kt, vt = (torch.zeros(n_own, page, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    P.paged_append(_bf16(k), _bf16(v), kt, vt, at[0], at[1], _i32(own), norm=False)
    got_k, got_v = _np(kt), _np(vt)
    count = 0
    for b, (q0, n, m) in enumerate(seqs):
        for i in range(n):
            p = i + m - n
            if p >= 0:
                at_ = own[b, p // page], p % page
                assert np.array_equal(got_k[at_], k[q0 + i]) and np.array_equal(got_v[at_], v[q0 + i])
                count += 1
    assert np.count_nonzero(np.any(got_k != 0, (2, 3))) == count


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    """Shapes drawn over everything that the operators take."""
    g = np.random.default_rng(1000 + seed)
    D, page, Hkv = int(g.choice([64, 128, 256])), int(g.choice([16, 32, 64, 128])), int(g.choice([1, 2, 3, 4]))
    Hq = Hkv * int(g.choice([1, 2, 3, 4, 5, 7, 8, 16, 33]))
    B = int(g.integers(1, 7))
    lq = [int(n) for n in (np.ones(B, int) if seed % 3 == 0 else g.integers(0, 4 + 70 * (seed % 2), B))]
    lk = [n + int(g.integers(0, 500)) if g.random() < 0.9 else int(g.integers(0, n + 1)) for n in lq]
    _say("random", seed, D, page, Hq, Hkv, lq, lk)
    cu = np.unique(np.r_[0, g.integers(0, B + 1, 2), B])
    prefix = [int(g.integers(-3, 1 + max(min(lk[b] for b in range(i, j)), 0) + 1)) for i, j in zip(cu, cu[1:])]
    table, n_pages = _group_table(g, lk, page, cu, prefix)
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D, layout=("pshd", "phsd", "both")[seed % 3])
    seqs = _seqs(lq, lk)
    q = AR.bf16(g.normal(0, 1.5, (sum(lq), Hq, D)))
    see = PR.visible(seqs, table, page, n_pages, Hkv)
    for kw in ({}, dict(cu_group=_i32(cu), prefix_len=_i32(prefix), max_prefix=max(max(prefix), 0))):
        out, lse = _run(_bf16(q), kt, vt, table, seqs, **kw)
        _check(out, lse, q, kp, vp, table, seqs, see, D ** -0.5)
    n = int(g.integers(1, 12))
    last = int(g.integers(1, n + 1))
    first = int(g.integers(0, n - last + 1))
    bounds = torch.stack([kt.amin(1), kt.amax(1)], 1).contiguous()
    blocks = P.select_blocks(_bf16(q), bounds, _i32(np.r_[0, np.cumsum(lq)]), _i32(lk), _i32(table), max(lq), max(lk), page, n,
                             first=first, last=last)
    want = PR.select(q, _np(bounds), table, seqs, page, n, first, last)
    assert np.array_equal(blocks.cpu().numpy(), want)
    out, lse = _run(_bf16(q), kt, vt, table, seqs, blocks=blocks)
    _check(out, lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv, want), D ** -0.5)


@pytest.mark.parametrize("lq,lk,prefix,Hq,Hkv,D,page", [([1, 1, 1], [20, 90, 64], 70, 4, 2, 64, 16), ([5, 30], [7, 200], 128, 2, 1, 128, 64)])
def test_the_first_sequence_of_a_group_is_the_shortest(lq, lk, prefix, Hq, Hkv, D, page):
    """Its row of the table names all of the prefix's pages, though it holds fewer keys itself."""
    _say("short first sequence", lq, lk, prefix, Hq, Hkv, D, page)
    g = np.random.default_rng(sum(lk))
    table, n_pages = _table(g, [max(lk)] + lk[1:], page)
    for b, n in enumerate(lk):
        full = prefix // page if n >= prefix else -(-n // page)
        table[b, :full] = table[0, :full]
    kp, vp, kt, vt = _pool(g, n_pages, page, Hkv, D)
    q = AR.bf16(g.normal(0, 2, (sum(lq), Hq, D)))
    seqs = _seqs(lq, lk)
    out, lse = _run(_bf16(q), kt, vt, table, seqs, cu_group=_i32([0, len(lk)]), prefix_len=_i32([prefix]), max_prefix=prefix,
                    max_kv=max(max(m - prefix, 0) for m in lk))
    _check(out, lse, q, kp, vp, table, seqs, PR.visible(seqs, table, page, n_pages, Hkv), D ** -0.5)
