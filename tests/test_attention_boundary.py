"""Host-side tests of the attention-side C ABI: the library exports what the
header declares, every refusal returns its status without touching a GPU, and
the float64 reference of the GPU tests agrees with formulas written apart from it."""
import ctypes
import os
import re

import numpy as np
import pytest

from mxfp4_routed_expert_moe_amd import attention as A
from mxfp4_routed_expert_moe_amd import binding as B
from tests import attention_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_attention.h")
OK, EINVAL, EALIGN, ELAYOUT, ESHAPE, EWORKSPACE = 0, 1, 2, 3, 4, 5
FAKE = 0x7F0000000000


def _v(p):
    return None if p is None else ctypes.c_void_p(p)


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src))
    assert names == set(A.EXPORTED)
    for n in names:
        assert hasattr(A.lib(), n), n


def test_struct_layout():
    # three 8-byte fields; twelve 4-byte ones, four tensors, four pointers
    assert ctypes.sizeof(A.moe_heads) == 24 and ctypes.sizeof(A.moe_attn) == 48 + 4 * 24 + 4 * 8


def _linear(T=4, N=256, K=512, x=FAKE, xs=None, w=FAKE, s=FAKE, kind=0, y=FAKE, ys=None, ws=FAKE, ws_bytes=1 << 40):
    return A.lib().moe_fp8_linear(_v(x), K if xs is None else xs, T, K, _v(w), _v(s), kind, N, _v(y),
                                  N if ys is None else ys, _v(ws), ws_bytes, None)


def test_fp8_linear_checks():
    assert _linear(T=0) == OK
    assert _linear(T=-1) == EINVAL
    assert _linear(T=B.MOE_MAX_TOKENS + 1) == ESHAPE
    for bad in (dict(N=0), dict(N=-1), dict(N=B.MOE_MAX_DIM + 1), dict(K=0), dict(K=-16), dict(K=24),
                dict(K=B.MOE_MAX_DIM + 16)):
        assert _linear(**bad) == ESHAPE, bad
    assert _linear(kind=2) == EINVAL and _linear(kind=-1) == EINVAL
    for name in ("x", "w", "s", "y", "ws"):
        assert _linear(**{name: None}) == EINVAL, name
    assert _linear(xs=504) == EINVAL and _linear(ys=255) == EINVAL
    assert _linear(xs=516) == EALIGN
    assert _linear(x=FAKE + 8) == EALIGN and _linear(w=FAKE + 8) == EALIGN and _linear(y=FAKE + 1) == EALIGN
    assert _linear(ws=FAKE + 128) == EALIGN and _linear(s=FAKE + 2, kind=1) == EALIGN
    need = A.fp8_linear_workspace_size(4, 256, 512)
    assert need >= 4 * 512 + 4 * 4 * 4 and _linear(ws_bytes=need - 1) == EWORKSPACE
    assert A.fp8_linear_workspace_size(0, 256, 512) == 0 and A.fp8_linear_workspace_size(4, 256, 500) == 0


def _heads(base=FAKE, row=1024, head=128):
    return A.moe_heads(base, row, head)


def _rope(T=4, Hq=8, Hk=2, D=128, q=None, k=None, qw=None, kw=None, eps=1e-6, pos=FAKE, cs=FAKE, P=64, R=128, off=0,
          inter=0, qo=None, ko=None):
    mk = lambda h: None if h is False else ctypes.byref(_heads() if h is None else h)  # noqa: E731
    return A.lib().moe_qk_norm_rope(mk(q), Hq, mk(k), Hk, T, D, _v(qw), _v(kw), eps, _v(pos), _v(cs), P, R, off, inter,
                                    mk(qo), mk(ko), None)


def test_qk_norm_rope_checks():
    assert _rope(T=0) == OK
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hk=-1), dict(R=-16), dict(off=-8), dict(P=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(inter=2)):
        assert _rope(**bad) == EINVAL, bad
    for bad in (dict(T=B.MOE_MAX_TOKENS + 1), dict(Hq=0), dict(Hq=1025), dict(Hq=1000, Hk=25), dict(D=4, R=0),
                dict(D=520), dict(D=100, R=0), dict(R=24), dict(R=144), dict(R=64, off=72), dict(R=64, off=4)):
        assert _rope(**bad) == ESHAPE, bad
    for name in ("q", "k", "qo", "ko"):
        assert _rope(**{name: False}) == EINVAL
        assert _rope(**{name: _heads(base=None)}) == EINVAL
        assert _rope(**{name: _heads(base=FAKE + 8)}) == EALIGN
        assert _rope(**{name: _heads(row=1028)}) == EALIGN and _rope(**{name: _heads(head=100)}) == EALIGN
        assert _rope(**{name: _heads(row=0)}) == EINVAL and _rope(**{name: _heads(head=-128)}) == EINVAL
    assert _rope(pos=None) == EINVAL and _rope(cs=None) == EINVAL
    assert _rope(cs=FAKE + 4) == EALIGN and _rope(qw=FAKE + 4) == EALIGN and _rope(kw=FAKE + 8) == EALIGN


def _desc(**kw):
    a = A.moe_attn()
    st = A.lib().moe_attn_init(ctypes.byref(a), _v(FAKE), _v(FAKE), _v(FAKE), _v(FAKE), _v(FAKE), 3, 100, 200, 8, 2, 128)
    assert st == OK
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _attn(ws=FAKE, ws_bytes=1 << 40, **kw):
    return A.lib().moe_attention(ctypes.byref(_desc(**kw)), _v(ws), ws_bytes, None)


def test_attn_init():
    a = _desc()
    assert (a.abi_version, a.head_dim, a.q_heads, a.kv_heads, a.n_seqs, a.q_rows, a.kv_rows, a.max_q, a.max_kv) == (
        1, 128, 8, 2, 3, 100, 200, 100, 200)
    assert a.causal == 1 and a.reserved == 0 and abs(a.scale - 128 ** -0.5) < 1e-7
    assert (a.q.row_stride, a.k.row_stride, a.v.row_stride, a.out.row_stride) == (1024, 256, 256, 1024)
    assert a.q.head_stride == a.k.head_stride == 128 and a.kv_start is None and a.lse is None
    L = A.lib()
    for i in range(6):
        args = [ctypes.byref(a)] + [_v(FAKE)] * 5
        args[i] = None
        assert L.moe_attn_init(*args, 3, 100, 200, 8, 2, 128) == EINVAL
    assert L.moe_attn_init(ctypes.byref(a), *[_v(FAKE)] * 5, 3, 100, 200, 8, 2, 0) == OK
    assert L.moe_attention(ctypes.byref(a), None, 0, None) == ESHAPE


def test_attention_checks():
    assert A.lib().moe_attention(None, None, 0, None) == EINVAL
    assert _attn(n_seqs=0) == OK and _attn(max_q=0) == OK and _attn(q_rows=0, max_q=0) == OK
    assert _attn(abi_version=2) == ELAYOUT
    for bad in (dict(n_seqs=-1), dict(q_rows=-1), dict(kv_rows=-1), dict(max_q=-1), dict(max_kv=-1), dict(max_q=101),
                dict(max_kv=201), dict(causal=2), dict(reserved=1), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(kv_start=FAKE), dict(kv_len=FAKE),
                dict(cu_q=None)):
        assert _attn(**bad) == EINVAL, bad
    for bad in (dict(head_dim=96), dict(head_dim=512), dict(kv_heads=0), dict(kv_heads=3), dict(q_heads=0),
                dict(q_heads=1026), dict(n_seqs=65537), dict(q_rows=B.MOE_MAX_TOKENS + 1)):
        assert _attn(**bad) == ESHAPE, bad
    for name in ("q", "k", "v", "out"):
        assert _attn(**{name: _heads(base=None)}) == EINVAL
        assert _attn(**{name: _heads(row=0)}) == EINVAL
        assert _attn(**{name: _heads(base=FAKE + 8)}) == EALIGN
        assert _attn(**{name: _heads(row=1028)}) == EALIGN
    assert _attn(k=_heads(row=(1 << 23) + 8)) == ESHAPE
    long = dict(kv_rows=8192, max_kv=8192)
    need = A.lib().moe_attention_workspace_size(ctypes.byref(_desc(**long)))
    assert need > 0
    assert _attn(ws=None, **long) == EINVAL and _attn(ws=FAKE + 64, **long) == EALIGN
    assert _attn(ws_bytes=need - 1, **long) == EWORKSPACE


def test_attention_workspace():
    size = lambda **kw: A.lib().moe_attention_workspace_size(ctypes.byref(_desc(**kw)))  # noqa: E731
    assert size(head_dim=96) == 0 and size(n_seqs=0) == 0
    # a long prompt fills the card by itself: one pass, no workspace
    assert size(q_rows=16384, max_q=16384, kv_rows=16384, max_kv=16384, q_heads=32, kv_heads=8, n_seqs=1) == 0
    # a single token over a long cache is split, and the shares of a row are D + 2 floats each
    one = dict(q_rows=1, max_q=1, kv_rows=1 << 17, max_kv=1 << 17, n_seqs=1)
    assert size(**one) >= 8 * 130 * 4 * 8


@pytest.mark.parametrize("name", ["fp8_linear", "qk_norm_rope", "attention"])
def test_binding_refuses_host_tensors(name):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        if name == "fp8_linear":
            A.fp8_linear(x[:, 0], torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.uint8))
        elif name == "qk_norm_rope":
            A.qk_norm_rope(x, x, None, None, None, None)
        else:
            A.attention(x, x, x, torch.zeros(2, dtype=torch.int32), 4)


# ---------------------------------------------------------------- the reference itself
def test_reference_e4m3():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, R.E4M3, equal_nan=True)
    g = np.random.default_rng(3)
    x = np.concatenate([g.uniform(-448, 448, 4000), g.normal(0, 0.02, 4000), [0, 0.5 * 2 ** -9, 1.5 * 2 ** -9, 17, 19, 464]])
    x = np.float32(x)
    assert np.array_equal(torch.from_numpy(x[:-1]).to(torch.float8_e4m3fn).double().numpy(), R.round_e4m3(x[:-1]))


def test_reference_quantiser():
    x = R.bf16(np.random.default_rng(4).normal(0, 1, (3, 300)))
    x[1] = 0
    for kind in ("e8m0", "float32"):
        q, s = R.quantise(x, kind)
        assert s.shape == (3, 3) and np.all(np.abs(q) <= 448)
        back = q * np.repeat(s, 128, 1)[:, :300]
        assert np.all(np.abs(back - x) <= np.abs(x) * 2.0 ** -4 + np.repeat(s, 128, 1)[:, :300] * 2.0 ** -10)
        if kind == "e8m0":
            m, _ = np.frexp(s)
            assert np.all(m == 0.5)


def test_reference_attention_is_softmax():
    g = np.random.default_rng(5)
    q, k, v = g.normal(size=(5, 4, 8)), g.normal(size=(7, 2, 8)), g.normal(size=(7, 2, 8))
    out, lse, _, _ = R.attention(q, k, v, [(0, 5, 0, 7)], 0.3, True)
    for h in range(4):
        z = q[:, h] @ k[:, h // 2].T * 0.3
        z[np.triu(np.ones((5, 7), bool), 3)] = -np.inf
        p = np.exp(z)
        assert np.allclose(out[:, h], p @ v[:, h // 2] / p.sum(1, keepdims=True), rtol=1e-12)
        assert np.allclose(lse[:, h], np.log(p.sum(1)), rtol=1e-12)


def test_reference_rope_keeps_norms_and_relative_angles():
    g = np.random.default_rng(6)
    x = g.normal(size=(2, 1, 32))
    ang = np.arange(40)[:, None] * 0.3 ** np.arange(16)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        y, _ = R.norm_rope(x, None, [5, 9], cs, 0, inter, 0.0)
        z, _ = R.norm_rope(x, None, [25, 29], cs, 0, inter, 0.0)
        assert np.allclose((y * y).sum(-1), 32)
        assert np.isclose(y[0, 0] @ y[1, 0], z[0, 0] @ z[1, 0])


def test_qk_norm_rope_refuses_more_heads_than_a_grid_has():
    assert B.MOE_MAX_TOKENS * 1024 == 1 << 28
    assert _rope(T=B.MOE_MAX_TOKENS, Hq=1000, Hk=24) == ESHAPE


def test_fp8_linear_workspace_grows_with_every_size():
    """A workspace for up to T tokens serves fewer of them, as for N and K."""
    sizes = (1, 16, 17, 64, 65, 130, 500, 700, 5000, 20000)
    f = A.fp8_linear_workspace_size
    for n, k in ((16, 16), (1000, 2064), (4096, 4096), (16384, 16384)):
        got = [f(t, n, k) for t in sizes]
        assert got == sorted(got)
        for t in sizes:
            assert f(t, n, k) <= f(t, n + 1000 if n < 15000 else n, k) and f(t, n, k) <= f(t, n, min(k + 1600, 16384))


def test_attention_scale_whose_base_two_form_overflows():
    assert _attn(scale=2.0 ** 127 * 1.5) == EINVAL


def test_qk_norm_rope_grid_of_wide_heads():
    """A group of 64 lanes takes four heads wider than 256: 2^18 tokens of 1021 to 1023 heads are 2^32 threads."""
    for D in (264, 512):
        for Hk in (21, 22, 23):
            assert _rope(T=B.MOE_MAX_TOKENS, Hq=1000, Hk=Hk, D=D) == ESHAPE
