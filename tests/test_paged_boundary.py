"""Host-side tests of the paged C ABI: the library exports what the header declares,
every refusal returns its status without touching a GPU, the binding's packed
structs are the header's, and the float64 reference of the GPU tests agrees with
formulas written apart from it."""
import ctypes
import os
import re

import numpy as np
import pytest

from mxfp4_routed_expert_moe_amd import attention as A
from mxfp4_routed_expert_moe_amd import binding as B
from mxfp4_routed_expert_moe_amd import paged as P
from tests import attention_reference as AR
from tests import paged_reference as PR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_paged.h")
OK, EINVAL, EALIGN, ELAYOUT, ESHAPE, EWORKSPACE = 0, 1, 2, 3, 4, 5
FAKE = 0x7F0000000000


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src))
    assert names == set(P.EXPORTED)
    for n in names:
        assert hasattr(P.lib(), n), n


def test_struct_layout():
    """The structs' fields stand in the header's order, and the packed forms have their sizes."""
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name in ("moe_pages", "moe_paged", "moe_append", "moe_paged_attn", "moe_select"):
        body = re.search(r"typedef struct %s \{(.*?)\}" % name, src, re.S).group(1)
        fields = []
        for line in body.split(";"):
            words = line.strip().split(None, 2 if line.strip().startswith("const") else 1)
            if words:
                fields += [f.strip(" *") for f in words[-1].split(",")]
        assert fields == [f for f, _ in getattr(P, name)._fields_], name
    assert (P._APPEND.size, P._ATTN.size, P._SELECT.size) == tuple(
        ctypes.sizeof(s) for s in (P.moe_append, P.moe_paged_attn, P.moe_select))


def _paged(**kw):
    p = P.moe_paged(1, 128, 8, 2, 3, 40, 100, 64, 20, 0, 20, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _heads(base=FAKE, row=1024, head=128):
    return A.moe_heads(base, row, head)


def _pool(base=FAKE, page=16384, row=256, head=128):
    return P.moe_pages(base, page, row, head)


def _set(a, kw):
    for k, v in kw.items():
        if hasattr(a, k):
            setattr(a, k, v)
        else:
            setattr(a.p, k, v)
    return a


def _append(**kw):
    a = P.moe_append(_paged(), 1, 1e-6, 64, 128, 0, 0, _heads(), _heads(), _heads(), _heads(), _pool(), _pool(), FAKE, None,
                     None, None, FAKE)
    return P.lib().moe_paged_append(ctypes.byref(_set(a, kw)), None)


def _attn_desc(**kw):
    return _set(P.moe_paged_attn(_paged(), 1, 1280, 0, 0, 0, 0.1, _heads(), _heads(), _pool(), _pool(), None, None, None,
                                 None), kw)


def _attn(ws=FAKE, ws_bytes=1 << 40, **kw):
    return P.lib().moe_paged_attention(ctypes.byref(_attn_desc(**kw)), ctypes.c_void_p(ws), ws_bytes, None)


def _select_desc(**kw):
    return _set(P.moe_select(_paged(), 1, 1280, 8, 1, 1, 0, _heads(), FAKE, FAKE), kw)


def _select(ws=FAKE, ws_bytes=1 << 40, **kw):
    return P.lib().moe_select_blocks(ctypes.byref(_select_desc(**kw)), ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("call", [_append, _attn, _select])
def test_shared_checks(call):
    assert call(n_seqs=0) == OK
    assert call(q_rows=0, **({} if call is _append else dict(max_q=0))) == OK
    assert call(abi_version=2) == ELAYOUT
    for bad in (dict(n_seqs=-1), dict(q_rows=-1), dict(n_pages=-1), dict(table_pages=-1), dict(q_heads=-2), dict(cu_q=None),
                dict(kv_len=None), dict(page_table=None), dict(table_stride=19)):
        assert call(**bad) == EINVAL, bad
    a = _paged(reserved=1)
    if call is not _select:
        assert call(p=a) == EINVAL
    for bad in (dict(head_dim=96), dict(head_dim=512), dict(page_size=8), dict(page_size=48), dict(page_size=256),
                dict(kv_heads=0), dict(kv_heads=3), dict(q_heads=1026), dict(n_seqs=65537),
                dict(q_rows=B.MOE_MAX_TOKENS + 1), dict(table_pages=1 << 24, table_stride=1 << 24)):
        assert call(**bad) == ESHAPE, bad
    assert P.lib().moe_paged_append(None, None) == EINVAL
    assert P.lib().moe_paged_attention(None, None, 0, None) == EINVAL
    assert P.lib().moe_select_blocks(None, None, 0, None) == EINVAL


def test_append_checks():
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(norm=2), dict(interleaved=2), dict(n_positions=-1),
                dict(rot_dim=-16), dict(rot_offset=-8), dict(cos_sin=None), dict(norm=0, q_weight=FAKE),
                dict(norm=0, k_weight=FAKE)):
        assert _append(**bad) == EINVAL, bad
    for bad in (dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=64, rot_offset=72), dict(rot_dim=64, rot_offset=4),
                dict(q_rows=200000, q_heads=1024, kv_heads=1, head_dim=256)):
        assert _append(**bad) == ESHAPE, bad
    for name in ("q", "q_out", "k", "v"):
        assert _append(**{name: _heads(base=None)}) == EINVAL and _append(**{name: _heads(row=0)}) == EINVAL
        assert _append(**{name: _heads(base=FAKE + 8)}) == EALIGN and _append(**{name: _heads(head=100)}) == EALIGN
    for name in ("k_pages", "v_pages"):
        assert _append(**{name: _pool(base=None)}) == EINVAL and _append(**{name: _pool(page=0)}) == EINVAL
        assert _append(**{name: _pool(base=FAKE + 2)}) == EALIGN and _append(**{name: _pool(page=16388)}) == EALIGN
        assert _append(**{name: _pool(row=(1 << 22) + 8)}) == ESHAPE
    for name in ("bounds", "q_weight", "k_weight", "cos_sin"):
        assert _append(**{name: FAKE + 4}) == EALIGN, name


def test_attention_checks():
    assert _attn(max_q=0) == OK
    for bad in (dict(max_q=-1), dict(max_q=41), dict(max_kv=-1), dict(max_kv=1281), dict(max_prefix=-1),
                dict(max_prefix=1281), dict(n_groups=-1), dict(n_groups=4), dict(n_groups=1), dict(n_blocks=-1),
                dict(n_blocks=4), dict(n_blocks=4, n_groups=1, cu_group=FAKE, prefix_len=FAKE, blocks=FAKE),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(n_groups=1, cu_group=FAKE), dict(n_groups=1, prefix_len=FAKE)):
        assert _attn(**bad) == EINVAL, bad
    assert _attn(q_heads=0) == ESHAPE and _attn(n_blocks=1025, blocks=FAKE) == ESHAPE
    big = dict(table_pages=32769, table_stride=32769, max_kv=32769 * 16, page_size=16, n_blocks=4, blocks=FAKE)
    assert _attn(**big) == ESHAPE
    for name in ("q", "out"):
        assert _attn(**{name: _heads(base=None)}) == EINVAL and _attn(**{name: _heads(row=1028)}) == EALIGN
    for name in ("k", "v"):
        assert _attn(**{name: _pool(base=None)}) == EINVAL and _attn(**{name: _pool(head=4)}) == EALIGN
    need = P.lib().moe_paged_attention_workspace_size(ctypes.byref(_attn_desc()))
    assert need > 0 and _attn(ws_bytes=need - 1) == EWORKSPACE and _attn(ws=None) == EINVAL and _attn(ws=FAKE + 8) == EALIGN
    assert P.lib().moe_paged_attention_workspace_size(ctypes.byref(_attn_desc(max_q=0))) == 0
    assert P.lib().moe_paged_attention_workspace_size(ctypes.byref(_attn_desc(head_dim=96))) == 0


def test_select_checks():
    assert _select(max_q=0) == OK
    for bad in (dict(max_q=-1), dict(max_q=41), dict(max_kv=-1), dict(max_kv=1281), dict(n_blocks=0), dict(first=-1),
                dict(last=0), dict(first=4, last=5), dict(first=9), dict(bounds=None), dict(blocks=None), dict(reserved=1)):
        assert _select(**bad) == EINVAL, bad
    assert _select(n_blocks=1025) == ESHAPE and _select(q_heads=0) == ESHAPE
    assert _select(table_pages=32769, table_stride=32769, page_size=16, max_kv=32769 * 16) == ESHAPE
    assert _select(q=_heads(base=None)) == EINVAL and _select(q=_heads(row=4)) == EALIGN
    assert _select(q_rows=B.MOE_MAX_TOKENS, kv_heads=128, q_heads=128) == ESHAPE and _select(bounds=FAKE + 8) == EALIGN
    for long in (dict(table_pages=3000, table_stride=3000, max_kv=192000), dict(q_rows=256, max_q=256, n_seqs=1)):
        need = P.lib().moe_select_blocks_workspace_size(ctypes.byref(_select_desc(**long)))
        assert need > 0 and _select(ws_bytes=need - 1, **long) == EWORKSPACE
        assert _select(ws=FAKE + 8, **long) == EALIGN and _select(ws=None, **long) == EINVAL


def test_workspaces_hang_on_shapes_alone():
    """The workspace queries of the binding pack the same shapes as its calls."""
    import torch
    q = torch.empty(40, 8, 128, dtype=torch.bfloat16)
    pool = torch.empty(100, 64, 2, 128, dtype=torch.bfloat16, device="meta")
    need = P.lib().moe_paged_attention_workspace_size(ctypes.byref(_attn_desc(max_kv=1280)))
    assert P.paged_attention_workspace_size(q, pool, 3, 1, 1280) == need
    need = P.lib().moe_paged_attention_workspace_size(ctypes.byref(_attn_desc(max_kv=640, n_groups=2, max_prefix=1280)))
    assert P.paged_attention_workspace_size(q, pool, 3, 1, 640, n_groups=2, max_prefix=1280) == need
    bounds = torch.empty(100, 2, 2, 128, dtype=torch.bfloat16)
    need = P.lib().moe_select_blocks_workspace_size(ctypes.byref(_select_desc()))
    assert P.select_blocks_workspace_size(q, bounds, 3, 1, 1280, 64) == need


# ---------------------------------------------------------------- the references
def test_reference_attention_is_the_contiguous_one():
    g = np.random.default_rng(1)
    seqs, page = [(0, 3, 20), (3, 5, 5), (8, 1, 33)], 16
    table = g.permutation(12).reshape(3, 4)
    kp, vp = g.normal(0, 1, (2, 12, page, 2, 8))
    q = g.normal(0, 1, (9, 4, 8))
    see = PR.visible(seqs, table, page, 12, 2)
    out, lse, *_ = PR.attention(q, kp, vp, table, seqs, see, 0.3)
    k = kp[table].reshape(3 * 4 * page, 2, 8)
    v = vp[table].reshape(3 * 4 * page, 2, 8)
    ref, rl, *_ = AR.attention(q, k, v, [(a, n, b * 64, m) for b, (a, n, m) in enumerate(seqs)], 0.3, True)
    assert np.allclose(out, ref) and np.allclose(lse, rl)
    # every block listed, twice and out of order, is no list at all
    blocks = np.tile(np.r_[3, 0, 1, 2, 2, -1, 99], (9, 2, 1))
    assert np.allclose(PR.attention(q, kp, vp, table, seqs, PR.visible(seqs, table, page, 12, 2, blocks), 0.3)[0], ref)


def test_reference_scores_bound_every_product():
    """The score of a page is at least the sum over the heads of any of its keys' products."""
    g = np.random.default_rng(2)
    q, keys = g.normal(0, 1, (6, 16)), g.normal(0, 1, (30, 16))
    low, high = keys.min(0), keys.max(0)
    score = np.maximum(q, 0).sum(0) @ high + np.minimum(q, 0).sum(0) @ low
    assert np.isclose(score, np.maximum(q * low, q * high).sum())
    assert np.all(keys @ q.sum(0) <= score)


def test_reference_selection():
    """Against a choice by hand: first and last blocks, ties to the lower block, scores that are not finite first, pages that are
    none last."""
    q = np.ones((1, 2, 8))
    bounds = np.zeros((9, 2, 1, 8))
    for page, s in enumerate([1, 5, 5, 2, np.inf, 3, 5, 0, 9]):
        bounds[page, 1] = s
    table = np.array([[0, 1, 2, 3, 4, 5, 6, 99, 8]])
    pick = lambda n, first, last: PR.select(q, bounds, table, [(0, 1, 9 * 16)], 16, n, first, last)[0, 0].tolist()  # noqa: E731
    assert pick(3, 1, 1) == [0, 4, 8] and pick(4, 0, 1) == [1, 2, 4, 8] and pick(3, 0, 1) == [1, 4, 8]
    assert pick(8, 0, 1) == [0, 1, 2, 3, 4, 5, 6, 8] and pick(10, 0, 1) == [0, 1, 2, 3, 4, 5, 6, 7, 8, -1]


def test_attention_join_fits_a_launch():
    """Rows in shares whose join would need 2^32 threads are refused before anything runs, and need no workspace; as many
    rows of one share are not."""
    rows = dict(q_rows=B.MOE_MAX_TOKENS, head_dim=64, q_heads=1024, kv_heads=1024)
    many = dict(rows, n_groups=1, cu_group=FAKE, prefix_len=FAKE, max_prefix=1280)
    spread = dict(n_seqs=65536, q_rows=65536, max_q=32, head_dim=128, q_heads=64, kv_heads=64, table_pages=1024, table_stride=1024,
                  max_kv=65536, n_blocks=32, blocks=FAKE)
    for bad in (spread, many):
        assert _attn(**bad) == ESHAPE
        assert P.lib().moe_paged_attention_workspace_size(ctypes.byref(_attn_desc(**bad))) == 0
    fits = dict(many, q_heads=512, kv_heads=512)
    assert P.lib().moe_paged_attention_workspace_size(ctypes.byref(_attn_desc(**fits))) == 2 * B.MOE_MAX_TOKENS * 512 * (64 * 4 + 8)
