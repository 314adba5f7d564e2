"""Python binding of the paged key/value cache (include/moe_paged.h).

Argument marshalling only, as in `attention`: a call checks its tensors,
allocates what the caller does not pass, and hands raw pointers and the current
HIP stream to the library; a refused call raises MoeError.

  paged_append     new keys (normed, rotated) and values into their pages, the queries beside them
  paged_attention  causal attention over the pages, with shared prefixes or listed blocks
  select_blocks    the blocks whose bounds promise a token's queries the largest products

A cache is two tensors [n_pages, page_size, kv_heads, head_dim] (parts of one, or in another
order of dimensions in memory); a row of the int32 page table names a sequence's pages in order.

`block.PagedAttentionBlock` runs them in a decoder block.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import attention as A
from . import binding as B
from .attention import _BF16, _F32, _HEADS, _I32, _NO_HEADS, _U8, _current, _flat, _heads, _refuse, _stream
from .binding import MoeError, _check  # noqa: F401

EXPORTED = ("moe_paged_append", "moe_paged_attention_workspace_size", "moe_paged_attention",
            "moe_select_blocks_workspace_size", "moe_select_blocks")


class moe_pages(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class moe_paged(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32)] + [
        (n, ctypes.c_int32) for n in ("head_dim", "q_heads", "kv_heads", "n_seqs", "q_rows", "n_pages", "page_size",
                                      "table_pages", "reserved")] + [
        ("table_stride", ctypes.c_int64), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p)]


class moe_append(ctypes.Structure):
    _fields_ = [("p", moe_paged), ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("n_positions", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("rot_offset", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("q", A.moe_heads), ("q_out", A.moe_heads), ("k", A.moe_heads), ("v", A.moe_heads),
                ("k_pages", moe_pages), ("v_pages", moe_pages), ("bounds", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("cos_sin", ctypes.c_void_p)]


class moe_paged_attn(ctypes.Structure):
    _fields_ = [("p", moe_paged)] + [
        (n, ctypes.c_int32) for n in ("max_q", "max_kv", "n_groups", "max_prefix", "n_blocks")] + [
        ("scale", ctypes.c_float), ("q", A.moe_heads), ("out", A.moe_heads), ("k", moe_pages), ("v", moe_pages),
        ("cu_group", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p), ("blocks", ctypes.c_void_p),
        ("lse", ctypes.c_void_p)]


class moe_select(ctypes.Structure):
    _fields_ = [("p", moe_paged)] + [
        (n, ctypes.c_int32) for n in ("max_q", "max_kv", "n_blocks", "first", "last", "reserved")] + [
        ("q", A.moe_heads), ("bounds", ctypes.c_void_p), ("blocks", ctypes.c_void_p)]


_typed = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so with the argument types of these entry points."""
    global _typed
    L = A.lib()
    if _typed is L:
        return L
    sz, vp = ctypes.c_size_t, ctypes.c_void_p  # a struct by reference, or its packed bytes
    sig = {
        "moe_paged_append": (ctypes.c_int, [vp, vp]),
        "moe_paged_attention_workspace_size": (sz, [vp]),
        "moe_paged_attention": (ctypes.c_int, [vp, vp, sz, vp]),
        "moe_select_blocks_workspace_size": (sz, [vp]),
        "moe_select_blocks": (ctypes.c_int, [vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _typed = L
    return L


# ---------------------------------------------------------------- argument checks
_PAGED = "I9iq3Q"
_APPEND = struct.Struct("=" + _PAGED + "if4i" + 4 * "Qqq" + 2 * "Qqqq" + "5Q")
_ATTN = struct.Struct("=" + _PAGED + "5if" + 2 * "Qqq" + 2 * "Qqqq" + "4Q")
_SELECT = struct.Struct("=" + _PAGED + "6i" + "Qqq" + "2Q")


def _pages(t, name, dev, shape=None):
    """Address and the three strides of a [n_pages, page_size, heads, head_dim] tensor."""
    if t.dtype not in _BF16 or t.get_device() != dev:
        _refuse(t, _BF16, name, dev)
    have = t.shape
    if len(have) != 4:
        raise ValueError(f"{name} must have four dimensions (pages, page_size, heads, head_dim)")
    if shape is not None and have != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(have)}")
    page, row, head, one = t.stride()
    if one != 1 and have[3] > 1:
        raise ValueError(f"{name} must have unit stride inside a head")
    # a dimension of one entry may carry any stride
    if have[2] <= 1:
        head = max(have[3], 8)
    if have[0] <= 1:
        page = max(page, 8) // 8 * 8
    return t.data_ptr(), page, row, head


def _vector(t, dtypes, name, dev, n):
    """The address of a contiguous vector of n elements (None: 0)."""
    if t is None:
        return 0
    if t.dtype not in dtypes or t.get_device() != dev:
        _refuse(t, dtypes, name, dev)
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape ({n},), got {tuple(t.shape)}")
    return t.data_ptr()


def _seqs(cu_q, kv_len, page_table, dev):
    """n_seqs, table_pages, the table's row stride and the three addresses."""
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [n_seqs + 1]")
    n = cu_q.numel() - 1
    if page_table.dtype not in _I32 or page_table.get_device() != dev:
        _refuse(page_table, _I32, "page_table", dev)
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [{n}, pages], got {tuple(page_table.shape)}")
    rows, width = page_table.shape
    if rows != n:
        raise ValueError(f"page_table must be [{n}, pages], got {(rows, width)}")
    row, one = page_table.stride()
    if one != 1 and width > 1:
        raise ValueError("page_table must have unit stride along its rows")
    return (n, width, row if n > 1 else width, _flat(cu_q, _I32, "cu_q", dev), _vector(kv_len, _I32, "kv_len", dev, n),
            page_table.data_ptr())


# ---------------------------------------------------------------- append
def paged_append(k, v, k_pages, v_pages, cu_q, kv_len, page_table, *, q=None, q_out=None, bounds=None, q_weight=None,
                 k_weight=None, norm=True, eps=1e-6, positions=None, cos_sin=None, rot_offset=0, interleaved=False):
    """moe_paged_append: k and v [T, Hkv, D] (any row and head strides that are multiples of 8) to the
    slots of k_pages and v_pages that cu_q [B + 1], kv_len [B] (the new rows included) and
    page_table [B, pages] name, k normed (norm=False: not) and rotated on the way; q [T, Hq, D]
    alike, to q_out (a new tensor unless given; q itself: in place) -> q_out, or None without q.

    bounds: bf16 [n_pages, 2, Hkv, D], the smallest and largest key elements of every page, kept for
    select_blocks, or None.  positions int32 [T]: the rotary positions, by default those in the
    cache; cos_sin float32 [n_positions, rot_dim] as in qk_norm_rope, or None: no rotation."""
    dev = _current(k, _BF16, "k")
    hk = _heads(k, "k", dev)
    T, Hk, D = shape = k.shape
    hv = _heads(v, "v", dev, shape)
    pk = _pages(k_pages, "k_pages", dev)
    pshape = k_pages.shape
    if pshape[2:] != shape[1:]:
        raise ValueError(f"k_pages must have heads of shape {tuple(shape[1:])}, got {tuple(pshape)}")
    pv = _pages(v_pages, "v_pages", dev, pshape)
    n, width, stride, cu, length, table = _seqs(cu_q, kv_len, page_table, dev)
    Hq, hq, hqo = 0, (0, 0, 0), (0, 0, 0)
    if q is not None:
        hq = _heads(q, "q", dev)
        qshape = q.shape
        Hq = qshape[1]
        if qshape[0] != T or qshape[2] != D:
            raise ValueError(f"q must have shape {(T, Hq, D)}, got {tuple(qshape)}")
        if q_out is None:
            q_out = torch.empty(qshape, dtype=torch.bfloat16, device=q.device)
        hqo = _heads(q_out, "q_out", dev, qshape)
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q")
    bp = cs = P = R = 0
    if bounds is not None:
        bp = _flat(bounds, _BF16, "bounds", dev, (pshape[0], 2, Hk, D))
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [n_positions, rot_dim]")
        P, R = cos_sin.shape
        cs = _flat(cos_sin, _F32, "cos_sin", dev)
    a = _APPEND.pack(B.MOE_ABI_VERSION, D, Hq, Hk, n, T, pshape[0], pshape[1], width, 0, stride, cu, length, table,
                     1 if norm else 0, eps, P, R, rot_offset, 1 if interleaved else 0, *hq, *hqo, *hk, *hv, *pk, *pv,
                     bp, _vector(q_weight, _F32, "q_weight", dev, D), _vector(k_weight, _F32, "k_weight", dev, D),
                     _vector(positions, _I32, "positions", dev, T), cs)
    st = lib().moe_paged_append(a, _stream(dev))
    if st:
        raise MoeError("moe_paged_append", st)
    return q_out


# ---------------------------------------------------------------- attention
def _attn_shape(q, k_pages, n_seqs, table_pages, max_q, max_kv, n_groups, max_prefix, n_blocks):
    return _ATTN.pack(B.MOE_ABI_VERSION, q.shape[2], q.shape[1], k_pages.shape[2], n_seqs, q.shape[0], k_pages.shape[0],
                      k_pages.shape[1], table_pages, 0, table_pages, 0, 0, 0, max_q, max_kv, n_groups, max_prefix,
                      n_blocks, 1.0, *(22 - 8) * (0,), 0, 0, 0, 0)


def paged_attention_workspace_size(q, k_pages, n_seqs: int, max_q: int, max_kv: int, *, n_groups=0, max_prefix=0,
                                   n_blocks=0) -> int:
    """Bytes paged_attention() needs for q and a cache of these shapes and these bounds."""
    pages = -(-max(max_kv, max_prefix) // k_pages.shape[1])
    return int(lib().moe_paged_attention_workspace_size(
        _attn_shape(q, k_pages, n_seqs, pages, max_q, max_kv, n_groups, max_prefix, n_blocks)))


def paged_attention_workspace(q, k_pages, n_seqs: int, max_q: int, max_kv: int, *, n_groups=0, max_prefix=0, n_blocks=0):
    need = paged_attention_workspace_size(q, k_pages, n_seqs, max_q, max_kv, n_groups=n_groups, max_prefix=max_prefix,
                                          n_blocks=n_blocks)
    return torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)


def paged_attention(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q: int, max_kv: int, *, cu_group=None,
                    prefix_len=None, max_prefix=0, blocks=None, scale=None, out=None, lse=None, ws=None):
    """moe_paged_attention: q [T, Hq, D] over the keys that kv_len [B] (the new rows included) and
    page_table [B, pages] name in k_pages and v_pages -> out [T, Hq, D], causal.

    max_q: the bound on a sequence's new rows; max_kv: on its keys, behind its shared prefix where there is one.
    cu_group int32 [groups + 1] with prefix_len int32 [groups] and their bound max_prefix: the sequences of a
    group, consecutive ones, hold the same first prefix_len keys in the same pages, all of them named by the
    first one's row of the table.
    blocks int32 [T, Hkv, n]: the blocks that each token and key head sees (select_blocks).
    scale: default D ** -0.5.  lse: float32 [T, Hq] to fill, or None.  Rows of out that belong
    to no sequence are left as they are (new: undefined)."""
    dev = _current(q, _BF16, "q")
    hq = _heads(q, "q", dev)
    T, Hq, D = shape = q.shape
    pk = _pages(k_pages, "k_pages", dev)
    pshape = k_pages.shape
    pv = _pages(v_pages, "v_pages", dev, pshape)
    if pshape[3] != D:
        raise ValueError(f"q and k_pages have different head sizes: {D}, {pshape[3]}")
    n, width, stride, cu, length, table = _seqs(cu_q, kv_len, page_table, dev)
    groups = n_blocks = gp = pp = bp = lp = 0
    if cu_group is not None and prefix_len is not None:
        groups = prefix_len.numel()
        gp = _vector(cu_group, _I32, "cu_group", dev, groups + 1)
        pp = _vector(prefix_len, _I32, "prefix_len", dev, groups)
    elif cu_group is not None or prefix_len is not None:
        raise ValueError("cu_group and prefix_len go together")
    if blocks is not None:
        if blocks.dim() != 3 or blocks.shape[2] < 1:
            raise ValueError(f"blocks must be [{T}, {pshape[2]}, n]")
        n_blocks = blocks.shape[2]
        bp = _flat(blocks, _I32, "blocks", dev, (T, pshape[2], n_blocks))
    if lse is not None:
        lp = _flat(lse, _F32, "lse", dev, (T, Hq))
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    ho = _heads(out, "out", dev, shape)
    a = _ATTN.pack(B.MOE_ABI_VERSION, D, Hq, pshape[2], n, T, pshape[0], pshape[1], width, 0, stride, cu, length, table,
                   max_q, max_kv, groups, max_prefix, n_blocks, D ** -0.5 if scale is None else scale, *hq, *ho, *pk, *pv,
                   gp, pp, bp, lp)
    L = lib()
    if ws is None:
        need = int(L.moe_paged_attention_workspace_size(a))
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = L.moe_paged_attention(a, _flat(ws, _U8, "ws", dev), ws.numel(), _stream(dev))
    if st:
        raise MoeError("moe_paged_attention", st)
    return out


# ---------------------------------------------------------------- selection
def select_blocks_workspace_size(q, bounds, n_seqs: int, max_q: int, max_kv: int, page_size: int) -> int:
    """Bytes select_blocks() needs for q and bounds of these shapes and these bounds on lengths."""
    a = _SELECT.pack(B.MOE_ABI_VERSION, q.shape[2], q.shape[1], bounds.shape[2], n_seqs, q.shape[0], bounds.shape[0],
                     page_size, -(-max_kv // page_size), 0, 0, 0, 0, 0, max_q, max_kv, 1, 0, 1, 0, 0, 0, 0, 0, 0)
    return int(lib().moe_select_blocks_workspace_size(a))


def select_blocks_workspace(q, bounds, n_seqs: int, max_q: int, max_kv: int, page_size: int):
    return torch.empty(max(select_blocks_workspace_size(q, bounds, n_seqs, max_q, max_kv, page_size), 256),
                       dtype=torch.uint8, device=q.device)


def select_blocks(q, bounds, cu_q, kv_len, page_table, max_q: int, max_kv: int, page_size: int, n_blocks: int, *,
                  first=1, last=1, blocks=None, ws=None):
    """moe_select_blocks: for every token of q [T, Hq, D] and key head the n_blocks blocks of highest score
    by bounds [n_pages, 2, Hkv, D] -> blocks int32 [T, Hkv, n_blocks], ascending, -1 where there are fewer;
    the first `first` blocks and the token's last `last` ones are always among them.

    max_q, max_kv: the bounds on a sequence's new rows and cached length.  Rows of blocks that belong to no
    sequence are left as they are (new: -1)."""
    dev = _current(q, _BF16, "q")
    hq = _heads(q, "q", dev)
    T, Hq, D = q.shape
    if bounds.dim() != 4:
        raise ValueError("bounds must be [n_pages, 2, heads, head_dim]")
    pages, _, Hk, _ = bounds.shape
    bp = _flat(bounds, _BF16, "bounds", dev, (pages, 2, Hk, D))
    n, width, stride, cu, length, table = _seqs(cu_q, kv_len, page_table, dev)
    if blocks is None:
        blocks = torch.full((T, Hk, n_blocks), -1, dtype=torch.int32, device=q.device)
    op = _flat(blocks, _I32, "blocks", dev, (T, Hk, n_blocks))
    a = _SELECT.pack(B.MOE_ABI_VERSION, D, Hq, Hk, n, T, pages, page_size, width, 0, stride, cu, length, table, max_q,
                     max_kv, n_blocks, first, last, 0, *hq, bp, op)
    L = lib()
    if ws is None:
        need = int(L.moe_select_blocks_workspace_size(a))
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = L.moe_select_blocks(a, _flat(ws, _U8, "ws", dev), ws.numel(), _stream(dev))
    if st:
        raise MoeError("moe_select_blocks", st)
    return blocks
