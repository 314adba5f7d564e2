"""Python binding of the attention half of a block (include/moe_attention.h).

Argument marshalling only, as in `binding`: tensor dtypes, devices and shapes
are checked here, outputs and workspaces are allocated as torch tensors unless
the caller passes its own, raw pointers and the current HIP stream go to the
library, and a non-zero status raises MoeError.  There is no fallback path.

  fp8_linear     y = x W^T, E4M3 weights with one scale per 128 x 128 block
  qk_norm_rope   RMS norm and rotary position of every query and key head
  attention      packed causal attention with grouped heads

`block.AttentionBlock` runs them together, in front of the MoE layer.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import binding as B
from .binding import MoeError, _check  # noqa: F401

MOE_SCALE_E8M0 = 0  # one byte per block, value 2^(e - 127)
MOE_SCALE_F32 = 1   # one float32 per block

EXPORTED = ("moe_fp8_linear_workspace_size", "moe_fp8_linear", "moe_qk_norm_rope", "moe_attn_init",
            "moe_attention_workspace_size", "moe_attention")


class moe_heads(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class moe_attn(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("head_dim", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("n_seqs", ctypes.c_int32), ("q_rows", ctypes.c_int32),
                ("kv_rows", ctypes.c_int32), ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q", moe_heads), ("k", moe_heads), ("v", moe_heads), ("out", moe_heads),
                ("cu_q", ctypes.c_void_p), ("kv_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("lse", ctypes.c_void_p)]


_typed = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so with the argument types of these entry points."""
    global _typed
    L = B.lib()
    if _typed is L:
        return L
    i32, i64, sz, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    heads = attn = vp  # a struct by reference, or its packed bytes
    sig = {
        "moe_fp8_linear_workspace_size": (sz, [i32, i32, i32]),
        "moe_fp8_linear": (ctypes.c_int, [vp, i64, i32, i32, vp, vp, i32, i32, vp, i64, vp, sz, vp]),
        "moe_qk_norm_rope": (ctypes.c_int, [heads, i32, heads, i32, i32, i32, vp, vp, f32, vp, vp, i32, i32, i32, i32,
                                            heads, heads, vp]),
        "moe_attn_init": (ctypes.c_int, [attn, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32]),
        "moe_attention_workspace_size": (sz, [attn]),
        "moe_attention": (ctypes.c_int, [attn, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _typed = L
    return L


# ---------------------------------------------------------------- argument checks
# A call of a few microseconds on the GPU should not wait for its checks: each
# looks at a tensor once, and the structs are packed in one go.
_BF16 = (torch.bfloat16, torch.int16)
_I32, _F32, _U8 = (torch.int32,), (torch.float32,), (torch.uint8,)
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_SCALE = (torch.uint8, torch.float8_e8m0fnu, torch.float32)
_HEADS = struct.Struct("=Qqq")
_ATTN = struct.Struct("=I9ifi" + 4 * "Qqq" + "4Q")
_NO_HEADS = _HEADS.pack(0, 0, 0)
_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice


def _refuse(t, dtypes, name, dev):
    """The error of a tensor that failed a check of its device or type."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _current(t, dtypes, name):
    """The device of the call: t's, which must be the current one."""
    dev = t.get_device()
    if dev < 0 or t.dtype not in dtypes:
        _refuse(t, dtypes, name, dev)
    if dev != _device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_device()}")
    return dev


def _flat(t, dtypes, name, dev, shape=None):
    """The address of a contiguous tensor."""
    if t.dtype not in dtypes or t.get_device() != dev:
        _refuse(t, dtypes, name, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _heads(t, name, dev, shape=None):
    """Address, row stride and head stride of a [rows, heads, head_dim] tensor."""
    if t.dtype not in _BF16 or t.get_device() != dev:
        _refuse(t, _BF16, name, dev)
    have = t.shape
    if len(have) != 3:
        raise ValueError(f"{name} must have three dimensions (rows, heads, head_dim)")
    if shape is not None and have != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(have)}")
    rows, heads, d = have
    row, head, one = t.stride()
    if one != 1 and d > 1:
        raise ValueError(f"{name} must have unit stride inside a head")
    # a dimension of one entry may carry any stride
    if heads <= 1:
        head = max(d, 8)
    if rows <= 1:
        row = max(heads, 1) * max(d, 8)
    return t.data_ptr(), row, head


def _rows(t, name, dev, shape):
    """Address and row stride of a [rows, columns] tensor."""
    if t.dtype not in _BF16 or t.get_device() != dev:
        _refuse(t, _BF16, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    row, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return t.data_ptr(), row if shape[0] > 1 else -(-shape[1] // 8) * 8


# ---------------------------------------------------------------- fp8 linear
def fp8_linear_workspace_size(T: int, N: int, K: int) -> int:
    return int(lib().moe_fp8_linear_workspace_size(T, N, K))


def fp8_linear_workspace(T: int, N: int, K: int, device="cuda"):
    """A workspace that fp8_linear takes for up to T tokens of this weight."""
    return torch.empty(max(fp8_linear_workspace_size(T, N, K), 256), dtype=torch.uint8, device=device)


def fp8_linear(x, w, w_scale, y=None, ws=None):
    """moe_fp8_linear: bf16 x [T, K], E4M3 w [N, K] with w_scale
    [ceil(N / 128), ceil(K / 128)] -> bf16 y [T, N].

    w is float8_e4m3fn or its bytes (uint8); w_scale is float8_e8m0fnu or its
    bytes (uint8), or float32.  Rows of x and y may be strided."""
    dev = _current(x, _BF16, "x")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must have two dimensions")
    T, K = shape = x.shape
    N, Kw = w.shape
    if K != Kw:
        raise ValueError(f"x [T, K] and w [N, K] do not fit: {tuple(shape)}, {(N, Kw)}")
    if y is None:
        y = torch.empty((T, N), dtype=torch.bfloat16, device=x.device)
    xp, xs = _rows(x, "x", dev, shape)
    yp, ys = _rows(y, "y", dev, (T, N))
    wp = _flat(w, _E4M3, "w", dev)
    sp = _flat(w_scale, _SCALE, "w_scale", dev, (-(-N // 128), -(-K // 128)))
    if ws is None:
        ws = fp8_linear_workspace(T, N, K, x.device)
    kind = MOE_SCALE_F32 if w_scale.dtype == torch.float32 else MOE_SCALE_E8M0
    st = lib().moe_fp8_linear(xp, xs, T, K, wp, sp, kind, N, yp, ys, _flat(ws, _U8, "ws", dev), ws.numel(),
                              _stream(dev))
    if st:
        raise MoeError("moe_fp8_linear", st)
    return y


# ---------------------------------------------------------------- norm and rotation
def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, *, rot_offset=0, interleaved=False, eps=1e-6,
                 q_out=None, k_out=None):
    """moe_qk_norm_rope on q [T, Hq, D] and k [T, Hkv, D] (k may be None)
    -> (q_out, k_out), new tensors unless given (q and k themselves: in place).

    q_weight, k_weight: float32 [D] or None; positions: int32 [T]; cos_sin:
    float32 [n_positions, rot_dim], the cosines of the rot_dim / 2 pairs, then
    their sines.  positions and cos_sin None: no rotation."""
    dev = _current(q, _BF16, "q")
    hq = _heads(q, "q", dev)
    T, Hq, D = shape = q.shape
    if q_out is None:
        q_out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    hq, hqo = _HEADS.pack(*hq), _HEADS.pack(*_heads(q_out, "q_out", dev, shape))
    hk = hko = _NO_HEADS
    Hk = 0
    if k is not None:
        hk = _heads(k, "k", dev)
        kshape = k.shape
        Hk = kshape[1]
        if kshape[0] != T or kshape[2] != D:
            raise ValueError(f"k must have shape {(T, Hk, D)}, got {tuple(kshape)}")
        if k_out is None:
            k_out = torch.empty(kshape, dtype=torch.bfloat16, device=q.device)
        hk, hko = _HEADS.pack(*hk), _HEADS.pack(*_heads(k_out, "k_out", dev, kshape))
    qw = None if q_weight is None else _flat(q_weight, _F32, "q_weight", dev, (D,))
    kw = None if k_weight is None else _flat(k_weight, _F32, "k_weight", dev, (D,))
    P = R = 0
    pos = cs = None
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [n_positions, rot_dim]")
        if positions is None:
            raise ValueError("cos_sin needs positions")
        P, R = cos_sin.shape
        cs = _flat(cos_sin, _F32, "cos_sin", dev)
        pos = _flat(positions, _I32, "positions", dev, (T,))
    st = lib().moe_qk_norm_rope(hq, Hq, hk, Hk, T, D, qw, kw, eps, pos, cs, P, R, rot_offset, 1 if interleaved else 0,
                                hqo, hko, _stream(dev))
    if st:
        raise MoeError("moe_qk_norm_rope", st)
    return q_out, k_out


# ---------------------------------------------------------------- attention
def attention_workspace_size(q, k, n_seqs: int, max_q: int, max_kv: int) -> int:
    """Bytes attention() needs for q and k of these shapes and bounds."""
    a = moe_attn()
    a.abi_version = B.MOE_ABI_VERSION
    a.q_rows, a.q_heads, a.head_dim = q.shape
    a.kv_rows, a.kv_heads = k.shape[0], k.shape[1]
    a.n_seqs, a.max_q, a.max_kv = n_seqs, max_q, max_kv
    return int(lib().moe_attention_workspace_size(ctypes.byref(a)))


def attention_workspace(q, k, n_seqs: int, max_q: int, max_kv: int):
    return torch.empty(max(attention_workspace_size(q, k, n_seqs, max_q, max_kv), 256), dtype=torch.uint8,
                       device=q.device)


def attention(q, k, v, cu_q, max_q: int, *, kv_start=None, kv_len=None, max_kv=None, scale=None, causal=True, out=None,
              lse=None, ws=None):
    """moe_attention: q [q_rows, Hq, D], k and v [kv_rows, Hkv, D], all bf16 with
    any row and head strides (multiples of 8) -> out [q_rows, Hq, D].

    cu_q int32 [B + 1]: the rows of q of each sequence; max_q (and max_kv): the
    caller's bounds on their lengths.  max_kv None: every key (a call over a cache, or
    over several prompts that is not causal, is split better where max_kv names the longest
    sequence; a workspace is for the bound that was given).  Without kv_start and kv_len the keys of
    a sequence are the rows that cu_q names; with them (int32 [B]) they are
    rows kv_start[b] .. kv_start[b] + kv_len[b] - 1 of a cache, the new rows included.
    scale: default D ** -0.5.  lse: float32 [q_rows, Hq] to fill, or None.  Rows
    of out that belong to no sequence are left as they are (new: undefined)."""
    dev = _current(q, _BF16, "q")
    hq = _heads(q, "q", dev)
    hk = _heads(k, "k", dev)
    qshape, kshape = q.shape, k.shape
    hv = _heads(v, "v", dev, kshape)
    Tq, Hq, D = qshape
    Tk, Hk, Dk = kshape
    if Dk != D:
        raise ValueError(f"q and k have different head sizes: {D}, {Dk}")
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [n_seqs + 1]")
    n_seqs = cu_q.numel() - 1
    cu = _flat(cu_q, _I32, "cu_q", dev)
    start = length = lp = 0
    if kv_start is not None and kv_len is not None:
        start = _flat(kv_start, _I32, "kv_start", dev, (n_seqs,))
        length = _flat(kv_len, _I32, "kv_len", dev, (n_seqs,))
    elif kv_start is not None or kv_len is not None:
        raise ValueError("kv_start and kv_len go together")
    if lse is not None:
        lp = _flat(lse, _F32, "lse", dev, (Tq, Hq))
    if out is None:
        out = torch.empty(qshape, dtype=torch.bfloat16, device=q.device)
    ho = _heads(out, "out", dev, qshape)
    if max_kv is None:  # no row below max_q of a causal prompt sees a key from max_q on
        max_kv = min(max_q, Tk) if causal and not start else Tk
    a = _ATTN.pack(B.MOE_ABI_VERSION, D, Hq, Hk, n_seqs, Tq, Tk, max_q, max_kv, 1 if causal else 0,
                   D ** -0.5 if scale is None else scale, 0, *hq, *hk, *hv, *ho, cu, start, length, lp)
    L = lib()
    if ws is None:
        need = int(L.moe_attention_workspace_size(a))
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = L.moe_attention(a, _flat(ws, _U8, "ws", dev), ws.numel(), _stream(dev))
    if st:
        raise MoeError("moe_attention", st)
    return out
