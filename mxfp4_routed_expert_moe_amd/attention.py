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

from . import binding as B
from .binding import MoeError, _check, _dev, _ptr, _stream, _torch  # noqa: F401

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
    heads, attn = ctypes.POINTER(moe_heads), ctypes.POINTER(moe_attn)
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
def _on(t, dtypes, name, device=None):
    """A device tensor of one of the dtypes, on `device` where one is given."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in (dtypes if isinstance(dtypes, tuple) else (dtypes,)):
        raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _current(t, name):
    """The calls go to the current device's stream: the tensors must be there."""
    cur = _torch().cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{cur}")
    return t.device


def _flat(t, dtypes, name, device, shape=None):
    _on(t, dtypes, name, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _bf16():
    torch = _torch()
    return (torch.bfloat16, torch.int16)


def _heads(t, name, device, shape=None):
    """A [rows, heads, head_dim] tensor as a moe_heads."""
    _on(t, _bf16(), name, device)
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions (rows, heads, head_dim)")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride inside a head")
    # a dimension of one entry may carry any stride
    d = max(t.shape[2], 8)
    head = t.stride(1) if t.shape[1] > 1 else d
    row = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1) * d
    return moe_heads(t.data_ptr(), row, head)


def _workspace(ws, need, device):
    torch = _torch()
    if ws is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return _flat(ws, torch.uint8, "ws", device)


# ---------------------------------------------------------------- fp8 linear
def fp8_linear_workspace_size(T: int, N: int, K: int) -> int:
    return int(lib().moe_fp8_linear_workspace_size(T, N, K))


def fp8_linear_workspace(T: int, N: int, K: int, device="cuda"):
    """A workspace that fp8_linear takes for up to T tokens of this weight."""
    torch = _torch()
    return torch.empty(max(fp8_linear_workspace_size(T, N, K), 256), dtype=torch.uint8, device=device)


def fp8_linear(x, w, w_scale, y=None, ws=None):
    """moe_fp8_linear: bf16 x [T, K], E4M3 w [N, K] with w_scale
    [ceil(N / 128), ceil(K / 128)] -> bf16 y [T, N].

    w is float8_e4m3fn or its bytes (uint8); w_scale is float8_e8m0fnu or its
    bytes (uint8), or float32.  Rows of x and y may be strided."""
    torch = _torch()
    _on(x, _bf16(), "x")
    dev = _current(x, "x")
    if x.dim() != 2 or w.dim() != 2 or w.shape[1] != x.shape[1]:
        raise ValueError(f"x [T, K] and w [N, K] do not fit: {tuple(x.shape)}, {tuple(w.shape)}")
    T, K = x.shape
    N = w.shape[0]
    _flat(w, (torch.uint8, torch.float8_e4m3fn), "w", dev)
    _flat(w_scale, (torch.uint8, torch.float8_e8m0fnu, torch.float32), "w_scale", dev, (-(-N // 128), -(-K // 128)))
    if y is None:
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    _on(y, _bf16(), "y", dev)
    if tuple(y.shape) != (T, N):
        raise ValueError(f"y must have shape {(T, N)}, got {tuple(y.shape)}")
    for t, name in ((x, "x"), (y, "y")):
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit stride along its rows")
    ws = _workspace(ws, fp8_linear_workspace_size(T, N, K), dev)
    kind = MOE_SCALE_F32 if w_scale.dtype == torch.float32 else MOE_SCALE_E8M0
    xs, ys = (x.stride(0), y.stride(0)) if T > 1 else (-(-K // 8) * 8, N)
    _check("moe_fp8_linear", lib().moe_fp8_linear(x.data_ptr(), xs, T, K, w.data_ptr(), w_scale.data_ptr(), kind, N,
                                                  y.data_ptr(), ys, ws.data_ptr(), ws.numel(), _stream()))
    return y


# ---------------------------------------------------------------- norm and rotation
def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, *, rot_offset=0, interleaved=False, eps=1e-6,
                 q_out=None, k_out=None):
    """moe_qk_norm_rope on q [T, Hq, D] and k [T, Hkv, D] (k may be None)
    -> (q_out, k_out), new tensors unless given (q and k themselves: in place).

    q_weight, k_weight: float32 [D] or None; positions: int32 [T]; cos_sin:
    float32 [n_positions, rot_dim], the cosines of the rot_dim / 2 pairs, then
    their sines.  positions and cos_sin None: no rotation."""
    torch = _torch()
    _on(q, _bf16(), "q")
    dev = _current(q, "q")
    hq = _heads(q, "q", dev)
    T, Hq, D = q.shape
    q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev) if q_out is None else q_out
    hqo = _heads(q_out, "q_out", dev, (T, Hq, D))
    hk, hko, Hk = moe_heads(), moe_heads(), 0
    if k is not None:
        Hk = k.shape[1]
        hk = _heads(k, "k", dev, (T, Hk, D))
        k_out = torch.empty((T, Hk, D), dtype=torch.bfloat16, device=dev) if k_out is None else k_out
        hko = _heads(k_out, "k_out", dev, (T, Hk, D))
    for wt, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if wt is not None:
            _flat(wt, torch.float32, name, dev, (D,))
    P = R = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [n_positions, rot_dim]")
        P, R = _flat(cos_sin, torch.float32, "cos_sin", dev).shape
        if positions is None:
            raise ValueError("cos_sin needs positions")
        _flat(positions, torch.int32, "positions", dev, (T,))
    _check("moe_qk_norm_rope", lib().moe_qk_norm_rope(
        ctypes.byref(hq), Hq, ctypes.byref(hk), Hk, T, D, _ptr(q_weight), _ptr(k_weight), eps, _ptr(positions),
        _ptr(cos_sin), P, R, rot_offset, int(bool(interleaved)), ctypes.byref(hqo), ctypes.byref(hko), _stream()))
    return q_out, k_out


# ---------------------------------------------------------------- attention
def _attn(q_shape, kv_shape, n_seqs, max_q, max_kv):
    """A descriptor with the shape fields set."""
    a = moe_attn()
    a.abi_version = B.MOE_ABI_VERSION
    a.q_rows, a.q_heads, a.head_dim = q_shape
    a.kv_rows, a.kv_heads = kv_shape[0], kv_shape[1]
    a.n_seqs, a.max_q, a.max_kv = n_seqs, max_q, max_kv
    return a


def attention_workspace_size(q, k, n_seqs: int, max_q: int, max_kv: int) -> int:
    """Bytes attention() needs for q and k of these shapes and bounds."""
    return int(lib().moe_attention_workspace_size(ctypes.byref(_attn(q.shape, k.shape, n_seqs, max_q, max_kv))))


def attention_workspace(q, k, n_seqs: int, max_q: int, max_kv: int):
    torch = _torch()
    return torch.empty(max(attention_workspace_size(q, k, n_seqs, max_q, max_kv), 256), dtype=torch.uint8,
                       device=q.device)


def attention(q, k, v, cu_q, max_q: int, *, kv_start=None, kv_len=None, max_kv=None, scale=None, causal=True, out=None,
              lse=None, ws=None):
    """moe_attention: q [q_rows, Hq, D], k and v [kv_rows, Hkv, D], all bf16 with
    any row and head strides (multiples of 8) -> out [q_rows, Hq, D].

    cu_q int32 [B + 1]: the rows of q of each sequence; max_q (and max_kv): the
    caller's bounds on their lengths.  Without kv_start and kv_len the keys of
    a sequence are the rows that cu_q names; with them (int32 [B]) they are
    rows kv_start[b] .. kv_start[b] + kv_len[b] - 1 of a cache, the new rows included.
    scale: default D ** -0.5.  lse: float32 [q_rows, Hq] to fill, or None.  Rows
    of out that belong to no sequence are left as they are (new: undefined)."""
    torch = _torch()
    _on(q, _bf16(), "q")
    dev = _current(q, "q")
    hq = _heads(q, "q", dev)
    hk = _heads(k, "k", dev)
    hv = _heads(v, "v", dev, k.shape)
    if k.shape[2] != q.shape[2]:
        raise ValueError(f"q and k have different head sizes: {q.shape[2]}, {k.shape[2]}")
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [n_seqs + 1]")
    n_seqs = cu_q.numel() - 1
    _flat(cu_q, torch.int32, "cu_q", dev)
    if (kv_start is None) != (kv_len is None):
        raise ValueError("kv_start and kv_len go together")
    if kv_start is not None:
        _flat(kv_start, torch.int32, "kv_start", dev, (n_seqs,))
        _flat(kv_len, torch.int32, "kv_len", dev, (n_seqs,))
    if lse is not None:
        _flat(lse, torch.float32, "lse", dev, q.shape[:2])
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev) if out is None else out
    if max_kv is None:
        max_kv = min(max_q, k.shape[0]) if kv_start is None else k.shape[0]
    a = _attn(q.shape, k.shape, n_seqs, max_q, max_kv)
    a.causal = int(bool(causal))
    a.scale = q.shape[2] ** -0.5 if scale is None else scale
    a.q, a.k, a.v, a.out = hq, hk, hv, _heads(out, "out", dev, q.shape)
    a.cu_q = cu_q.data_ptr()
    if kv_start is not None:
        a.kv_start, a.kv_len = kv_start.data_ptr(), kv_len.data_ptr()
    if lse is not None:
        a.lse = lse.data_ptr()
    L = lib()
    if ws is None:
        need = int(L.moe_attention_workspace_size(ctypes.byref(a)))
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        _flat(ws, torch.uint8, "ws", dev)
    _check("moe_attention", L.moe_attention(ctypes.byref(a), _ptr(ws), 0 if ws is None else ws.numel(), _stream()))
    return out
