"""Rotary positions, the paged key/value cache and its attention: the binding
of the entry points on head rows (include/rmsnorm.h).

Argument checks and marshalling only. A call's structure is packed with one
``struct`` call, since for a few tokens the host's share is most of the time.
"""
from __future__ import annotations

import contextlib
import math
import struct

import torch

from ._binding import RMSNORM_WEIGHT_F32, TORCH_DTYPE, _raise, _stream_handle, lib

# rope_rows_t: in, out, in_token, in_head, out_token, out_head
# rope_angles_t: positions, inv_freq, axis_stride, position_bytes, n_axes, rotary_dim, pairing
# paged_cache_t: k, v, pages, k_page, k_slot, k_head, v_page, v_slot, v_head, page_size, heads
_ROWS, _ANGLES, _CACHE = "QQqqqq", "QQqiiii", "QQqqqqqqqii"
_ROPE = struct.Struct("<" + 2 * _ROWS + _ANGLES + "qiiii")
_APPEND = struct.Struct("<" + 3 * _ROWS + _ANGLES + _CACHE + "QQQqffiiii")
_ATTN = struct.Struct("<QQQqqqq" + _CACHE + "QQQqqQQfiiiiiiii4x")

_PAIRING = {"half": 0, "adjacent": 1}
_NO_ROWS = (0, 0, 0, 0, 0, 0)
_NO_ANGLES = (0, 0, 0, 0, 0, 0, 0)


def rope_axes(sections, interleaved: bool = False) -> bytes:
    """The axis of each rotary frequency, one byte each, as the ``axes``
    argument takes it: sections[a] frequencies turn by axis a's position.
    Blocks of neighbouring frequencies, or (interleaved) dealt one by one to
    the axes that have frequencies left."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= 4 or min(left) < 0:
        raise ValueError("sections must give 1 to 4 axes' frequency counts")
    if not interleaved:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    out = bytearray()
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return bytes(out)


def _heads(t, name: str, like=None):
    """Strides of a [T, heads, head_dim] CUDA tensor with head_dim contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [tokens, heads, head_dim]")
    st = t.stride()
    if st[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must match dtype/device of the other head rows")
    return st


def _code(t) -> int:
    code = TORCH_DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}; use torch.float32, torch.bfloat16 or torch.float16")
    return code


def _rows(x, out, name: str, like):
    """rope_rows_t's fields for rows x written to `out` (made when None)."""
    st = _heads(x, name, like)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    so = _heads(out, name + "_out", x)
    if out.shape != x.shape:
        raise ValueError(f"{name}_out must have {name}'s shape {tuple(x.shape)}, has {tuple(out.shape)}")
    return out, (x.data_ptr(), out.data_ptr(), st[0], st[1], so[0], so[1])


def _small(t, name: str, dtypes, device, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on the input's device")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, is {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_INTS = (torch.int32, torch.int64)
_F32 = (torch.float32,)


def _angles(positions, inv_freq, axes, pairing, tokens: int, head_dim: int, device):
    """rope_angles_t's fields."""
    _small(positions, "positions", _INTS, device, contiguous=False)
    _small(inv_freq, "inv_freq", _F32, device)
    n = positions.shape[0] if positions.dim() == 2 else 1
    if positions.dim() not in (1, 2) or positions.shape[-1] != tokens or not 1 <= n <= 4:
        raise ValueError(f"positions must be [{tokens}] or [axes, {tokens}] with 1 to 4 axes, "
                         f"has {tuple(positions.shape)}")
    if tokens > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must be contiguous over the tokens")
    half = inv_freq.numel()
    if inv_freq.dim() != 1 or not 1 <= half <= head_dim // 2:
        raise ValueError(f"inv_freq must have 1 to {head_dim // 2} frequencies for head_dim {head_dim}, "
                         f"has {tuple(inv_freq.shape)}")
    if axes is None:
        if n > 1:
            raise ValueError("several axes need `axes` (rope_axes(sections))")
    elif not isinstance(axes, bytes) or len(axes) != half or max(axes) >= n:
        raise ValueError(f"axes must be {half} bytes below {n} (rope_axes(sections))")
    if pairing not in _PAIRING:
        raise ValueError(f"pairing must be 'half' or 'adjacent', is {pairing!r}")
    return (positions.data_ptr(), inv_freq.data_ptr(), positions.stride(0) if positions.dim() == 2 else 0,
            positions.element_size(), n, 2 * half, _PAIRING[pairing])


def _cache(k_cache, v_cache, like, head_dim: int):
    """paged_cache_t's fields."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 4 or t.shape[3] != head_dim:
            raise ValueError(f"{name} must be [pages, page_size, heads, {head_dim}], has {tuple(t.shape)}")
        if t.dtype != like.dtype or t.device != like.device:
            raise ValueError(f"{name} must match dtype/device of the head rows")
        if t.stride(3) != 1 and head_dim > 1:
            raise ValueError(f"{name}'s last dimension must be contiguous")
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    sk, sv, shape = k_cache.stride(), v_cache.stride(), k_cache.shape
    return (k_cache.data_ptr(), v_cache.data_ptr(), shape[0], sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], shape[1],
            shape[2])


_HERE = contextlib.nullcontext()


def _on(device):
    """Makes `device` current; nothing where it is already."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _call(fn, what: str, device, stream, *args):
    """fn(*args, stream) with the tensors' device current."""
    with _on(device):
        st = fn(*args, _stream_handle(stream, device))
    if st:
        _raise(st, what)


def _rope(fn, what, q, k, positions, inv_freq, axes, pairing, q_out, k_out, stream):
    code = _code(q)
    q_out, q_rows = _rows(q, q_out, "q", None)
    T, hq, D = q.shape
    k_rows, hk = _NO_ROWS, 0
    if k is not None:
        k_out, k_rows = _rows(k, k_out, "k", q)
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"k must be [{T}, heads, {D}], has {tuple(k.shape)}")
        hk = k.shape[1]
    ang = _angles(positions, inv_freq, axes, pairing, T, D, q.device)
    _call(fn, what, q.device, stream, _ROPE.pack(*q_rows, *k_rows, *ang, T, hq, hk, D, code), axes)
    return q_out, (k_out if k is not None else None)


def rope_fwd(q, k, positions, inv_freq, *, axes=None, pairing="half", q_out=None, k_out=None, stream=None):
    """q, k rotated by their tokens' positions. q [T, heads, D] and k (or
    None) [T, kv_heads, D] may be strided views of a fused projection, and
    q_out / k_out the inputs themselves.

    positions: int32 or int64 [T], or [axes, T] with ``axes`` (from
    ``rope_axes``) naming the axis of each frequency. inv_freq: fp32, one per
    pair; 2 * len(inv_freq) values of each head are rotated, the rest pass.
    pairing: "half" pairs (i, i + len(inv_freq)), "adjacent" (2i, 2i + 1)."""
    return _rope(lib().rope_fwd, "rope_fwd", q, k, positions, inv_freq, axes, pairing, q_out, k_out, stream)


def rope_bwd(dq, dk, positions, inv_freq, *, axes=None, pairing="half", dq_out=None, dk_out=None, stream=None):
    """The gradients of rope_fwd's q and k, from those of its results."""
    return _rope(lib().rope_bwd, "rope_bwd", dq, dk, positions, inv_freq, axes, pairing, dq_out, dk_out, stream)


def paged_kv_append(k, v, k_cache, v_cache, slots, positions=None, inv_freq=None, *, axes=None, pairing="half",
                    q=None, q_out=None, wq=None, wk=None, eps: float = 1e-6, offset: float = 0.0, stream=None):
    """Appends k and v [T, kv_heads, D] to a paged cache [pages, page_size,
    kv_heads, D] at ``slots`` (int64 [T]: page * page_size + place; negative:
    the token is left out). k is first normalised per head where ``wk`` is
    given and rotated where ``positions`` are (as rope_fwd); q (optional) is
    normalised by ``wq`` and rotated in the same launch and returned (None
    without q). Two tokens of a call must not share a slot."""
    code = _code(k)
    sk, sv = _heads(k, "k"), _heads(v, "v", k)
    T, hk, D = k.shape
    if v.shape != k.shape:
        raise ValueError(f"v must have k's shape {tuple(k.shape)}, has {tuple(v.shape)}")
    dev = k.device
    q_rows, hq = _NO_ROWS, 0
    if q is not None:
        q_out, q_rows = _rows(q, q_out, "q", k)
        if q.shape[0] != T or q.shape[2] != D:
            raise ValueError(f"q must be [{T}, heads, {D}], has {tuple(q.shape)}")
        hq = q.shape[1]
    elif wq is not None or q_out is not None:
        raise ValueError("wq and q_out need q")
    if positions is None:
        if inv_freq is not None or axes is not None:
            raise ValueError("inv_freq and axes need positions")
        ang = _NO_ANGLES
    else:
        ang = _angles(positions, inv_freq, axes, pairing, T, D, dev)
    cache = _cache(k_cache, v_cache, k, D)
    if cache[-1] != hk:
        raise ValueError(f"the cache holds {cache[-1]} heads, k has {hk}")
    _small(slots, "slots", (torch.int64,), dev)
    if slots.numel() != T:
        raise ValueError(f"slots must have {T} elements, has {slots.numel()}")
    wp = [0, 0]
    wdt = None
    for i, (w, name) in enumerate(((wq, "wq"), (wk, "wk"))):
        if w is not None:
            _small(w, name, (k.dtype, torch.float32), dev)
            if w.numel() != D or (wdt is not None and w.dtype != wdt):
                raise ValueError(f"{name} must have {D} elements and wq, wk one type")
            wdt = w.dtype
            wp[i] = w.data_ptr()
    if wdt is torch.float32 and code != 0:
        code |= RMSNORM_WEIGHT_F32
    _call(lib().paged_kv_append, "paged_kv_append", dev, stream,
          _APPEND.pack(*q_rows, k.data_ptr(), 0, sk[0], sk[1], 0, 0, v.data_ptr(), 0, sv[0], sv[1], 0, 0, *ang, *cache,
                       slots.data_ptr(), wp[0], wp[1], T, eps, offset, hq, D, code, 0), axes)
    return q_out if q is not None else None


def _attn_call(q, out, lse, sq, so, cache, block_table, kv_lens, cu_q, max_q, max_kv, scale, causal, code, ws, wsb):
    T, hq, D = q.shape
    return _ATTN.pack(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), sq[0], sq[1], so[0], so[1],
                      *cache, block_table.data_ptr(), kv_lens.data_ptr(), cu_q.data_ptr(), block_table.stride(0), T,
                      ws, wsb, scale, kv_lens.shape[0], block_table.shape[1], hq, D, max_q, max_kv, int(causal), code)


def paged_attn_fwd(q, k_cache, v_cache, block_table, kv_lens, cu_q, *, max_q: int, max_kv: int, scale=None,
                   causal: bool = True, out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache; returns out, lse.

    q [T, heads, D] (bf16 or fp16) holds the sequences' new tokens one after
    the other, sequence b's in rows cu_q[b] .. cu_q[b + 1] (int32 [batch + 1]).
    k_cache, v_cache [pages, page_size, kv_heads, D], block_table int32
    [batch, width] names each sequence's pages, kv_lens int32 [batch] its
    length with the new tokens (already appended). Causal: a new token sees
    the keys up to itself. max_q and max_kv bound the sequences' new tokens
    and lengths. scale defaults to 1 / sqrt(D). lse: True, or an fp32 tensor
    [T, heads], for the log of each row's sum of exponentials (None: not
    written). Rows behind the last sequence are left as they were.
    workspace: a tensor of at least paged_attn_workspace_bytes() bytes."""
    sq = _heads(q, "q")
    T, hq, D = q.shape
    code = _code(q)
    dev = q.device
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    elif not isinstance(out, torch.Tensor) or out.shape != q.shape:
        raise ValueError(f"out must have q's shape {tuple(q.shape)}")
    so = _heads(out, "out", q)
    cache = _cache(k_cache, v_cache, q, D)
    i32 = (torch.int32,)
    _small(block_table, "block_table", i32, dev, contiguous=False)
    _small(kv_lens, "kv_lens", i32, dev)
    _small(cu_q, "cu_q", i32, dev)
    batch = kv_lens.shape[0] if kv_lens.dim() == 1 else -1
    if block_table.dim() != 2 or block_table.shape[0] != batch or (block_table.shape[1] > 1
                                                                  and block_table.stride(1) != 1):
        raise ValueError("block_table must be [batch, width] with contiguous rows, kv_lens [batch]")
    if cu_q.dim() != 1 or cu_q.shape[0] != batch + 1:
        raise ValueError(f"cu_q must have {batch + 1} elements")
    if lse is False:
        lse = None
    elif lse is True:
        lse = torch.empty((T, hq), dtype=torch.float32, device=dev)
    elif lse is not None:
        _small(lse, "lse", _F32, dev)
        if lse.numel() != T * hq:
            raise ValueError(f"lse must have {T * hq} elements, has {lse.numel()}")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ws, wsb = 0, 0
    if workspace is not None:
        if not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the input's device")
        ws, wsb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    call = _attn_call(q, out, lse, sq, so, cache, block_table, kv_lens, cu_q, max_q, max_kv, scale, causal, code, ws,
                      wsb)
    if workspace is None and stream is None:
        # torch's own allocator, on the current stream; with another stream
        # the library takes stream-ordered memory there
        with _on(dev):
            n = lib().paged_attn_workspace_bytes(call)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
            call = _attn_call(q, out, lse, sq, so, cache, block_table, kv_lens, cu_q, max_q, max_kv, scale, causal,
                              code, workspace.data_ptr(), n)
    _call(lib().paged_attn_fwd, "paged_attn_fwd", dev, stream, call)
    return out, lse


def paged_attn_workspace_bytes(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int, max_q: int,
                               max_kv: int) -> int:
    """Bytes of workspace paged_attn_fwd takes for these sizes on the current device."""
    c = _ATTN.pack(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, kv_heads, 0, 0, 0, 0, tokens, 0, 0, 1.0, batch,
                   0, heads, head_dim, max_q, max_kv, 1, 1)
    return int(lib().paged_attn_workspace_bytes(c))
