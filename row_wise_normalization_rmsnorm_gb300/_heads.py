"""Rotary positions, the paged key/value cache and its attention (the entry
points on head rows of include/rmsnorm.h).

The arguments are checked and marshalled by the module ``_heads_ext``
(csrc/heads_ext.cpp): for a few tokens the host's share is most of a call.
There is no CPU fallback.

``stream`` names the stream to launch on (an object or a handle; None: the
device's current one). The call waits for nothing there, so what it reads has
to be ready in that stream's order. Results that it makes for a named stream
lie in that stream's memory, and the current stream may read them once it has
waited for the named one.
"""
from __future__ import annotations

from . import _binding

_ext = None


def _load():
    """The native module, loaded on the first call (after the library)."""
    global _ext
    _binding.lib()
    try:
        from . import _heads_ext
    except ImportError as e:
        raise RuntimeError(
            "the native module _heads_ext is not built; run `python -m row_wise_normalization_rmsnorm_gb300.build` "
            f"(or __graft_entry__.build()): {e}") from e
    _ext = _heads_ext
    return _ext


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


def rope_fwd(q, k, positions, inv_freq, *, axes=None, pairing="half", q_out=None, k_out=None, stream=None):
    """q, k rotated by their tokens' positions. q [T, heads, D] and k (or
    None) [T, kv_heads, D] may be strided views of a fused projection, and
    q_out / k_out the inputs themselves. Returns (q_out, k_out).

    positions: int32 or int64 [T], or [axes, T] with ``axes`` (from
    ``rope_axes``) naming the axis of each frequency. inv_freq: fp32, one per
    pair; 2 * len(inv_freq) values of each head are rotated, the rest pass.
    pairing: "half" pairs (i, i + len(inv_freq)), "adjacent" (2i, 2i + 1)."""
    return (_ext or _load()).rope(False, q, k, positions, inv_freq, axes, pairing, q_out, k_out, stream)


def rope_bwd(dq, dk, positions, inv_freq, *, axes=None, pairing="half", dq_out=None, dk_out=None, stream=None):
    """The gradients of rope_fwd's q and k, from those of its results."""
    return (_ext or _load()).rope(True, dq, dk, positions, inv_freq, axes, pairing, dq_out, dk_out, stream)


def paged_kv_append(k, v, k_cache, v_cache, slots, positions=None, inv_freq=None, *, axes=None, pairing="half",
                    q=None, q_out=None, wq=None, wk=None, eps: float = 1e-6, offset: float = 0.0, stream=None):
    """Appends k and v [T, kv_heads, D] to a paged cache [pages, page_size,
    kv_heads, D] at ``slots`` (int64 [T]: page * page_size + place; negative:
    the token is left out). k is first normalised per head where ``wk`` is
    given and rotated where ``positions`` are (as rope_fwd); q (optional) is
    normalised by ``wq`` and rotated in the same launch and returned (None
    without q). Two tokens of a call must not share a slot. What paged_attn_fwd
    reads is narrower: bf16 or fp16, D a multiple of 8 up to 128, page_size a
    multiple of 8."""
    return (_ext or _load()).append(k, v, k_cache, v_cache, slots, positions, inv_freq, axes, pairing, q, q_out, wq, wk,
                                    eps, offset, stream)


def paged_attn_fwd(q, k_cache, v_cache, block_table, kv_lens, cu_q, *, max_q: int, max_kv: int, scale=None,
                   causal: bool = True, out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache; returns out, lse.

    q [T, heads, D] (bf16 or fp16) holds the sequences' new tokens one after
    the other, sequence b's in rows cu_q[b] .. cu_q[b + 1] (int32 [batch + 1]).
    k_cache, v_cache [pages, page_size, kv_heads, D], block_table int32
    [batch, width] names each sequence's pages, kv_lens int32 [batch] its
    length with the new tokens (already appended). Causal: a new token sees
    the keys up to itself. max_q and max_kv bound the sequences' new tokens
    and lengths (bounds far above them cost time: the work is cut by them).
    scale defaults to 1 / sqrt(D). lse: True, or an fp32 tensor [T, heads], for
    the log of each row's sum of exponentials (None: not written). Rows behind
    the last sequence are left as they were.
    workspace: a tensor of at least paged_attn_workspace_bytes() bytes."""
    return (_ext or _load()).attn(q, k_cache, v_cache, block_table, kv_lens, cu_q, max_q, max_kv, scale, causal, out, lse,
                                  workspace, stream)


def paged_attn_workspace_bytes(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int, max_q: int,
                               max_kv: int) -> int:
    """Bytes of workspace paged_attn_fwd takes for these sizes on the current device."""
    return (_ext or _load()).attn_workspace(tokens, batch, heads, kv_heads, head_dim, max_q, max_kv)
