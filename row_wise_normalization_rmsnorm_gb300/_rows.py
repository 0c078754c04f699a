"""Rows of a training step beside the norms: what a norm's input is kept as
for the backward pass (8-bit checkpoints), group norm with an activation, and
embedding rows with their gradient (entry points of include/rmsnorm.h).

Row arrays are contiguous CUDA tensors in bf16, fp16 or fp32, weights in the
rows' type or fp32. ``stream`` and the memory of results are as in the calls
on head rows; results are made here unless they are given, and a workspace is
taken from PyTorch's allocator unless one is given. There is no CPU fallback.
"""
from __future__ import annotations

import torch

from . import _heads
from ._binding import TORCH_DTYPE


def _ext():
    return _heads._ext or _heads._load()


def ckpt8_pack(x, *, codes=None, scales=None, stream=None):
    """x's rows (last dimension N) in 8 bits: codes (int8, x's shape) and
    scales (uint8 [..., ceil(N / 32)]). A code c of a block with scale byte b
    stands for c 2^(b - 127), at most 2^-7 of the block's largest magnitude off;
    a block with an infinity or a NaN stands for NaN."""
    return _ext().pack(x, codes, scales, stream)


def ckpt8_unpack(codes, scales, dtype, *, x=None, stream=None):
    """The rows that ``ckpt8_pack`` kept, in ``dtype``."""
    return _ext().unpack(codes, scales, dtype, x, stream)


def rmsnorm_fwd_ckpt8(x, w, *, residual=None, eps: float = 1e-6, offset: float = 0.0, y=None, residual_out=None,
                      rstd=None, codes=None, scales=None, stream=None) -> dict:
    """rmsnorm_fwd, or (with ``residual``) rmsnorm_add_fwd, with the row that
    is normalised kept in 8 bits in the same pass. Returns a dict with y,
    residual_out (fused only), rstd, codes, scales."""
    out = _ext().norm_keep(x, w, residual, eps, offset, y, residual_out, rstd, codes, scales, stream)
    return dict(zip(("y", "residual_out", "rstd", "codes", "scales"), out))


def rmsnorm_bwd_ckpt8(dy, codes, scales, w, rstd, *, dresidual_out=None, offset: float = 0.0, dx=None, dw=None,
                      workspace=None, stream=None):
    """dx, dw of rmsnorm_fwd_ckpt8 from what it kept and its rstd; with
    ``dresidual_out`` dx is the gradient of x and of residual. w None is
    non-affine (dw None)."""
    return _ext().norm_bwd(dy, codes, scales, w, rstd, dresidual_out, offset, dx, dw, workspace, stream)


def rmsnorm_bwd_ckpt8_workspace_bytes(M: int, N: int, dtype) -> int:
    return _ext().workspace(M, N, _code(dtype), None)


def groupnorm_fwd(x, gamma, beta, groups: int, *, act=None, eps: float = 1e-5, y=None, mean=None, rstd=None,
                  workspace=None, stream=None) -> dict:
    """Group norm over channels that come last, x [batch, ..., channels] (a
    channels_last image as [batch, height, width, channels]), with an
    activation (None, "silu" or "gelu") behind it. gamma / beta [channels] may
    be None. Returns a dict with y, and mean and rstd [batch, groups]."""
    out = _ext().gn_fwd(x, gamma, beta, groups, act, eps, False, y, mean, rstd, None, None, workspace, stream)
    return {"y": out[0], "mean": out[1], "rstd": out[2]}


def groupnorm_fwd_ckpt8(x, gamma, beta, groups: int, *, act=None, eps: float = 1e-5, y=None, mean=None, rstd=None,
                        codes=None, scales=None, workspace=None, stream=None) -> dict:
    """groupnorm_fwd with x kept in 8 bits: also codes and scales. (The work may
    be cut another way: y, mean and rstd may differ in their last bits from
    those of groupnorm_fwd.)"""
    out = _ext().gn_fwd(x, gamma, beta, groups, act, eps, True, y, mean, rstd, codes, scales, workspace, stream)
    return dict(zip(("y", "mean", "rstd", "codes", "scales"), out))


def groupnorm_bwd(dy, x, gamma, beta, mean, rstd, groups: int, *, act=None, want_dgamma=True, want_dbeta=True,
                  dx=None, dgamma=None, dbeta=None, workspace=None, stream=None) -> dict:
    """dx, dgamma and dbeta of groupnorm_fwd given its mean and rstd (dgamma
    None without gamma or when not wanted, dbeta when not wanted: a tensor
    given for it is then left as it is, as in layernorm_bwd)."""
    out = _ext().gn_bwd(dy, x, None, None, gamma, beta, mean, rstd, groups, act, bool(want_dgamma), bool(want_dbeta),
                        dx, dgamma, dbeta, workspace, stream)
    return dict(zip(("dx", "dgamma", "dbeta"), out))


def groupnorm_bwd_ckpt8(dy, codes, scales, gamma, beta, mean, rstd, groups: int, *, act=None, want_dgamma=True,
                        want_dbeta=True, dx=None, dgamma=None, dbeta=None, workspace=None, stream=None) -> dict:
    """groupnorm_bwd from what groupnorm_fwd_ckpt8 kept of x."""
    out = _ext().gn_bwd(dy, None, codes, scales, gamma, beta, mean, rstd, groups, act, bool(want_dgamma),
                        bool(want_dbeta), dx, dgamma, dbeta, workspace, stream)
    return dict(zip(("dx", "dgamma", "dbeta"), out))


def groupnorm_workspace_bytes(batch: int, places: int, channels: int, groups: int, dtype, *, backward=False) -> int:
    """Bytes of workspace that groupnorm_fwd (or _bwd) and its _ckpt8 form take at most for these sizes on the current
    device, wherever the arrays lie."""
    return _ext().workspace(batch, places, channels, groups, _code(dtype), bool(backward))


def embed_fwd(ids, table, *, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids], rounded once: ids int32 or int64 of any shape,
    table [rows, N]. An id that is negative or not below rows (padding) gives
    a row of zeros."""
    return _ext().embed(ids, table, None, False, scale, 0.0, 0.0, None, out, None, stream)


def rmsnorm_embed_fwd(ids, table, w, *, scale: float = 1.0, eps: float = 1e-6, offset: float = 0.0, y=None,
                      residual_out=None, rstd=None, stream=None):
    """h = embed_fwd(ids, table), y = RMSNorm(h) in one pass; returns y, h,
    rstd as rmsnorm_add_fwd does (rmsnorm_add_bwd and embed_bwd are its
    gradient)."""
    return _ext().embed(ids, table, w, True, scale, eps, offset, y, residual_out, rstd, stream)


def embed_bwd(dh, ids, rows: int, *, scale: float = 1.0, dtype=None, dtable=None, accumulate=False, workspace=None,
              stream=None):
    """The table's gradient [rows, N] from that of its looked-up rows: for
    each row scale times the sum of dh over the row's tokens, in an order that
    depends on the ids, their number and N alone. In dh's type or (``dtype``, or a given
    ``dtable``) fp32. accumulate: added to ``dtable``, of which only the rows
    with tokens are touched; otherwise every row is written."""
    return _ext().embed_grad(dh, ids, rows, scale, dtype, dtable, accumulate, workspace, stream)


def embed_bwd_workspace_bytes(tokens: int, columns: int, rows: int) -> int:
    return _ext().workspace(tokens, columns, rows)


def _code(dtype) -> int:
    return TORCH_DTYPE[dtype] if isinstance(dtype, torch.dtype) else dtype
