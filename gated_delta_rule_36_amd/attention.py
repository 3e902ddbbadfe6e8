"""Python binding of the attention layers' operators: ``qk_norm_rotary``,
``append_kv`` and ``paged_attention``.

Argument marshalling only, by the layer operators' rules: the caller gives
the output tensors and the cache, the call is enqueued on the current stream
of the tensors' device, and an argument the library refuses raises
:class:`KdaArgumentError` before anything is enqueued.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .layer import _BF16, _FP32, _call, _call_with_workspace, _dense, _device, _tensor, _tokens, _typed

_INT32, _INT64 = torch.int32, torch.int64


def _rotation(positions, inv_freq, device, shape):
    """(positions' pointer, frequencies' pointer, rotated channels), 0 for none."""
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    if positions is None:
        return 0, 0, 0
    pp = _dense("positions", positions, device, shape, _INT64)
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype is not _FP32 or inv_freq.device != device:
        _tensor("inv_freq", inv_freq, device, _FP32)
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be contiguous [R/2], got {list(inv_freq.shape)} with strides {inv_freq.stride()}")
    return pp, inv_freq.data_ptr(), 2 * inv_freq.shape[0]


def _cache(name, t, device, heads, channels):
    """(pointer, strides of page, token and head) of a paged cache [pages, page_size, heads, channels]."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.device != device:
        _tensor(name, t, device, _BF16)
    shape, strides = t.shape, t.stride()
    if len(shape) != 4 or shape[2] != heads or shape[3] != channels:
        raise ValueError(f"{name} must be [pages,page_size,{heads},{channels}], got {list(shape)}")
    if channels != 1 and strides[3] != 1:
        raise ValueError(f"{name}: the channels of a head must be adjacent, got strides {strides}")
    return t.data_ptr(), strides[0], strides[1], strides[2]


def qk_norm_rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                   inv_freq: Optional[torch.Tensor], q_out: torch.Tensor, k_out: Optional[torch.Tensor] = None,
                   q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, *,
                   eps: float = 1e-6, interleaved: bool = False, rotary_scale: float = 1.0) -> torch.Tensor:
    """RMS norm of every query and key head and its position rotation, in one
    pass; writes ``q_out`` and ``k_out``.

    ``y = x / sqrt(mean x^2 + eps) * weight`` (``x`` where the weight is None),
    then the pairs of the first R = ``2 len(inv_freq)`` channels are turned by
    the angles ``positions inv_freq`` (formed in 64 bits) and scaled by
    ``rotary_scale``: channels f and f + R/2, or ``interleaved`` 2 f and
    2 f + 1; the others stay.  ``q`` and ``q_out`` are bf16 ``[B, T, Hq, D]``,
    ``k`` and ``k_out`` ``[B, T, Hk, D]`` or None, D an even number up to 512;
    ``positions`` int64 ``[B, T]`` and ``inv_freq`` fp32 ``[R/2]``, or both None
    (norm alone); the weights ``[D]`` bf16 or fp32.  ``q`` and ``k`` may be
    slices of a fused projection; contiguous ones may be their own output.
    """
    device = _device(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must be [B,T,H,D], got {list(q.shape)}")
    B, T, Hq, D = shape = q.shape
    pq, qb, qt = _tokens("q", q, device, shape)
    po = _dense("q_out", q_out, device, shape, _BF16)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    pk = pko = kb = kt = Hk = 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            _tensor("k", k, device, _BF16)
            raise ValueError(f"k must be [B,T,H,D], got {list(k.shape)}")
        Hk = k.shape[2]
        pk, kb, kt = _tokens("k", k, device, (B, T, Hk, D))
        pko = _dense("k_out", k_out, device, (B, T, Hk, D), _BF16)
    pp, pf, R = _rotation(positions, inv_freq, device, (B, T))
    pw, wcode = _typed("q_weight", q_weight, device, (D,))
    pu, ucode = _typed("k_weight", k_weight, device, (D,))
    _call("kda_qk_norm_rotary", (pq, pk, po, pko, qb, qt, kb, kt, pp, pf, pw, pu, B, T, Hq, Hk, D, R, wcode, ucode,
                                 1 if interleaved else 0, 0, eps, rotary_scale), device)
    return q_out


def append_kv(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
              positions: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
              weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6, interleaved: bool = False,
              rotary_scale: float = 1.0) -> None:
    """Writes new tokens' keys and values into their slots of a paged cache.

    ``k`` and ``v`` are bf16 ``[B, T, Hk, D]``; the keys go through the norm
    (``weight``) and rotation (``positions``, ``inv_freq``) of
    :func:`qk_norm_rotary` on the way, each left out where it is None.  The
    caches are bf16 ``[pages, page_size, Hk, D]`` with adjacent channels and any
    other strides.  ``slots`` (int64 ``[B, T]``) says where: slot s is token
    ``s % page_size`` of page ``s // page_size``.  Tokens with a slot outside the
    cache (-1 for padding) are left out; tokens of one call have distinct slots
    otherwise.  Nothing else in the caches is written.
    """
    device = _device(k, "k")
    if k.dim() != 4:
        raise ValueError(f"k must be [B,T,H,D], got {list(k.shape)}")
    B, T, H, D = shape = k.shape
    pk, kb, kt = _tokens("k", k, device, shape)
    if v is None:
        _tensor("v", v, device, _BF16)
    pv, vb, vt = _tokens("v", v, device, shape)
    pkc, kp, ks, kh = _cache("k_cache", k_cache, device, H, D)
    pvc, vp, vs, vh = _cache("v_cache", v_cache, device, H, D)
    pages, page_size = k_cache.shape[:2]
    if v_cache.shape[:2] != k_cache.shape[:2]:
        raise ValueError(f"the caches differ in pages: {list(k_cache.shape)} and {list(v_cache.shape)}")
    if slots is None:
        _tensor("slots", slots, device, _INT64)
    ps = _dense("slots", slots, device, (B, T), _INT64)
    pp, pf, R = _rotation(positions, inv_freq, device, (B, T))
    pw, wcode = _typed("weight", weight, device, (D,))
    _call("kda_append_kv", (pk, pv, pkc, pvc, kb, kt, vb, vt, kp, ks, kh, vp, vs, vh, ps, pp, pf, pw, B, T, H, D, R,
                            pages, page_size, wcode, 1 if interleaved else 0, 0, eps, rotary_scale), device)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    lengths: torch.Tensor, out: torch.Tensor, scale: float, *, lse: Optional[torch.Tensor] = None,
                    window: Optional[int] = None) -> torch.Tensor:
    """Softmax attention of one new token per sequence over a paged cache;
    writes ``out`` (and ``lse``).

    ``out[n, h] = sum_t p_t v_t`` with p the softmax of ``scale q[n, h] . k_t``
    over the sequence's first ``lengths[n]`` tokens, or the last ``window`` of
    them.  ``q`` and ``out`` are bf16 ``[N, Hq, D]`` (q's rows may be slices),
    the caches bf16 ``[pages, page_size, Hk, D]`` with adjacent channels and any
    other strides; Hk divides Hq, and query heads share a key head.  D is a
    multiple of 16 up to 256.  ``block_table`` int32 ``[N, width]`` names the
    pages of each sequence in order, ``lengths`` int32 ``[N]`` counts its tokens,
    the new one among them; neither is read on the host.  ``lse`` fp32
    ``[N, Hq]`` takes the logarithm of the softmax's sum.  A sequence without a
    visible token gets zeros and -inf; pages outside the cache are not read and
    their tokens not visible.  The workspace is a temporary allocation on the
    same stream, sized by ``width``, by which a sequence is also split: a table far
    wider than the lengths need costs time.
    """
    device = _device(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must be [N,Hq,D], got {list(q.shape)}")
    N, Hq, D = shape = q.shape
    strides = q.stride()
    if (strides[2] != 1 and D != 1) or (strides[1] != D and Hq != 1):
        raise ValueError(f"q: the channels of a sequence must be adjacent, got strides {strides}")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        _tensor("k_cache", k_cache, device, _BF16)
        raise ValueError(f"k_cache must be [pages,page_size,Hk,D], got {list(k_cache.shape)}")
    pages, page_size, Hk, _ = k_cache.shape
    pk, kp, ks, kh = _cache("k_cache", k_cache, device, Hk, D)
    pv, vp, vs, vh = _cache("v_cache", v_cache, device, Hk, D)
    if v_cache.shape[:2] != k_cache.shape[:2]:
        raise ValueError(f"the caches differ in pages: {list(k_cache.shape)} and {list(v_cache.shape)}")
    if not isinstance(block_table, torch.Tensor) or block_table.dtype is not _INT32 or block_table.device != device:
        _tensor("block_table", block_table, device, _INT32)
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError(f"block_table must be [{N},width], got {list(block_table.shape)}")
    width = block_table.shape[1]
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError(f"block_table: a sequence's pages must be adjacent, got strides {block_table.stride()}")
    if lengths is None or out is None:
        _tensor("out" if out is None else "lengths", None, device)
    pl = _dense("lengths", lengths, device, (N,), _INT32)
    po = _dense("out", out, device, shape, _BF16)
    pe = _dense("lse", lse, device, (N, Hq), _FP32)
    if window is not None and (not isinstance(window, int) or isinstance(window, bool) or window < 1):
        raise ValueError(f"window must be a positive int or None, got {window!r}")
    values = (q.data_ptr(), pk, pv, block_table.data_ptr(), pl, po, pe, strides[0], block_table.stride(0), kp, ks, kh, vp, vs, vh,
              N, Hq, Hk, D, pages, page_size, width, window or 0, 0, scale)
    _call_with_workspace("kda_paged_attention", "kda_paged_attention_workspace_bytes", values, device)
    return out
