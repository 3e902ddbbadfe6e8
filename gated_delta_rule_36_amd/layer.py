"""Python binding of the layer operators: ``short_conv``, ``ssm_fwd``,
``gated_norm`` and ``residual_norm``.

Argument marshalling only, like :func:`gated_delta_rule_36_amd.fwd`: the
caller gives the output tensors, the call is enqueued on the current stream
of the tensors' device, and an argument the library refuses raises
:class:`KdaArgumentError` before anything is enqueued.  Inputs may be slices
of wider rows (a fused projection's output): the channels of a token have to
be adjacent, the tokens may lie anywhere.
"""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import _lib
from .api import KdaArgumentError, KdaError

_CODES = {torch.bfloat16: _lib.KDA_DTYPE_BF16, torch.float32: _lib.KDA_DTYPE_FP32}
_ACTIVATIONS = {None: _lib.KDA_ACT_NONE, "silu": _lib.KDA_ACT_SILU, "sigmoid": _lib.KDA_ACT_SIGMOID}
_BF16 = torch.bfloat16


def _tensor(name, t, device, *dtypes):
    """A tensor of one of `dtypes` on `device`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _device(x):
    """x's device, which must be a GPU; x must be bf16."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dtype != _BF16:
        raise TypeError(f"x must be {_BF16}, got {x.dtype}")
    if x.device.type != "cuda":
        raise ValueError(f"x must be on a GPU device, got {x.device}")
    return x.device


def _dense(name, t, device, shape, *dtypes):
    """The pointer of a contiguous tensor of exactly `shape`, or 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.device != device:
        _tensor(name, t, device, *dtypes)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _tokens(name, t, device, shape):
    """(pointer, batch stride, token stride) of bf16 [B, T, ...] whose trailing dimensions are adjacent."""
    if t is None:
        return 0, 0, 0
    _tensor(name, t, device, _BF16)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    strides, width = t.stride(), 1
    for size, stride in zip(reversed(shape[2:]), reversed(strides[2:])):
        if size != 1 and stride != width:
            raise ValueError(f"{name}: the channels of a token must be adjacent, got strides {strides}")
        width *= size
    return t.data_ptr(), strides[0], strides[1]


def _row_stride(name, t):
    """The one stride of the rows [..., D] of t, whose channels are adjacent."""
    shape, strides = t.shape, t.stride()
    if shape[-1] != 1 and strides[-1] != 1:
        raise ValueError(f"{name}: the channels of a row must be adjacent, got strides {strides}")
    if t.is_contiguous():
        return shape[-1]
    found, step = None, None
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if step is not None and stride != step:
            raise ValueError(f"{name}: the rows must be evenly spaced, got strides {strides}")
        found = stride if found is None else found
        step = stride * size
    return shape[-1] if found is None else found


def _sequences(cu_seqlens, device, B, T, check):
    """(pointer, number of sequences, states) of a call."""
    if cu_seqlens is None:
        return 0, 0, B
    _tensor("cu_seqlens", cu_seqlens, device, torch.int64)
    if cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be contiguous [N+1] with N+1 >= 1 entries")
    if check:
        host = cu_seqlens.cpu()
        if int(host[0]) != 0 or int(host[-1]) != T or bool((host[1:] < host[:-1]).any()):
            raise ValueError("cu_seqlens must be nondecreasing from 0 to T")
    n = cu_seqlens.numel() - 1
    return cu_seqlens.data_ptr(), n, n


def _typed(name, t, device, shape):
    """(pointer, dtype code) of a contiguous bf16 or fp32 tensor of exactly `shape`, or of None."""
    if t is None:
        return 0, _lib.KDA_DTYPE_NONE
    return _dense(name, t, device, shape, _BF16, torch.float32), _CODES[t.dtype]


def _pack(pack, values):
    """The bytes of an argument struct; a field of the wrong type is a TypeError."""
    try:
        return pack(*values)
    except struct.error as e:
        raise TypeError(f"an argument has the wrong type: {e}") from None


def _entry(name):
    found = _lib.LAYER.get(name)
    if found is None:
        _lib.load()
        found = _lib.LAYER[name]
    return found


def _call(name, values, device, args=None):
    """Enqueue `values` (or what they were packed to) on the current stream of `device` (its handle straight from
    torch's C layer: the Stream object that torch.cuda.current_stream builds costs as much as the launch)."""
    entry, pack = _entry(name)
    if args is None:
        args = _pack(pack, values)
    index = device.index
    if torch._C._cuda_getDevice() == index:
        status = entry(args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = entry(args, torch._C._cuda_getCurrentRawStream(index))
    if status != _lib.KDA_OK:
        raise (KdaError if status == _lib.KDA_ERR_LAUNCH else KdaArgumentError)(status)


def short_conv(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor,
               bias: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
               l2norm: Optional[int] = None, l2norm_eps: float = 1e-6,
               initial_state: Optional[torch.Tensor] = None,
               final_state: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None,
               check_cu_seqlens: bool = True) -> torch.Tensor:
    """Short causal depthwise convolution; writes ``out`` (and ``final_state``).

    ``y[t, c] = act(bias[c] + sum_j weight[c, j] x[t - W + 1 + j, c])``, with
    the inputs before a sequence's first token from ``initial_state``
    ``[N, W-1, D]`` (bf16 or fp32, oldest first; None: zeros).  ``x`` and
    ``out`` are bf16 ``[B, T, D]`` or ``[B, T, H, K]`` (D = H K), ``weight``
    ``[D, W]`` and ``bias`` ``[D]`` both bf16 or both fp32, W at most 8;
    ``activation`` is "silu" or None.  ``l2norm`` (64, 128 or 256) divides
    every group of that many channels by ``sqrt(sum y^2 + l2norm_eps)``: with
    128 the queries and keys come out as :func:`fwd` takes them.
    ``final_state`` takes the last W - 1 inputs of each sequence and may be
    ``initial_state``; a single token with the state carried is T = 1.
    ``cu_seqlens`` and ``check_cu_seqlens`` are those of :func:`fwd`.
    """
    device = _device(x)
    if x.dim() not in (3, 4):
        raise ValueError(f"x must be [B,T,D] or [B,T,H,K], got {list(x.shape)}")
    shape = x.shape
    B, T = shape[0], shape[1]
    D = shape[2] if len(shape) == 3 else shape[2] * shape[3]
    px, sb, st = _tokens("x", x, device, shape)
    po = _dense("out", out, device, shape, _BF16)
    _tensor("weight", weight, device, _BF16, torch.float32)
    if weight.dim() != 2:
        raise ValueError(f"weight must be [D,W], got {list(weight.shape)}")
    W = weight.shape[1]
    pw, wcode = _typed("weight", weight, device, (D, W))
    pb = _dense("bias", bias, device, (D,), weight.dtype)
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    pc, num, N = _sequences(cu_seqlens, device, B, T, check_cu_seqlens)
    pi, icode = _typed("initial_state", initial_state, device, (N, W - 1, D))
    pf, fcode = _typed("final_state", final_state, device, (N, W - 1, D))
    _call("kda_short_conv", (px, sb, st, pw, pb, po, pi, pf, pc, num, B, T, D, W, wcode, icode, fcode,
                             _ACTIVATIONS[activation], l2norm or 0, l2norm_eps, 0), device)
    return out


def ssm_fwd(x: torch.Tensor, dt: torch.Tensor, b: torch.Tensor, c: torch.Tensor, out: torch.Tensor,
            A_log: torch.Tensor, D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
            z: Optional[torch.Tensor] = None, *, initial_state: Optional[torch.Tensor] = None,
            final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
            dt_softplus: bool = True, check_cu_seqlens: bool = True,
            segment_tokens: Optional[int] = None) -> torch.Tensor:
    """Selective state space scan; writes ``out`` (and ``final_state``).

    Per head, with a state S of [P, N]: ``dt = softplus(dt + dt_bias)``,
    ``S = exp(-exp(A_log) dt) S + dt x b^T``, ``y = S c + D x``, and
    ``out = y silu(z)``.  ``x``, ``z`` and ``out`` are bf16 ``[B, T, H, P]``,
    ``dt`` bf16 ``[B, T, H]``, ``b`` and ``c`` bf16 ``[B, T, G, N]`` (G
    divides H; heads share a group's b and c), ``A_log``, ``D`` and
    ``dt_bias`` fp32 ``[H]``.  P is a multiple of 32 up to 256, N 32, 64, 128
    or 256.  The states are ``[N, H, P, N]`` (sequences first) in bf16 or
    fp32 and may be one buffer.  ``cu_seqlens`` and ``check_cu_seqlens`` are
    those of :func:`fwd`.  ``segment_tokens`` (a multiple of 32) cuts long
    sequences into segments that run in parallel; None lets the library
    choose.  The workspace is a temporary allocation on the same stream.
    """
    device = _device(x)
    if x.dim() != 4:
        raise ValueError(f"x must be [B,T,H,P], got {list(x.shape)}")
    B, T, H, P = shape = x.shape
    _tensor("b", b, device, _BF16)
    if b.dim() != 4:
        raise ValueError(f"b must be [B,T,G,N], got {list(b.shape)}")
    G, N = b.shape[2], b.shape[3]
    px, xb, xt = _tokens("x", x, device, shape)
    pd, db, dtt = _tokens("dt", dt, device, (B, T, H))
    pb, bb, bt = _tokens("b", b, device, (B, T, G, N))
    pc, cb, ct = _tokens("c", c, device, (B, T, G, N))
    pz, zb, zt = _tokens("z", z, device, shape)
    po = _dense("out", out, device, shape, _BF16)
    _tensor("A_log", A_log, device, torch.float32)
    pA = _dense("A_log", A_log, device, (H,), torch.float32)
    pD = _dense("D", D, device, (H,), torch.float32)
    pt = _dense("dt_bias", dt_bias, device, (H,), torch.float32)
    pu, num, seqs = _sequences(cu_seqlens, device, B, T, check_cu_seqlens)
    pi, icode = _typed("initial_state", initial_state, device, (seqs, H, P, N))
    pf, fcode = _typed("final_state", final_state, device, (seqs, H, P, N))
    if segment_tokens is not None and (not isinstance(segment_tokens, int) or isinstance(segment_tokens, bool)
                                       or segment_tokens < 1):
        raise ValueError(f"segment_tokens must be a positive int or None, got {segment_tokens!r}")
    values = (px, pd, pb, pc, pz, po, xb, xt, db, dtt, bb, bt, cb, ct, zb, zt, pA, pD, pt, pi, pf, pu,
              num, B, T, H, P, G, N, icode, fcode, 1 if dt_softplus else 0, 0, segment_tokens or 0)
    workspace_bytes, pack = _entry("kda_ssm_workspace_bytes")
    args = _pack(pack, values + (0, 0))
    nbytes = workspace_bytes(args)
    if nbytes > 0:
        # freed right after the call: the caching allocator hands it out
        # again only to work ordered after this call on the same stream
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        args = _pack(pack, values + (workspace.data_ptr(), nbytes))
    _call("kda_ssm_fwd", values, device, args)
    return out


def gated_norm(x: torch.Tensor, gate: Optional[torch.Tensor], weight: torch.Tensor, out: torch.Tensor, *,
               group_size: Optional[int] = None, eps: float = 1e-6, activation: str = "sigmoid",
               gate_first: bool = False) -> torch.Tensor:
    """RMS norm of a mixer's output with its gate; writes ``out``.

    ``out = v / sqrt(mean v^2 + eps) * weight * act(gate)`` with ``v = x``,
    or with ``gate_first`` ``out = v / sqrt(mean v^2 + eps) * weight`` with
    ``v = x act(gate)``.  ``x``, ``gate`` and ``out`` are bf16 ``[..., D]``,
    ``weight`` ``[D]`` bf16 or fp32.  The mean runs over groups of
    ``group_size`` channels (None: D; at most 16384).  ``activation`` is
    "sigmoid" or "silu"; without ``gate`` (None) it is a plain RMS norm.
    The rows of ``x`` and ``gate`` may be slices of wider ones, evenly spaced.
    """
    device = _device(x)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    shape = x.shape
    D = shape[-1]
    xs = _row_stride("x", x)
    gs = 0
    if gate is not None:
        _tensor("gate", gate, device, _BF16)
        if gate.shape != shape:
            raise ValueError(f"gate must be {list(shape)}, got {list(gate.shape)}")
        gs = _row_stride("gate", gate)
    po = _dense("out", out, device, shape, _BF16)
    if weight is None:
        raise TypeError("weight must be a torch.Tensor")
    pw, wcode = _typed("weight", weight, device, (D,))
    if activation not in ("sigmoid", "silu"):
        raise ValueError(f"activation must be 'sigmoid' or 'silu', got {activation!r}")
    if D == 0:
        return out
    _call("kda_gated_norm", (x.data_ptr(), 0 if gate is None else gate.data_ptr(), pw, po, xs, gs,
                             x.numel() // D, D, D if group_size is None else group_size, wcode,
                             _ACTIVATIONS[activation], 1 if gate_first else 0, 0, eps), device)
    return out


def _gate_rows(gate, shape):
    """(rows that share a gate row, its stride) of a gate that broadcasts to rows [..., D] of `shape`: its
    leading sizes are those of x up to some dimension and 1 from there on."""
    if gate.shape[-1] != shape[-1]:
        raise ValueError(f"gate must end in {shape[-1]} channels, got {list(gate.shape)}")
    rows = 1
    for size in shape[:-1]:
        rows *= size
    if gate.numel() == shape[-1]:
        _row_stride("gate", gate)
        return max(rows, 1), 0
    lead = gate.shape[:-1]
    if len(lead) != len(shape) - 1:
        raise ValueError(f"gate must be [D] or have the dimensions of x, got {list(gate.shape)}")
    k = len(lead)
    while k > 0 and lead[k - 1] == 1:
        k -= 1
    if lead[:k] != shape[:k]:
        raise ValueError(f"gate {list(gate.shape)} must match x {list(shape)} up to some dimension, then be 1")
    period = 1
    for size in shape[k:-1]:
        period *= size
    return max(period, 1), _row_stride("gate", gate)


def residual_norm(x: torch.Tensor, residual: Optional[torch.Tensor], weight: Optional[torch.Tensor],
                  out: Optional[torch.Tensor], residual_out: Optional[torch.Tensor] = None, *,
                  post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  block_scale: float = 1.0, residual_scale: float = 1.0,
                  eps: float = 1e-6) -> Optional[torch.Tensor]:
    """Residual update between two blocks, with the norms after the one and
    before the next; writes ``residual_out`` and ``out``.

    ``y = x``, or with ``post_weight`` ``x / sqrt(mean x^2 + eps) * post_weight``;
    ``r = residual_scale * residual + block_scale * gate * y`` is written to
    ``residual_out``, and ``out = r / sqrt(mean r^2 + eps) * weight``, from the
    unrounded r.  ``x`` (a block's output) and ``out`` (the next one's input)
    are bf16 ``[..., D]``, D at most 16384; ``residual`` and ``residual_out``
    bf16 or fp32 of the same shape, and may be one buffer; the weights ``[D]``
    bf16 or fp32.  ``gate`` (bf16 or fp32) is ``[D]``, or of x's shape with 1
    in its last leading dimensions (``[B, 1, D]``: one a sequence).  Without
    ``residual`` (None) the stream starts here; ``weight`` and ``out`` are
    both None where no norm follows, and one of the outputs may be left out.
    The scales are 0 or normal numbers of fp32.
    """
    device = _device(x)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    shape = x.shape
    D = shape[-1]
    xs = _row_stride("x", x)
    if (weight is None) != (out is None):
        raise ValueError("weight and out go together")
    if out is None and residual_out is None:
        raise ValueError("out or residual_out must be given")
    pr, rcode = _typed("residual", residual, device, shape)
    pq, qcode = _typed("residual_out", residual_out, device, shape)
    pp, pcode = _typed("post_weight", post_weight, device, (D,))
    pw, wcode = _typed("weight", weight, device, (D,))
    po = _dense("out", out, device, shape, _BF16)
    pg, gcode, period, gs = 0, _lib.KDA_DTYPE_NONE, 0, 0
    if gate is not None:
        _tensor("gate", gate, device, _BF16, torch.float32)
        if gate.dim() < 1:
            raise ValueError("gate must have at least one dimension")
        period, gs = _gate_rows(gate, shape)
        pg, gcode = gate.data_ptr(), _CODES[gate.dtype]
    if D == 0:
        return out
    _call("kda_residual_norm", (x.data_ptr(), pr, pq, pp, pg, pw, po, xs, gs, period, x.numel() // D, D,
                                rcode, qcode, pcode, gcode, wcode, 0, residual_scale, block_scale, eps), device)
    return out
