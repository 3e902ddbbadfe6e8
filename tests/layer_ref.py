"""Plain 64-bit forms of the layer operators for the tests, token by token
and row by row, on CPU tensors; each also gives the scale that rounding
errors are measured against (the same sum over absolute values)."""
from __future__ import annotations

import torch

F64 = torch.float64


def spans(B, T, cu):
    """(batch row, begin, end) of every sequence."""
    if cu is None:
        return [(r, 0, T) for r in range(B)]
    cu = [int(c) for c in cu]
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def silu(v):
    return v * torch.sigmoid(v)


def short_conv(x, weight, bias=None, activation="silu", l2norm=None, eps=1e-6, initial=None, cu=None):
    """(out, final state, scale of out) in 64 bits; rows outside every sequence are NaN."""
    B, T, D = x.shape
    W = weight.shape[1]
    x, w = x.to(F64), weight.to(F64)
    out = torch.full((B, T, D), float("nan"), dtype=F64)
    scale = torch.zeros(B, T, D, dtype=F64)
    ss = spans(B, T, cu)
    final = torch.zeros(len(ss), W - 1, D, dtype=F64)
    for n, (r, a, b) in enumerate(ss):
        past = initial[n].to(F64) if initial is not None else torch.zeros(W - 1, D, dtype=F64)
        line = torch.cat([past, x[r, a:b]])
        for t in range(b - a):
            terms = line[t:t + W] * w.T
            y, s = terms.sum(0), terms.abs().sum(0)
            if bias is not None:
                y, s = y + bias.to(F64), s + bias.to(F64).abs()
            if activation == "silu":
                y = silu(y)
            if l2norm:
                h = y.reshape(-1, l2norm)
                norm = torch.sqrt((h * h).sum(-1, keepdim=True) + eps)
                y = (h / norm).reshape(-1)
                s = (s.reshape(-1, l2norm) / norm).reshape(-1)
            out[r, a + t], scale[r, a + t] = y, s
        final[n] = line[len(line) - (W - 1):]
    return out, final, scale


def ssm(x, dt, b, c, A_log, D=None, dt_bias=None, z=None, initial=None, cu=None, softplus=True):
    """(out, final state, scale of out, scale of the state) in 64 bits."""
    B, T, H, P = x.shape
    G, N = b.shape[2:]
    x, dt, b, c = (v.to(F64) for v in (x, dt, b, c))
    if dt_bias is not None:
        dt = dt + dt_bias.to(F64)
    if softplus:
        dt = torch.nn.functional.softplus(dt, threshold=1e9)
    keep = torch.exp(-torch.exp(A_log.to(F64)) * dt)
    out, scale = torch.full((B, T, H, P), float("nan"), dtype=F64), torch.zeros(B, T, H, P, dtype=F64)
    ss = spans(B, T, cu)
    final, fscale = torch.zeros(len(ss), H, P, N, dtype=F64), torch.zeros(len(ss), H, P, N, dtype=F64)
    for n, (r, first, last) in enumerate(ss):
        S = initial[n].to(F64).clone() if initial is not None else torch.zeros(H, P, N, dtype=F64)
        M = S.abs()
        for t in range(first, last):
            bt, ct = (v[r, t].repeat_interleave(H // G, 0)[:, None] for v in (b, c))
            k, add = keep[r, t][:, None, None], (dt[r, t][:, None] * x[r, t])[..., None] * bt
            S, M = k * S + add, k * M + add.abs()
            y, s = (S * ct).sum(-1), (M * ct.abs()).sum(-1)
            if D is not None:
                y, s = y + D.to(F64)[:, None] * x[r, t], s + (D.to(F64)[:, None] * x[r, t]).abs()
            if z is not None:
                g = silu(z[r, t].to(F64))
                y, s = y * g, s * g.abs()
            out[r, t], scale[r, t] = y, s
        final[n], fscale[n] = S, M
    return out, final, scale, fscale


def gated_norm(x, gate, weight, group=None, eps=1e-6, activation="sigmoid", gate_first=False):
    x, w = x.to(F64), weight.to(F64)
    group = group or x.shape[-1]
    a = torch.ones_like(x)
    if gate is not None:
        a = torch.sigmoid(gate.to(F64)) if activation == "sigmoid" else silu(gate.to(F64))
    v = (x * a if gate_first else x).unflatten(-1, (-1, group))
    y = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)).flatten(-2) * w
    return y if gate_first else y * a


def residual_norm(x, residual, weight, post_weight=None, gate=None, block_scale=1.0, residual_scale=1.0, eps=1e-6):
    """(out, residual_out, scale of residual_out) in 64 bits; out is None without weight."""
    y = x.to(F64)
    if post_weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * post_weight.to(F64)
    if gate is not None:
        y = y * gate.to(F64)
    r, s = block_scale * y, (block_scale * y).abs()
    if residual is not None:
        r, s = r + residual_scale * residual.to(F64), s + (residual_scale * residual.to(F64)).abs()
    out = None
    if weight is not None:
        out = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * weight.to(F64)
    return out, r, s
