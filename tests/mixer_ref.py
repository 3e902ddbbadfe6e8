"""Plain 64-bit forms of the delta rule and the attention layers' operators for
the tests, token by token, on CPU tensors, with the bounds on rounding errors
that the tests hold the kernels to."""
from __future__ import annotations

import math

import torch

from layer_ref import F64, spans

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


def delta(q, k, v, g, beta, scale, A_log, dt_bias=None, initial=None, cu=None):
    """(out, final state, bound on out before it is rounded, bound on the norm of the final state's rows).

    S <- a S, u = b (v - S k), S <- S + u k^T, out = scale S q with S [V, K].

    The bounds: let M be the sum of the absolute values of what S is made of
    (M <- a M + |u| |k|^T).  A kernel forms S k from K products and, in a chunk,
    from up to 64 earlier tokens whose own sums it solves for in up to 64
    steps, so S k is off by at most (K + 128) 2^-24 M |k|, u by that and a few
    roundings of b and v, and S by |u| |k|^T's and a's.  An error e of a row of
    S goes on as a (I - b k k^T) e, which for |k| <= 1 is no longer than e."""
    B, T, H, V = v.shape
    G, K = k.shape[2:]
    q, k, v, g, beta = (x.to(F64) for x in (q, k, v, g, beta))
    if dt_bias is not None:
        g = g + dt_bias.to(F64)
    a = torch.exp(-torch.exp(A_log.to(F64)) * torch.nn.functional.softplus(g, threshold=1e9))
    b = torch.sigmoid(beta)
    ss = spans(B, T, cu)
    out = torch.full((B, T, H, V), float("nan"), dtype=F64)
    bound = torch.zeros(B, T, H, V, dtype=F64)
    final, fbound = torch.zeros(len(ss), H, V, K, dtype=F64), torch.zeros(len(ss), H, V, dtype=F64)
    for n, (r, first, last) in enumerate(ss):
        S = initial[n].to(F64).clone() if initial is not None else torch.zeros(H, V, K, dtype=F64)
        M, E = S.abs(), torch.zeros(H, V, dtype=F64)
        for t in range(first, last):
            qt, kt = (x[r, t].repeat_interleave(H // G, 0)[:, None] for x in (q, k))  # [H, 1, K]
            at, bt = a[r, t][:, None], b[r, t][:, None]
            S, M = at[..., None] * S, at[..., None] * M
            u = bt * (v[r, t] - (S * kt).sum(-1))
            du = U32 * ((K + 128) * bt * ((M * kt.abs()).sum(-1) + v[r, t].abs()) + 16 * u.abs())
            norm = kt.norm(dim=-1)
            E = at * E + du * norm + 16 * U32 * M.norm(dim=-1)
            S, M = S + u[..., None] * kt, M + u.abs()[..., None] * kt.abs()
            out[r, t] = scale * (S * qt).sum(-1)
            bound[r, t] = abs(scale) * (E * qt.norm(dim=-1) + 2.0 ** -16 * (M * qt.abs()).sum(-1))
        final[n], fbound[n] = S, E
    return out, final, bound, fbound


def rms(x, weight, eps):
    x = x.to(F64)
    return x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(F64)


def rotary(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False, scale=1.0):
    """(out, bound before it is rounded) of x [B, T, H, D].

    The norm's factors are good to a few 2^-24, cosine and sine of a reduced
    angle to 2^-22 of 1."""
    y = rms(x, weight, eps)
    if positions is None:
        return y, 16 * U32 * y.abs()
    R = 2 * len(inv_freq)
    angle = positions.to(F64)[..., None] * inv_freq.to(F64)
    cos, sin = torch.cos(angle)[:, :, None] * scale, torch.sin(angle)[:, :, None] * scale
    i = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    j = i + 1 if interleaved else i + R // 2
    out, size = y.clone(), y.abs()
    out[..., i], out[..., j] = y[..., i] * cos - y[..., j] * sin, y[..., j] * cos + y[..., i] * sin
    both = (y[..., i].abs() + y[..., j].abs()) * abs(scale)
    size[..., i], size[..., j] = both, both
    return out, 32 * U32 * size


def append(k, v, k_cache, v_cache, slots, positions=None, inv_freq=None, weight=None, **kw):
    """(k_cache, v_cache, bound on k_cache) after the call; slots outside the cache are left out."""
    y, bound = rotary(k, positions, inv_freq, weight, **kw)
    kc, vc, kb = k_cache.to(F64), v_cache.to(F64), torch.zeros(k_cache.shape, dtype=F64)
    pages, size = kc.shape[:2]
    for b in range(k.shape[0]):
        for t in range(k.shape[1]):
            s = int(slots[b, t])
            if 0 <= s < pages * size:
                kc[s // size, s % size], vc[s // size, s % size], kb[s // size, s % size] = y[b, t], v[b, t].to(F64), bound[b, t]
    return kc, vc, kb


def attention(q, k_cache, v_cache, table, lengths, scale, window=None):
    """(out, lse, bound on out before it is rounded, bound on lse).

    A score of D products is off by e <= (D + 8) 2^-24 |scale| sum |q| |k|, a
    probability by 2 e and what its parts leave out (the first is cut from 1 -
    2^-10 of it and leaves less than 2^-7 of the number's power of two, of which
    the second holds all but half a step, 2^-9 of it: 2^-16), a sum of n of
    them by n 2^-24 (splits and waves only make it less)."""
    N, Hq, D = q.shape
    pages, size, Hk = k_cache.shape[:3]
    out, bound = torch.zeros(N, Hq, D, dtype=F64), torch.zeros(N, Hq, D, dtype=F64)
    lse, lbound = torch.full((N, Hq), -math.inf, dtype=F64), torch.zeros(N, Hq, dtype=F64)
    for n in range(N):
        length = min(max(int(lengths[n]), 0), table.shape[1] * size)
        first = max(0, length - window) if window else 0
        t = torch.arange(first, length)
        page = table[n].long()[t // size] if length > first else t
        keep = (page >= 0) & (page < pages)
        t, page = t[keep], page[keep]
        if len(t) == 0:
            continue
        k, v = (c[page, t % size].to(F64).movedim(1, 0).repeat_interleave(Hq // Hk, 0) for c in (k_cache, v_cache))
        x = q[n].to(F64)
        s = scale * (k * x[:, None]).sum(-1)                                        # [Hq, t]
        e = (D + 8) * U32 * abs(scale) * (k.abs() * x.abs()[:, None]).sum(-1).amax(-1, keepdim=True)
        e = e + 4 * U32 * s.abs().amax(-1, keepdim=True)
        lse[n] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[n][:, None])[..., None]
        off = 2 * e + 2.0 ** -16 + (len(t) + 16) * U32
        out[n], bound[n] = (p * v).sum(1), off * (p * v.abs()).sum(1)
        lbound[n] = (e + (len(t) + 16) * U32)[:, 0] + 8 * U32 * lse[n].abs()
    return out, lse, bound, lbound


def check(name, got, want, bound):
    """|got - want| within bound and half a step of got's type; NaN only where want has it."""
    got = got.detach().cpu()
    half = torch.finfo(got.dtype).eps / 2
    got = got.to(F64)
    assert torch.equal(got.isnan(), want.isnan()), f"{name}: NaN in other places"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), f"{name}: infinities"
    got, want, bound = got[fine], want[fine], bound.expand(fine.shape)[fine]
    # the rounding is half a step of what is rounded, which is off by the bound itself
    room = half * (want.abs() + bound) + bound + 2.0 ** -133
    far = (got - want).abs() / room
    worst = float(far.max()) if far.numel() else 0.0
    print(f"[check] {name}: worst {worst:.3f} of what is allowed", flush=True)
    assert worst <= 1.0, f"{name}: {worst} of what is allowed"
