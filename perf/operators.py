"""The layer operators beside the KDA forward pass, as measurable cases.

Four operators surround a recurrent token mixer in a model: the short causal
convolution in front of it, the selective state space scan (the scalar-decay
sibling of the KDA recurrence, which a hybrid model alternates with it), the
gated norm of the mixer's heads, and the residual update with the norms
before and after a block.  ``listed`` and ``draw`` give cases, ``prepare``
the tensors a program holds before the call, ``run`` one call in the plain
form or (``own``) through the package, ``exact`` the definition in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
BF16 = torch.bfloat16
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _conv(name, B, T, D, W, l2norm=0, bias=False, activation="silu", state="bf16", weight="bf16", seqs=0,
          shortest=1):
    return dict(name=name, op="short_conv", B=B, T=T, D=D, W=W, l2norm=l2norm, bias=bias,
                activation=activation, state=state, weight=weight, seqs=seqs, shortest=shortest)


def _ssm(name, B, T, H, P, G, N, gate=True, state="fp32", initial=True, seqs=0, shortest=1):
    return dict(name=name, op="ssm_fwd", B=B, T=T, H=H, P=P, G=G, N=N, gate=gate, state=state, initial=initial,
                seqs=seqs, shortest=shortest)


def _gated(name, rows, D, group, activation, gate_first=False, weight="bf16"):
    return dict(name=name, op="gated_norm", rows=rows, D=D, group=group, activation=activation,
                gate_first=gate_first, weight=weight)


def _resid(name, B, T, D, post, gate, residual, weight="bf16"):
    return dict(name=name, op="residual_norm", B=B, T=T, D=D, post=post, gate=gate, residual=residual,
                weight=weight)


def listed():
    return [
        # one decoding step of 64 requests: q, k and v of 32 heads of 128, states carried
        _conv("conv_decode_b64", 64, 1, 12288, 4),
        # packed prompts, the query heads: convolution, SiLU and the per-head L2 norm that KDA expects
        _conv("conv_prompt_l2norm", 1, 19595, 4096, 4, l2norm=128, seqs=8, shortest=100),
        # one prompt through an odd channel count (inner channels and both projections of a small scan)
        _conv("conv_odd_channels", 1, 4097, 1283, 3, bias=True, state="fp32", weight="fp32"),
        # one decoding step of 64 requests: the state read and written once dominates
        _ssm("ssm_decode_b64", 64, 1, 32, 64, 1, 128),
        # packed prompts of U[100, 4000] tokens, bf16 states
        _ssm("ssm_varlen_n8", 1, 19595, 32, 64, 1, 128, state="bf16", seqs=8, shortest=100),
        # one long prompt, few heads, two groups: parallel only along the sequence
        _ssm("ssm_long_b1", 1, 8192, 16, 128, 2, 64, gate=False),
        # the throughput case: a batch of long sequences
        _ssm("ssm_large_b8", 8, 16384, 32, 64, 1, 128, initial=False),
        # one decoding step: the 32 heads of 64 requests
        _gated("gated_norm_decode", 64 * 32, 128, 128, "sigmoid"),
        # every head row of the large KDA workload
        _gated("gated_norm_large", 8 * 16384 * 32, 128, 128, "sigmoid"),
        # one decoding step of 64 requests, pre-norm only
        _resid("residual_norm_decode", 64, 1, 4096, False, "none", "bf16"),
        # prompts through a sandwich-norm block: post norm, per-channel gate, fp32 residual stream
        _resid("residual_norm_prompt", 8, 4096, 4096, True, "channel", "fp32"),
        # an odd width, gate per sequence
        _resid("residual_norm_odd", 3, 1001, 2561, True, "sequence", "bf16", weight="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("short_conv", "ssm_fwd", "gated_norm", "residual_norm"))
    if op == "short_conv":
        W = rng.choice((2, 3, 4, 4, 4))
        l2norm = rng.choice((0, 0, 64, 128))
        D = l2norm * _log_int(rng, 1, 12288 // l2norm) if l2norm else _log_int(rng, 16, 12288)
        T = rng.choice((1, _log_int(rng, 2, 16384)))
        B = _log_int(rng, 1, max(1, min(128, (1 << 27) // (T * D))))
        seqs = rng.randint(2, 16) if T > 64 and rng.random() < 0.5 else 0
        c = _conv("", 1 if seqs else B, T, D, W, l2norm, rng.random() < 0.5, rng.choice(("silu", "silu", "none")),
                  rng.choice(("bf16", "fp32")), rng.choice(("bf16", "fp32")), seqs)
    elif op == "ssm_fwd":
        G = rng.choice((1, 1, 2, 4))
        H = G * _log_int(rng, 1, 48 // G)
        P, N = rng.choice((32, 64, 64, 128)), rng.choice((32, 64, 128, 128, 256))
        T = rng.choice((1, rng.randint(2, 16), _log_int(rng, 17, 16384), _log_int(rng, 17, 16384)))
        B = _log_int(rng, 1, max(1, min(128, (1 << 27) // (T * H * P), (1 << 28) // (H * P * N))))
        seqs = rng.randint(2, 12) if T > 64 and rng.random() < 0.5 else 0
        c = _ssm("", 1 if seqs else B, T, H, P, G, N, rng.random() < 0.5, rng.choice(("bf16", "fp32")),
                 rng.random() < 0.7, seqs)
    elif op == "gated_norm":
        group = rng.choice((64, 128, 128, _log_int(rng, 16, 8192)))
        D = group * rng.choice((1, 1, 2, 4)) if group <= 2048 else group
        rows = _log_int(rng, 1, (1 << 28) // D)
        c = _gated("", rows, D, group, rng.choice(("sigmoid", "silu")), rng.random() < 0.5, rng.choice(("bf16", "fp32")))
    else:
        D = _log_int(rng, 64, 16384)
        T = rng.choice((1, _log_int(rng, 2, 16384)))
        B = _log_int(rng, 1, max(1, min(128, (1 << 27) // (T * D))))
        c = _resid("", B, T, D, rng.random() < 0.5, rng.choice(("none", "channel", "sequence", "token")),
                   rng.choice(("bf16", "fp32")), rng.choice(("bf16", "fp32")))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case, seed):
    """`seqs` lengths of at least `shortest` tokens that fill T tokens."""
    g = torch.Generator().manual_seed(seed)
    n, spare = case["seqs"], case["T"] - case["seqs"] * case["shortest"]
    share = torch.rand(n, generator=g, dtype=torch.float64) + 0.05
    cut = torch.floor(torch.cumsum(share, 0) / share.sum() * spare + 0.5).long()
    cut[-1] = spare
    return torch.diff(cut, prepend=cut.new_zeros(1)) + case["shortest"]


def _offsets(lengths):
    """Sequence offsets on the GPU (packed), or None (a batch of equal lengths)."""
    if lengths is None:
        return None
    return torch.cat([lengths.new_zeros(1), torch.cumsum(lengths, 0)]).to(DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape, dtype=BF16, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEVICE) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=DEVICE) * (hi - lo) + lo

    s = {"case": case}
    op = case["op"]
    if op in ("short_conv", "ssm_fwd"):
        lengths = _lengths(case, seed) if case["seqs"] else None
        s["longest"] = int(lengths.max()) if case["seqs"] else case["T"]
        s["cu"] = _offsets(lengths)
        B, T, n = case["B"], case["T"], case["seqs"] or case["B"]
    if op == "short_conv":
        D, W, wt = case["D"], case["W"], DTYPES[case["weight"]]
        s["x"] = normal(B, T, D)
        s["weight"] = normal(D, W, dtype=wt, scale=W ** -0.5)
        s["bias"] = normal(D, dtype=wt, scale=0.1) if case["bias"] else None
        s["initial"] = normal(n, W - 1, D).to(DTYPES[case["state"]])
        s["final"] = torch.empty_like(s["initial"])
        s["out"] = torch.empty_like(s["x"])
    elif op == "ssm_fwd":
        H, P, G, N, st = case["H"], case["P"], case["G"], case["N"], DTYPES[case["state"]]
        # x, b and c are slices of the convolution's output, z and dt of the input projection's
        xbc = normal(B, T, H * P + 2 * G * N)
        s["x"] = xbc[..., :H * P].unflatten(-1, (H, P))
        s["b"] = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        s["c"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
        if case["gate"]:
            zdt = normal(B, T, H * P + H)
            s["z"], s["dt"] = zdt[..., :H * P].unflatten(-1, (H, P)), zdt[..., H * P:]
        else:
            s["z"], s["dt"] = None, normal(B, T, H)
        s["A_log"] = torch.log(uniform(H, lo=1.0, hi=16.0))
        step = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
        s["D"] = uniform(H, lo=0.5, hi=1.5)
        s["initial"] = normal(n, H, P, N, dtype=st, scale=0.3) if case["initial"] else None
        s["final"] = torch.empty(n, H, P, N, dtype=st, device=DEVICE)
        s["out"] = torch.empty(B, T, H, P, dtype=BF16, device=DEVICE)
    elif op == "gated_norm":
        rows, D = case["rows"], case["D"]
        s["x"], s["gate"] = normal(rows, D), normal(rows, D)
        s["weight"] = uniform(D, lo=0.5, hi=1.5).to(DTYPES[case["weight"]])
        s["out"] = torch.empty_like(s["x"])
    else:
        B, T, D, wt = case["B"], case["T"], case["D"], DTYPES[case["weight"]]
        s["x"] = normal(B, T, D)
        s["residual"] = normal(B, T, D, dtype=DTYPES[case["residual"]], scale=3.0)
        s["post_weight"] = uniform(D, lo=0.5, hi=1.5).to(wt) if case["post"] else None
        s["weight"] = uniform(D, lo=0.5, hi=1.5).to(wt)
        shape = {"none": None, "channel": (D,), "sequence": (B, 1, D), "token": (B, T, D)}[case["gate"]]
        s["gate"] = normal(*shape, scale=0.5) if shape else None
        s["out"] = torch.empty_like(s["x"])
        s["residual_out"] = torch.empty_like(s["residual"])
    return s


# the constants of the operators' keyword arguments that every case uses
EPS = 1e-6
BLOCK_SCALE, RESIDUAL_SCALE = 0.7, 0.9


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import gated_delta_rule_36_amd as kda
        if op == "short_conv":
            kda.short_conv(s["x"], s["weight"], s["out"], s["bias"],
                           activation=None if case["activation"] == "none" else case["activation"],
                           l2norm=case["l2norm"] or None, l2norm_eps=EPS, initial_state=s["initial"],
                           final_state=s["final"], cu_seqlens=s["cu"], check_cu_seqlens=False)
            return {"out": s["out"], "final_state": s["final"]}
        if op == "ssm_fwd":
            kda.ssm_fwd(s["x"], s["dt"], s["b"], s["c"], s["out"], s["A_log"], s["D"], s["dt_bias"], s["z"],
                        initial_state=s["initial"], final_state=s["final"], cu_seqlens=s["cu"],
                        check_cu_seqlens=False)
            return {"out": s["out"], "final_state": s["final"]}
        if op == "gated_norm":
            kda.gated_norm(s["x"], s["gate"], s["weight"], s["out"], group_size=case["group"], eps=EPS,
                           activation=case["activation"], gate_first=case["gate_first"])
            return {"out": s["out"]}
        kda.residual_norm(s["x"], s["residual"], s["weight"], s["out"], s["residual_out"],
                          post_weight=s["post_weight"], gate=s["gate"], block_scale=BLOCK_SCALE,
                          residual_scale=RESIDUAL_SCALE, eps=EPS)
        return {"out": s["out"], "residual_out": s["residual_out"]}
    return {"short_conv": _plain_conv, "ssm_fwd": _plain_ssm, "gated_norm": _plain_gated,
            "residual_norm": _plain_resid}[op](s)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _places(case, cu):
    """For every packed row its sequence and its place in it, and the sequences' offsets."""
    if cu is None:
        cu = torch.arange(case["B"] + 1, device=DEVICE) * case["T"]
    rows = torch.arange(case["B"] * case["T"], device=DEVICE)
    n = torch.searchsorted(cu, rows, right=True) - 1
    return rows, n, rows - cu[n], cu


def _taps(x, state, rows, n, i, W, j):
    """Tap j of every row: the input W - 1 - j tokens earlier, from the state before the sequence's start."""
    past = (i + j < W - 1)[:, None]
    return torch.where(past, state[n, (i + j).clamp(max=W - 2)], x[(rows + j - (W - 1)).clamp(min=0)])


def _plain_conv(s):
    case = s["case"]
    W, D = case["W"], case["D"]
    rows, n, i, cu = _places(case, s["cu"])
    x, state, w = s["x"].reshape(-1, D).float(), s["initial"].float(), s["weight"].float()
    y = sum(_taps(x, state, rows, n, i, W, j) * w[:, j] for j in range(W))
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if case["activation"] == "silu":
        y = _silu(y)
    if case["l2norm"]:
        h = y.unflatten(-1, (-1, case["l2norm"]))
        y = (h * torch.rsqrt((h * h).sum(-1, keepdim=True) + EPS)).flatten(-2)
    # the state after a sequence: the last W - 1 of (state, inputs)
    at = torch.diff(cu)[:, None] + torch.arange(W - 1, device=DEVICE)
    seq = torch.arange(len(cu) - 1, device=DEVICE)[:, None].expand_as(at)
    final = torch.where((at < W - 1)[..., None], state[seq, at.clamp(max=W - 2)],
                        x[(cu[:-1, None] + at - (W - 1)).clamp(min=0)])
    return {"out": y.reshape(s["x"].shape).to(BF16), "final_state": final.to(s["initial"].dtype)}


def _padded(s):
    """Row numbers [n, longest] of a packed batch and which of them exist; None for a batch of equal lengths."""
    cu = s["cu"]
    if cu is None:
        return None
    t = torch.arange(s["longest"], device=DEVICE)
    return (cu[:-1, None] + t).clamp(max=s["case"]["T"] - 1), t < torch.diff(cu)[:, None]


def _plain_ssm(s):
    """Chunks of Q tokens: products inside a chunk, the chunks' states joined by one product over chunks."""
    case = s["case"]
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    pad = _padded(s)
    take = (lambda v: v[0][pad[0]]) if pad else (lambda v: v)
    x, b, c = (take(s[k]).float() for k in "xbc")
    dt = torch.logaddexp(take(s["dt"]).float() + s["dt_bias"], x.new_zeros(()))
    if pad:
        dt = dt * pad[1][..., None]  # a row past the end neither decays nor writes
    n, T = dt.shape[:2]
    Q = min(256, T)
    k = -(-T // Q)

    def chunks(v):
        if k * Q > T:
            v = torch.cat([v, v.new_zeros(n, k * Q - T, *v.shape[2:])], 1)
        return v.unflatten(1, (k, Q))

    xc, bc, cc, dc = chunks(x), chunks(b), chunks(c), chunks(dt)
    # log decays up to and with each token; sums in 64 bits, since their differences are what counts
    g = torch.cumsum(-torch.exp(s["A_log"].double()) * dc.double(), 2).movedim(-1, 2)     # [n, k, H, Q]
    lower = torch.ones(Q, Q, dtype=torch.bool, device=DEVICE).tril()
    decay = torch.where(lower, g[..., :, None] - g[..., None, :], -math.inf).float().exp()  # [n, k, H, Q, Q]
    bg, cg = bc.movedim(3, 2).contiguous(), cc.movedim(3, 2).contiguous()                  # [n, k, G, Q, N]
    scores = torch.matmul(cg, bg.transpose(-1, -2)).repeat_interleave(H // G, 2)
    xd = (xc * dc[..., None]).movedim(3, 2)                                                # [n, k, H, Q, P]
    y = torch.matmul(scores * decay, xd)
    # each chunk's own state, then the state in front of each chunk
    to_end = torch.exp(g[..., -1:] - g).float()
    own_state = torch.matmul((xd * to_end[..., None]).reshape(n, k, G, H // G, Q, P).transpose(-1, -2).flatten(3, 4),
                             bg).reshape(n, k, H, P * N)
    first = s["initial"].float() if s["initial"] is not None else x.new_zeros(n, H, P, N)
    every = torch.cat([first.reshape(n, 1, H, P * N), own_state], 1).movedim(2, 1)         # [n, H, k+1, P N]
    e = torch.cumsum(torch.cat([g.new_zeros(n, H, 1), g[..., -1].movedim(2, 1)], -1), -1)  # [n, H, k+1]
    joined = torch.ones(k + 1, k + 1, dtype=torch.bool, device=DEVICE).tril()
    span = torch.where(joined, e[..., :, None] - e[..., None, :], -math.inf).exp().float()
    before = torch.matmul(span, every)                                                     # [n, H, k+1, P N]
    start = before[:, :, :k].movedim(1, 2).reshape(n, k, G, H // G * P, N)
    carried = torch.matmul(cg, start.transpose(-1, -2)).unflatten(-1, (H // G, P))         # [n, k, G, Q, H/G, P]
    y = y + carried.movedim(4, 3).flatten(2, 3) * torch.exp(g).float()[..., None]
    y = y.movedim(2, 3).flatten(1, 2)[:, :T] + x * s["D"][:, None]
    if s["z"] is not None:
        y = y * _silu(take(s["z"]).float())
    y = y[pad[1]][None] if pad else y
    return {"out": y.to(BF16), "final_state": before[:, :, k].reshape(n, H, P, N).to(s["final"].dtype)}


def _rms(v, weight):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * weight


def _plain_gated(s):
    case = s["case"]
    x, gate, w = (s[k].float().unflatten(-1, (-1, case["group"])) for k in ("x", "gate", "weight"))
    gate = _silu(gate) if case["activation"] == "silu" else 1 / (1 + torch.exp(-gate))
    y = _rms(x * gate, w) if case["gate_first"] else _rms(x, w) * gate
    return {"out": y.flatten(-2).to(BF16)}


def _plain_resid(s):
    y = s["x"].float()
    if s["post_weight"] is not None:
        y = _rms(y, s["post_weight"].float())
    if s["gate"] is not None:
        y = y * s["gate"].float()
    r = RESIDUAL_SCALE * s["residual"].float() + BLOCK_SCALE * y
    return {"out": _rms(r, s["weight"].float()).to(BF16), "residual_out": r.to(s["residual"].dtype)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "short_conv":
        cells, n = case["B"] * case["T"] * case["D"], case["seqs"] or case["B"]
        wb = 2 if case["weight"] == "bf16" else 4
        state = n * (case["W"] - 1) * case["D"] * (2 if case["state"] == "bf16" else 4)
        return {"bytes": 4 * cells + case["D"] * (case["W"] + case["bias"]) * wb + 2 * state,
                "flops": cells * (2 * case["W"] + 5)}
    if op == "ssm_fwd":
        H, P, G, N, tokens = case["H"], case["P"], case["G"], case["N"], case["B"] * case["T"]
        state = (case["seqs"] or case["B"]) * H * P * N * (2 if case["state"] == "bf16" else 4)
        return {"bytes": tokens * 2 * (H * P * (3 if case["gate"] else 2) + 2 * G * N + H) + 12 * H
                + state * (2 if case["initial"] else 1),
                "flops": tokens * H * P * (5 * N + 8)}
    if op == "gated_norm":
        return {"bytes": 6 * case["rows"] * case["D"] + case["D"] * (2 if case["weight"] == "bf16" else 4),
                "flops": 10 * case["rows"] * case["D"]}
    cells, D = case["B"] * case["T"] * case["D"], case["D"]
    gate = {"none": 0, "channel": D, "sequence": case["B"] * D, "token": cells}[case["gate"]]
    return {"bytes": cells * (4 + 2 * (2 if case["residual"] == "bf16" else 4)) + 2 * gate
            + D * (2 if case["weight"] == "bf16" else 4) * (2 if case["post"] else 1),
            "flops": 12 * cells}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one token or one row at a time where the plain form uses products
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"short_conv": _exact_conv, "ssm_fwd": _exact_ssm, "gated_norm": _exact_gated,
            "residual_norm": _exact_resid}[case["op"]](s)


def _sequences(s):
    case = s["case"]
    if s["cu"] is None:
        return [(r, 0, case["T"]) for r in range(case["B"])]
    cu = s["cu"].tolist()
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def _exact_conv(s):
    case = s["case"]
    W, w = case["W"], s["weight"].double()
    out, final = torch.empty(s["x"].shape, dtype=torch.float64, device=DEVICE), torch.empty_like(s["final"])
    for n, (row, a, b) in enumerate(_sequences(s)):
        line = torch.cat([s["initial"][n].double(), s["x"][row, a:b].double()])
        y = torch.zeros(b - a, case["D"], dtype=torch.float64, device=DEVICE)
        for j in range(W):
            y += line[j:j + b - a] * w[:, j]
        if s["bias"] is not None:
            y += s["bias"].double()
        if case["activation"] == "silu":
            y = y * torch.sigmoid(y)
        if case["l2norm"]:
            h = y.unflatten(-1, (-1, case["l2norm"]))
            y = (h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) + EPS)).flatten(-2)
        out[row, a:b] = y
        final[n] = line[len(line) - (W - 1):].to(final.dtype)
    return {"out": out, "final_state": final.double()}


def _exact_ssm(s):
    case = s["case"]
    H, P, G, N = case["H"], case["P"], case["G"], case["N"]
    spans = _sequences(s)
    lengths = torch.tensor([b - a for _, a, b in spans])
    longest = int(lengths.max())
    n = len(spans)
    flat = torch.stack([row * case["T"] + (a + torch.arange(longest)).clamp(max=max(a, b - 1))
                        for row, a, b in spans]).to(DEVICE)                                 # [n, longest]
    alive = (torch.arange(longest) < lengths[:, None]).to(DEVICE)
    rows = lambda v: v.reshape(-1, *v.shape[2:])  # noqa: E731
    dt = torch.nn.functional.softplus(rows(s["dt"]).double() + s["dt_bias"].double(), threshold=1000.0)
    keep = torch.exp(-torch.exp(s["A_log"].double()) * dt)
    h = s["initial"].double() if s["initial"] is not None else torch.zeros(n, H, P, N, dtype=torch.float64, device=DEVICE)
    h = h.clone()
    out = torch.empty(case["B"] * case["T"], H, P, dtype=torch.float64, device=DEVICE)
    x, b, c = rows(s["x"]), rows(s["b"]), rows(s["c"])
    for t in range(longest):
        at, on = flat[:, t], alive[:, t]
        step, xt = (dt[at] * on[:, None])[..., None], x[at].double()
        h = torch.where(on[:, None], keep[at], 1.0)[..., None, None] * h
        bt, ct = (v[at].double().repeat_interleave(H // G, 1) for v in (b, c))
        h += (step * xt)[..., None] * bt[:, :, None]
        yt = (h * ct[:, :, None]).sum(-1) + s["D"].double()[:, None] * xt
        if s["z"] is not None:
            zt = rows(s["z"])[at].double()
            yt = yt * zt * torch.sigmoid(zt)
        if case["seqs"]:
            yt = torch.where(on[:, None, None], yt, out[at])
        out[at] = yt
    return {"out": out.reshape(case["B"], case["T"], H, P), "final_state": h}


def _exact_gated(s):
    case = s["case"]
    x, gate = s["x"].double(), s["gate"].double()
    gate = gate * torch.sigmoid(gate) if case["activation"] == "silu" else torch.sigmoid(gate)
    v = (x * gate if case["gate_first"] else x).unflatten(-1, (-1, case["group"]))
    y = (v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + EPS)).flatten(-2) * s["weight"].double()
    return {"out": y if case["gate_first"] else y * gate}


def _exact_resid(s):
    y = s["x"].double()
    if s["post_weight"] is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + EPS) * s["post_weight"].double()
    if s["gate"] is not None:
        y = y * s["gate"].double()
    r = s["residual"].double() * RESIDUAL_SCALE + y * BLOCK_SCALE
    out = r / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + EPS) * s["weight"].double()
    return {"out": out, "residual_out": r}
