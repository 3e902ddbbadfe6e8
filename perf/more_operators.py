"""The gated delta rule and the attention layers beside it, as measurable cases.

A hybrid decoder alternates recurrent mixers with full attention.  Four
operators serve it: the gated delta rule with one decay per head over prompts
and single tokens, the per-head norms and position rotation of queries and
keys, the append of keys and values to a paged cache, and the attention of one
new token over that cache.  ``listed`` and ``draw`` give cases, ``prepare``
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

def _delta(name, B, T, G, H, K, V, state="fp32", initial=True, seqs=0, shortest=1):
    return dict(name=name, op="delta_fwd", B=B, T=T, G=G, H=H, K=K, V=V, state=state, initial=initial, seqs=seqs,
                shortest=shortest)


def _rotary(name, B, T, Hq, Hk, D, R, norm=True, interleaved=False, weight="bf16", start=0):
    return dict(name=name, op="qk_norm_rotary", B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, norm=norm,
                interleaved=interleaved, weight=weight, start=start)


def _append(name, B, T, H, D, page, pages, R, norm=True, start=0):
    return dict(name=name, op="append_kv", B=B, T=T, H=H, D=D, page=page, pages=pages, R=R, norm=norm, start=start)


def _attn(name, seqs, tokens, Hq, Hk, D, page, shortest=1, window=0):
    return dict(name=name, op="paged_attention", seqs=seqs, tokens=tokens, Hq=Hq, Hk=Hk, D=D, page=page,
                shortest=shortest, window=window)


def listed():
    return [
        # one decoding step of 64 requests: the fp32 state read and written once dominates
        _delta("delta_decode_b64", 64, 1, 16, 32, 128, 128),
        # packed prompts of unequal lengths, bf16 states
        _delta("delta_varlen_n8", 1, 19595, 16, 32, 128, 128, state="bf16", seqs=8, shortest=100),
        # one long prompt of few narrow heads, an odd length: little runs in parallel
        _delta("delta_long_b1", 1, 8191, 4, 12, 64, 96),
        # the throughput case: a batch of long sequences
        _delta("delta_large_b8", 8, 16384, 16, 32, 128, 128, initial=False),
        # one decoding step of 64 requests far into their contexts
        _rotary("rotary_decode_b64", 64, 1, 32, 4, 128, 128, start=100000),
        # prompts, a quarter of each head rotated
        _rotary("rotary_prompt", 8, 4096, 32, 8, 128, 32, weight="fp32"),
        # one decoding step of 64 requests: 8 key and value heads each
        _append("append_decode_b64", 64, 1, 8, 128, 64, 1024, 128, start=100000),
        # a packed prompt into small pages that lie anywhere
        _append("append_prompt", 1, 19595, 8, 128, 16, 2048, 128),
        # one request with a short context: latency
        _attn("attention_short_b1", 1, 333, 16, 16, 64, 16),
        # 64 requests of unequal lengths, eight query heads a key head
        _attn("attention_decode_b64", 64, 262144, 32, 4, 128, 64, shortest=100),
        # one request with a long context: parallel only along its length
        _attn("attention_long_b1", 1, 131071, 16, 2, 128, 16),
        # the throughput case: as many long contexts as a server keeps
        _attn("attention_large_b64", 64, 1048576, 32, 8, 128, 64, shortest=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("delta_fwd", "delta_fwd", "qk_norm_rotary", "append_kv", "paged_attention", "paged_attention"))
    if op == "delta_fwd":
        G = rng.choice((1, 2, 4, 8, 16))
        H = G * rng.choice((1, 2, 3))
        K, V = rng.choice((64, 128, 128, 256)), rng.choice((32, 64, 96, 128, 128, 256))
        T = rng.choice((1, rng.randint(2, 32), _log_int(rng, 33, 16384), _log_int(rng, 33, 16384)))
        B = _log_int(rng, 1, max(1, min(128, (1 << 28) // (T * H * max(K, V)), (1 << 28) // (H * K * V))))
        seqs = rng.randint(2, 12) if T > 64 and rng.random() < 0.5 else 0
        c = _delta("", 1 if seqs else B, T, G, H, K, V, rng.choice(("bf16", "fp32")), rng.random() < 0.7, seqs)
    elif op in ("qk_norm_rotary", "append_kv"):
        D = rng.choice((64, 80, 96, 128, 128, 128, 192, 256))
        R = rng.choice((D, D, D // 2, D // 4))
        T = rng.choice((1, _log_int(rng, 2, 16384)))
        start = rng.choice((0, _log_int(rng, 1, 1000000)))
        Hk = _log_int(rng, 1, 16)
        if op == "qk_norm_rotary":
            Hq = Hk * rng.choice((1, 2, 4, 8))
            B = _log_int(rng, 1, max(1, min(128, (1 << 27) // (T * (Hq + Hk) * D))))
            c = _rotary("", B, T, Hq, Hk, D, R, rng.random() < 0.7, rng.random() < 0.4, rng.choice(("bf16", "fp32")),
                        start)
        else:
            B = _log_int(rng, 1, max(1, min(128, (1 << 26) // (T * Hk * D))))
            page = rng.choice((16, 32, 64, 128))
            c = _append("", B, T, Hk, D, page, -(-B * T // page) + rng.randint(1, 64), R, rng.random() < 0.7, start)
    else:
        Hk = _log_int(rng, 1, 16)
        Hq = Hk * rng.choice((1, 1, 2, 4, 5, 8, 16))
        D = rng.choice((64, 96, 128, 128, 128, 192, 256))
        seqs = _log_int(rng, 1, 128)
        tokens = _log_int(rng, seqs, max(seqs, min(1 << 20, (1 << 30) // (Hk * D))))
        c = _attn("", seqs, tokens, Hq, Hk, D, rng.choice((16, 32, 64, 128)), window=rng.choice((0, 0, 0, 1024)))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(n, total, shortest, seed):
    """`n` lengths of at least `shortest` tokens that fill `total` tokens."""
    g = torch.Generator().manual_seed(seed)
    spare = total - n * shortest
    share = torch.rand(n, generator=g, dtype=torch.float64) + 0.05
    cut = torch.floor(torch.cumsum(share, 0) / share.sum() * spare + 0.5).long()
    cut[-1] = spare
    return torch.diff(cut, prepend=cut.new_zeros(1)) + shortest


def _silu(v):
    return v / (1 + torch.exp(-v))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape, dtype=BF16, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEVICE) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=DEVICE) * (hi - lo) + lo

    s = {"case": case}
    op = case["op"]
    if op == "delta_fwd":
        B, T, G, H, K, V, st = *(case[c] for c in "BTGHKV"), DTYPES[case["state"]]
        lengths = _lengths(case["seqs"], T, case["shortest"], seed) if case["seqs"] else None
        n = case["seqs"] or B
        s["longest"] = int(lengths.max()) if case["seqs"] else T
        s["cu"] = torch.cat([lengths.new_zeros(1), torch.cumsum(lengths, 0)]).to(DEVICE) if case["seqs"] else None
        # the queries and keys of one convolution with its L2 norm, the values of another
        qk = _silu(normal(B, T, 2 * G, K, dtype=torch.float32))
        qk = (qk * torch.rsqrt((qk * qk).sum(-1, keepdim=True) + 1e-6)).to(BF16)
        s["q"], s["k"] = qk[:, :, :G], qk[:, :, G:]
        s["v"] = _silu(normal(B, T, H, V, dtype=torch.float32)).to(BF16)
        # gate and beta logits are slices of the input projection's
        gb = normal(B, T, 2 * H)
        s["g"], s["beta"] = gb[..., :H], gb[..., H:]
        s["scale"] = K ** -0.5
        s["A_log"] = torch.log(uniform(H, lo=1.0, hi=16.0))
        step = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
        s["initial"] = normal(n, H, V, K, dtype=st, scale=0.3) if case["initial"] else None
        s["final"] = torch.empty(n, H, V, K, dtype=st, device=DEVICE)
        s["out"] = torch.empty(B, T, H, V, dtype=BF16, device=DEVICE)
        return s
    if op == "paged_attention":
        n, Hq, Hk, D, page = case["seqs"], case["Hq"], case["Hk"], case["D"], case["page"]
        lengths = _lengths(n, case["tokens"], case["shortest"], seed)
        used = -(-lengths // page)
        width, pages = int(used.max()), int(used.sum()) + 1
        # pages lie anywhere in the cache; the table's unused entries name none
        order = torch.randperm(pages, generator=gen, device=DEVICE)[:pages - 1].int()
        table = torch.full((n, width), -1, dtype=torch.int32, device=DEVICE)
        table[torch.arange(width, device=DEVICE) < used.to(DEVICE)[:, None]] = order
        s["table"], s["lengths"] = table, lengths.int().to(DEVICE)
        s["q"] = normal(n, Hq, D)
        s["k_cache"], s["v_cache"] = normal(pages, page, Hk, D), normal(pages, page, Hk, D)
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(n, Hq, D, dtype=BF16, device=DEVICE)
        s["lse"] = torch.empty(n, Hq, dtype=torch.float32, device=DEVICE)
        return s
    B, T, D, R = case["B"], case["T"], case["D"], case["R"]
    s["positions"] = torch.arange(T, device=DEVICE).expand(B, T) + case["start"]
    if T == 1:
        s["positions"] = s["positions"] + torch.randint(0, 4096, (B, 1), generator=gen, device=DEVICE)
    s["positions"] = s["positions"].contiguous()
    s["inv_freq"] = 10000.0 ** (-torch.arange(0, R, 2, device=DEVICE, dtype=torch.float32) / R)
    if op == "qk_norm_rotary":
        Hq, Hk, wt = case["Hq"], case["Hk"], DTYPES[case["weight"]]
        qkv = normal(B, T, Hq + 2 * Hk, D)  # one projection's output
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        s["q_weight"], s["k_weight"] = ((uniform(D, lo=0.5, hi=1.5).to(wt), uniform(D, lo=0.5, hi=1.5).to(wt))
                                        if case["norm"] else (None, None))
        s["q_out"] = torch.empty(B, T, Hq, D, dtype=BF16, device=DEVICE)
        s["k_out"] = torch.empty(B, T, Hk, D, dtype=BF16, device=DEVICE)
    else:
        H, page, pages = case["H"], case["page"], case["pages"]
        kv = normal(B, T, 2 * H, D)
        s["k"], s["v"] = kv[:, :, :H], kv[:, :, H:]
        s["weight"] = uniform(D, lo=0.5, hi=1.5).to(BF16) if case["norm"] else None
        s["k_cache"], s["v_cache"] = normal(pages, page, H, D), normal(pages, page, H, D)
        if T == 1:  # every request's newest page is another one
            at = torch.randperm(pages, generator=gen, device=DEVICE)[:B] if pages >= B else None
            where = (at * page + torch.randint(0, page, (B,), generator=gen, device=DEVICE) if at is not None
                     else torch.randperm(pages * page, generator=gen, device=DEVICE)[:B])
            s["slots"] = where[:, None].contiguous()
        else:  # prompts fill page after page
            t = torch.arange(B * T, device=DEVICE)
            s["slots"] = (torch.randperm(pages, generator=gen, device=DEVICE)[t // page] * page + t % page).view(B, T)
    return s


EPS = 1e-6


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import gated_delta_rule_36_amd as kda
        if op == "delta_fwd":
            kda.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["out"], s["A_log"], s["dt_bias"],
                          initial_state=s["initial"], final_state=s["final"], cu_seqlens=s["cu"],
                          check_cu_seqlens=False)
            return {"out": s["out"], "final_state": s["final"]}
        if op == "qk_norm_rotary":
            kda.qk_norm_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"], s["q_weight"],
                               s["k_weight"], eps=EPS, interleaved=case["interleaved"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "append_kv":
            kda.append_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["inv_freq"],
                          s["weight"], eps=EPS)
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        kda.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["out"], s["scale"],
                            lse=s["lse"], window=case["window"] or None)
        return {"out": s["out"], "lse": s["lse"]}
    return {"delta_fwd": _plain_delta, "qk_norm_rotary": _plain_rotary, "append_kv": _plain_append,
            "paged_attention": _plain_attention}[op](s)


CHUNK = 64


def _plain_delta(s):
    """Chunks of 64 tokens: the tokens of a chunk are solved together, the state is carried from chunk to chunk."""
    case = s["case"]
    G, H, K, V, T = case["G"], case["H"], case["K"], case["V"], s["longest"]
    pad = None
    if s["cu"] is not None:
        t = torch.arange(T, device=DEVICE)
        pad = (s["cu"][:-1, None] + t).clamp(max=case["T"] - 1), t < torch.diff(s["cu"])[:, None]
    take = (lambda v: v[0][pad[0]]) if pad else (lambda v: v)
    q, k, v, raw, logit = (take(s[c]).float() for c in ("q", "k", "v", "g", "beta"))
    # log decay and write strength; a row past the end neither decays nor writes
    g = -torch.exp(s["A_log"]) * torch.logaddexp(raw + s["dt_bias"], raw.new_zeros(()))
    beta = 1 / (1 + torch.exp(-logit))
    if pad:
        g, beta = g * pad[1][..., None], beta * pad[1][..., None]
    n = g.shape[0]
    Q = min(CHUNK, 1 << (T - 1).bit_length())
    c = -(-T // Q)

    def chunks(x):  # [n, T, heads, ...] -> [n, chunk, heads, Q, ...]
        if c * Q > T:
            x = torch.cat([x, x.new_zeros(n, c * Q - T, *x.shape[2:])], 1)
        return x.unflatten(1, (c, Q)).movedim(3, 2)

    q, k, v, beta = chunks(q), chunks(k), chunks(v), chunks(beta)
    # log decays up to and with each token; sums in 64 bits, since their differences are what counts
    g = torch.cumsum(chunks(g).double(), -1)                                               # [n, c, H, Q]
    lower = torch.ones(Q, Q, dtype=torch.bool, device=DEVICE).tril()
    decay = torch.where(lower, g[..., :, None] - g[..., None, :], -math.inf).float().exp()  # [n, c, H, Q, Q]
    heads = lambda x: x.repeat_interleave(H // G, 2)  # noqa: E731
    kt = k.transpose(-1, -2).contiguous()
    inner = heads(torch.matmul(q, kt)) * decay
    a = heads(torch.matmul(k, kt)) * decay * beta[..., None]
    # (I + strictly lower a)^-1, blocks of twice the size at each step
    eye = torch.eye(Q, device=DEVICE)
    inv = eye.expand_as(a).clone()
    size = 1
    while size < Q:
        i = torch.arange(Q, device=DEVICE) // size
        below = (i[:, None] % 2 == 1) & (i[:, None] == i[None] + 1)
        inv = inv - torch.matmul(inv, torch.matmul(a * below, inv))
        size *= 2
    eg = torch.exp(g).float()[..., None]
    k, q = heads(k), heads(q)
    u0 = torch.matmul(inv, v * beta[..., None])
    w = torch.matmul(inv, k * (beta[..., None] * eg))
    q = q * eg
    ke = (k * torch.exp(g[..., -1:] - g).float()[..., None]).transpose(-1, -2)
    end = torch.exp(g[..., -1]).float()[..., None, None]
    S = s["initial"].float().transpose(-1, -2) if s["initial"] is not None else q.new_zeros(n, H, K, V)
    out = []
    for i in range(c):
        u = u0[:, i] - torch.matmul(w[:, i], S)
        out.append(torch.matmul(q[:, i], S) + torch.matmul(inner[:, i], u))
        S = end[:, i] * S + torch.matmul(ke[:, i], u)
    o = (torch.stack(out, 1).movedim(3, 2).flatten(1, 2)[:, :T] * s["scale"]).to(BF16)
    return {"out": o[pad[1]][None] if pad else o, "final_state": S.transpose(-1, -2).to(s["final"].dtype).contiguous()}


def _rms(x, weight):
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _rotate(x, cos, sin, interleaved):
    """The first 2 R' channels of x [B, T, H, D] by the angles [B, T, R'] of their pairs."""
    half = cos.shape[-1]
    cos, sin = cos[:, :, None], sin[:, :, None]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _angles(s):
    """Cosines and sines; far positions times frequencies in 64 bits."""
    angle = s["positions"].double()[..., None] * s["inv_freq"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _plain_rotary(s):
    cos, sin = _angles(s)
    return {x: _rotate(_rms(s[x].float(), s[x + "_weight"]), cos, sin, s["case"]["interleaved"]).to(BF16) for x in "qk"}


def _plain_append(s):
    cos, sin = _angles(s)
    k = _rotate(_rms(s["k"].float(), s["weight"]), cos, sin, False).to(BF16)
    at = s["slots"].flatten()
    s["k_cache"].flatten(0, 1)[at] = k.flatten(0, 1)
    s["v_cache"].flatten(0, 1)[at] = s["v"].flatten(0, 1)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    case = s["case"]
    n, Hq, Hk, D = case["seqs"], case["Hq"], case["Hk"], case["D"]
    rows = s["table"].clamp(min=0).long()
    k = s["k_cache"][rows].flatten(1, 2).float()                                            # [n, t, Hk, D]
    length = s["lengths"].long()[:, None]
    t = torch.arange(k.shape[1], device=DEVICE)
    seen = t < length
    if case["window"]:
        seen = seen & (t >= length - case["window"])
    q = s["q"].float().unflatten(1, (Hk, Hq // Hk)) * s["scale"]
    score = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous())                              # [n, Hk, Hq / Hk, t]
    del k
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][rows].flatten(1, 2).movedim(2, 1).float()                              # [n, Hk, t, D]
    out = torch.matmul(p / total, v)
    return {"out": out.flatten(1, 2).to(BF16), "lse": (top + torch.log(total)).flatten(1)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "delta_fwd":
        G, H, K, V, tokens = case["G"], case["H"], case["K"], case["V"], case["B"] * case["T"]
        state = (case["seqs"] or case["B"]) * H * K * V * (2 if case["state"] == "bf16" else 4)
        return {"bytes": tokens * 2 * (2 * G * K + 2 * H * V + 2 * H) + 8 * H + state * (2 if case["initial"] else 1),
                "flops": tokens * H * K * V * 7}
    if op == "paged_attention":
        seen = min(case["tokens"], case["seqs"] * case["window"]) if case["window"] else case["tokens"]
        rows = case["seqs"] * case["Hq"]
        return {"bytes": 4 * seen * case["Hk"] * case["D"] + 4 * rows * case["D"] + 4 * rows + 4 * seen // case["page"],
                "flops": 4 * seen * case["Hq"] * case["D"]}
    tokens, D, R = case["B"] * case["T"], case["D"], case["R"]
    if op == "qk_norm_rotary":
        cells = tokens * (case["Hq"] + case["Hk"]) * D
        return {"bytes": 4 * cells + 8 * tokens + 2 * R + (2 * D * (2 if case["weight"] == "bf16" else 4)
                                                           if case["norm"] else 0),
                "flops": 8 * cells}
    cells = tokens * case["H"] * D
    return {"bytes": 8 * cells + 16 * tokens + 2 * R + (2 * D if case["norm"] else 0), "flops": 8 * cells}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one token or one sequence at a time where the plain form uses products
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"delta_fwd": _exact_delta, "qk_norm_rotary": _exact_rotary, "append_kv": _exact_append,
            "paged_attention": _exact_attention}[case["op"]](s)


def _exact_delta(s):
    case = s["case"]
    B, T, G, H, K, V = (case[c] for c in "BTGHKV")
    bounds = s["cu"].tolist() if s["cu"] is not None else [T * i for i in range(B + 1)]
    begin = torch.tensor(bounds[:-1], device=DEVICE)
    size = torch.diff(torch.tensor(bounds, device=DEVICE))
    flat = {c: s[c].flatten(0, 1) for c in ("q", "k", "v", "g", "beta")}
    keep = torch.exp(-torch.exp(s["A_log"].double())
                     * torch.nn.functional.softplus(flat["g"].double() + s["dt_bias"].double(), threshold=1000.0))
    strength = torch.sigmoid(flat["beta"].double())
    n = len(size)
    S = (s["initial"].double().clone() if s["initial"] is not None
         else torch.zeros(n, H, V, K, dtype=torch.float64, device=DEVICE))
    out = torch.zeros(B * T, H, V, dtype=torch.float64, device=DEVICE)
    for t in range(s["longest"]):
        on = size > t
        at = (begin + t).clamp(max=B * T - 1)
        k, q = (flat[c][at].double().repeat_interleave(H // G, 1) for c in "kq")
        alpha = torch.where(on[:, None], keep[at], 1.0)
        b = torch.where(on[:, None], strength[at], 0.0)
        S *= alpha[..., None, None]
        u = b[..., None] * (flat["v"][at].double() - torch.matmul(S, k[..., None])[..., 0])
        S += u[..., None] * k[..., None, :]
        y = s["scale"] * torch.matmul(S, q[..., None])[..., 0]
        if s["cu"] is not None:
            y = torch.where(on[:, None, None], y, out[at])
        out[at] = y
    return {"out": out.view(B, T, H, V), "final_state": S}


def _exact_turn(x, weight, s, interleaved):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * weight.double()
    R = s["case"]["R"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                       s["positions"].double()[..., None, None] * s["inv_freq"].double())
    pairs = x[..., :R].unflatten(-1, (-1, 2)) if interleaved else x[..., :R].unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = z if interleaved else z.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., R:]], -1)


def _exact_rotary(s):
    return {x: _exact_turn(s[x], s[x + "_weight"], s, s["case"]["interleaved"]) for x in "qk"}


def _exact_append(s):
    page = s["case"]["page"]
    at = s["slots"].flatten()
    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[at // page, at % page] = _exact_turn(s["k"], s["weight"], s, False).flatten(0, 1)
    v[at // page, at % page] = s["v"].double().flatten(0, 1)
    return {"k_cache": k, "v_cache": v}


def _exact_attention(s):
    case = s["case"]
    Hq, Hk, page = case["Hq"], case["Hk"], case["page"]
    outs, lses = [], []
    for i, length in enumerate(s["lengths"].tolist()):
        first = max(0, length - case["window"]) if case["window"] else 0
        t = torch.arange(first, length, device=DEVICE)
        at = s["table"][i].long()[t // page]
        k, v = (s[c][at, t % page].double().movedim(1, 0).contiguous() for c in ("k_cache", "v_cache"))  # [Hk, t, D]
        q = s["q"][i].double().view(Hk, Hq // Hk, -1)
        score = torch.matmul(k, q.transpose(1, 2).contiguous()).transpose(1, 2) * s["scale"]
        lse = torch.logsumexp(score, -1)
        outs.append(torch.matmul(torch.exp(score - lse[..., None]), v).flatten(0, 1))
        lses.append(lse.flatten())
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
