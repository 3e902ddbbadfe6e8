"""The layer operators on the GPU against their plain 64-bit forms.

Tolerances, per element.  A value rounded to bf16 is off by at most 2^-8 of
itself.  What goes before the rounding is fp32: every sum of n terms is off
by at most (n + 2) 2^-24 of the sum of the terms' absolute values ("scale"),
and exp2, rcp, rsq are good to a few units, under 2^-20 together.  So

  |out - ref| <= 2^-8 |ref| + c scale

with c = 1.1 (W + 2) 2^-23 + 2^-20 for the convolution (silu has slope at
most 1.1; the L2 norm divides value and scale alike and its sum of squares
adds 256 2^-24, within 2^-15 of |ref|).  The scan's matrix operands are split
into two bf16 parts, so each is good to 2^-16 of itself; a product chain
holds at most three of them and the decays' exponents (up to a few hundred in
base 2, fp32) add up to 2^-16 more: c = 2^-14 for out, 2^-15 of its scale for
the fp32 state.  The recurrent form is plain fp32: c = 2^-17.
"""
import math

import pytest
import torch

import gated_delta_rule_36_amd as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def normal(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def check(name, got, want, slack):
    """|got - want| <= half a step of got's type + slack, where `want` is finite."""
    got64, half = got.double().cpu(), HALF[got.dtype]
    bad = (got64 - want).abs() > half * want.abs() + slack
    bad |= ~torch.isfinite(got64)
    assert not bool(bad.any()), (
        f"{name}: {int(bad.sum())} of {bad.numel()} off; worst "
        f"{float(((got64 - want).abs() / (half * want.abs() + slack + 1e-300)).max()):.3g} of the tolerance")


def cuda(t):
    return None if t is None else t.cuda()


# ---------------------------------------------------------------------------
# short_conv
# ---------------------------------------------------------------------------

def conv_case(B, T, D, W, *, seed=0, bias=True, activation="silu", l2norm=None, state=BF16, weight=BF16,
              initial=True, cu=None, in_place=False, odd_rows=False, heads=None, eps=1e-6):
    g = torch.Generator().manual_seed(seed)
    n = len(cu) - 1 if cu is not None else B
    wide = normal(g, B, T, D + (3 if odd_rows else 0))
    x = wide[..., 1:1 + D] if odd_rows else wide
    w = normal(g, D, W, dtype=weight, scale=W ** -0.5)
    bi = normal(g, D, dtype=weight, scale=0.3) if bias else None
    st = normal(g, n, W - 1, D).to(state) if initial else None
    want, final, scale = ref.short_conv(x, w, bi, activation, l2norm, eps, st, cu)
    xg = wide.cuda()[..., 1:1 + D] if odd_rows else x.cuda()
    shape = x.shape if heads is None else (B, T, heads, D // heads)
    out = torch.full(shape, 7.0, dtype=BF16, device="cuda")
    sg = cuda(st)
    fin = sg if in_place else torch.full((n, W - 1, D), 7.0, dtype=state, device="cuda")
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int64, device="cuda")
    kda.short_conv(xg if heads is None else xg.unflatten(-1, (heads, -1)), w.cuda(), out, cuda(bi),
                   activation=activation, l2norm=l2norm, l2norm_eps=eps, initial_state=sg, final_state=fin,
                   cu_seqlens=cug, check_cu_seqlens=False)
    out = out.reshape(B, T, D)
    inside = ~torch.isnan(want[..., 0])
    assert bool((out.cpu()[~inside] == 7.0).all()), "rows outside every sequence were written"
    c = 1.1 * (W + 2) * 2.0 ** -23 + 2.0 ** -20
    slack = c * scale[inside] + (2.0 ** -15 * want[inside].abs() if l2norm else 0)
    check("out", out.cpu()[inside], want[inside], slack)
    assert torch.equal(fin.double().cpu(), final.to(state).double()), "final_state"


@pytest.mark.parametrize("T", [1, 2, 3, 31, 32, 33, 67])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 7, 8])
def test_conv_lengths_and_taps(T, W):
    conv_case(2, T, 40, W, seed=T * 10 + W)


@pytest.mark.parametrize("D", [1, 7, 8, 9, 127, 511, 512, 513, 1283])
@pytest.mark.parametrize("odd_rows", [False, True])
def test_conv_channels(D, odd_rows):
    conv_case(2, 5, D, 4, seed=D, odd_rows=odd_rows, weight=F32, state=F32)


@pytest.mark.parametrize("l2norm,D", [(64, 64), (64, 576), (128, 128), (128, 1408), (256, 256), (256, 768)])
@pytest.mark.parametrize("odd_rows", [False, True])
def test_conv_l2norm(l2norm, D, odd_rows):
    conv_case(1, 37, D, 4, seed=D, l2norm=l2norm, odd_rows=odd_rows, bias=False)
    conv_case(1, 3, D, 2, seed=D + 1, l2norm=l2norm, activation=None, initial=False, heads=D // l2norm)


CUS = [[0, 0], [0, 1, 2, 3], [0, 0, 5, 5, 5, 38, 70, 70], [0, 32, 64, 96], [0, 31, 33, 97, 98],
       [0] + [3 * i for i in range(1, 40)], [0] * 70 + [5] * 70 + [41]]


@pytest.mark.parametrize("cu", CUS)
@pytest.mark.parametrize("in_place", [False, True])
def test_conv_packed(cu, in_place):
    conv_case(1, cu[-1], 24, 4, seed=len(cu), cu=cu, in_place=in_place)
    conv_case(1, cu[-1] + 9, 24, 3, seed=len(cu) + 1, cu=cu, in_place=in_place, state=F32)  # rows behind the last


def test_conv_many_sequences():
    cu = [i // 2 for i in range(5000)]
    conv_case(1, cu[-1], 8, 4, seed=3, cu=cu, in_place=True)


def test_conv_in_place_state_of_long_sequences():
    conv_case(3, 200, 520, 8, seed=4, in_place=True)


def test_conv_empty_batch_passes_the_state_through():
    conv_case(2, 0, 24, 4, seed=5)
    conv_case(2, 0, 24, 4, seed=6, in_place=True)


def test_conv_token_by_token_equals_the_prompt():
    g = torch.Generator().manual_seed(7)
    B, T, D, W = 3, 21, 256, 4
    x, w = normal(g, B, T, D).cuda(), normal(g, D, W).cuda()
    whole, steps = torch.empty_like(x), torch.empty_like(x)
    state = torch.zeros(B, W - 1, D, dtype=BF16, device="cuda")
    last = torch.empty_like(state)
    kda.short_conv(x, w, whole, l2norm=128, final_state=last)
    for t in range(T):
        one = torch.empty(B, 1, D, dtype=BF16, device="cuda")
        kda.short_conv(x[:, t:t + 1], w, one, l2norm=128, initial_state=state, final_state=state)
        steps[:, t:t + 1] = one
    assert torch.equal(whole, steps) and torch.equal(last, state)


def test_conv_special_values_stay_in_their_channel_and_window():
    g = torch.Generator().manual_seed(8)
    x, w = normal(g, 1, 40, 16), normal(g, 16, 4)
    clean = torch.empty_like(x, device="cuda")
    kda.short_conv(x.cuda(), w.cuda(), clean, activation=None)
    x[0, 11, 3], x[0, 20, 5] = float("nan"), float("inf")
    out = torch.empty_like(clean)
    kda.short_conv(x.cuda(), w.cuda(), out, activation=None)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[0, 11:15, 3] = touched[0, 20:24, 5] = True
    assert torch.equal(out.cpu()[~touched], clean.cpu()[~touched])
    assert not torch.isfinite(out.cpu()[touched].float()).any()


# ---------------------------------------------------------------------------
# gated_norm, residual_norm
# ---------------------------------------------------------------------------

SIZES = [1, 7, 8, 63, 64, 65, 100, 128, 129, 256, 257, 512, 513, 1000, 2048, 2049, 2561, 4096, 5000, 8192, 16384]


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("activation,gate_first", [("sigmoid", False), ("silu", True), ("silu", False)])
def test_gated_norm_sizes(D, activation, gate_first):
    g = torch.Generator().manual_seed(D)
    rows = 37 if D < 600 else 5
    x, gate, w = normal(g, rows, D), normal(g, rows, D), normal(g, D, dtype=F32 if D % 2 else BF16)
    out = torch.empty(rows, D, dtype=BF16, device="cuda")
    kda.gated_norm(x.cuda(), gate.cuda(), w.cuda(), out, activation=activation, gate_first=gate_first, eps=1e-5)
    want = ref.gated_norm(x, gate, w, None, 1e-5, activation, gate_first)
    # the mean's sum: (D + 2) 2^-24 at most, half of it after the root
    check("out", out, want, (2.0 ** -19 + D * 2.0 ** -25) * want.abs())


@pytest.mark.parametrize("D,group", [(256, 64), (384, 128), (1024, 256), (4096, 1024), (4096, 512), (60, 20), (8192, 4096)])
def test_gated_norm_groups(D, group):
    g = torch.Generator().manual_seed(D + group)
    x, gate, w = normal(g, 2, 9, D, scale=3.0), normal(g, 2, 9, D), normal(g, D)
    out = torch.empty(2, 9, D, dtype=BF16, device="cuda")
    kda.gated_norm(x.cuda(), gate.cuda(), w.cuda(), out, group_size=group, activation="silu", gate_first=True)
    want = ref.gated_norm(x, gate, w, group, 1e-6, "silu", True)
    check("out", out, want, (2.0 ** -19 + group * 2.0 ** -25) * want.abs())


def test_gated_norm_heads_slices_and_no_gate():
    g = torch.Generator().manual_seed(1)
    wide = normal(g, 2, 5, 4 * 128 + 3)
    x = wide[..., 3:].unflatten(-1, (4, 128))
    gate, w = normal(g, 2, 5, 4, 128), normal(g, 128)
    out = torch.empty(2, 5, 4, 128, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="evenly"):  # heads inside slices of wider rows: two strides
        kda.gated_norm(wide.cuda()[..., 3:].unflatten(-1, (4, 128)), gate.cuda(), w.cuda(), out)
    # one row of heads per token is evenly spaced
    flat = torch.empty(2, 5, 512, dtype=BF16, device="cuda")
    w4 = w.repeat(4)
    kda.gated_norm(wide.cuda()[..., 3:], gate.cuda().flatten(-2), w4.cuda(), flat, group_size=128)
    want = ref.gated_norm(x, gate, w).flatten(-2)
    check("out", flat, want, 2.0 ** -18 * want.abs())
    kda.gated_norm(x.contiguous().cuda(), None, w.cuda(), out)
    want = ref.gated_norm(x, None, w)
    check("out", out, want, 2.0 ** -18 * want.abs())


def test_norms_zero_rows_and_rows_of_zeros():
    w = torch.ones(128, dtype=BF16, device="cuda")
    out = torch.empty(0, 128, dtype=BF16, device="cuda")
    assert kda.gated_norm(out, None, w, torch.empty_like(out)).shape == (0, 128)
    x = torch.zeros(4, 128, dtype=BF16, device="cuda")
    out, r = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    kda.gated_norm(x, x, w, out)
    assert not out.any()
    kda.residual_norm(x, x, w, out.fill_(7.0), r, post_weight=w, gate=x)
    assert not out.any() and not r.any()


def test_norms_keep_special_values_in_their_row():
    g = torch.Generator().manual_seed(2)
    for D in (128, 2048):
        x, gate, w = normal(g, 6, D).cuda(), normal(g, 6, D).cuda(), normal(g, D).cuda()
        clean, out = torch.empty_like(x), torch.empty_like(x)
        kda.gated_norm(x, gate, w, clean)
        x[1, 3], x[4, 5] = float("nan"), float("-inf")
        kda.gated_norm(x, gate, w, out)
        keep = [0, 2, 3, 5]
        assert torch.equal(out[keep], clean[keep]) and bool(out[1].isnan().all()) and bool(out[4, 5].isnan())


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("gate,post,residual", [("none", False, BF16), ("channel", True, F32), ("token", True, BF16),
                                                ("sequence", False, F32)])
def test_residual_norm_sizes(D, gate, post, residual):
    g = torch.Generator().manual_seed(D)
    B, T = 3, 7 if D < 600 else 2
    wt = BF16 if D % 2 else F32
    x, r = normal(g, B, T, D), normal(g, B, T, D, dtype=residual, scale=2.0)
    pw, w = (normal(g, D, dtype=wt) if post else None), normal(g, D, dtype=wt)
    shape = {"none": None, "channel": (D,), "sequence": (B, 1, D), "token": (B, T, D)}[gate]
    a = normal(g, *shape, dtype=wt) if shape else None
    out, ro = torch.empty(B, T, D, dtype=BF16, device="cuda"), torch.empty(B, T, D, dtype=residual, device="cuda")
    kda.residual_norm(x.cuda(), r.cuda(), w.cuda(), out, ro, post_weight=cuda(pw), gate=cuda(a), block_scale=0.7,
                      residual_scale=0.9, eps=1e-5)
    want, wr, scale = ref.residual_norm(x, r, w, pw, a, 0.7, 0.9, 1e-5)
    # the scales are rounded to fp32 too; the post norm's mean as in gated_norm
    c = 2.0 ** -19 + (D * 2.0 ** -25 if post else 0)
    check("residual_out", ro, wr, c * scale)
    rms = torch.sqrt((wr * wr).mean(-1, keepdim=True) + 1e-5)
    check("out", out, want, (2.0 ** -19 + D * 2.0 ** -25) * want.abs() + c * scale / rms * w.double().abs()
          + want.abs() * (c * scale / rms).max(-1, keepdim=True).values)


def test_residual_norm_optional_parts_and_in_place():
    g = torch.Generator().manual_seed(5)
    for D in (96, 2000):
        x, r, w = normal(g, 10, D).cuda(), normal(g, 10, D, dtype=F32).cuda(), normal(g, D).cuda()
        out, ro, out2, alone = torch.empty_like(x), torch.empty_like(r), torch.empty_like(x), torch.empty_like(r)
        kda.residual_norm(x, r, w, out, ro)
        kda.residual_norm(x, r, None, None, alone)   # no norm follows
        kda.residual_norm(x, r, w, out2)             # the stream is not kept
        assert torch.equal(ro, alone) and torch.equal(out, out2)
        kda.residual_norm(x, None, w, out2, alone)   # the stream starts here
        assert torch.equal(alone, x.float())
        want = ref.gated_norm(x.cpu(), None, w.cpu())
        check("out", out2, want, 2.0 ** -18 * want.abs())
        kda.residual_norm(x, r, w, out2, r)          # in place
        assert torch.equal(r, ro) and torch.equal(out2, out)
        wide = torch.empty(10, D + 5, dtype=BF16, device="cuda")
        wide[:, 5:] = x
        kda.residual_norm(wide[:, 5:], ro, w, out2, alone)
        kda.residual_norm(x, ro, w, out, ro)
        assert torch.equal(out, out2) and torch.equal(alone, ro)


def test_residual_norm_gate_of_leading_dimensions():
    g = torch.Generator().manual_seed(6)
    x, w = normal(g, 2, 3, 5, 72), normal(g, 72)
    for shape in ((2, 1, 1, 72), (2, 3, 1, 72), (1, 1, 1, 72)):
        a = normal(g, *shape, dtype=F32)
        ro = torch.empty(2, 3, 5, 72, device="cuda")
        kda.residual_norm(x.cuda(), None, None, None, ro, gate=a.cuda())
        _, wr, scale = ref.residual_norm(x, None, None, None, a)
        check("residual_out", ro, wr, 2.0 ** -22 * scale)


# ---------------------------------------------------------------------------
# ssm_fwd
# ---------------------------------------------------------------------------

def ssm_inputs(g, B, T, H, P, G, N, n, *, state=F32, gate=True, initial=True, slices=True):
    """CPU tensors of a scan call; x, b, c (and z, dt) as slices of fused rows."""
    xbc = normal(g, B, T, H * P + 2 * G * N)
    x = xbc[..., :H * P].unflatten(-1, (H, P))
    b = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    c = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
    zdt = normal(g, B, T, H * P + H)
    z, dt = (zdt[..., :H * P].unflatten(-1, (H, P)) if gate else None), zdt[..., H * P:]
    A_log = torch.log(torch.rand(H, generator=g) * 15 + 1)
    D, bias = torch.rand(H, generator=g) + 0.5, torch.rand(H, generator=g) * 4 - 5
    st = normal(g, n, H, P, N, scale=0.5).to(state) if initial else None
    return dict(x=x, dt=dt, b=b, c=c, A_log=A_log, D=D, dt_bias=bias, z=z, initial=st)


def on_gpu(v):
    """A copy on the GPU with the same strides (slices stay slices)."""
    if v is None:
        return None
    base = torch.empty(v.untyped_storage().nbytes() // v.element_size(), dtype=v.dtype, device="cuda")
    return base.as_strided(v.shape, v.stride(), v.storage_offset()).copy_(v)


def ssm_case(B, T, H, P, G, N, *, seed=0, state=F32, gate=True, initial=True, cu=None, in_place=False,
             softplus=True, segment_tokens=None, extra=True, recurrent=None):
    g = torch.Generator().manual_seed(seed)
    n = len(cu) - 1 if cu is not None else B
    a = ssm_inputs(g, B, T, H, P, G, N, n, state=state, gate=gate, initial=initial)
    if not extra:
        a["D"] = a["dt_bias"] = None
    if not softplus:
        a["dt"], a["dt_bias"] = (a["dt"].float().abs() * 0.2).to(BF16), None
    want, final, scale, fscale = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], a["dt_bias"], a["z"],
                                         a["initial"], cu, softplus)
    d = {k: on_gpu(v) for k, v in a.items()}
    out = torch.full((B, T, H, P), 7.0, dtype=BF16, device="cuda")
    fin = d["initial"] if in_place else torch.full((n, H, P, N), 7.0, dtype=state, device="cuda")
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int64, device="cuda")
    kda.ssm_fwd(d["x"], d["dt"], d["b"], d["c"], out, d["A_log"], d["D"], d["dt_bias"], d["z"],
                initial_state=d["initial"], final_state=fin, cu_seqlens=cug, dt_softplus=softplus,
                check_cu_seqlens=False, segment_tokens=segment_tokens)
    inside = ~torch.isnan(want[..., 0, 0])
    assert bool((out.cpu()[~inside] == 7.0).all()), "rows outside every sequence were written"
    if recurrent is None:
        recurrent = cu is None and T <= 8
    co, cf = (2.0 ** -17, 2.0 ** -17) if recurrent else (2.0 ** -14, 2.0 ** -15)
    check("final_state", fin, final, cf * fscale)
    check("out", out.cpu()[inside], want[inside], co * scale[inside])


@pytest.mark.parametrize("T", [1, 2, 7, 8])
@pytest.mark.parametrize("P,N", [(32, 32), (64, 64), (64, 128), (128, 256), (96, 128), (256, 64)])
def test_ssm_few_tokens(T, P, N):
    ssm_case(2, T, 4, P, 2, N, seed=T + N, state=BF16 if T % 2 else F32)


@pytest.mark.parametrize("T", [9, 31, 32, 33, 63, 64, 65, 130])
@pytest.mark.parametrize("P,N", [(32, 32), (64, 128)])
def test_ssm_lengths(T, P, N):
    ssm_case(2, T, 3, P, 1, N, seed=T)


@pytest.mark.parametrize("P,N", [(32, 64), (32, 256), (64, 32), (64, 64), (64, 256), (96, 128), (128, 64), (128, 128), (256, 128),
                                 (160, 32)])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 2), (10, 1)])
def test_ssm_head_layouts(P, N, H, G):
    ssm_case(1, 70, H, P, G, N, seed=P + N + H, state=BF16 if H == 6 else F32, initial=H != 1)


@pytest.mark.parametrize("cu", [[0, 0], [0, 1, 2, 3], [0, 0, 5, 5, 5, 38, 102, 102], [0, 32, 64, 96], [0, 31, 33, 97, 98],
                                [0] + [3 * i for i in range(1, 20)]])
@pytest.mark.parametrize("in_place", [False, True])
def test_ssm_packed(cu, in_place):
    ssm_case(1, cu[-1], 2, 64, 1, 64, seed=len(cu), cu=cu, in_place=in_place)
    ssm_case(1, cu[-1] + 40, 2, 32, 2, 128, seed=len(cu) + 1, cu=cu, in_place=in_place, state=BF16)


@pytest.mark.parametrize("segment_tokens", [32, 64, 96, 4096])
def test_ssm_segments(segment_tokens):
    ssm_case(2, 301, 2, 64, 1, 128, seed=segment_tokens, segment_tokens=segment_tokens, in_place=True)
    ssm_case(1, 333, 2, 64, 1, 64, seed=segment_tokens + 1, segment_tokens=segment_tokens, in_place=True,
             cu=[0, 0, 30, 190, 191, 333], state=BF16)
    ssm_case(1, 340, 2, 32, 1, 64, seed=segment_tokens + 2, segment_tokens=segment_tokens, initial=False,
             cu=[0, 64, 128, 333])


def test_ssm_optional_parts():
    for T in (5, 50):
        ssm_case(2, T, 4, 64, 1, 64, seed=T, gate=False, extra=False, initial=False)
        ssm_case(2, T, 4, 64, 4, 64, seed=T + 1, softplus=False)


def test_ssm_empty_batch_passes_the_state_through():
    ssm_case(2, 0, 2, 64, 1, 128, seed=1)
    ssm_case(2, 0, 2, 64, 1, 128, seed=2, in_place=True, state=BF16)


def test_ssm_strong_and_weak_decay():
    """Decays from 1 - 2^-20 to 0 within a chunk; a step of 0 leaves the state."""
    g = torch.Generator().manual_seed(3)
    for T in (6, 75):
        B, H, P, G, N = 1, 4, 64, 1, 64
        a = ssm_inputs(g, B, T, H, P, G, N, B)
        dt = torch.full((B, T, H), 1e-6)
        dt[..., 1], dt[..., 2], dt[..., 3] = 30.0, 0.0, 0.5
        dt[:, ::3, 3] = 200.0
        a["dt"], a["dt_bias"] = dt.to(BF16), None
        a["A_log"] = torch.tensor([0.0, 3.0, 1.0, 2.0])
        want, final, scale, fscale = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], None, a["z"], a["initial"],
                                             None, False)
        d = {k: on_gpu(v) for k, v in a.items()}
        out, fin = torch.empty(B, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
        kda.ssm_fwd(d["x"], d["dt"], d["b"], d["c"], out, d["A_log"], d["D"], None, d["z"], initial_state=d["initial"],
                    final_state=fin, dt_softplus=False)
        check("final_state", fin, final, 2.0 ** -15 * fscale)
        check("out", out, want, 2.0 ** -14 * scale)
        assert torch.equal(fin[:, 2].cpu(), a["initial"][:, 2])


def test_ssm_softplus_over_its_range():
    g = torch.Generator().manual_seed(4)
    ssm_in = ssm_inputs(g, 1, 1, 64, 32, 1, 32, 1)
    ssm_in["dt"] = torch.linspace(-40, 40, 64).to(BF16).reshape(1, 1, 64)
    ssm_in["A_log"] = torch.full((64,), -9.0)
    ssm_in["dt_bias"] = None
    _, final, _, fscale = ref.ssm(ssm_in["x"], ssm_in["dt"], ssm_in["b"], ssm_in["c"], ssm_in["A_log"], ssm_in["D"])
    d = {k: on_gpu(v) for k, v in ssm_in.items()}
    out, fin = torch.empty(1, 1, 64, 32, dtype=BF16, device="cuda"), torch.empty(1, 64, 32, 32, device="cuda")
    kda.ssm_fwd(d["x"], d["dt"], d["b"], d["c"], out, d["A_log"], d["D"], None, None, final_state=fin)
    check("final_state", fin, final, 2.0 ** -20 * fscale)


def test_ssm_token_by_token_continues_a_prompt():
    g = torch.Generator().manual_seed(9)
    B, T, H, P, G, N = 2, 45, 4, 64, 2, 128
    a = ssm_inputs(g, B, T, H, P, G, N, B)
    want, final, scale, fscale = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], a["dt_bias"], a["z"], a["initial"])
    d = {k: on_gpu(v) for k, v in a.items()}
    state = d["initial"]
    outs = []
    for lo, hi in [(0, 40)] + [(t, t + 1) for t in range(40, T)]:
        out = torch.empty(B, hi - lo, H, P, dtype=BF16, device="cuda")
        kda.ssm_fwd(d["x"][:, lo:hi], d["dt"][:, lo:hi], d["b"][:, lo:hi], d["c"][:, lo:hi], out, d["A_log"], d["D"],
                    d["dt_bias"], d["z"][:, lo:hi], initial_state=state, final_state=state)
        outs.append(out)
    check("out", torch.cat(outs, 1), want, 2.0 ** -14 * scale)
    check("final_state", state, final, 2.0 ** -15 * fscale)


def test_ssm_never_mixes_sequences():
    """A NaN or infinity in one sequence leaves the others' outputs bit for bit, and its own earlier chunks."""
    g = torch.Generator().manual_seed(10)
    cu = [0, 50, 51, 150, 200]
    a = ssm_inputs(g, 1, 200, 2, 64, 1, 64, 4)
    d = {k: on_gpu(v) for k, v in a.items()}
    cug = torch.tensor(cu, device="cuda")

    def run():
        out, fin = torch.empty(1, 200, 2, 64, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
        kda.ssm_fwd(d["x"], d["dt"], d["b"], d["c"], out, d["A_log"], d["D"], d["dt_bias"], d["z"], cu_seqlens=cug,
                    initial_state=d["initial"], final_state=fin, segment_tokens=64)
        return out, fin

    clean, cf = run()
    d["x"][0, 100, 0, 5], d["b"][0, 110, 0, 7] = float("nan"), float("inf")
    out, fin = run()
    for lo, hi in ((0, 50), (50, 51), (51, 83), (150, 200)):
        assert torch.equal(out[:, lo:hi], clean[:, lo:hi]), (lo, hi)
    assert torch.equal(fin[[0, 1, 3]], cf[[0, 1, 3]]) and bool(fin[2].isnan().any())


# ---------------------------------------------------------------------------
# together, streams, graphs
# ---------------------------------------------------------------------------

class Block:
    """One layer of a hybrid model on the operators: norm, projection, convolution, mixer, gated norm,
    projection, residual.  `mixer` is "kda" or "ssm"."""

    def __init__(self, mixer, hidden=256, H=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.mixer, self.H, self.hidden = mixer, H, hidden
        inner = H * 128
        width = {"kda": 5 * inner + H, "ssm": 2 * inner + 2 * 128 + H}[mixer]
        self.w_in = normal(g, hidden, width, scale=hidden ** -0.5).cuda()
        self.w_out = normal(g, inner, hidden, scale=inner ** -0.5).cuda()
        self.conv = normal(g, {"kda": 3 * inner, "ssm": inner + 256}[mixer], 4, scale=0.5).cuda()
        self.norm, self.head, self.post = (torch.ones(n, dtype=BF16, device="cuda") for n in (hidden, 128, hidden))
        self.A_log = torch.zeros(H, device="cuda")
        self.dt_bias = torch.zeros(H, 128, device="cuda") if mixer == "kda" else torch.full((H,), -2.0, device="cuda")
        self.D = torch.ones(H, device="cuda")

    def states(self, B):
        return (torch.zeros(B, 3, self.conv.shape[0], dtype=BF16, device="cuda"),
                torch.zeros(B, self.H, 128, 128, device="cuda"))

    def __call__(self, normed, residual, conv_state, state):
        """(next block's input, residual) of [B, T, hidden]; the states are updated in place."""
        B, T, _ = normed.shape
        H, inner = self.H, self.H * 128
        new = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")
        proj = normed @ self.w_in
        mixed = new(B, T, H, 128)
        if self.mixer == "kda":
            qk, v = new(B, T, 2 * H, 128), new(B, T, H, 128)
            # the channels of q, k and v hold their own parts of the state
            sq, sv = conv_state[..., :2 * inner].contiguous(), conv_state[..., 2 * inner:].contiguous()
            kda.short_conv(proj[..., :2 * inner].unflatten(-1, (2 * H, 128)), self.conv[:2 * inner], qk, l2norm=128,
                           initial_state=sq, final_state=sq)
            kda.short_conv(proj[..., 2 * inner:3 * inner].unflatten(-1, (H, 128)), self.conv[2 * inner:], v,
                           initial_state=sv, final_state=sv)
            conv_state.copy_(torch.cat([sq, sv], -1))
            q, k = qk[:, :, :H].contiguous(), qk[:, :, H:].contiguous()
            decay, gate = (proj[..., i * inner:(i + 1) * inner].unflatten(-1, (H, 128)).contiguous() for i in (3, 4))
            kda.fwd(q, k, v, decay, proj[..., 5 * inner:].contiguous(), 128 ** -0.5, mixed, self.A_log, self.dt_bias,
                    -5.0, initial_state=state, final_state=state)
            y = torch.empty_like(mixed)
            kda.gated_norm(mixed, gate, self.head, y)
        else:
            xbc = new(B, T, inner + 256)
            kda.short_conv(proj[..., inner:2 * inner + 256], self.conv, xbc, initial_state=conv_state,
                           final_state=conv_state)
            kda.ssm_fwd(xbc[..., :inner].unflatten(-1, (H, 128)), proj[..., 2 * inner + 256:],
                        xbc[..., inner:inner + 128].unflatten(-1, (1, 128)), xbc[..., inner + 128:].unflatten(-1, (1, 128)),
                        mixed, self.A_log, self.D, self.dt_bias, initial_state=state, final_state=state)
            y = torch.empty_like(mixed)
            kda.gated_norm(mixed.flatten(-2), proj[..., :inner], self.head.repeat(H), y.flatten(-2), group_size=128,
                           activation="silu", gate_first=True)
        out, res = new(B, T, self.hidden), torch.empty_like(residual)
        kda.residual_norm(y.flatten(-2) @ self.w_out, residual, self.norm, out, res, post_weight=self.post)
        return out, res


def test_hybrid_layers_prompt_then_tokens():
    """KDA and scan layers in turn: a prompt and then single tokens give what the whole sequence gives,
    to the bf16 rounding of the layers between."""
    g = torch.Generator().manual_seed(11)
    B, T, hidden = 2, 40, 256
    layers = [Block("kda", seed=1), Block("ssm", seed=2), Block("kda", seed=3)]
    x = normal(g, B, T, hidden).cuda()

    def run(pieces):
        states = [m.states(B) for m in layers]
        got = []
        for lo, hi in pieces:
            part = x[:, lo:hi].contiguous()
            normed, res = torch.empty_like(part), torch.empty(part.shape, device="cuda")
            kda.residual_norm(part, None, layers[0].norm, normed, res)
            for m, s in zip(layers, states):
                normed, res = m(normed, res, *s)
            got.append(res)
        return torch.cat(got, 1), states

    whole, ws = run([(0, T)])
    steps, ss = run([(0, 30)] + [(t, t + 1) for t in range(30, T)])
    assert bool(torch.isfinite(whole).all())
    assert float((whole - steps).norm() / whole.norm()) < 2e-2
    for (wc, wm), (sc, sm) in zip(ws, ss):
        assert float((wm - sm).norm() / wm.norm()) < 3e-2
        assert float((wc - sc).float().norm() / wc.float().norm()) < 3e-2


def calls(g):
    """name -> (call, outputs, inputs that may change between replays) of every operator, prompts and single tokens."""
    found = {}
    for T in (1, 70):
        x, w, st = normal(g, 2, T, 256).cuda(), normal(g, 256, 4).cuda(), normal(g, 2, 3, 256).cuda()
        out, fin = torch.empty_like(x), torch.empty_like(st)
        found[f"conv T={T}"] = (lambda x=x, w=w, out=out, st=st, fin=fin: kda.short_conv(
            x, w, out, l2norm=128, initial_state=st, final_state=fin), [out, fin], [x, st])
        a = {k: on_gpu(v) for k, v in ssm_inputs(g, 2, T, 4, 64, 1, 128, 2).items()}
        so, sf = torch.empty(2, T, 4, 64, dtype=BF16, device="cuda"), torch.empty_like(a["initial"])
        found[f"ssm T={T}"] = (lambda a=a, so=so, sf=sf: kda.ssm_fwd(
            a["x"], a["dt"], a["b"], a["c"], so, a["A_log"], a["D"], a["dt_bias"], a["z"], initial_state=a["initial"],
            final_state=sf, segment_tokens=32), [so, sf], [a["x"], a["initial"], a["dt"]])
    x, gate, w = normal(g, 33, 512).cuda(), normal(g, 33, 512).cuda(), normal(g, 512).cuda()
    out = torch.empty_like(x)
    found["gated"] = (lambda: kda.gated_norm(x, gate, w, out, group_size=128), [out], [x, gate])
    r = normal(g, 33, 2560, dtype=F32).cuda()
    y, w2 = normal(g, 33, 2560).cuda(), normal(g, 2560).cuda()
    o2, r2 = torch.empty_like(y), torch.empty_like(r)
    found["residual"] = (lambda: kda.residual_norm(y, r, w2, o2, r2, post_weight=w2), [o2, r2], [y, r])
    return found


def test_captured_calls_replay_with_new_inputs():
    """Every operator captured together in one graph: each replay equals the eager calls on its inputs."""
    g = torch.Generator().manual_seed(12)
    found = calls(g)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for call, _, _ in found.values():
            call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _, _ in found.values():
            call()
    for seed in range(3):
        gg = torch.Generator().manual_seed(100 + seed)
        for _, _, inputs in found.values():
            for t in inputs:
                t.copy_(torch.randn(t.shape, generator=gg))
        for _, outs, _ in found.values():
            for t in outs:
                t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        replayed = {k: [t.clone() for t in outs] for k, (_, outs, _) in found.items()}
        for name, (call, outs, _) in found.items():
            call()
            torch.cuda.synchronize()
            for a, b in zip(replayed[name], outs):
                assert torch.equal(a, b), (name, seed)


def test_calls_on_several_streams_at_once():
    g = torch.Generator().manual_seed(13)
    found = calls(g)
    want = {}
    for name, (call, outs, _) in found.items():
        call()
        torch.cuda.synchronize()
        want[name] = [t.clone() for t in outs]
        for t in outs:
            t.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in found]
    for s, (call, _, _) in zip(streams, found.values()):
        with torch.cuda.stream(s):
            call()
    torch.cuda.synchronize()
    for name, (_, outs, _) in found.items():
        for a, b in zip(want[name], outs):
            assert torch.equal(a, b), name


def test_offsets_beyond_32_bits():
    """Token strides that put the last rows past 2^32 elements: the same results as the rows packed together."""
    g = torch.Generator().manual_seed(14)
    T, H, P, N, far = 40, 2, 64, 64, 1 << 27
    base = torch.zeros(far * (T - 1) + 4096, dtype=BF16, device="cuda")  # 10 GiB
    a = {k: on_gpu(v) for k, v in ssm_inputs(g, 1, T, H, P, 1, N, 1, gate=False).items()}
    width = H * P

    def place(v, at):
        w = v[0, 0].numel()
        t = base.as_strided((1, T, w), (0, far, 1), at)
        t.copy_(v.reshape(1, T, w))
        return t.reshape(v.shape) if v.dim() == 3 else t.unflatten(-1, v.shape[2:])

    x, b, c = place(a["x"], 0), place(a["b"], 512), place(a["c"], 1024)
    out, far_out = (torch.empty(1, T, H, P, dtype=BF16, device="cuda") for _ in range(2))
    rest = (a["A_log"], a["D"], a["dt_bias"])
    kda.ssm_fwd(a["x"], a["dt"], a["b"], a["c"], out, *rest, segment_tokens=32)
    kda.ssm_fwd(x, a["dt"], b, c, far_out, *rest, segment_tokens=32)
    assert torch.equal(out, far_out)
    w = normal(g, width, 4).cuda()
    co, cfar = torch.empty(1, T, width, dtype=BF16, device="cuda"), torch.empty(1, T, width, dtype=BF16, device="cuda")
    kda.short_conv(a["x"].flatten(-2).contiguous(), w, co)
    kda.short_conv(x.flatten(-2), w, cfar)
    assert torch.equal(co, cfar)
    n, nfar = torch.empty(T, width, dtype=BF16, device="cuda"), torch.empty(T, width, dtype=BF16, device="cuda")
    wn = torch.ones(width, dtype=BF16, device="cuda")
    kda.gated_norm(a["x"][0].flatten(-2).contiguous(), None, wn, n)
    kda.gated_norm(x[0].flatten(-2), None, wn, nfar)
    assert torch.equal(n, nfar)


def test_ssm_largest_token_strides():
    """x, b, c and z at the largest token strides the chunked scan takes, with the widest rows of lanes (N = 32)."""
    g = torch.Generator().manual_seed(15)
    T, H, P, N, far = 70, 2, 32, 32, 1 << 26
    a = {k: on_gpu(v) for k, v in ssm_inputs(g, 1, T, H, P, 1, N, 1).items()}
    base = torch.zeros(2 * far * (T // 2) + 4096, dtype=BF16, device="cuda")  # 8.8 GiB

    def place(v, at, stride, count):
        w = v[0, 0].numel()
        t = base.as_strided((1, count, w), (0, stride, 1), at)
        t.copy_(v[:, :count].reshape(1, count, w))
        return t.unflatten(-1, v.shape[2:])

    rest = (a["A_log"], a["D"], a["dt_bias"])
    for near, count, stride in (("z", T, far), ("xbc", T // 2, 2 * far)):
        got = {k: place(a[k], 512 * i, stride, count) if k in near else a[k][:, :count] for i, k in enumerate("xbcz")}
        out, far_out = (torch.empty(1, count, H, P, dtype=BF16, device="cuda") for _ in range(2))
        dt = a["dt"][:, :count]
        kda.ssm_fwd(a["x"][:, :count], dt, a["b"][:, :count], a["c"][:, :count], out, *rest, a["z"][:, :count])
        kda.ssm_fwd(got["x"], dt, got["b"], got["c"], far_out, *rest, got["z"])
        assert torch.equal(out, far_out)


# ---------------------------------------------------------------------------
# calls at the edges of what is allowed
# ---------------------------------------------------------------------------
def scan(a, out, fin, **kw):
    kda.ssm_fwd(a["x"], a["dt"], a["b"], a["c"], out, a["A_log"], a["D"], a["dt_bias"], a["z"],
                initial_state=a["initial"], final_state=fin, **kw)


def scan_against_formula(a, cu, softplus, **kw):
    """A chunked scan of CPU inputs `a` against the formula, with the tolerances of ssm_case."""
    B, T, H, P = a["x"].shape
    want, final, scale, fscale = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], a["dt_bias"], a["z"],
                                         a["initial"], cu, softplus)
    d = {k: on_gpu(v) for k, v in a.items()}
    out, fin = torch.empty(B, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int64, device="cuda")
    scan(d, out, fin, cu_seqlens=cug, dt_softplus=softplus, **kw)
    check("final_state", fin, final, 2.0 ** -15 * fscale)
    check("out", out, want, 2.0 ** -14 * scale)


@pytest.mark.parametrize("segment_tokens", [None, 64, 352])
@pytest.mark.parametrize("cu", [None, [0, 40, 400, 400, 640]])
def test_ssm_decays_that_end_a_segment_early(segment_tokens, cu):
    """Eight heads of one workgroup, from a step that keeps all to one that forgets at once: tiles on both sides of
    every choice by decay, and segments whose first tiles leave nothing."""
    g = torch.Generator().manual_seed(21)
    T, H = 640, 8
    a = ssm_inputs(g, 1, T, H, 32, 1, 64, 1 if cu is None else len(cu) - 1)
    per_token = torch.tensor([2.0 ** -14, 0.11, 0.14, 0.6, 0.64, 1.3, 5.0, 100.0])  # halvings, about
    a["A_log"] = torch.log(per_token * 0.6931)
    a["dt"] = (1 + 0.1 * torch.randn(1, T, H, generator=g)).abs().to(BF16)
    a["dt_bias"] = None
    scan_against_formula(a, cu, False, segment_tokens=segment_tokens)
    a["A_log"] = torch.full((H,), 2.0)  # all of them forget: workgroups stop early
    scan_against_formula(a, cu, True, segment_tokens=segment_tokens)


def test_ssm_negative_steps_grow_the_state():
    g = torch.Generator().manual_seed(22)
    for T, segment_tokens in ((6, None), (200, None), (200, 96)):
        a = ssm_inputs(g, 2, T, 4, 64, 1, 128, 2)
        a["dt"] = (torch.randn(2, T, 4, generator=g) * 0.3).to(BF16)
        a["dt_bias"], a["A_log"] = None, torch.tensor([-2.0, -1.0, 0.0, 0.5])
        scan_against_formula(a, None, False, segment_tokens=segment_tokens)


@pytest.mark.parametrize("P,H,G", [(96, 5, 1), (160, 4, 2), (32, 9, 1), (256, 2, 2)])
def test_ssm_heads_across_workgroups_in_segments(P, H, G):
    ssm_case(1, 260, H, P, G, 32, seed=P, segment_tokens=96, cu=[0, 100, 100, 259], in_place=True)
    ssm_case(2, 200, H, P, G, 128, seed=P + 1, segment_tokens=64)


def test_broadcast_inputs():
    """Inputs expanded over the batch or the tokens (strides of 0) equal their copies."""
    g = torch.Generator().manual_seed(23)
    B, T, H, P, N = 2, 70, 3, 64, 64
    a = {k: on_gpu(v) for k, v in ssm_inputs(g, B, T, H, P, 1, N, B).items()}
    a["b"], a["c"] = a["b"][:, :1].expand(B, T, 1, N), a["c"][:1].expand(B, T, 1, N)
    a["x"], a["z"] = a["x"][:, :1].expand(B, T, H, P), a["z"][:1, :1].expand(B, T, H, P)
    whole = {k: v if v is None else v.clone(memory_format=torch.contiguous_format) for k, v in a.items()}
    for n in (T, 5):
        outs = []
        for v in (a, whole):
            v = {k: t if t is None or k in ("A_log", "D", "dt_bias", "initial") else t[:, :n] for k, t in v.items()}
            out, fin = torch.empty(B, n, H, P, dtype=BF16, device="cuda"), torch.empty_like(a["initial"])
            scan(v, out, fin)
            outs.append((out, fin))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    row, w4 = normal(g, 1, 1, 192).cuda(), normal(g, 192, 4).cuda()
    wide, copy = row.expand(B, T, 192), row.expand(B, T, 192).contiguous()
    for f in (lambda x, o: kda.short_conv(x, w4, o), lambda x, o: kda.gated_norm(x, x, w4[:, 0].contiguous(), o),
              lambda x, o: kda.residual_norm(x, None, w4[:, 1].contiguous(), o)):
        one, two = torch.empty_like(copy), torch.empty_like(copy)
        f(wide, one)
        f(copy, two)
        assert torch.equal(one, two)


@pytest.mark.parametrize("cu", [[0, 50, 20, 130], [0, -7, 60, 130], [3, 200, 1 << 40, 130], [130, 90, 40, 0],
                                [-(1 << 62), 1 << 62, -5, 1 << 33]])
def test_offsets_out_of_order_write_nothing_else(cu):
    """cu_seqlens that the caller did not check: the results mean nothing, but no other memory is written."""
    g = torch.Generator().manual_seed(24)
    T, H, P, N, n, edge = 130, 2, 64, 64, len(cu) - 1, 1 << 16
    cug = torch.tensor(cu, dtype=torch.int64, device="cuda")
    a = {k: on_gpu(v) for k, v in ssm_inputs(g, 1, T, H, P, 1, N, n).items()}

    def guarded(*shape, dtype=BF16):
        whole = torch.full((2 * edge + torch.Size(shape).numel(),), 7.0, dtype=dtype, device="cuda")
        return whole, whole[edge:-edge].view(shape)

    made = []
    for segment_tokens in (None, 32):
        (ow, out), (fw, fin) = guarded(1, T, H, P), guarded(n, H, P, N, dtype=F32)
        scan(a, out, fin, cu_seqlens=cug, check_cu_seqlens=False, segment_tokens=segment_tokens)
        made += [ow, fw]
    x, w, st = normal(g, 1, T, 13).cuda(), normal(g, 13, 8).cuda(), normal(g, n, 7, 13).cuda()
    (ow, out), (fw, fin) = guarded(1, T, 13), guarded(n, 7, 13)
    kda.short_conv(x, w, out, initial_state=st, final_state=fin, cu_seqlens=cug, check_cu_seqlens=False)
    for whole in made + [ow, fw]:
        assert bool((whole[:edge] == 7.0).all()) and bool((whole[-edge:] == 7.0).all())


@pytest.mark.parametrize("D", [3, 13, 515, 1027])
def test_conv_in_place_states_of_odd_widths(D):
    conv_case(1, 60, D, 8, seed=D, cu=[0, 1, 1, 4, 30, 60], in_place=True, state=F32)
    conv_case(3, 1, D, 4, seed=D + 1, in_place=True, odd_rows=True)


def test_norms_of_more_rows_than_one_grid_dimension():
    """2^29 rows of one channel: as in slices."""
    rows, piece = (1 << 29) + 5, 1 << 24
    x = torch.empty(rows, 1, dtype=BF16, device="cuda")
    for at in range(0, rows, piece):
        x[at:at + piece].normal_()
    w, out = torch.full((1,), 1.5, dtype=BF16, device="cuda"), torch.empty_like(x)
    v = x[-piece:].double()
    plain = v * (v * v + 1e-6).rsqrt() * 1.5
    for f, want in ((lambda x, o: kda.gated_norm(x, x, w, o), plain * torch.sigmoid(v)),
                    (lambda x, o: kda.residual_norm(x, None, w, o), plain)):
        out.fill_(7.0)
        f(x, out)
        for at in (0, rows // 2, rows - piece):
            part = torch.empty(piece, 1, dtype=BF16, device="cuda")
            f(x[at:at + piece], part)
            assert torch.equal(part, out[at:at + piece])
        # fp32 arithmetic: below 2^-20 of values up to 1.5
        assert bool(((out[-piece:].double() - want).abs() <= HALF[BF16] * want.abs() + 2.0 ** -19).all())


def test_two_graphs_replayed_in_turn():
    """Two captures of the same calls on inputs of their own, replayed in turn and at once on two streams."""
    sets = []
    for seed in (31, 32):
        found = calls(torch.Generator().manual_seed(seed))
        for call, _, _ in found.values():
            call()
        torch.cuda.synchronize()
        want = {k: [t.clone() for t in outs] for k, (_, outs, _) in found.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for call, _, _ in found.values():
                call()
        sets.append((found, want, graph))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for found, _, _ in sets:
            for _, outs, _ in found.values():
                for t in outs:
                    t.fill_(7.0)
        torch.cuda.synchronize()
        for stream, (_, _, graph) in zip(streams, sets):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for found, want, _ in sets:
            for name, (_, outs, _) in found.items():
                for got, expected in zip(outs, want[name]):
                    assert torch.equal(got, expected), name


@pytest.mark.parametrize("n", [63, 64, 65, 130])
@pytest.mark.parametrize("segment_tokens", [None, 32])
def test_as_many_sequences_as_lanes_and_more(n, segment_tokens):
    """Random lengths, some of 0, around the number at which tiles are found another way."""
    g = torch.Generator().manual_seed(n)
    lengths = torch.randint(0, 12, (n,), generator=g)
    lengths[[0, 7, n // 2, n - 2]] = torch.tensor([0, 100, 70, 33])
    cu = [0] + torch.cumsum(lengths, 0).tolist()
    ssm_case(1, cu[-1] + 3, 2, 32, 1, 32, seed=n, cu=cu, segment_tokens=segment_tokens, in_place=True)
    conv_case(1, cu[-1] + 3, 24, 4, seed=n, cu=cu, in_place=True)


@pytest.mark.parametrize("call", [
    lambda x, w, o: kda.gated_norm(x, None, w, o, group_size=2.5),
    lambda x, w, o: kda.gated_norm(x, None, w, o, eps="small"),
    lambda x, w, o: kda.residual_norm(x, None, w, o, block_scale=None),
    lambda x, w, o: kda.short_conv(x[None], w[:, None], o[None], l2norm="all"),
])
def test_arguments_of_the_wrong_type(call):
    x, w, o = torch.zeros(2, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda"), \
        torch.full((2, 64), 7.0, dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        call(x, w, o)
    assert bool((o == 7.0).all())


def test_host_refusals_on_the_gpu():
    """What the library refuses raises before anything is enqueued: the outputs stay as they were."""
    x = torch.zeros(1, 9, 2, 32, dtype=BF16, device="cuda")
    bc, dt, a = torch.zeros(1, 9, 1, 32, dtype=BF16, device="cuda"), torch.zeros(1, 9, 2, dtype=BF16, device="cuda"), torch.zeros(2, device="cuda")
    out = torch.full_like(x, 7.0)
    for segment_tokens in (16, 33):
        with pytest.raises(kda.KdaArgumentError):
            kda.ssm_fwd(x, dt, bc, bc, out, a, segment_tokens=segment_tokens)
    with pytest.raises(kda.KdaArgumentError):
        kda.ssm_fwd(x, dt, bc, bc, x, a)  # out is an input
    with pytest.raises(kda.KdaArgumentError):
        kda.short_conv(x.flatten(-2), torch.zeros(64, 9, dtype=BF16, device="cuda"), out.flatten(-2))  # nine taps
    with pytest.raises(kda.KdaArgumentError):
        kda.gated_norm(x, None, torch.ones(32, dtype=BF16, device="cuda"), out, group_size=5)
    with pytest.raises(kda.KdaArgumentError):
        kda.residual_norm(x, None, torch.ones(32, dtype=BF16, device="cuda"), out, eps=-1.0)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("D", [513, 640, 1025, 1536, 1999, 2560, 2561, 3590, 4095, 4097, 5120, 5121, 7168, 8191, 8193, 10240, 12289, 16383])
def test_norms_of_rows_of_every_number_of_waves(D):
    test_gated_norm_sizes(D, "silu", D % 2 == 0)
    test_residual_norm_sizes(D, "channel", True, F32)
    test_residual_norm_sizes(D, "none", False, BF16)


@pytest.mark.parametrize("P,N,G", [(64, 128, 1), (128, 64, 2), (64, 256, 1)])
@pytest.mark.parametrize("segment_tokens", [None, 4096])
def test_ssm_state_is_as_exact_as_fp32(P, N, G, segment_tokens):
    """The fp32 state of a chunked scan from decays that forget in a token to ones that keep all.  Some thirty
    roundings of 2^-24 reach an element (steps 4, weights 6, products 1, sums over 300 tokens in sixteens); they are
    independent, so their sum is sqrt(30) 2^-24 or 2^-21.5 of it."""
    g = torch.Generator().manual_seed(N)
    for per_token in (0.003, 0.1, 2.0):
        a = ssm_inputs(g, 1, 300, 8, P, G, N, 1, gate=False)
        a["A_log"] = torch.log(torch.linspace(1, 16, 8) * per_token)
        want, final, _, _ = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], a["dt_bias"], None, a["initial"])
        d = {k: on_gpu(v) for k, v in a.items()}
        out, fin = torch.empty(1, 300, 8, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
        scan(d, out, fin, segment_tokens=segment_tokens)
        for h in range(8):
            error = (fin[:, h].double().cpu() - final[:, h]).norm() / final[:, h].norm()
            assert float(error) <= 2.0 ** -20, (per_token, h, float(error))
