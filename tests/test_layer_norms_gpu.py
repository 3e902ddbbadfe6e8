"""The norms (gated_norm, residual_norm, short_conv's L2 norm) of rows whose
squares fp32 does not hold, and with an eps of 0 or far from 1.

Tolerances as in the parity tests: a sum of n squares is off by (n + 2) 2^-24 at
most and half of that after the root, the rest is under 2^-19 together, and
the output's rounding half a step.  Inputs are bf16 or fp32 numbers times a
power of two, so outputs are of order 1 wherever eps is small beside them."""
import pytest
import torch

import gated_delta_rule_36_amd as kda
import layer_ref as ref
from test_layer_gpu import BF16, F32, check, normal

pytestmark = pytest.mark.gpu

SHIFTS = [-126, -100, -70, -64, -50, -43, -40, -30, 0, 40, 62, 64, 90, 120]
SIZES = [7, 64, 100, 128, 512, 600, 2048, 5000, 16384]


def shifted(t, k):
    """t 2^k in t's type (exact but for bf16's denormals, which are inputs like any other)."""
    return (t.double() * 2.0 ** k).to(t.dtype)


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("gate_first", [False, True])
def test_gated_norm_of_rows_beyond_fp32_squares(D, gate_first):
    """A row of every size at once, so that the rows of a wave differ; eps = 0."""
    g = torch.Generator().manual_seed(D)
    x = torch.cat([shifted(normal(g, 1, D), k) for k in SHIFTS])
    gate, w = normal(g, len(SHIFTS), D), normal(g, D, dtype=F32)
    out = torch.empty_like(x, device="cuda")
    kda.gated_norm(x.cuda(), gate.cuda(), w.cuda(), out, gate_first=gate_first, eps=0.0)
    want = ref.gated_norm(x, gate, w, None, 0.0, "sigmoid", gate_first)
    # below 2^-126 x act(gate) is rounded to a step of 2^-149, which is 2^-149 / rms of the row in the output
    rms = (x.double() ** 2).mean(-1, keepdim=True).sqrt() * 0.25
    lost = 2.0 ** -149 / rms * w.double().abs() if gate_first else 0.0
    check("out", out, want, (2.0 ** -19 + D * 2.0 ** -25) * want.abs() + lost)


@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("post", [False, True])
def test_residual_norm_of_rows_beyond_fp32_squares(D, post):
    g = torch.Generator().manual_seed(D + 1)
    x = torch.cat([shifted(normal(g, 1, D), k) for k in SHIFTS])
    r = normal(g, len(SHIFTS), D, dtype=F32) if post else torch.cat([shifted(normal(g, 1, D, dtype=F32), k) for k in SHIFTS])
    w, pw = normal(g, D), normal(g, D) if post else None
    out, ro = torch.empty_like(x, device="cuda"), torch.empty_like(r, device="cuda")
    kda.residual_norm(x.cuda(), r.cuda(), w.cuda(), out, ro, post_weight=None if pw is None else pw.cuda(), eps=0.0)
    want, wr, scale = ref.residual_norm(x, r, w, pw, None, 1.0, 1.0, 0.0)
    c = 2.0 ** -19 + (D * 2.0 ** -25 if post else 0)
    check("residual_out", ro, wr, c * scale + 2.0 ** -149)
    rms = torch.sqrt((wr * wr).mean(-1, keepdim=True))
    off = (c * scale + 2.0 ** -149) / rms
    check("out", out, want, (2.0 ** -19 + D * 2.0 ** -25) * want.abs() + off * w.double().abs()
          + want.abs() * off.max(-1, keepdim=True).values)


@pytest.mark.parametrize("D", [64, 600, 5000])
@pytest.mark.parametrize("eps,k", [(1e-40, -66), (1e-50, -83), (1e-25, -41), (1e-24, -40), (1e30, 50), (1e38, 63), (1e39, 64),
                                   (1e45, 75), (1e300, 120)])
def test_norms_with_eps_far_from_one(D, eps, k):
    """eps beside mean squares of its own order, also where fp32 does not hold it."""
    g = torch.Generator().manual_seed(D)
    x, w = shifted(normal(g, 3, D), k), normal(g, D)
    out, two = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    kda.gated_norm(x.cuda(), None, w.cuda(), out, eps=eps)
    kda.residual_norm(x.cuda(), None, w.cuda(), two, eps=eps)
    want = ref.gated_norm(x, None, w, None, eps)
    slack = (2.0 ** -19 + D * 2.0 ** -25) * want.abs() + 2.0 ** -133  # bf16's least step
    check("gated", out, want, slack)
    check("residual", two, want, slack)


@pytest.mark.parametrize("l2norm,D", [(64, 576), (128, 384), (256, 512)])
@pytest.mark.parametrize("W", [1, 4])
def test_conv_l2norm_of_groups_beyond_fp32_squares(l2norm, D, W):
    """Tokens of every size; behind a larger one the window holds numbers that are far apart, whose sum is off by
    2^-24 of the largest and its norm as well."""
    g = torch.Generator().manual_seed(D + W)
    x = torch.zeros(1, W * len(SHIFTS), D, dtype=BF16)
    for i, k in enumerate(SHIFTS):
        x[0, i * W:(i + 1) * W] = shifted(normal(g, W, D), min(k, 118))
    w = normal(g, D, W, dtype=F32, scale=W ** -0.5)
    out = torch.empty_like(x, device="cuda")
    kda.short_conv(x.cuda(), w.cuda(), out, activation=None, l2norm=l2norm, l2norm_eps=0.0)
    want, _, scale = ref.short_conv(x, w, None, None, l2norm, 0.0)
    # a product of a number below 2^-102 is rounded to 2^-149 at its least
    size = (x.double().abs().amax(-1, keepdim=True) * 2.0 ** -6).clamp(min=2.0 ** -149)
    check("out", out, want, 1.1 * (W + 2) * 2.0 ** -23 * scale + 2.0 ** -15 * want.abs() + 2.0 ** -20 * scale
          + (W + 1) * 2.0 ** -149 / size)


def test_norms_of_the_lowest_number_and_zeros():
    """A row of bf16's lowest number (a mask's fill) has rms 3.4e38; a row of zeros is 0 with eps > 0 and NaN without."""
    for D in (64, 128, 512, 4096):
        x = torch.full((2, D), torch.finfo(BF16).min, dtype=BF16, device="cuda")
        w, out = torch.ones(D, dtype=BF16, device="cuda"), torch.zeros(2, D, dtype=BF16, device="cuda")
        kda.gated_norm(x, None, w, out)
        assert bool((out == -1.0).all())
        kda.residual_norm(x, None, w, out.zero_())
        assert bool((out == -1.0).all())
        kda.gated_norm(torch.zeros_like(x), None, w, out)
        assert not bool(out.any())
        kda.gated_norm(torch.zeros_like(x), None, w, out, eps=0.0)
        assert bool(out.isnan().all())
