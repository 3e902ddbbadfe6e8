"""qk_norm_rotary and append_kv where a row's size and its weights lie far from 1."""
import pytest
import torch

import gated_delta_rule_36_amd as kda
import mixer_ref as ref
from mixer_ref import check
from test_attention_gpu import BF, freqs, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weight", [1e30, 1e-30])
@pytest.mark.parametrize("size", [1e-30, 1e-11, 1.0, 1e11, 1e30])
@pytest.mark.parametrize("D", [6, 36, 128, 300])
def test_large_and_small_weights(D, size, weight):
    """The normalised row is near 1, and its product with the weights is what fp32 holds, whatever the row's size."""
    x = [(rand(1, 3, 2, D, seed=i, dtype=torch.float32) * size).to(BF) for i in (1, 2, 3)]
    qw, kw = (rand(D, seed=4, dtype=torch.float32) * weight).to(BF), rand(D, seed=5, dtype=torch.float32) * weight
    pos, f = torch.tensor([[0, 7, 70000]]), freqs(2)
    q, k, v, pos_, f_ = (t.cuda() for t in (*x, pos, f))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kda.qk_norm_rotary(q, k, pos_, f_, qo, ko, qw.cuda(), kw.cuda(), eps=0.0)
    check("q", qo, *ref.rotary(x[0], pos, f, qw, eps=0.0))
    check("k", ko, *ref.rotary(x[1], pos, f, kw, eps=0.0))
    kc, vc = torch.zeros(2, 3, 2, D, dtype=BF, device="cuda"), torch.zeros(2, 3, 2, D, dtype=BF, device="cuda")
    slots = torch.tensor([[4, 0, 2]])
    want_k, want_v, bound = ref.append(x[1], x[2], kc.cpu(), vc.cpu(), slots, pos, f, kw, eps=0.0)
    kda.append_kv(k, v, kc, vc, slots.cuda(), pos_, f_, kw.cuda(), eps=0.0)
    check("k_cache", kc, want_k, bound)
    assert torch.equal(vc.cpu().double(), want_v)
