"""The operators together, as a server of a hybrid decoder calls them: packed
prompts of three requests, then single tokens, through a recurrent layer
(short_conv, delta_fwd, gated_norm) and an attention layer (qk_norm_rotary,
append_kv, paged_attention), with residual_norm between.  Every operator's
results are held against its 64-bit form on what it was really given."""
import pytest
import torch

import gated_delta_rule_36_amd as kda
import layer_ref
import mixer_ref as ref
from mixer_ref import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
G, H, K, V, W = 2, 4, 64, 32, 4
HQ, HK, D, R, PAGE = 8, 2, 64, 32, 16
DIM = H * V


class Model:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        def n(*s): return torch.randn(*s, generator=g)
        self.w_in = (n(DIM, 2 * G * K + 2 * H * V + 2 * H) * DIM ** -0.5).cuda()
        self.w_qkv = (n(DIM, (HQ + 2 * HK) * D) * DIM ** -0.5).cuda()
        self.w_out = (n(HQ * D, DIM) * (HQ * D) ** -0.5).cuda()
        self.conv_qk = (n(2 * G * K, W) * 0.5).to(BF).cuda()
        self.conv_v = (n(H * V, W) * 0.5).to(BF).cuda()
        self.A_log, self.dt_bias = torch.rand(H, generator=g).cuda(), (n(H) - 3).cuda()
        self.norm_v = torch.rand(H * V, generator=g).to(BF).cuda()
        self.norm_1, self.norm_2 = (torch.rand(DIM, generator=g) + 0.5).cuda(), (torch.rand(DIM, generator=g) + 0.5).cuda()
        self.q_norm, self.k_norm = (torch.rand(D, generator=g) + 0.5).to(BF).cuda(), (torch.rand(D, generator=g) + 0.5).to(BF).cuda()
        self.inv_freq = (10000.0 ** (-torch.arange(0, R, 2) / R)).float().cuda()


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def project(x, w):
    return (x.float() @ w).to(BF)


def recurrent_layer(m, x, states, cu):
    """The mixer's output [B, T, H V]; the states are updated in place."""
    B, T = x.shape[:2]
    p = project(x, m.w_in)
    a, b, c = 2 * G * K, 2 * G * K + H * V, 2 * G * K + 2 * H * V
    qk, v = empty(B, T, 2 * G, K), empty(B, T, H, V)
    check_cu = dict(cu_seqlens=cu, check_cu_seqlens=False)
    kda.short_conv(p[..., :a].unflatten(-1, (2 * G, K)), m.conv_qk, qk, l2norm=64, initial_state=states["qk"],
                   final_state=states["qk"], **check_cu)
    kda.short_conv(p[..., a:b].unflatten(-1, (H, V)), m.conv_v, v, initial_state=states["v"], final_state=states["v"], **check_cu)
    o = empty(B, T, H, V)
    args = (qk[:, :, :G], qk[:, :, G:], v, p[..., c:c + H], p[..., c + H:], K ** -0.5)
    before = states["S"].clone()
    kda.delta_fwd(*args, o, m.A_log, m.dt_bias, initial_state=states["S"], final_state=states["S"], **check_cu)
    want = ref.delta(*(t.cpu() if isinstance(t, torch.Tensor) else t for t in args), m.A_log.cpu(), m.dt_bias.cpu(),
                     before.cpu(), None if cu is None else cu.tolist())
    check("delta", o, want[0], want[2])
    assert float((states["S"].cpu().double() - want[1]).norm() / want[1].norm()) < 1e-6
    y = empty(B, T, H * V)
    kda.gated_norm(o.flatten(2), p[..., b:c], m.norm_v, y, group_size=V)
    # some ten roundings of numbers below 30 before the last one
    check("gated norm", y, layer_ref.gated_norm(o.flatten(2).cpu(), p[..., b:c].cpu(), m.norm_v.cpu(), V),
          torch.tensor(300 * 2.0 ** -24, dtype=torch.float64))
    return y


def rotate(m, x, cache, positions, slots):
    """The queries [B, T, HQ, D] of an attention layer; its keys and values go into the cache."""
    B, T = x.shape[:2]
    qkv = project(x, m.w_qkv).unflatten(-1, (HQ + 2 * HK, D))
    q = empty(B, T, HQ, D)
    kda.qk_norm_rotary(qkv[:, :, :HQ], None, positions, m.inv_freq, q, None, m.q_norm)
    before = [c.cpu() for c in cache]
    kda.append_kv(qkv[:, :, HQ:HQ + HK], qkv[:, :, HQ + HK:], *cache, slots, positions, m.inv_freq, m.k_norm)
    pos, f = positions.cpu(), m.inv_freq.cpu()
    check("q", q, *ref.rotary(qkv[:, :, :HQ].cpu(), pos, f, m.q_norm.cpu()))
    kc, vc, kb = ref.append(qkv[:, :, HQ:HQ + HK].cpu(), qkv[:, :, HQ + HK:].cpu(), *before, slots.cpu(), pos, f, m.k_norm.cpu())
    check("k_cache", cache[0], kc, kb)
    # copies, and what no token wrote is still NaN
    torch.testing.assert_close(cache[1].cpu().double(), vc, rtol=0, atol=0, equal_nan=True)
    # the same keys as through qk_norm_rotary, bit for bit
    both = empty(B, T, HQ, D), empty(B, T, HK, D)
    kda.qk_norm_rotary(qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HK], positions, m.inv_freq, *both, m.q_norm, m.k_norm)
    assert torch.equal(both[0], q)
    s = slots.flatten()
    kept = s >= 0
    assert torch.equal(cache[0].flatten(0, 1)[s[kept]], both[1].flatten(0, 1)[kept])
    return q


def test_prompts_and_then_tokens():
    m = Model(1)
    lengths, steps = [5, 37, 100], 4
    N, T = len(lengths), sum(lengths)
    gen = torch.Generator().manual_seed(2)
    cu = torch.tensor([0, 5, 42, 142]).cuda()
    width = 8
    order = torch.randperm(N * width + 3, generator=gen)
    table = order[:N * width].view(N, width).int()
    cache = tuple(torch.full((N * width + 3, PAGE, HK, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    states = {"qk": torch.zeros(N, W - 1, 2 * G * K, device="cuda"), "v": torch.zeros(N, W - 1, H * V, device="cuda"),
              "S": torch.zeros(N, H, V, K, device="cuda")}

    def slot(n, t):
        return int(table[n, t // PAGE]) * PAGE + t % PAGE

    def layers(x, cu, positions, slots, visible):
        """A recurrent layer, the residual update with the next norm, and the attention layer's cache; with
        `visible` lengths also its attention and the update behind it."""
        stream, h = empty(*x.shape, dtype=F32), empty(*x.shape)
        kda.residual_norm(x, None, m.norm_1, h, stream)
        y = recurrent_layer(m, h, states, cu)
        kda.residual_norm(y, stream, m.norm_2, h, stream)
        q = rotate(m, h, cache, positions, slots)
        if visible is None:
            return None
        out, lse = empty(N, HQ, D), empty(N, HQ, dtype=F32)
        kda.paged_attention(q[:, 0], *cache, table.cuda(), visible, out, D ** -0.5, lse=lse)
        wo, wl, bo, bl = ref.attention(q[:, 0].cpu(), cache[0].cpu(), cache[1].cpu(), table, visible.cpu(), D ** -0.5)
        check("attention", out, wo, bo)
        check("lse", lse, wl, bl)
        final = empty(*x.shape)
        kda.residual_norm(project(out.flatten(1), m.w_out)[:, None].contiguous(), stream, m.norm_1, final, stream)
        return final

    positions = torch.cat([torch.arange(n) for n in lengths])[None].cuda()
    slots = torch.tensor([[slot(n, t) for n in range(N) for t in range(lengths[n])]]).cuda()
    layers(torch.randn(1, T, DIM, generator=gen).to(BF).cuda(), cu, positions, slots, None)
    x = torch.randn(N, 1, DIM, generator=gen).to(BF).cuda()
    for step in range(steps):
        at = [n + step for n in lengths]
        x = layers(x, None, torch.tensor(at)[:, None].cuda(), torch.tensor([[slot(n, t)] for n, t in enumerate(at)]).cuda(),
                   torch.tensor(at, dtype=torch.int32).cuda() + 1)
        assert torch.isfinite(x.float()).all()
