"""delta_fwd on the GPU against the token recurrence in 64 bits: lengths, head
layouts, states, packed sequences, strides, strong and weak decays, inputs that
are not finite."""
import math

import pytest
import torch

import gated_delta_rule_36_amd as kda
import mixer_ref as ref
from mixer_ref import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def inputs(B, T, G, H, K, V, seed=0, n=None, state=F32, initial=True, alike=0.0):
    """q and k as a convolution with SiLU and its L2 norm leaves them; `alike` mixes one direction into every key."""
    g = torch.Generator().manual_seed(seed)
    def normal(*shape): return torch.randn(*shape, generator=g)
    def unit(x): return (x / x.norm(dim=-1, keepdim=True)).to(BF)
    silu = torch.nn.functional.silu
    x = dict(q=unit(silu(normal(B, T, G, K))), k=unit(silu(normal(B, T, G, K)) + alike * normal(K)),
             v=silu(normal(B, T, H, V)).to(BF), g=normal(B, T, H).to(BF), beta=normal(B, T, H).to(BF), scale=K ** -0.5,
             A_log=torch.log(1 + 15 * torch.rand(H, generator=g)))
    step = torch.exp(torch.rand(H, generator=g) * math.log(100.0) + math.log(1e-3))
    x["dt_bias"] = step + torch.log(-torch.expm1(-step))
    x["initial"] = (0.3 * normal(n or B, H, V, K)).to(state) if initial else None
    return x


def call(x, cu=None, state=F32, final=True, seg=None, **over):
    """(out, final state) of a call with x's tensors on the GPU; unwritten outputs stay NaN."""
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in {**x, **over}.items()}
    B, T, H, V = y["v"].shape
    n = B if cu is None else len(cu) - 1
    out = torch.full((B, T, H, V), NAN, dtype=BF, device="cuda")
    fin = torch.full((n, H, V, y["k"].shape[-1]), NAN, dtype=state, device="cuda") if final else None
    kda.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["scale"], out, y["A_log"], y["dt_bias"],
                  initial_state=y["initial"], final_state=fin,
                  cu_seqlens=None if cu is None else torch.tensor(cu, device="cuda"), check_cu_seqlens=False,
                  segment_tokens=seg)
    return out, fin


def row_bound(fin, want, fbound):
    """Rows of the state as one number each, the length of the error, against the bound."""
    half = torch.finfo(fin.dtype).eps / 2 if fin.dtype == BF else 2.0 ** -24
    err = (fin.cpu().double() - want).norm(dim=-1)
    room = fbound + half * want.norm(dim=-1) * 1.001 + 2.0 ** -100
    worst = float((err / room).max())
    print(f"[check] state: worst {worst:.3f} of what is allowed", flush=True)
    assert worst <= 1.0


def hold(x, cu=None, state=F32, seg=None):
    out, fin = call(x, cu, state, seg=seg)
    wo, wf, bo, bf = ref.delta(**x, cu=cu)
    check("out", out, wo, bo)
    row_bound(fin, wf, bf)
    return out, fin, wf


@pytest.mark.parametrize("T", [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 48, 63, 64, 65, 79, 127, 128, 129, 200, 321])
def test_lengths(T):
    hold(inputs(2, T, 1, 2, 128, 32, seed=T))


@pytest.mark.parametrize("G,H,K,V", [(1, 1, 64, 16), (2, 2, 64, 48), (1, 3, 128, 128), (2, 4, 128, 96), (4, 4, 256, 64),
                                     (1, 2, 256, 256), (1, 1, 64, 512), (3, 9, 64, 80), (1, 1, 128, 272)])
@pytest.mark.parametrize("T", [3, 150])
def test_heads(G, H, K, V, T):
    hold(inputs(1, T, G, H, K, V, seed=K + V))


@pytest.mark.parametrize("state", [F32, BF])
@pytest.mark.parametrize("T", [5, 130])
def test_states(state, T):
    x = inputs(2, T, 1, 2, 128, 64, seed=3, state=state)
    out, fin, _ = hold(x, state=state)
    # in place
    s = x["initial"].cuda()
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    again = torch.empty_like(out)
    kda.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["scale"], again, y["A_log"], y["dt_bias"],
                  initial_state=s, final_state=s)
    assert torch.equal(again, out) and torch.equal(s, fin)
    # without either state, without a bias
    x["initial"] = x["dt_bias"] = None
    hold(x, state=state)
    out, fin = call(x, final=False)
    check("out", out, *ref.delta(**x)[0:3:2])


@pytest.mark.parametrize("cu", [[0, 100], [0, 0, 1, 1, 30, 100], [0, 64, 65, 100], [5, 20, 20, 90], [0] * 70 + [100],
                                list(range(101)), [0, 3, 6, 9, 40, 57, 89, 100]])
def test_packed(cu):
    x = inputs(1, 100, 1, 2, 64, 32, seed=len(cu), n=len(cu) - 1)
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    out = torch.full((1, 100, 2, 32), NAN, dtype=BF, device="cuda")
    fin = torch.full((len(cu) - 1, 2, 32, 64), NAN, dtype=F32, device="cuda")
    kda.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["scale"], out, y["A_log"], y["dt_bias"],
                  initial_state=y["initial"], final_state=fin, cu_seqlens=torch.tensor(cu, device="cuda"),
                  check_cu_seqlens=False)
    wo, wf, bo, bf = ref.delta(**x, cu=cu)
    check("out", out, wo, bo)  # rows outside every sequence stay as they were
    row_bound(fin, wf, bf)


def test_packed_offsets_that_are_out_of_order_stay_inside():
    x = inputs(1, 90, 1, 1, 64, 16, seed=9, n=3)
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    out = torch.zeros(1, 90, 1, 16, dtype=BF, device="cuda")
    fin = torch.zeros(3, 1, 16, 64, device="cuda")
    kda.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["scale"], out, y["A_log"], initial_state=y["initial"],
                  final_state=fin, cu_seqlens=torch.tensor([-5, 40, 20, 1 << 40], device="cuda"), check_cu_seqlens=False)
    assert torch.isfinite(fin).all()


def test_slices_of_projections():
    """Odd places and strides; the same numbers as from contiguous tensors."""
    x = inputs(2, 70, 1, 2, 64, 32, seed=21)
    out, fin = call(x)
    def within(t, before, after):
        return torch.cat([torch.full((*t.shape[:2], before), NAN, dtype=BF), t.flatten(2),
                          torch.full((*t.shape[:2], after), NAN, dtype=BF)], 2).cuda()[..., before:before + t[0, 0].numel()].view_as(t) \
            if t.dim() == 3 else torch.cat([torch.full((*t.shape[:2], before), NAN, dtype=BF), t.flatten(2),
                                            torch.full((*t.shape[:2], after), NAN, dtype=BF)],
                                           2).cuda()[..., before:before + t[0, 0].numel()].unflatten(-1, t.shape[2:])
    y = {k: within(x[k], 3, 4) for k in ("q", "k", "v")}
    y.update({k: within(x[k], 1, 2) for k in ("g", "beta")})
    again, fin2 = call(x, **y)
    assert torch.equal(out, again) and torch.equal(fin, fin2)


@pytest.mark.parametrize("T", [6, 200])
@pytest.mark.parametrize("A,shift", [(-20.0, 0.0), (3.0, 6.0), (8.0, 10.0), (2.77, -8.0)])
def test_decays(A, shift, T):
    """From none at all to a state that is gone after each token, and both in one chunk."""
    x = inputs(1, T, 1, 2, 64, 32, seed=31)
    x["A_log"] = torch.full((2,), A)
    x["g"] = (x["g"].float() * 3 + shift).to(BF)
    x["g"][:, ::17] = 30.0  # a strong one now and then among weak ones
    hold(x)


@pytest.mark.parametrize("alike", [0.0, 1.0, 5.0])
@pytest.mark.parametrize("strength", [-20.0, 0.0, 20.0])
def test_keys_alike_and_write_strengths(alike, strength):
    x = inputs(1, 200, 1, 2, 128, 32, seed=41, alike=alike)
    x["beta"] = (x["beta"].float() + strength).to(BF)
    x["A_log"] -= 4.0
    hold(x)


def test_the_same_key_every_time():
    """Keys all equal, full strength, hardly any decay: every token replaces the one before."""
    x = inputs(1, 140, 1, 1, 64, 16, seed=51)
    x["k"] = x["k"][:, :1].expand(1, 140, 1, 64).contiguous()
    x["beta"][:] = 30.0
    x["A_log"] -= 10.0
    hold(x)


def test_fp32_state_accuracy():
    """The fp32 state is good to fp32's own digits: 2^-20 of its length after 2000 tokens."""
    x = inputs(1, 2000, 1, 2, 128, 32, seed=61)
    x["A_log"] -= 3.0
    _, fin = call(x)
    want = ref.delta(**x)[1]
    rel = float((fin.cpu().double() - want).norm() / want.norm())
    print(f"[check] state after 2000 tokens: {rel:.3g}", flush=True)
    assert rel <= 2.0 ** -20


@pytest.mark.parametrize("T", [8, 180])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
def test_non_finite_inputs_reach_no_earlier_token_and_no_other_sequence(where, value, T):
    x = inputs(3, T, 1, 2, 64, 32, seed=71)
    clean, clean_fin = call(x)
    t = T // 2 + 3
    bad = x[where].clone()
    bad[1, t, 0] = value if where in ("g", "beta") else bad[1, t, 0]
    if where not in ("g", "beta"):
        bad[1, t, 0, 5] = value
    out, fin = call(x, **{where: bad})
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert torch.equal(fin[0], clean_fin[0]) and torch.equal(fin[2], clean_fin[2])
    assert torch.equal(out[1, :t], clean[1, :t])
    if where == "q":
        assert torch.equal(out[1, t + 1:], clean[1, t + 1:]) and torch.equal(fin, clean_fin)
        assert not torch.isfinite(out[1, t].float()).any()
    elif where != "k":
        assert torch.equal(out[1, :, 1], clean[1, :, 1]) and torch.equal(fin[1, 1], clean_fin[1, 1])
    if where in ("k", "v"):
        assert not torch.isfinite(fin[1, 0, 5]).all()


def test_large_values_stay_finite_where_the_recurrence_does():
    x = inputs(1, 150, 1, 1, 64, 16, seed=81)
    x["v"] = (x["v"].float() * 1e30).to(BF)
    x["initial"] = x["initial"] * 1e30
    hold(x)
    x["v"] = (x["v"].float() * 1e-66).to(BF)
    x["initial"] = x["initial"] * 1e-66
    x["scale"] = 1.0
    out, fin = call(x)
    assert torch.isfinite(out.float()).all() and torch.isfinite(fin).all()


def test_two_captured_graphs_and_eager_calls_between():
    x = inputs(2, 100, 1, 2, 128, 64, seed=91)
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    want, want_fin = call(x)
    def run(out, fin):
        kda.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["scale"], out, y["A_log"], y["dt_bias"],
                      initial_state=y["initial"], final_state=fin)
    outs = [(torch.empty_like(want), torch.empty_like(want_fin)) for _ in range(2)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(*outs[0])
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in outs]
    for graph, o in zip(graphs, outs):
        with torch.cuda.graph(graph):
            run(*o)
    for _ in range(4):
        for graph, (o, f) in zip(graphs, outs):
            o.fill_(NAN)
            f.fill_(NAN)
            graph.replay()
        eager = call(x)
        torch.cuda.synchronize()
        for o, f in (*outs, eager):
            assert torch.equal(o, want) and torch.equal(f, want_fin)


def test_two_streams():
    a, b = inputs(1, 300, 1, 2, 64, 32, seed=101), inputs(1, 170, 1, 2, 64, 32, seed=102)
    want = [call(x) for x in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(10):
        for s, x, o in zip(streams, (a, b), got):
            with torch.cuda.stream(s):
                o.append(call(x))
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(w[0], y) and torch.equal(w[1], f) for y, f in o)


# ---------------------------------------------------------------------------
# segments
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("K,V", [(64, 16), (64, 96), (128, 32), (128, 144), (256, 48)])
@pytest.mark.parametrize("T,seg", [(64, 64), (65, 64), (128, 64), (129, 64), (300, 64), (640, 128), (700, 256)])
def test_segments(K, V, T, seg):
    hold(inputs(2, T, 1, 2, K, V, seed=T + V), seg=seg)


@pytest.mark.parametrize("state", [F32, BF])
def test_segments_without_and_with_states_in_place(state):
    x = inputs(1, 400, 1, 2, 64, 32, seed=111, state=state)
    out, fin, _ = hold(x, state=state, seg=64)
    s = x["initial"].cuda()
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    again = torch.empty_like(out)
    kda.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["scale"], again, y["A_log"], y["dt_bias"],
                  initial_state=s, final_state=s, segment_tokens=64)
    assert torch.equal(again, out) and torch.equal(s, fin)
    x["initial"] = None
    hold(x, state=state, seg=64)
    out, _ = call(x, final=False, seg=64)
    check("out", out, *ref.delta(**x)[0:3:2])


@pytest.mark.parametrize("cu", [[0, 500], [0, 64, 128, 500], [0, 1, 1, 200, 327, 500], [7, 300, 310, 480],
                                [0] + [5 * i for i in range(1, 70)] + [500], list(range(0, 501, 100))])
def test_packed_segments(cu):
    hold(inputs(1, 500, 1, 2, 64, 32, seed=len(cu), n=len(cu) - 1), cu=cu, seg=64)


def test_packed_segments_with_offsets_that_are_out_of_order_stay_inside():
    x = inputs(1, 390, 1, 1, 64, 16, seed=9, n=4)
    out, fin = call(x, cu=[-5, 340, 20, 1 << 40, 3], seg=64)
    assert out.shape == (1, 390, 1, 16) and fin.shape == (4, 1, 16, 64)


def test_the_library_cuts_one_long_sequence_of_few_heads():
    from gated_delta_rule_36_amd import _lib
    size = lambda **kw: _lib.load().kda_delta_workspace_bytes(_lib.DeltaArgs(B=1, H=2, G=1, K=128, V=128, **kw))  # noqa: E731
    assert size(T=4096) > 0 and size(T=512) == 0 and size(T=4096, seg_tokens=4096) == 0
    x = inputs(1, 4096, 1, 2, 128, 32, seed=121)
    x["A_log"] -= 4.0
    out, fin, _ = hold(x)
    whole, whole_fin = call(x, seg=4096)
    print(f"[check] segments against one: {float((fin - whole_fin).norm() / whole_fin.norm()):.3g}", flush=True)
    want = ref.delta(**x)[1]
    assert float((fin.cpu().double() - want).norm() / want.norm()) <= 2.0 ** -20


@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta"])
def test_non_finite_inputs_in_a_segment(where):
    x = inputs(2, 500, 1, 2, 64, 32, seed=131)
    clean, clean_fin = call(x, seg=64)
    t = 200
    bad = x[where].clone()
    if where in ("g", "beta"):
        bad[1, t, 0] = NAN
    else:
        bad[1, t, 0, 5] = NAN
    out, fin = call(x, seg=64, **{where: bad})
    assert torch.equal(out[0], clean[0]) and torch.equal(fin[0], clean_fin[0])
    assert torch.equal(out[1, :t], clean[1, :t])
    if where == "q":
        assert torch.equal(out[1, t + 1:], clean[1, t + 1:]) and torch.equal(fin, clean_fin)
    elif where != "k":
        assert torch.equal(out[1, :, 1], clean[1, :, 1]) and torch.equal(fin[1, 1], clean_fin[1, 1])
    if where in ("k", "v"):
        assert not torch.isfinite(fin[1, 0, 5]).all()


def test_segments_replay_from_a_graph():
    x = inputs(1, 600, 1, 2, 128, 64, seed=141)
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    want, want_fin = call(x, seg=64)
    out, fin = torch.empty_like(want), torch.empty_like(want_fin)
    def run():
        kda.delta_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], y["scale"], out, y["A_log"], y["dt_bias"],
                      initial_state=y["initial"], final_state=fin, segment_tokens=64)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(4):
        out.fill_(NAN)
        fin.fill_(NAN)
        graph.replay()
        eager = call(x, seg=64)
        torch.cuda.synchronize()
        for o, f in ((out, fin), eager):
            assert torch.equal(o, want) and torch.equal(f, want_fin)


# ---------------------------------------------------------------------------
# many packed sequences
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("cu", [list(range(9)), [0, 1, 2, 5, 5, 8, 12, 14, 14], [3] * 20 + [40], [0] + [1 + i // 2 for i in range(80)]])
@pytest.mark.parametrize("seg", [None, 64])
def test_packed_single_tokens(cu, seg):
    """A decoding step of packed requests: one or two tokens each, some of none, one of more; rows behind the last."""
    T = cu[-1] + 2
    hold(inputs(1, T, 2, 4, 128, 96, seed=T, n=len(cu) - 1), cu=cu, seg=seg)


@pytest.mark.parametrize("state", [F32, BF])
def test_more_packed_sequences_than_lanes(state):
    cu = [0]
    for i in range(70):
        cu.append(cu[-1] + (i * 37) % 90 * (i % 3 != 1))
    hold(inputs(1, cu[-1] + 3, 1, 2, 64, 32, seed=151, n=70, state=state), cu=cu, state=state)


def test_segments_on_two_streams():
    a, b = inputs(1, 600, 1, 2, 64, 32, seed=161), inputs(1, 470, 1, 2, 64, 32, seed=162)
    want = [call(x, seg=64) for x in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(10):
        for s, x, o in zip(streams, (a, b), got):
            with torch.cuda.stream(s):
                o.append(call(x, seg=64))
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(w[0], y) and torch.equal(w[1], f) for y, f in o)


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T", [4, 8200])
def test_outputs_past_32_bits(T):
    """Values and outputs of 2^31 elements and more: the last sequence as it is by itself."""
    H, V, K = 32, 512, 64
    B = (1 << 31) // (T * H * V) + 2
    g = torch.Generator("cuda").manual_seed(171)
    def normal(*shape): return torch.randn(*shape, generator=g, device="cuda", dtype=BF)
    k = torch.nn.functional.normalize(normal(B, T, 1, K).float(), dim=-1).to(BF)
    q, gate, beta = normal(B, T, 1, K), normal(B, T, H), normal(B, T, H)
    v = torch.empty(B, T, H, V, device="cuda", dtype=BF)
    v[0].normal_(generator=g)
    v[1:] = v[:1]  # every sequence has the first one's values
    A = torch.zeros(H, device="cuda")
    out = torch.empty_like(v)
    kda.delta_fwd(q, k, v, gate, beta, 0.125, out, A)
    for b in (0, B - 2, B - 1):
        alone = torch.full((1, T, H, V), NAN, device="cuda", dtype=BF)
        one = slice(b, b + 1)
        kda.delta_fwd(q[one], k[one], v[:1], gate[one], beta[one], 0.125, alone, A, segment_tokens=8256)
        assert torch.equal(out[b], alone[0]), b


def test_batch_strides_past_32_bits():
    x = inputs(2, 100, 1, 2, 64, 32, seed=181)
    want, want_fin = call(x)
    room = torch.empty((1 << 32) + (1 << 20), dtype=BF, device="cuda")  # 8 GiB, of which two ends are used
    def far(name, at):
        t = x[name].cuda()
        n = t[0].numel()
        y = room.as_strided(t.shape, ((1 << 32) + 2, *t.stride()[1:]), at)
        y.copy_(t)
        assert n < 1 << 17
        return y
    y = {name: far(name, 1 + (i << 17)) for i, name in enumerate(("q", "k", "v", "g", "beta"))}
    out, fin = call(x, **y)
    assert torch.equal(out, want) and torch.equal(fin, want_fin)


# ---------------------------------------------------------------------------
# workgroups of every width
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T", [9, 150])
@pytest.mark.parametrize("B,G,H,K,V", [(33, 2, 4, 64, 256), (33, 4, 4, 128, 128), (17, 4, 8, 256, 128), (16, 8, 8, 128, 128),
                                       (16, 2, 4, 128, 160), (65, 1, 2, 128, 272), (40, 1, 2, 64, 96), (33, 4, 4, 256, 80)])
def test_many_chains(B, G, H, K, V, T):
    """So many chains that a workgroup takes 32 to 128 columns."""
    hold(inputs(B, T, G, H, K, V, seed=B + T))


@pytest.mark.parametrize("K", [64, 128, 256])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta"])
def test_non_finite_inputs_with_many_chains(where, K):
    x = inputs(65, 150, 2, 4, K, 128, seed=191)
    clean, clean_fin = call(x)
    t, b = 77, 31
    bad = x[where].clone()
    if where in ("g", "beta"):
        bad[b, t, 0] = NAN
    else:
        bad[b, t, 0, 5] = NAN
    out, fin = call(x, **{where: bad})
    other = torch.arange(65, device="cuda") != b
    assert torch.equal(out[other], clean[other]) and torch.equal(fin[other], clean_fin[other])
    assert torch.equal(out[b, :t], clean[b, :t]) and torch.equal(out[b, :, 2:], clean[b, :, 2:])
    if where == "q":
        assert torch.equal(out[b, t + 1:], clean[b, t + 1:]) and torch.equal(fin, clean_fin)
        assert out[b, t, :2].isnan().all()
    elif where == "k":
        assert out[b, t:, :2].isnan().all() and fin[b, :2].isnan().all()
    elif where == "v":
        rest = torch.arange(128, device="cuda") != 5
        assert torch.equal(out[b, :, 0][:, rest], clean[b, :, 0][:, rest]) and torch.equal(fin[b, 0][rest], clean_fin[b, 0][rest])
        assert out[b, t:, 0, 5].isnan().all() and fin[b, 0, 5].isnan().all()
    else:
        assert out[b, t:, 0].isnan().all() and torch.equal(out[b, :, 1], clean[b, :, 1])


def test_the_library_cuts_packed_sequences():
    from gated_delta_rule_36_amd import _lib
    cu = [0, 100, 3000, 3001, 4500]
    args = _lib.DeltaArgs(B=1, T=4500, H=2, G=1, K=128, V=128, cu_seqlens=256, num_seqs=4)
    assert _lib.load().kda_delta_workspace_bytes(args) > 0
    x = inputs(1, 4500, 1, 2, 128, 128, seed=201, n=4)
    x["A_log"] -= 4.0
    _, fin, want = hold(x, cu=cu)
    assert float((fin.cpu().double() - want).norm() / want.norm()) <= 2.0 ** -20
