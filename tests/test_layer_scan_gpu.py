"""The chunked scan where its arithmetic and its masks can go wrong: operand
splits under cancellation, quiet tails, non-finite inputs, workspaces."""
import pytest
import torch

import layer_ref as ref
from gated_delta_rule_36_amd import _lib
from test_layer_gpu import BF16, F32, check, normal, on_gpu, scan, ssm_case, ssm_inputs

pytestmark = pytest.mark.gpu


def still(T, H, P, N):
    """Inputs of a scan whose state never decays (exp(A_log) = 0) and whose x, dt, b and c are 0."""
    z = lambda *s: torch.zeros(*s, dtype=BF16)  # noqa: E731
    return dict(x=z(1, T, H, P), dt=z(1, T, H), b=z(1, T, 1, N), c=z(1, T, 1, N), A_log=torch.full((H,), -200.0), D=None,
                dt_bias=None, z=None, initial=torch.zeros(1, H, P, N))


def mantissas(n, g):
    """n numbers in [1, 2) of 24 bits, and the nearest bf16 numbers."""
    v = 1 + torch.randint(0, 1 << 23, (n,), generator=g).float() * 2.0 ** -23
    return v, v.to(BF16).float()


# A value v of 24 bits less its nearest bf16 number r, an operand that is exact: two parts of v, each rounded to
# nearest, leave 2^-8 2^-9 v at most (|v - r| <= 2^-8 in [1, 2), half a step of which is 2^-17); the sums are exact up
# to 2^-24 of |v|, a handful of times.
def check_rest(name, got, v, r):
    want = v.double() - r.double()
    check(name, got, want, (2.0 ** -17 + 2.0 ** -20) * torch.ones_like(want))


@pytest.mark.parametrize("N", [64, 128, 256])
def test_scan_state_operand_is_good_to_two_rounded_parts(N):
    T, H, P = 70, 2, 64
    a, g = still(T, H, P, N), torch.Generator().manual_seed(N)
    v, r = mantissas(H * P, g)
    a["initial"][0, :, :, 3], a["initial"][0, :, :, 9] = v.view(H, P), r.view(H, P)
    a["c"][..., 3], a["c"][..., 9] = 1.0, -1.0
    d = {k: on_gpu(t) for k, t in a.items()}
    out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty(1, H, P, N, device="cuda")
    scan(d, out, fin, dt_softplus=False)
    assert torch.equal(fin.cpu(), a["initial"])
    for t in range(T):
        check_rest(f"token {t}", out[0, t].flatten(), v, r)


@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("s,t", [(0, 0), (3, 20), (3, 40), (35, 60), (35, 35), (5, 69)])
def test_scan_weighted_operand_is_good_to_two_rounded_parts(N, s, t):
    """Token s writes v = dt x, and token t reads it beside -r from the initial state."""
    T, H, P = 70, 64, 32
    a, g = still(T, H, P, N), torch.Generator().manual_seed(N + s)
    v, r = mantissas(H, g)
    a["dt_bias"] = v                   # dt = v at every token; x is 0 but at s
    a["x"][0, s] = 1.0
    a["b"][0, s, 0, 3] = 1.0
    a["initial"][0, :, :, 9] = r[:, None]
    a["c"][0, t, 0, 3], a["c"][0, t, 0, 9] = 1.0, -1.0
    d = {k: on_gpu(u) for k, u in a.items()}
    out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty(1, H, P, N, device="cuda")
    scan(d, out, fin, dt_softplus=False)
    check_rest(f"token {t}", out[0, t].flatten(), v[:, None].expand(H, P).flatten(), r[:, None].expand(H, P).flatten())
    assert torch.equal(fin[0, :, :, 3].cpu(), v[:, None].expand(H, P))


@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("s,t", [(2, 2), (3, 30), (3, 50), (40, 63)])
def test_scan_product_operand_is_good_to_two_rounded_parts(N, s, t):
    """c_t . b_s is a number of 24 bits; the token's x takes it as it is, beside the nearest bf16 number less."""
    T, H, P = 70, 2, 32
    g = torch.Generator().manual_seed(s + t)
    for _ in range(24):
        a = still(T, H, P, N)
        v, r = mantissas(1, g)
        a["dt_bias"] = torch.ones(H)
        a["x"][0, s] = 1.0
        rest = v.double()
        for n in range(3):             # v in three bf16 numbers
            a["b"][0, s, 0, n] = rest.to(BF16).item()
            rest = rest - rest.to(BF16).double()
            a["c"][0, t, 0, n] = 1.0
        a["initial"][..., 9] = r.item()
        a["c"][0, t, 0, 9] = -1.0
        d = {k: on_gpu(u) for k, u in a.items()}
        out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty(1, H, P, N, device="cuda")
        scan(d, out, fin, dt_softplus=False)
        check_rest(f"token {t}", out[0, t].flatten(), v.expand(H * P), r.expand(H * P))


@pytest.mark.parametrize("P,N", [(64, 128), (64, 64), (32, 256)])
@pytest.mark.parametrize("segment_tokens", [None, 4096])
@pytest.mark.parametrize("T,tail", [(320, 32), (320, 64), (300, 32), (300, 64)])
def test_scan_state_of_a_quiet_tail_is_as_exact_as_fp32(P, N, segment_tokens, T, tail):
    """Tokens whose x is zero or small at a prompt's end (padding, masked ones): the state is what earlier ones left,
    and as exact.  Independent roundings leave 2^-20 (as where no token is quiet); the log decay d from the tail's start
    carries up to six relative roundings common to all tokens (e^A_log, log2 e, their product, the steps, their product
    and sums), which are 6 d ln 2 2^-24 of the state."""
    g = torch.Generator().manual_seed(N + T + tail)
    H = 8
    per_block = torch.linspace(4.2, 12.0, H)
    for scale in (0.0, 0.01):
        a = ssm_inputs(g, 1, T, H, P, 1, N, 1, gate=False)
        a["x"][:, T - tail:] *= scale
        a["dt"], a["dt_bias"] = torch.full((1, T, H), 0.125, dtype=BF16), None
        a["A_log"] = torch.log(per_block / 32 / 0.125 * 0.693147181)
        want, final, _, _ = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], None, None, a["initial"], None, False)
        d = {k: on_gpu(v) for k, v in a.items()}
        out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
        scan(d, out, fin, segment_tokens=segment_tokens, dt_softplus=False)
        for h in range(H):
            error = float((fin[:, h].double().cpu() - final[:, h]).norm() / final[:, h].norm())
            bound = 2.0 ** -20 + 6 * 0.6931 * 2.0 ** -24 * float(per_block[h]) * tail / 32
            assert error <= bound, (scale, h, error, bound)


@pytest.mark.parametrize("T,segment_tokens", [(4, None), (70, None), (300, 64), (300, None)])
@pytest.mark.parametrize("N", [64, 256])
def test_scan_decay_parameters_that_are_not_finite(T, segment_tokens, N):
    """A_log = NaN makes its head's outputs and state NaN, at any length; A_log = inf forgets everything before a
    token (exp(-inf dt) = 0), so its state is the last token's, also where the last tile is not full."""
    g = torch.Generator().manual_seed(T + N)
    H, P = 3, 32
    a = ssm_inputs(g, 1, T, H, P, 1, N, 1)
    d = {k: on_gpu(v) for k, v in a.items()}

    def run():
        out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
        scan(d, out, fin, segment_tokens=segment_tokens)
        return out, fin

    clean, cf = run()
    d["A_log"][1] = a["A_log"][1] = float("nan")
    out, fin = run()
    assert bool(out[:, :, 1].isnan().all()) and bool(fin[:, 1].isnan().all())
    assert torch.equal(out[:, :, [0, 2]], clean[:, :, [0, 2]]) and torch.equal(fin[:, [0, 2]], cf[:, [0, 2]])
    d["A_log"][1] = a["A_log"][1] = float("inf")
    out, fin = run()
    want, final, scale, fscale = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], a["dt_bias"], a["z"],
                                         a["initial"])
    # the tolerances of the parity tests
    check("final_state", fin, final, 2.0 ** -15 * fscale)
    check("out", out, want, 2.0 ** -14 * scale)


NAN, INF, LOWEST = float("nan"), float("inf"), torch.finfo(BF16).min


@pytest.mark.parametrize("T,segment_tokens", [(6, None), (150, None), (150, 64), (150, 96)])
@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("kind,value", [("x", NAN), ("x", INF), ("x", -INF), ("x", LOWEST), ("dt", NAN), ("dt", INF),
                                        ("dt", LOWEST), ("b", NAN), ("b", -INF), ("c", NAN), ("c", INF)])
def test_scan_inputs_that_are_not_finite_never_reach_earlier_tokens(T, segment_tokens, N, kind, value):
    """One value of a padded or masked token: the outputs before it are those without it, its own and later ones of its
    column (x), head (dt) or group (b; c: its own token) are not finite, and everything else stays as it was.  The
    first head decays little, the second by some 2^-60 in 64 tokens.  LOWEST: with dt a growth by 2^(10^38) (a step
    without softplus); x times its step is beyond fp32, but not what the decay leaves of it, which need not be infinite."""
    g = torch.Generator().manual_seed(T + N)
    H, P = 2, 64
    a = ssm_inputs(g, 1, T, H, P, 1, N, 1)
    a["dt"], a["dt_bias"] = (1 + 0.2 * torch.randn(1, T, H, generator=g)).abs().to(BF16), None
    a["A_log"] = torch.log(torch.tensor([0.1, 0.95]) * 0.6931)
    for s in [0, 3, 5] if T == 6 else [0, 7, 31, 32, 45, 63, 64, 100, 149]:
        a["dt"][0, s] = 2.0
        d = {k: on_gpu(v) for k, v in a.items()}

        def run():
            out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
            scan(d, out, fin, segment_tokens=segment_tokens, dt_softplus=False)
            return out.cpu(), fin.cpu()

        clean, cf = run()
        where = {"x": (0, s, 1, 9), "dt": (0, s, 1), "b": (0, s, 0, 3), "c": (0, s, 0, 3)}[kind]
        for h in range(H if kind in ("x", "dt") else 1):
            at = (*where[:2], h, *where[3:]) if kind in ("x", "dt") else where
            kept = d[kind][at].clone()
            d[kind][at] = value
            out, fin = run()
            d[kind][at] = kept
            touched = torch.zeros(out.shape, dtype=torch.bool)
            if kind == "x":
                touched[:, s:, h, 9] = True
            elif kind == "dt":
                touched[:, s:, h] = True
            else:
                touched[:, s:s + 1 if kind == "c" else T] = True
            if kind == "dt":   # the other tokens' decays are rounded in other units: the parity tests' tolerance
                want, _, scale, _ = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], None, a["z"],
                                            a["initial"], None, False)
                check("out", out[:, :s, h], want[:, :s, h], 2.0 ** -14 * scale[:, :s, h])
                touched[:, :s, h] = True
            assert torch.equal(out[~touched], clean[~touched]), (s, h)
            assert (kind, value) == ("x", LOWEST) or not bool(out[:, s:][touched[:, s:]].isfinite().any()), (s, h)
            if kind == "x":
                assert value == LOWEST or not bool(fin[0, h, 9].isfinite().any())
                fin[0, h, 9] = cf[0, h, 9]
            if kind == "dt":
                assert not bool(fin[0, h].isfinite().any())
                fin[0, h] = cf[0, h]
            if kind != "b":
                assert torch.equal(fin, cf), (s, h)


@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("up,down", [((0, 16), (32, 48)), ((2, 30), (31, 60)), ((32, 40), (48, 64)), ((0, 30), (64, 90))])
def test_scan_growth_that_a_decay_takes_back(N, up, down):
    """Negative steps (without softplus) grow the state by 2^100 and positive ones take 2^138 of it, within a block, a
    tile or from one to the next: the tolerances of the parity tests hold, relative to the sums' absolute values."""
    g = torch.Generator().manual_seed(N)
    T, H, P = 100, 2, 32
    a = ssm_inputs(g, 1, T, H, P, 1, N, 1, gate=False)
    a["dt"], a["dt_bias"] = torch.full((1, T, H), 2.0 ** -7, dtype=BF16), None
    a["A_log"] = torch.log(torch.tensor([0.6931, 0.6931]))
    a["dt"][:, up[0]:up[1]] = -100.0 / (up[1] - up[0])
    a["dt"][:, down[0]:down[1]] = 138.0 / (down[1] - down[0])
    want, final, scale, fscale = ref.ssm(a["x"], a["dt"], a["b"], a["c"], a["A_log"], a["D"], None, None, a["initial"], None,
                                         False)
    d = {k: on_gpu(v) for k, v in a.items()}
    out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
    scan(d, out, fin, dt_softplus=False)
    check("final_state", fin, final, 2.0 ** -15 * fscale)
    check("out", out, want, 2.0 ** -14 * scale)


def ssm_args(a, out, initial, final, segment_tokens, cu=None):
    """The C arguments of a scan of GPU tensors `a`, without a workspace."""
    (B, T, H, P), N = a["x"].shape, a["b"].shape[3]
    args = _lib.SsmArgs(out=out.data_ptr(), A_log=a["A_log"].data_ptr(), D=a["D"].data_ptr(), dt_bias=a["dt_bias"].data_ptr(),
                        initial_state=initial.data_ptr(), final_state=final.data_ptr(), B=B, T=T, H=H, P=P, G=1, N=N,
                        initial_state_dtype=_lib.KDA_DTYPE_FP32, final_state_dtype=_lib.KDA_DTYPE_FP32, softplus=1,
                        seg_tokens=segment_tokens)
    if cu is not None:
        args.cu_seqlens, args.num_seqs = cu.data_ptr(), cu.numel() - 1
    for k in ("x", "dt", "b", "c", "z"):
        setattr(args, k, a[k].data_ptr())
        setattr(args, f"{k}_stride_b", a[k].stride(0))
        setattr(args, f"{k}_stride_t", a[k].stride(1))
    return args


@pytest.mark.parametrize("cu", [[0, 130], list(range(131)), [0, 1, 2, 3, 100, 130], [0] + [2 * i for i in range(1, 66)], [0, 0, 64, 64, 130],
                                [130, 90, 40, 0], [0, 130, 0, 130, 0, 130], [5, 127, 3, 130, 64, 64, -9, 1 << 40]])
@pytest.mark.parametrize("segment_tokens", [32, 64, 96])
def test_scan_stays_in_its_workspace(cu, segment_tokens):
    """The workspace of exactly the bytes asked for lies between two guards, for offsets in order and not; the same
    results as with the library's own, in place too."""
    g = torch.Generator().manual_seed(len(cu))
    T, H, P, N, n, edge = 130, 3, 32, 32, len(cu) - 1, 1 << 16
    a = {k: on_gpu(v) for k, v in ssm_inputs(g, 1, T, H, P, 1, N, n).items()}
    cug = torch.tensor(cu, dtype=torch.int64, device="cuda")
    out, fin = torch.zeros(1, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(a["initial"])
    scan(a, out, fin, cu_seqlens=cug, check_cu_seqlens=False, segment_tokens=segment_tokens)
    state, again = a["initial"].clone(), torch.zeros_like(out)
    args = ssm_args(a, again, state, state, segment_tokens, cug)
    lib = _lib.load()
    nbytes = lib.kda_ssm_workspace_bytes(args)
    assert nbytes > 0
    whole = torch.full((2 * edge + nbytes,), 7, dtype=torch.uint8, device="cuda")
    args.workspace, args.workspace_bytes = whole.data_ptr() + edge, nbytes
    assert lib.kda_ssm_fwd(args, torch.cuda.current_stream().cuda_stream) == _lib.KDA_OK
    torch.cuda.synchronize()
    assert bool((whole[:edge] == 7).all()) and bool((whole[edge + nbytes:] == 7).all())
    if cu == sorted(cu):
        assert torch.equal(out, again) and torch.equal(fin, state)


@pytest.mark.parametrize("n,longest", [(200, 1), (300, 5), (60, 1), (150, 90)])
@pytest.mark.parametrize("state", [BF16, F32])
def test_scan_of_many_short_sequences(n, longest, state):
    """Packed single tokens and short prompts, with a longer one among them, states in place."""
    g = torch.Generator().manual_seed(n)
    lengths = torch.randint(0, longest + 1, (n,), generator=g)
    lengths[n // 3], lengths[n - 1] = 150, 1
    cu = [0] + torch.cumsum(lengths, 0).tolist()
    for segment_tokens in (None, 32):
        ssm_case(1, cu[-1], 2, 32, 1, 64, seed=n, cu=cu, state=state, in_place=True, segment_tokens=segment_tokens)


def test_scan_decay_of_a_head_over_two_workgroups_has_one_writer():
    """Heads of 96 columns, 8 units of 32 a workgroup: head 2 lies in two.  The first stops where all its heads have
    forgotten, the second has one that keeps all and goes on.  The head's sum of logarithms in the workspace is the
    first's, whichever ends last."""
    g = torch.Generator().manual_seed(1)
    T, H, P, N, seg = 1920, 6, 96, 32, 960
    a = ssm_inputs(g, 1, T, H, P, 1, N, 1)
    a["dt"], a["dt_bias"] = torch.full((1, T, H), 20.5, dtype=BF16), torch.zeros(H)
    a["A_log"] = torch.log(torch.tensor([40.0, 40.0, 40.0, 1e-3, 40.0, 40.0]) / 64 / 20.5 * 0.6931)  # 2^-40 a tile
    d = {k: on_gpu(v) for k, v in a.items()}
    out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["initial"])
    args = ssm_args(d, out, d["initial"], fin, seg)
    nbytes = _lib.load().kda_ssm_workspace_bytes(args)
    work = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    args.workspace, args.workspace_bytes = work.data_ptr(), nbytes
    for _ in range(4):
        assert _lib.load().kda_ssm_fwd(args, torch.cuda.current_stream().cuda_stream) == _lib.KDA_OK
        slabs = nbytes // (4 * (H * P * N + H))
        logs = work[4 * slabs * H * P * N:][:4 * H].view(torch.float32).cpu()
        assert bool((logs[:3] < -300).all()) and bool((logs[:3] > -420).all()), logs   # of 600 in all
        assert -1.0 < float(logs[3]) < 0.0


@pytest.mark.parametrize("N", [64, 128, 256])
@pytest.mark.parametrize("step", [1.0015, 1.0025, 1.0039, 1.5])
def test_scan_products_next_to_fp32s_largest_never_reach_earlier_tokens(N, step):
    """x = bf16's lowest number times a step just above 1: between bf16's largest number and fp32's, or beyond."""
    T, H, P = 90, 1, 32
    a, g = still(T, H, P, N), torch.Generator().manual_seed(N)
    a["b"], a["c"] = normal(g, 1, T, 1, N), normal(g, 1, T, 1, N)
    a["x"], a["initial"] = normal(g, 1, T, H, P), torch.randn(1, H, P, N, generator=g)
    a["dt_bias"] = torch.full((H,), step)
    for s in (1, 31, 40, 63, 64, 85):
        outs = []
        for value in (1.0, LOWEST):
            a["x"][0, s, 0, 5] = value
            d = {k: on_gpu(u) for k, u in a.items()}
            out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty(1, H, P, N, device="cuda")
            scan(d, out, fin, dt_softplus=False)
            outs.append(out.cpu())
        a["x"][0, s, 0, 5] = 1.0
        touched = torch.zeros(out.shape, dtype=torch.bool)
        touched[:, s:, 0, 5] = True
        assert torch.equal(outs[0][~touched], outs[1][~touched]), s


@pytest.mark.parametrize("N", [64, 128, 256])
def test_scan_large_numbers_of_both_signs_never_reach_earlier_tokens(N):
    """Neighbours of opposite sign in one load: what is looked for must not cancel."""
    T, H, P = 90, 2, 32
    a, g = still(T, H, P, N), torch.Generator().manual_seed(N)
    a["b"], a["c"], a["x"] = normal(g, 1, T, 1, N), normal(g, 1, T, 1, N), normal(g, 1, T, H, P)
    a["dt_bias"] = torch.full((H,), 1.5)
    for s, pairs in ((31, [(4, 5)]), (40, [(4, 5), (6, 7)]), (63, [(4, 6)]), (85, [(5, 6), (9, 24)])):
        outs, kept = [], a["x"].clone()
        for sign in (None, 1.0, -1.0):
            a["x"] = kept.clone()
            for i, j in pairs if sign else ():
                a["x"][0, s, 0, i], a["x"][0, s, 0, j] = sign * LOWEST, -sign * LOWEST
            d = {k: on_gpu(u) for k, u in a.items()}
            out, fin = torch.empty(1, T, H, P, dtype=BF16, device="cuda"), torch.empty(1, H, P, N, device="cuda")
            scan(d, out, fin, dt_softplus=False)
            outs.append(out.cpu())
        a["x"] = kept
        for out in outs[1:]:
            assert torch.equal(outs[0][:, :s], out[:, :s]) and torch.equal(outs[0][:, :, 1], out[:, :, 1]), s
