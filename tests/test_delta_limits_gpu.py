"""delta_fwd where its other tests are silent: what it writes beside its outputs,
the digits of the state for every K, and non-finite numbers behind the join of
segments and in the state a call starts with."""
import ctypes
import math

import pytest
import torch

import mixer_ref as ref
from gated_delta_rule_36_amd import _lib
from test_delta_gpu import BF, F32, NAN, call, inputs

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# what is written
# ---------------------------------------------------------------------------

GUARD = 1 << 14  # bytes


class Guarded:
    """A buffer of `nbytes` between two of GUARD bytes, all of one pattern."""

    def __init__(self, nbytes):
        self.nbytes = nbytes
        self.all = torch.full((nbytes + 2 * GUARD,), 0x5b, dtype=torch.uint8, device="cuda")
        self.bytes = self.all[GUARD:GUARD + nbytes]

    def intact(self):
        return bool((self.all[:GUARD] == 0x5b).all()) and bool((self.all[GUARD + self.nbytes:] == 0x5b).all())


@pytest.mark.parametrize("K,V", [(64, 16), (128, 144), (256, 48)])
@pytest.mark.parametrize("seg", [0, 64, 128])
@pytest.mark.parametrize("cu", [
    [0, 100, 390], [17, 230, 230, 371],                          # in order, with rows in front and behind
    [30, 10, 160, 50], [-5, 340, 20, 1 << 40, 3],                # out of order
    [(i * 131) % 400 - 5 for i in range(71)], [390] * 30 + [0] * 41 + [200] * 9])
def test_writes_nothing_but_its_outputs(cu, seg, K, V):
    """Outputs, final states and workspace between guards: only rows of some sequence are written, whatever order the
    offsets are in."""
    T, H, n = 390, 2, len(cu) - 1
    x = inputs(1, T, 1, H, K, V, seed=K + len(cu), n=n)
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    lib = _lib.load()
    offsets = torch.tensor(cu, device="cuda")
    args = _lib.DeltaArgs(B=1, T=T, H=H, G=1, K=K, V=V, num_seqs=n, seg_tokens=seg, cu_seqlens=offsets.data_ptr())
    work = Guarded(lib.kda_delta_workspace_bytes(ctypes.byref(args)))
    out, fin = Guarded(T * H * V * 2), Guarded(n * H * V * K * 4)
    for name, t in (("q", y["q"]), ("k", y["k"]), ("v", y["v"]), ("g", y["g"]), ("beta", y["beta"])):
        setattr(args, name, t.data_ptr())
        setattr(args, name + "_stride_b", t.stride(0))
        setattr(args, name + "_stride_t", t.stride(1))
    for name, t in (("out", out.bytes), ("A_log", y["A_log"]), ("dt_bias", y["dt_bias"]), ("initial_state", y["initial"]),
                    ("final_state", fin.bytes), ("workspace", work.bytes)):
        setattr(args, name, t.data_ptr())
    args.initial_state_dtype = args.final_state_dtype = _lib.KDA_DTYPE_FP32
    args.scale, args.workspace_bytes = x["scale"], work.nbytes
    assert lib.kda_delta_fwd(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == _lib.KDA_OK
    torch.cuda.synchronize()
    assert out.intact() and fin.intact() and work.intact()
    rows = torch.zeros(T, dtype=torch.bool)
    clamped = [min(max(c, 0), T) for c in cu]
    for a, b in zip(clamped, clamped[1:]):
        rows[a:b] = True
    o = out.bytes.view(T, -1)
    assert (o[~rows.cuda()] == 0x5b).all()
    if clamped != sorted(clamped):
        return  # sequences may overlap, or be more than the grid has slots for
    values, state = o.view(BF).view(1, T, H, V).cpu().double(), fin.bytes.view(F32).view(n, H, V, K).cpu().double()
    want, final, bound, fbound = ref.delta(**x, cu=cu)
    room = ref.HALF_BF16 * (want.abs() + bound) + bound
    assert ((values - want).abs() <= room)[:, rows].all()
    assert ((state - final).norm(dim=-1) <= fbound + 2.0 ** -24 * final.norm(dim=-1) * 1.001 + 2.0 ** -100).all()


# ---------------------------------------------------------------------------
# the state's digits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("seg", [None, 512])
@pytest.mark.parametrize("K", [64, 128, 256])
def test_state_accuracy(K, seg):
    """The fp32 state after 2000 tokens, whole and joined from segments, to 2^-20 of its length.

    A token writes u k^T; u takes on K / 32 sums of three parts and some 16 roundings of its own, of 2^-24 at most:
    sqrt(3 K / 32 + 16) 2^-25 to be expected, 3.2 2^-24 for K = 256.  Errors of different tokens do not add up in one
    direction and fade as what they wrote does, so five times that is room enough; a state in two parts, off by up to
    2^-17 in every u, is past it."""
    x = inputs(1, 2000, 1, 2, K, 32, seed=211 + K)
    x["A_log"] -= 3.0
    _, fin = call(x, seg=seg)
    want = ref.delta(**x)[1]
    rel = float((fin.cpu().double() - want).norm() / want.norm())
    print(f"[check] state after 2000 tokens, K {K}, segments {seg}: {rel:.3g}", flush=True)
    assert rel <= 2.0 ** -20


# ---------------------------------------------------------------------------
# what is not finite
# ---------------------------------------------------------------------------

def lost(t):
    return bool((~torch.isfinite(t.float())).all())


@pytest.mark.parametrize("K", [64, 128, 256])
@pytest.mark.parametrize("where,value", [(w, v) for w in ("q", "k", "v") for v in (NAN, math.inf, -math.inf)]
                         + [("g", NAN), ("beta", NAN)])
@pytest.mark.parametrize("t", [0, 63, 200, 448])
def test_non_finite_inputs_stay_lost_behind_the_join(where, value, K, t):
    """From its token on to the sequence's last and the final state, through the segments' join; nothing else."""
    T, V = 500, 48
    x = inputs(2, T, 2, 4, K, V, seed=221)
    x["A_log"] -= 4.0
    clean, clean_fin = call(x, seg=64)
    bad = x[where].clone()
    if where in ("g", "beta"):
        bad[1, t, 0] = value
    else:
        bad[1, t, 0, 5] = value
    out, fin = call(x, seg=64, **{where: bad})
    hit = torch.zeros(4, V, dtype=torch.bool, device="cuda")
    if where in ("q", "k"):
        hit[:2] = True          # the heads that share it
    elif where == "v":
        hit[0, 5] = True        # its column
    else:
        hit[0] = True           # its head
    last = t + 1 if where == "q" else T
    assert lost(out[1, t:last][:, hit])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, t:last] = ~hit
    assert torch.equal(out[keep], clean[keep])
    kept = torch.ones(2, 4, V, dtype=torch.bool, device="cuda")
    if where != "q":
        assert lost(fin[1][hit])
        kept[1] = ~hit
    assert torch.equal(fin[kept], clean_fin[kept])


@pytest.mark.parametrize("T,seg", [(0, None), (1, None), (6, None), (9, None), (150, None), (300, 64), (700, 256)])
@pytest.mark.parametrize("K", [64, 128, 256])
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("state", [F32, BF])
def test_non_finite_initial_states(value, K, T, seg, state):
    """A number of the state reaches its own row of it (a column of the outputs) alone, from the first token on."""
    V = 80
    x = inputs(2, T, 2, 4, K, V, seed=231, state=state)
    clean, clean_fin = call(x, state=state, seg=seg)
    bad = x["initial"].clone()
    bad[1, 2, 37, K - 3] = value
    out, fin = call(x, state=state, seg=seg, initial=bad)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, :, 2, 37] = False
    assert torch.equal(out[keep], clean[keep]) and lost(out[~keep])
    kept = torch.ones(2, 4, V, dtype=torch.bool, device="cuda")
    kept[1, 2, 37] = False
    assert torch.equal(fin[kept], clean_fin[kept])
    if T == 0:
        assert torch.equal(fin[1, 2, 37].cpu().nan_to_num(7.0, 8.0, 9.0), bad[1, 2, 37].nan_to_num(7.0, 8.0, 9.0))
    else:
        assert lost(fin[1, 2, 37])
