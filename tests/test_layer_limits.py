"""Limits and messages of the layer operators that no launch is needed for."""
import pytest

from gated_delta_rule_36_amd import _lib


def workspace(**over):
    fields = dict(B=1, T=0, H=32, P=64, G=1, N=128, softplus=1)
    fields.update(over)
    return _lib.load().kda_ssm_workspace_bytes(_lib.SsmArgs(**fields))


STATE = 4 * (32 * 64 * 128 + 32)  # of the heads above, with their log decays


@pytest.mark.parametrize("n,T", [(512, 512), (1000, 1000), (4096, 4096), (1000, 5000), (300, 40), (65, 64)])
def test_many_short_sequences_need_little_workspace(n, T):
    """Segments have 64 tokens at least and a sequence of one needs no slab, so T / 64 sequences at most have any, of
    twice as many segments as 64-token steps they cross: never one for every sequence."""
    assert 0 <= workspace(cu_seqlens=16, num_seqs=n, T=T) <= 2 * (T // 64) * STATE + 16


@pytest.mark.parametrize("n,T,seg", [(1, 4096, 64), (8, 19595, 704), (3, 1000, 32), (100, 1000, 32), (7, 33, 32), (2, 31, 32)])
def test_workspace_of_packed_segments(n, T, seg):
    whole = T // seg if T > seg else 0
    assert workspace(cu_seqlens=16, num_seqs=n, T=T, seg_tokens=seg) <= min(2 * whole, whole + n) * STATE + 16
    assert (workspace(cu_seqlens=16, num_seqs=n, T=T, seg_tokens=seg) > 0) == (T > seg)


def test_workspace_of_a_batch():
    """As many slabs as segments where there are several, none where there is one."""
    assert workspace(B=4, T=4096, seg_tokens=512) == 4 * 8 * STATE
    assert workspace(B=4, T=4090, seg_tokens=512) == 4 * 8 * STATE
    assert workspace(B=4, T=512, seg_tokens=512) == 0
    assert workspace(B=4, T=8) == 0


@pytest.mark.parametrize("over", [dict(), dict(seg_tokens=32), dict(seg_tokens=1 << 31), dict(cu_seqlens=1 << 44, num_seqs=1)])
def test_scan_token_counts_that_would_leave_32_bits_are_refused(over):
    """Inputs may be broadcast over tokens (strides of 0), so such a call can fit the memory.  Nothing is launched: the
    largest length allowed gets as far as the next check, here that of a pointer."""
    fields = dict(B=1, H=1, P=32, G=1, N=32, softplus=1)
    fields.update(over)
    lib = _lib.load()
    for T, code in (((1 << 31) - 129, _lib.KDA_ERR_NULL_POINTER), ((1 << 31) - 128, _lib.KDA_ERR_SIZE),
                    ((1 << 31) - 64, _lib.KDA_ERR_SIZE), ((1 << 31) - 1, _lib.KDA_ERR_SIZE)):
        args = _lib.SsmArgs(T=T, **fields)
        assert lib.kda_ssm_fwd(args, None) == code, T
        assert (lib.kda_ssm_workspace_bytes(args) < 0) == (code == _lib.KDA_ERR_SIZE), T


@pytest.mark.parametrize("scale,ok", [(0.0, True), (-0.0, True), (1.0, True), (-2.0 ** -126, True), (2.0 ** 127, True),
                                      (2.0 ** 128, False), (-1e39, False), (1e300, False), (2.0 ** -127, False), (1e-300, False)])
def test_residual_scales_are_numbers_of_fp32(scale, ok):
    """Beyond fp32 a scale would be infinite (and times 0 NaN) or lose its digits."""
    for name in ("residual_scale", "block_scale"):
        fields = dict(rows=0, D=64, gate_period=1, x_stride=64, eps=1e-6, residual_scale=1.0, block_scale=1.0)
        fields[name] = scale
        status = _lib.load().kda_residual_norm(_lib.ResidualNormArgs(**fields), None)
        assert status == (_lib.KDA_OK if ok else _lib.KDA_ERR_SCALE), name


@pytest.mark.parametrize("code,words", [
    (_lib.KDA_ERR_STRIDE, ("negative", "int64", "2^27", "2^26")),
    (_lib.KDA_ERR_SCALE, ("finite", "eps", ">= 0", "residual_scale", "block_scale")),
    (_lib.KDA_ERR_SIZE, ("2^31", "2^31 - 128", "2^32 threads", "gate_period", "rows")),
    (_lib.KDA_ERR_ALIGNMENT, ("16 bytes", "inputs 2", "inputs 4", "cu_seqlens 8", "residual_out")),
])
def test_messages_name_what_the_layer_operators_refuse(code, words):
    """The text that a KdaArgumentError shows."""
    text = _lib.status_string(code)
    assert all(w in text for w in words), text
