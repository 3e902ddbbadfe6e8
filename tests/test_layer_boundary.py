"""Host-side checks of the layer operators' C ABI and Python binding (no GPU):
argument errors before any launch, struct layouts, compiled code."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import gated_delta_rule_36_amd as kda
from gated_delta_rule_36_amd import _lib
from test_codegen import HIPCC, functions, kernel_metadata

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_36_amd", "csrc")

# dummies of 64 KiB, 16-byte aligned and far apart: the declared extents of
# the small calls below stay inside them
BUF = [ctypes.create_string_buffer((1 << 16) + 16) for _ in range(14)]
A = [(ctypes.addressof(b) + 15) & ~15 for b in BUF]
BF, F32 = _lib.KDA_DTYPE_BF16, _lib.KDA_DTYPE_FP32
HUGE = 1 << 61


def call(entry, struct, base, over):
    """The status of a call with well-formed dummies, some replaced; None means a NULL struct."""
    fields = dict(base)
    for k in over:
        assert k in dict(struct._fields_), k
    fields.update(over)
    return getattr(_lib.load(), entry)(struct(**fields), None)


# With T = 0 and no final state (or rows = 0) nothing is launched even when
# every check passes; calls with T > 0 below all carry a planted error.
CONV = dict(x=A[0], x_stride_b=8, x_stride_t=8, weight=A[1], bias=A[2], out=A[3], B=1, T=0, D=8, W=4,
            weight_dtype=BF, activation=_lib.KDA_ACT_SILU, l2norm_eps=1e-6)


@pytest.mark.parametrize("over,code", [
    (dict(), _lib.KDA_OK),
    (dict(l2norm=64, D=128), _lib.KDA_OK),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(activation=_lib.KDA_ACT_SIGMOID), _lib.KDA_ERR_OPTION),
    (dict(activation=9), _lib.KDA_ERR_OPTION),
    (dict(W=0), _lib.KDA_ERR_SHAPE),
    (dict(W=9), _lib.KDA_ERR_SHAPE),
    (dict(D=0), _lib.KDA_ERR_SHAPE),
    (dict(D=(1 << 24) + 1), _lib.KDA_ERR_SHAPE),
    (dict(l2norm=32, D=128), _lib.KDA_ERR_SHAPE),
    (dict(l2norm=128, D=192), _lib.KDA_ERR_SHAPE),
    (dict(l2norm=-64, D=128), _lib.KDA_ERR_SHAPE),
    (dict(l2norm=64, D=128, l2norm_eps=-1.0), _lib.KDA_ERR_SCALE),
    (dict(l2norm=64, D=128, l2norm_eps=math.nan), _lib.KDA_ERR_SCALE),
    (dict(weight_dtype=0), _lib.KDA_ERR_DTYPE),
    (dict(weight_dtype=3), _lib.KDA_ERR_DTYPE),
    (dict(B=0), _lib.KDA_ERR_SIZE),
    (dict(T=-1), _lib.KDA_ERR_SIZE),
    (dict(T=1 << 31), _lib.KDA_ERR_SIZE),
    (dict(B=1 << 40, T=1 << 30), _lib.KDA_ERR_SIZE),
    (dict(cu_seqlens=A[4], num_seqs=1, B=2), _lib.KDA_ERR_VARLEN_BATCH),
    (dict(cu_seqlens=A[4], num_seqs=-1), _lib.KDA_ERR_VARLEN_BATCH),
    (dict(x_stride_t=-8, T=4), _lib.KDA_ERR_STRIDE),
    (dict(x_stride_t=HUGE, T=16), _lib.KDA_ERR_STRIDE),
    (dict(x=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(out=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(weight=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(initial_state=A[5]), _lib.KDA_ERR_NULL_POINTER),
    (dict(initial_state=A[5], initial_state_dtype=7), _lib.KDA_ERR_STATE_DTYPE),
    (dict(initial_state=A[5], initial_state_dtype=BF, final_state=A[6], final_state_dtype=F32), _lib.KDA_ERR_STATE_DTYPE),
    (dict(out=A[0], T=4), _lib.KDA_ERR_ALIAS),
    (dict(out=A[1], T=4), _lib.KDA_ERR_ALIAS),
    (dict(initial_state=A[5], initial_state_dtype=BF, final_state=A[5] + 16, final_state_dtype=BF), _lib.KDA_ERR_ALIAS),
    (dict(final_state=A[0], final_state_dtype=BF, T=4), _lib.KDA_ERR_ALIAS),
    (dict(final_state=A[3], final_state_dtype=BF, T=4), _lib.KDA_ERR_ALIAS),
    (dict(x=A[0] + 1), _lib.KDA_ERR_ALIGNMENT),
    (dict(out=A[3] + 2), _lib.KDA_ERR_ALIGNMENT),
    (dict(weight=A[1] + 2, weight_dtype=F32), _lib.KDA_ERR_ALIGNMENT),
    (dict(initial_state=A[5] + 8, initial_state_dtype=BF), _lib.KDA_ERR_ALIGNMENT),
    (dict(cu_seqlens=A[4] + 4, num_seqs=1), _lib.KDA_ERR_ALIGNMENT),
])
def test_conv_argument_errors(over, code):
    assert call("kda_short_conv", _lib.ConvArgs, CONV, over) == code


SSM = dict(x=A[0], dt=A[1], b=A[2], c=A[3], z=A[4], out=A[5], A_log=A[6], D=A[7], dt_bias=A[8], B=1, T=0, H=2, P=64,
           G=1, N=64, softplus=1, x_stride_b=128, x_stride_t=128, dt_stride_b=2, dt_stride_t=2, b_stride_b=64,
           b_stride_t=64, c_stride_b=64, c_stride_t=64, z_stride_b=128, z_stride_t=128)


@pytest.mark.parametrize("over,code", [
    (dict(), _lib.KDA_OK),
    (dict(z=None, D=None, dt_bias=None, softplus=0), _lib.KDA_OK),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(softplus=2), _lib.KDA_ERR_OPTION),
    (dict(P=48), _lib.KDA_ERR_SHAPE),
    (dict(P=0), _lib.KDA_ERR_SHAPE),
    (dict(P=288), _lib.KDA_ERR_SHAPE),
    (dict(N=16), _lib.KDA_ERR_SHAPE),
    (dict(N=96), _lib.KDA_ERR_SHAPE),
    (dict(G=0), _lib.KDA_ERR_SHAPE),
    (dict(G=3), _lib.KDA_ERR_SHAPE),
    (dict(seg_tokens=-32), _lib.KDA_ERR_SHAPE),
    (dict(seg_tokens=48), _lib.KDA_ERR_SHAPE),
    (dict(H=0), _lib.KDA_ERR_SIZE),
    (dict(H=65537), _lib.KDA_ERR_SIZE),
    (dict(B=0), _lib.KDA_ERR_SIZE),
    (dict(T=-1), _lib.KDA_ERR_SIZE),
    (dict(B=1 << 40, T=1 << 30), _lib.KDA_ERR_SIZE),
    (dict(B=(1 << 31) - 1, H=2), _lib.KDA_ERR_SIZE),
    (dict(cu_seqlens=A[9], num_seqs=1, B=2), _lib.KDA_ERR_VARLEN_BATCH),
    (dict(b_stride_t=-1, T=9), _lib.KDA_ERR_STRIDE),
    (dict(z_stride_t=HUGE, T=90), _lib.KDA_ERR_STRIDE),
    (dict(x=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(c=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(A_log=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(final_state=A[10]), _lib.KDA_ERR_NULL_POINTER),
    (dict(initial_state=A[10], initial_state_dtype=5), _lib.KDA_ERR_STATE_DTYPE),
    (dict(initial_state=A[10], initial_state_dtype=BF, final_state=A[11], final_state_dtype=F32), _lib.KDA_ERR_STATE_DTYPE),
    (dict(out=A[4], T=4), _lib.KDA_ERR_ALIAS),
    (dict(out=A[7], T=4), _lib.KDA_ERR_ALIAS),
    (dict(final_state=A[2], final_state_dtype=F32, T=4), _lib.KDA_ERR_ALIAS),
    (dict(initial_state=A[10], initial_state_dtype=F32, final_state=A[10] + 16, final_state_dtype=F32), _lib.KDA_ERR_ALIAS),
    (dict(dt=A[1] + 1), _lib.KDA_ERR_ALIGNMENT),
    (dict(out=A[5] + 8), _lib.KDA_ERR_ALIGNMENT),
    (dict(A_log=A[6] + 2), _lib.KDA_ERR_ALIGNMENT),
    (dict(final_state=A[10] + 8, final_state_dtype=BF, T=4), _lib.KDA_ERR_ALIGNMENT),
])
def test_ssm_argument_errors(over, code):
    assert call("kda_ssm_fwd", _lib.SsmArgs, SSM, over) == code


GATED = dict(x=A[0], gate=A[1], weight=A[2], out=A[3], x_stride=64, gate_stride=64, rows=0, D=64, group=32,
             weight_dtype=BF, activation=_lib.KDA_ACT_SIGMOID, eps=1e-6)


@pytest.mark.parametrize("over,code", [
    (dict(), _lib.KDA_OK),
    (dict(gate=None, activation=0), _lib.KDA_OK),
    (dict(activation=0), _lib.KDA_ERR_OPTION),
    (dict(gate_first=2), _lib.KDA_ERR_OPTION),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(group=48), _lib.KDA_ERR_SHAPE),
    (dict(group=0), _lib.KDA_ERR_SHAPE),
    (dict(D=32768, group=32768), _lib.KDA_ERR_SHAPE),
    (dict(D=0), _lib.KDA_ERR_SHAPE),
    (dict(eps=-1e-9), _lib.KDA_ERR_SCALE),
    (dict(eps=math.inf), _lib.KDA_ERR_SCALE),
    (dict(weight_dtype=0), _lib.KDA_ERR_DTYPE),
    (dict(rows=-1), _lib.KDA_ERR_SIZE),
    (dict(rows=1 << 60), _lib.KDA_ERR_SIZE),
    (dict(rows=2, x_stride=-64), _lib.KDA_ERR_STRIDE),
    (dict(rows=20, gate_stride=HUGE), _lib.KDA_ERR_STRIDE),
    (dict(rows=2, x=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(weight=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(rows=2, out=A[0]), _lib.KDA_ERR_ALIAS),
    (dict(rows=2, out=A[1] + 16), _lib.KDA_ERR_ALIAS),
    (dict(x=A[0] + 1), _lib.KDA_ERR_ALIGNMENT),
    (dict(out=A[3] + 8), _lib.KDA_ERR_ALIGNMENT),
])
def test_gated_norm_argument_errors(over, code):
    assert call("kda_gated_norm", _lib.GatedNormArgs, GATED, over) == code


RESID = dict(x=A[0], residual=A[1], residual_out=A[2], post_weight=A[3], gate=A[4], weight=A[5], out=A[6], x_stride=64,
             gate_stride=0, gate_period=1, rows=0, D=64, residual_dtype=F32, residual_out_dtype=F32,
             post_weight_dtype=BF, gate_dtype=BF, weight_dtype=BF, residual_scale=1.0, block_scale=1.0, eps=1e-6)


@pytest.mark.parametrize("over,code", [
    (dict(), _lib.KDA_OK),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(D=0), _lib.KDA_ERR_SHAPE),
    (dict(D=16385), _lib.KDA_ERR_SHAPE),
    (dict(eps=-1.0), _lib.KDA_ERR_SCALE),
    (dict(block_scale=math.inf), _lib.KDA_ERR_SCALE),
    (dict(residual_scale=math.nan), _lib.KDA_ERR_SCALE),
    (dict(residual_dtype=0), _lib.KDA_ERR_DTYPE),
    (dict(gate_dtype=4), _lib.KDA_ERR_DTYPE),
    (dict(rows=-1), _lib.KDA_ERR_SIZE),
    (dict(gate_period=0), _lib.KDA_ERR_SIZE),
    (dict(rows=2, x_stride=-1), _lib.KDA_ERR_STRIDE),
    (dict(rows=20, gate_stride=HUGE), _lib.KDA_ERR_STRIDE),
    (dict(rows=2, x=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(rows=2, out=None, weight=None, residual_out=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(weight=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(rows=2, out=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(rows=2, out=A[0]), _lib.KDA_ERR_ALIAS),
    (dict(rows=2, out=A[2]), _lib.KDA_ERR_ALIAS),
    (dict(rows=2, residual_out=A[1] + 16), _lib.KDA_ERR_ALIAS),
    (dict(rows=2, residual_out=A[1], residual_out_dtype=BF), _lib.KDA_ERR_ALIAS),
    (dict(rows=2, residual_out=A[4]), _lib.KDA_ERR_ALIAS),
    (dict(residual=A[1] + 2), _lib.KDA_ERR_ALIGNMENT),
    (dict(residual_out=A[2] + 4), _lib.KDA_ERR_ALIGNMENT),
])
def test_residual_norm_argument_errors(over, code):
    assert call("kda_residual_norm", _lib.ResidualNormArgs, RESID, over) == code


def test_null_structs_and_status_strings():
    lib = _lib.load()
    for name in ("kda_short_conv", "kda_ssm_fwd", "kda_gated_norm", "kda_residual_norm"):
        assert getattr(lib, name)(None, None) == _lib.KDA_ERR_NULL_POINTER
    assert lib.kda_ssm_workspace_bytes(None) == -1
    msgs = {_lib.status_string(c) for c in range(16)}
    assert len(msgs) == 16 and "unknown status" not in msgs


STRUCTS = {"kda_conv_args": _lib.ConvArgs, "kda_ssm_args": _lib.SsmArgs, "kda_gated_norm_args": _lib.GatedNormArgs,
           "kda_residual_norm_args": _lib.ResidualNormArgs}


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_struct_layouts_match_the_header(tmp_path):
    lines = []
    for name, s in STRUCTS.items():
        lines.append(f'printf("{name} %zu", sizeof({name}));')
        lines += [f'printf(" %zu", offsetof({name}, {f}));' for f, _ in s._fields_]
        lines.append('printf("\\n");')
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda.h"\nint main(void) {' + "".join(lines)
                   + "return 0; }\n")
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.splitlines()
    want = [f"{n} {ctypes.sizeof(s)} " + " ".join(str(getattr(s, f).offset) for f, _ in s._fields_)
            for n, s in STRUCTS.items()]
    assert got == want


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", sorted(f for f in os.listdir(os.path.join(CSRC, "layer")) if f.endswith(".hip")))
def test_no_calls_scratch_or_spills(src, tmp_path):
    out = tmp_path / (src + ".s")
    subprocess.run([HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", f"-I{ROOT}/include", f"-I{CSRC}", f"-I{CSRC}/layer", "--cuda-device-only", "-S",
                    os.path.join(CSRC, "layer", src), "-o", str(out)], check=True, capture_output=True)
    asm = out.read_text()
    meta = kernel_metadata(asm)
    assert meta
    for name, m in meta.items():
        assert not any(m.values()), (name, m)
    assert "s_swappc" not in asm
    assert not [n for n in functions(asm) if n not in meta], "out-of-line device functions"


# --------------------------------------------------------------------------
# the Python binding, on host tensors (refused before any launch)
# --------------------------------------------------------------------------

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call,error,text", [
    (lambda: kda.short_conv(t(1, 2, 8), t(8, 4), t(1, 2, 8)), ValueError, "GPU"),
    (lambda: kda.short_conv(t(1, 2, 8, dtype=torch.float16), t(8, 4), t(1, 2, 8)), TypeError, "bfloat16"),
    (lambda: kda.short_conv(None, t(8, 4), t(1, 2, 8)), TypeError, "Tensor"),
    (lambda: kda.ssm_fwd(t(1, 2, 2, 64), t(1, 2, 2), t(1, 2, 1, 64), t(1, 2, 1, 64), t(1, 2, 2, 64), t(2)), ValueError, "GPU"),
    (lambda: kda.ssm_fwd(t(1, 2, 2, 64).float(), t(1, 2, 2), t(1, 2, 1, 64), t(1, 2, 1, 64), t(1, 2, 2, 64), t(2)),
     TypeError, "bfloat16"),
    (lambda: kda.gated_norm(t(2, 8), t(2, 8), t(8), t(2, 8)), ValueError, "GPU"),
    (lambda: kda.gated_norm([1.0], None, t(8), t(2, 8)), TypeError, "Tensor"),
    (lambda: kda.residual_norm(t(2, 8), None, t(8), t(2, 8)), ValueError, "GPU"),
])
def test_binding_refuses(call, error, text):
    with pytest.raises(error, match=text):
        call()


def test_row_and_gate_strides():
    from gated_delta_rule_36_amd.layer import _gate_rows, _row_stride, _tokens
    assert _row_stride("x", t(3, 5, 8)) == 8
    assert _row_stride("x", t(3, 5, 20)[..., 4:12]) == 20
    assert _row_stride("x", t(8)) == 8
    assert _row_stride("x", t(1, 7, 1, 8)) == 8
    assert _row_stride("x", t(8).expand(4, 8)) == 0
    for bad in (t(3, 6, 8)[:, :5], t(3, 8, 5).transpose(1, 2), t(3, 5, 16)[..., ::2], t(3, 1, 8).expand(3, 5, 8)):
        with pytest.raises(ValueError):
            _row_stride("x", bad)
    assert _gate_rows(t(8), (3, 5, 8)) == (15, 0)
    assert _gate_rows(t(1, 1, 8), (3, 5, 8)) == (15, 0)
    assert _gate_rows(t(3, 1, 8), (3, 5, 8)) == (5, 8)
    assert _gate_rows(t(3, 5, 8), (3, 5, 8)) == (1, 8)
    assert _gate_rows(t(3, 24)[:, None, 8:16], (3, 5, 8)) == (5, 24)
    for bad in (t(1, 5, 8), t(5, 8), t(2, 1, 8), t(7)):
        with pytest.raises(ValueError):
            _gate_rows(bad, (3, 5, 8))
    cpu = torch.device("cpu")
    wide = t(2, 3, 40)
    assert _tokens("x", wide[..., 8:24].unflatten(-1, (2, 8)), cpu, (2, 3, 2, 8))[1:] == (120, 40)
    with pytest.raises(ValueError, match="adjacent"):
        _tokens("x", t(2, 3, 8, 2).transpose(2, 3), cpu, (2, 3, 2, 8))


WIDE = [(i + 1) << 44 for i in range(14)]  # addresses with room for any size; nothing is launched with them


@pytest.mark.parametrize("entry,struct,base,over", [
    ("kda_short_conv", _lib.ConvArgs, "CONV", dict(cu_seqlens=WIDE[9], num_seqs=(1 << 31) - 1, T=1, D=1024)),
    ("kda_short_conv", _lib.ConvArgs, "CONV", dict(B=1 << 27, T=1)),
    ("kda_ssm_fwd", _lib.SsmArgs, "SSM", dict(B=(1 << 24), T=1, H=1, P=32, N=32)),
    ("kda_ssm_fwd", _lib.SsmArgs, "SSM", dict(B=1, T=1, cu_seqlens=WIDE[9], num_seqs=1 << 23)),
    ("kda_ssm_fwd", _lib.SsmArgs, "SSM", dict(B=1, T=2 << 20, cu_seqlens=WIDE[9], num_seqs=1 << 22, seg_tokens=32,
                                              H=16, workspace=WIDE[13], workspace_bytes=1 << 50)),
    ("kda_gated_norm", _lib.GatedNormArgs, "GATED", dict(rows=1 << 42, D=1, group=1)),
    ("kda_residual_norm", _lib.ResidualNormArgs, "RESID", dict(rows=1 << 42, D=1, residual=None, residual_out=None)),
])
def test_grids_beyond_the_launch_limit_are_refused(entry, struct, base, over):
    fields = dict(globals()[base])
    for i, k in enumerate(k for k, v in fields.items() if v in A):
        fields[k] = WIDE[i]
    fields.update({k: 0 for k in fields if "_stride" in k})
    assert call(entry, struct, fields, over) == _lib.KDA_ERR_SIZE


@pytest.mark.parametrize("over,code", [
    (dict(T=9, x_stride_t=(1 << 27) + 1), _lib.KDA_ERR_STRIDE),
    (dict(T=9, b_stride_t=(1 << 27) + 1), _lib.KDA_ERR_STRIDE),
    (dict(T=9, c_stride_t=(1 << 27) + 1), _lib.KDA_ERR_STRIDE),
    (dict(T=9, z_stride_t=(1 << 26) + 1), _lib.KDA_ERR_STRIDE),
    (dict(T=2, cu_seqlens=A[9], num_seqs=2, z_stride_t=(1 << 26) + 1), _lib.KDA_ERR_STRIDE),
    # allowed ones get as far as the next check, here that of a pointer
    (dict(T=9, x_stride_t=1 << 27, b_stride_t=1 << 27, c_stride_t=1 << 27, z_stride_t=1 << 26, A_log=None),
     _lib.KDA_ERR_NULL_POINTER),
    (dict(T=9, z=None, z_stride_t=1 << 30, A_log=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(T=8, x_stride_t=1 << 30, z_stride_t=1 << 30, A_log=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(T=1, cu_seqlens=A[9], num_seqs=2, x_stride_t=1 << 30, z_stride_t=1 << 30, A_log=None), _lib.KDA_ERR_NULL_POINTER),
])
def test_ssm_token_stride_limits(over, code):
    assert call("kda_ssm_fwd", _lib.SsmArgs, SSM, over) == code
