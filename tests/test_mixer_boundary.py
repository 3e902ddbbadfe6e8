"""Host-side checks of delta_fwd's and the attention layers' C ABI and Python
binding (no GPU): argument errors before any launch, struct layouts, sizes of
workspaces."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import gated_delta_rule_36_amd as kda
from gated_delta_rule_36_amd import _lib
from test_layer_boundary import A, BF, F32, HUGE, WIDE, call, t

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK = _lib.KDA_OK

# With no tokens (or no sequences) nothing is launched even when every check
# passes; calls with some below all carry a planted error.
DELTA = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], out=A[5], A_log=A[6], dt_bias=A[7], B=1, T=0, H=2, G=1, K=64, V=32,
             scale=0.125, q_stride_b=64, q_stride_t=64, k_stride_b=64, k_stride_t=64, v_stride_b=64, v_stride_t=64,
             g_stride_b=2, g_stride_t=2, beta_stride_b=2, beta_stride_t=2)
STATE = dict(initial_state=A[8], initial_state_dtype=F32)


@pytest.mark.parametrize("over,code", [
    (dict(), OK),
    (dict(dt_bias=None, scale=0.0), OK),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(K=32), _lib.KDA_ERR_SHAPE),
    (dict(K=96), _lib.KDA_ERR_SHAPE),
    (dict(K=512), _lib.KDA_ERR_SHAPE),
    (dict(V=8), _lib.KDA_ERR_SHAPE),
    (dict(V=24), _lib.KDA_ERR_SHAPE),
    (dict(V=528), _lib.KDA_ERR_SHAPE),
    (dict(G=0), _lib.KDA_ERR_SHAPE),
    (dict(G=4), _lib.KDA_ERR_SHAPE),
    (dict(H=0), _lib.KDA_ERR_SIZE),
    (dict(H=65537, G=1), _lib.KDA_ERR_SIZE),
    (dict(B=0), _lib.KDA_ERR_SIZE),
    (dict(T=-1), _lib.KDA_ERR_SIZE),
    (dict(T=(1 << 31) - 100), _lib.KDA_ERR_SIZE),
    (dict(B=1 << 40, T=1 << 30), _lib.KDA_ERR_SIZE),
    (dict(B=(1 << 31) - 1), _lib.KDA_ERR_SIZE),
    (dict(scale=math.nan), _lib.KDA_ERR_SCALE),
    (dict(scale=math.inf), _lib.KDA_ERR_SCALE),
    (dict(scale=1e39), _lib.KDA_ERR_SCALE),
    (dict(scale=1e-39), _lib.KDA_ERR_SCALE),
    (dict(cu_seqlens=A[9], num_seqs=1, B=2), _lib.KDA_ERR_VARLEN_BATCH),
    (dict(cu_seqlens=A[9], num_seqs=-1), _lib.KDA_ERR_VARLEN_BATCH),
    (dict(q_stride_t=-1, T=9), _lib.KDA_ERR_STRIDE),
    (dict(beta_stride_t=HUGE, T=90), _lib.KDA_ERR_STRIDE),
    (dict(T=9, v_stride_t=(1 << 24) + 1), _lib.KDA_ERR_STRIDE),
    (dict(T=9, g_stride_t=(1 << 24) + 1), _lib.KDA_ERR_STRIDE),
    (dict(T=2, cu_seqlens=A[9], num_seqs=1, k_stride_t=(1 << 24) + 1), _lib.KDA_ERR_STRIDE),
    (dict(T=8, k_stride_t=(1 << 24) + 1, A_log=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(T=9, k_stride_t=1 << 24, A_log=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(q=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(beta=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(out=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(A_log=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(initial_state=A[8]), _lib.KDA_ERR_NULL_POINTER),
    (dict(initial_state=A[8], initial_state_dtype=9), _lib.KDA_ERR_STATE_DTYPE),
    (dict(STATE, final_state=A[10], final_state_dtype=BF), _lib.KDA_ERR_STATE_DTYPE),
    (dict(out=A[2], T=4), _lib.KDA_ERR_ALIAS),
    (dict(out=A[7], T=4), _lib.KDA_ERR_ALIAS),
    (dict(final_state=A[1], final_state_dtype=F32, T=4), _lib.KDA_ERR_ALIAS),
    (dict(STATE, final_state=A[8] + 16, final_state_dtype=F32), _lib.KDA_ERR_ALIAS),
    (dict(k=A[1] + 1), _lib.KDA_ERR_ALIGNMENT),
    (dict(out=A[5] + 8), _lib.KDA_ERR_ALIGNMENT),
    (dict(A_log=A[6] + 2), _lib.KDA_ERR_ALIGNMENT),
    (dict(final_state=A[10] + 8, final_state_dtype=F32, T=4), _lib.KDA_ERR_ALIGNMENT),
    (dict(cu_seqlens=A[9] + 4, num_seqs=1), _lib.KDA_ERR_ALIGNMENT),
])
def test_delta_argument_errors(over, code):
    assert call("kda_delta_fwd", _lib.DeltaArgs, DELTA, over) == code


ROTARY = dict(q=A[0], k=A[1], q_out=A[2], k_out=A[3], positions=A[4], inv_freq=A[5], q_weight=A[6], k_weight=A[7], B=1, T=0,
              Hq=4, Hk=2, D=64, R=64, q_stride_b=256, q_stride_t=256, k_stride_b=128, k_stride_t=128, q_weight_dtype=BF,
              k_weight_dtype=F32, eps=1e-6, rotary_scale=1.0)


@pytest.mark.parametrize("over,code", [
    (dict(), OK),
    (dict(B=0, T=5), OK),
    (dict(k=None, k_out=None, Hk=0), OK),
    (dict(positions=None, inv_freq=None, R=0), OK),
    (dict(q_weight=None, q_weight_dtype=0), OK),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(interleaved=2), _lib.KDA_ERR_OPTION),
    (dict(D=0, R=0), _lib.KDA_ERR_SHAPE),
    (dict(D=65), _lib.KDA_ERR_SHAPE),
    (dict(D=514), _lib.KDA_ERR_SHAPE),
    (dict(R=66), _lib.KDA_ERR_SHAPE),
    (dict(R=0), _lib.KDA_ERR_SHAPE),
    (dict(R=33), _lib.KDA_ERR_SHAPE),
    (dict(eps=-1.0), _lib.KDA_ERR_SCALE),
    (dict(eps=math.nan), _lib.KDA_ERR_SCALE),
    (dict(rotary_scale=math.inf), _lib.KDA_ERR_SCALE),
    (dict(rotary_scale=1e-40), _lib.KDA_ERR_SCALE),
    (dict(q_weight_dtype=0), _lib.KDA_ERR_DTYPE),
    (dict(k_weight_dtype=5), _lib.KDA_ERR_DTYPE),
    (dict(Hq=0), _lib.KDA_ERR_SIZE),
    (dict(Hk=-1), _lib.KDA_ERR_SIZE),
    (dict(Hq=65537), _lib.KDA_ERR_SIZE),
    (dict(B=-1), _lib.KDA_ERR_SIZE),
    (dict(T=1 << 31), _lib.KDA_ERR_SIZE),
    (dict(B=1 << 40, T=1 << 30), _lib.KDA_ERR_SIZE),
    (dict(q_stride_t=-256, T=4), _lib.KDA_ERR_STRIDE),
    (dict(k_stride_t=HUGE, T=40), _lib.KDA_ERR_STRIDE),
    (dict(q=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(k_out=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(inv_freq=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(positions=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(q_out=A[1], T=4), _lib.KDA_ERR_ALIAS),
    (dict(q_out=A[0] + 16, T=4), _lib.KDA_ERR_ALIAS),
    (dict(q_out=A[0], q_stride_t=300, T=4), _lib.KDA_ERR_ALIAS),
    (dict(k_out=A[2], T=4), _lib.KDA_ERR_ALIAS),
    (dict(q_out=A[4], T=4), _lib.KDA_ERR_ALIAS),
    (dict(k_out=A[7], T=4), _lib.KDA_ERR_ALIAS),
    (dict(q=A[0] + 1), _lib.KDA_ERR_ALIGNMENT),
    (dict(q_out=A[2] + 8), _lib.KDA_ERR_ALIGNMENT),
    (dict(positions=A[4] + 4), _lib.KDA_ERR_ALIGNMENT),
    (dict(k_weight=A[7] + 2), _lib.KDA_ERR_ALIGNMENT),
])
def test_rotary_argument_errors(over, code):
    assert call("kda_qk_norm_rotary", _lib.RotaryArgs, ROTARY, over) == code


APPEND = dict(k=A[0], v=A[1], k_cache=A[2], v_cache=A[3], slots=A[4], positions=A[5], inv_freq=A[6], weight=A[7], B=1, T=0, Hk=2,
              D=64, R=64, pages=3, page_size=4, k_stride_b=128, k_stride_t=128, v_stride_b=128, v_stride_t=128,
              k_cache_stride_page=512, k_cache_stride_token=128, k_cache_stride_head=64, v_cache_stride_page=512,
              v_cache_stride_token=128, v_cache_stride_head=64, weight_dtype=BF, eps=1e-6, rotary_scale=1.0)
WOVEN = dict(k_cache=A[2], v_cache=A[2] + 1024, k_cache_stride_page=1024, v_cache_stride_page=1024)


@pytest.mark.parametrize("over,code", [
    (dict(), OK),
    (dict(positions=None, inv_freq=None, weight=None, weight_dtype=0), OK),
    (dict(k_cache_stride_token=64, k_cache_stride_head=256), OK),
    (dict(WOVEN), OK),
    (dict(pages=0, T=4), OK),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(interleaved=-1), _lib.KDA_ERR_OPTION),
    (dict(D=63), _lib.KDA_ERR_SHAPE),
    (dict(R=128), _lib.KDA_ERR_SHAPE),
    (dict(eps=math.inf), _lib.KDA_ERR_SCALE),
    (dict(weight_dtype=3), _lib.KDA_ERR_DTYPE),
    (dict(Hk=0), _lib.KDA_ERR_SIZE),
    (dict(page_size=0), _lib.KDA_ERR_SIZE),
    (dict(pages=-1), _lib.KDA_ERR_SIZE),
    (dict(pages=1 << 40, page_size=1 << 30), _lib.KDA_ERR_SIZE),
    (dict(k_cache_stride_page=-512), _lib.KDA_ERR_STRIDE),
    (dict(k_cache_stride_page=500), _lib.KDA_ERR_STRIDE),
    (dict(v_cache_stride_token=0), _lib.KDA_ERR_STRIDE),
    (dict(v_cache_stride_head=32), _lib.KDA_ERR_STRIDE),
    (dict(k_cache_stride_token=64), _lib.KDA_ERR_STRIDE),
    (dict(v_cache_stride_page=HUGE), _lib.KDA_ERR_STRIDE),
    (dict(k=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(slots=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(v_cache=None, T=4), _lib.KDA_ERR_NULL_POINTER),
    (dict(inv_freq=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(k_cache=A[0], T=4), _lib.KDA_ERR_ALIAS),
    (dict(v_cache=A[4], T=4), _lib.KDA_ERR_ALIAS),
    (dict(v_cache=A[2]), _lib.KDA_ERR_ALIAS),
    (dict(WOVEN, v_cache=A[2] + 512), _lib.KDA_ERR_ALIAS),
    (dict(WOVEN, v_cache_stride_page=2048), _lib.KDA_ERR_ALIAS),
    (dict(k_cache=A[2] + 1), _lib.KDA_ERR_ALIGNMENT),
    (dict(slots=A[4] + 4), _lib.KDA_ERR_ALIGNMENT),
])
def test_append_argument_errors(over, code):
    assert call("kda_append_kv", _lib.AppendArgs, APPEND, over) == code


ATTENTION = dict(q=A[0], k_cache=A[1], v_cache=A[2], block_table=A[3], lengths=A[4], out=A[5], lse=A[6], q_stride=256,
                 table_stride=4, k_cache_stride_page=512, k_cache_stride_token=128, k_cache_stride_head=64,
                 v_cache_stride_page=512, v_cache_stride_token=128, v_cache_stride_head=64, N=0, Hq=4, Hk=2, D=64, pages=3,
                 page_size=4, table_width=4, scale=0.125)


@pytest.mark.parametrize("over,code", [
    (dict(), OK),
    (dict(lse=None, window=7, D=16, scale=0.0), OK),
    (dict(reserved=1), _lib.KDA_ERR_OPTION),
    (dict(D=8), _lib.KDA_ERR_SHAPE),
    (dict(D=72), _lib.KDA_ERR_SHAPE),
    (dict(D=272), _lib.KDA_ERR_SHAPE),
    (dict(Hk=3), _lib.KDA_ERR_SHAPE),
    (dict(Hk=0), _lib.KDA_ERR_SHAPE),
    (dict(Hq=0), _lib.KDA_ERR_SHAPE),
    (dict(N=-1), _lib.KDA_ERR_SIZE),
    (dict(Hq=1 << 17), _lib.KDA_ERR_SIZE),
    (dict(pages=-1), _lib.KDA_ERR_SIZE),
    (dict(page_size=0), _lib.KDA_ERR_SIZE),
    (dict(window=-1), _lib.KDA_ERR_SIZE),
    (dict(table_width=-1), _lib.KDA_ERR_SIZE),
    (dict(table_width=1 << 30, page_size=2), _lib.KDA_ERR_SIZE),
    (dict(scale=math.nan), _lib.KDA_ERR_SCALE),
    (dict(scale=1e-40), _lib.KDA_ERR_SCALE),
    (dict(N=2, q_stride=-1), _lib.KDA_ERR_STRIDE),
    (dict(N=2, table_stride=-4), _lib.KDA_ERR_STRIDE),
    (dict(k_cache_stride_head=-1), _lib.KDA_ERR_STRIDE),
    (dict(v_cache_stride_page=HUGE), _lib.KDA_ERR_STRIDE),
    (dict(N=2, q=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(N=2, out=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(N=2, lengths=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(N=2, block_table=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(N=2, v_cache=None), _lib.KDA_ERR_NULL_POINTER),
    (dict(N=2, out=A[0]), _lib.KDA_ERR_ALIAS),
    (dict(N=2, out=A[1] + 16), _lib.KDA_ERR_ALIAS),
    (dict(N=2, lse=A[5]), _lib.KDA_ERR_ALIAS),
    (dict(N=2, lse=A[4]), _lib.KDA_ERR_ALIAS),
    (dict(out=A[5] + 8), _lib.KDA_ERR_ALIGNMENT),
    (dict(block_table=A[3] + 2), _lib.KDA_ERR_ALIGNMENT),
    (dict(N=1, table_width=4096), _lib.KDA_ERR_WORKSPACE),
    (dict(N=1, table_width=4096, workspace=A[7], workspace_bytes=64), _lib.KDA_ERR_WORKSPACE),
    (dict(N=1, table_width=4096, workspace=A[7] + 8, workspace_bytes=1 << 30), _lib.KDA_ERR_WORKSPACE),
    (dict(N=1, table_width=4096, workspace=A[5], workspace_bytes=1 << 30), _lib.KDA_ERR_WORKSPACE),
])
def test_attention_argument_errors(over, code):
    assert call("kda_paged_attention", _lib.AttentionArgs, ATTENTION, over) == code


def workspace(**over):
    args = _lib.AttentionArgs(**{**ATTENTION, **over})
    return _lib.load().kda_paged_attention_workspace_bytes(ctypes.byref(args))


def test_attention_workspace():
    assert _lib.load().kda_paged_attention_workspace_bytes(None) == -1
    assert workspace(D=8) == -1 and workspace(page_size=0) == -1
    assert workspace(N=0) == 0 and workspace(N=1, table_width=0) == 0
    assert workspace(N=1, table_width=16) == 0  # 64 tokens: one workgroup's
    assert workspace(N=1 << 16, table_width=4096) == 0  # enough sequences
    one = workspace(N=1, table_width=4096)
    assert one > 0 and one % (4 * (64 + 2) * 4) == 0
    assert workspace(N=1, table_width=4096, window=64) == 0
    # never more than the tokens there is room for
    assert workspace(N=1, table_width=1024) <= one


def test_null_structs():
    lib = _lib.load()
    for name in ("kda_delta_fwd", "kda_qk_norm_rotary", "kda_append_kv", "kda_paged_attention"):
        assert getattr(lib, name)(None, None) == _lib.KDA_ERR_NULL_POINTER


STRUCTS = {"kda_delta_args": _lib.DeltaArgs, "kda_rotary_args": _lib.RotaryArgs, "kda_append_args": _lib.AppendArgs,
           "kda_attention_args": _lib.AttentionArgs}


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


@pytest.mark.parametrize("entry,struct,base,over", [
    ("kda_delta_fwd", _lib.DeltaArgs, "DELTA", dict(B=1 << 24, T=1, H=1, V=16)),
    ("kda_qk_norm_rotary", _lib.RotaryArgs, "ROTARY", dict(B=1 << 26, T=1, Hq=32)),
    ("kda_append_kv", _lib.AppendArgs, "APPEND", dict(B=1 << 26, T=1, Hk=32)),
    ("kda_paged_attention", _lib.AttentionArgs, "ATTENTION", dict(N=1 << 24)),
])
def test_grids_beyond_the_launch_limit_are_refused(entry, struct, base, over):
    fields = dict(globals()[base])
    for i, k in enumerate(k for k, v in fields.items() if v in A):
        fields[k] = WIDE[i]
    fields.update({k: 0 for k in fields if k.endswith("_stride_b")})
    if base == "APPEND":
        fields.update(k_cache_stride_token=64 * 32, v_cache_stride_token=64 * 32, k_cache_stride_page=256 * 32,
                      v_cache_stride_page=256 * 32)
    if base == "ATTENTION":
        fields.update(q_stride=0, table_stride=0)
    assert call(entry, struct, fields, over) == _lib.KDA_ERR_SIZE


# --------------------------------------------------------------------------
# the Python binding, on host tensors (refused before any launch)
# --------------------------------------------------------------------------

def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("call,error,text", [
    (lambda: kda.delta_fwd(t(1, 2, 1, 64), t(1, 2, 1, 64), t(1, 2, 2, 32), t(1, 2, 2), t(1, 2, 2), 1.0, t(1, 2, 2, 32), t(2)),
     ValueError, "GPU"),
    (lambda: kda.delta_fwd(None, None, t(1, 2, 2, 32).float(), None, None, 1.0, None, None), TypeError, "v must be torch.bfloat16"),
    (lambda: kda.delta_fwd(None, None, None, None, None, 1.0, None, None), TypeError, "v must be a torch.Tensor"),
    (lambda: kda.qk_norm_rotary(t(1, 2, 2, 64), None, None, None, t(1, 2, 2, 64)), ValueError, "q must be on a GPU"),
    (lambda: kda.qk_norm_rotary([1.0], None, None, None, None), TypeError, "Tensor"),
    (lambda: kda.append_kv(t(1, 2, 2, 64), t(1, 2, 2, 64), t(2, 4, 2, 64), t(2, 4, 2, 64), i32(1, 2)), ValueError, "k must be on a GPU"),
    (lambda: kda.append_kv(t(1, 2, 2, 64).half(), None, None, None, None), TypeError, "bfloat16"),
    (lambda: kda.paged_attention(t(1, 2, 64), t(2, 4, 2, 64), t(2, 4, 2, 64), i32(1, 2), i32(1), t(1, 2, 64), 1.0), ValueError, "GPU"),
    (lambda: kda.paged_attention(None, None, None, None, None, None, 1.0), TypeError, "Tensor"),
])
def test_binding_refuses(call, error, text):
    with pytest.raises(error, match=text):
        call()


def test_rotation_and_cache_arguments():
    from gated_delta_rule_36_amd.attention import _cache, _rotation
    cpu = torch.device("cpu")
    pos, f = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(8)
    assert _rotation(None, None, cpu, (2, 3)) == (0, 0, 0)
    assert _rotation(pos, f, cpu, (2, 3)) == (pos.data_ptr(), f.data_ptr(), 16)
    for p, q, error in ((pos, None, ValueError), (None, f, ValueError), (pos.int(), f, TypeError), (pos[:, :2], f, ValueError),
                        (pos, f.double(), TypeError), (pos, f[None], ValueError), (pos, f[::2], ValueError)):
        with pytest.raises(error):
            _rotation(p, q, cpu, (2, 3))
    c = t(5, 4, 2, 16)
    assert _cache("c", c, cpu, 2, 16) == (c.data_ptr(), 128, 32, 16)
    heads = t(5, 2, 4, 16).transpose(1, 2)
    assert _cache("c", heads, cpu, 2, 16)[1:] == (128, 16, 64)
    for bad, error in ((t(5, 4, 2, 32)[..., ::2], ValueError), (t(5, 4, 3, 16), ValueError), (t(4, 2, 16), ValueError),
                       (c.float(), TypeError), (None, TypeError)):
        with pytest.raises(error):
            _cache("c", bad, cpu, 2, 16)


# --------------------------------------------------------------------------
# workspaces and segments of the gated delta rule
# --------------------------------------------------------------------------

def delta_workspace(**over):
    args = _lib.DeltaArgs(**{**DELTA, **over})
    return _lib.load().kda_delta_workspace_bytes(ctypes.byref(args))


def test_delta_workspace():
    assert _lib.load().kda_delta_workspace_bytes(None) == -1
    assert delta_workspace(K=32) == -1 and delta_workspace(T=-1) == -1 and delta_workspace(seg_tokens=48) == -1
    assert delta_workspace(T=8, seg_tokens=64) == 0 and delta_workspace(T=64, seg_tokens=64) == 0
    # of two segments: the end of the first and what it makes of K unit vectors; the second's end is the result
    H, K, V = (DELTA[k] for k in "HKV")
    slab = H * K * (V + K) * 4
    assert delta_workspace(T=65, seg_tokens=64) % slab == 0 and delta_workspace(T=65, seg_tokens=64) > 0
    assert delta_workspace(T=65, B=3, seg_tokens=64) == 3 * delta_workspace(T=65, seg_tokens=64)
    # packed: at most two tokens a sequence need none, unless asked for segments
    assert delta_workspace(T=200, cu_seqlens=A[9], num_seqs=100) == 0
    assert delta_workspace(T=200, cu_seqlens=A[9], num_seqs=100, seg_tokens=64) > 0
    # long sequences of few heads are cut without being asked
    assert delta_workspace(T=4096) > 0 and delta_workspace(T=4096, B=256) == 0 and delta_workspace(T=4096, H=512) == 0


@pytest.mark.parametrize("over,code", [
    (dict(seg_tokens=48), _lib.KDA_ERR_SHAPE),
    (dict(seg_tokens=-64), _lib.KDA_ERR_SHAPE),
    (dict(T=65, seg_tokens=64), _lib.KDA_ERR_WORKSPACE),
    (dict(T=65, seg_tokens=64, workspace=WIDE[0], workspace_bytes=64), _lib.KDA_ERR_WORKSPACE),
    (dict(T=65, seg_tokens=64, workspace=WIDE[0] + 8, workspace_bytes=1 << 30), _lib.KDA_ERR_WORKSPACE),
    (dict(T=65, seg_tokens=64, workspace=A[0], workspace_bytes=1 << 30), _lib.KDA_ERR_WORKSPACE),
    (dict(T=65, seg_tokens=64, workspace=A[5], workspace_bytes=1 << 30), _lib.KDA_ERR_WORKSPACE),
    (dict(T=200, cu_seqlens=A[9], num_seqs=100, seg_tokens=64), _lib.KDA_ERR_WORKSPACE),
])
def test_delta_segment_errors(over, code):
    assert call("kda_delta_fwd", _lib.DeltaArgs, DELTA, over) == code


def test_attention_of_more_heads_than_a_grid_takes():
    most = dict(N=(1 << 31) - 1, Hq=65536, Hk=65536, D=16, page_size=1 << 20, table_width=2000)
    assert workspace(**most) == 0
    fields = {**ATTENTION, **{k: WIDE[i] for i, k in enumerate(k for k, v in ATTENTION.items() if v in A)}}
    fields.update(q_stride=0, table_stride=0, k_cache_stride_head=0, v_cache_stride_head=0)
    assert call("kda_paged_attention", _lib.AttentionArgs, fields, most) != OK
