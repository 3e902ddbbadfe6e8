"""Checks on the layer kernels' compiled code that spills and scratch, which other
tests look at, do not show.  CPU only: hipcc cross-compiles."""
import os
import re
import subprocess

import pytest

from test_codegen import CSRC, HIPCC, ROOT, functions

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


def registers(operand):
    """(file, first, last) of v[0:3], a[4:7] or v9; None for a constant."""
    m = re.match(r"([va])\[(\d+):(\d+)\]$|([va])(\d+)$", operand)
    if not m:
        return None
    return (m[1], int(m[2]), int(m[3])) if m[1] else (m[4], int(m[5]), int(m[5]))


def overlap(a, b):
    return a and b and a[0] == b[0] and a[1] <= b[2] and b[1] <= a[2]


def close_products(body):
    """(slots between, the first, the second) of matrix products whose accumulator a product of another shape wrote."""
    found, done, slot = [], [], 0
    for line in body.splitlines():
        if not line.startswith("\t") or line.lstrip().startswith((";", ".")):
            continue
        op, _, rest = line.strip().partition(" ")
        operands = [x.strip() for x in rest.split(";")[0].split(",")]
        slot += 1 + (int(operands[0]) if op == "s_nop" else 0)
        if op.startswith("v_mfma"):
            taken = registers(operands[3].split()[0])
            for at, other, written in reversed(done):
                if overlap(written, taken):
                    if other != op:
                        found.append((slot - at, other, op))
                    break
            done.append((slot, op, registers(operands[0])))
    return found


def test_close_products_are_found():
    body = "\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0\n\ts_nop 1\n\tv_mfma_f32_16x16x16_bf16 v[0:3], v[8:9], v[10:11], v[0:3]\n"
    assert close_products(body) == [(3, "v_mfma_f32_16x16x32_bf16", "v_mfma_f32_16x16x16_bf16")]
    assert not close_products(body.replace("16x16x16_", "16x16x32_"))
    assert not close_products(body.replace("v[0:3]\n", "v[4:7]\n"))


LAYER = os.path.join(CSRC, "layer")


@pytest.mark.parametrize("src", sorted(f for f in os.listdir(LAYER) if f.endswith(".hip") and "_mfma_" in open(os.path.join(LAYER, f)).read()))
def test_products_of_two_shapes_stay_apart(src, tmp_path):
    """A product over 16 slots right behind one over 32 on the same accumulator, which the compiler does not keep apart,
    has given wrong sums here.  Such a pair needs eight slots between, the passes of the longest of these products; the
    layer kernels sum each shape by itself, so that what remains is over a hundred apart."""
    out = tmp_path / (src + ".s")
    subprocess.run([HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", f"-I{ROOT}/include", f"-I{CSRC}", f"-I{CSRC}/layer", "--cuda-device-only", "-S",
                    os.path.join(LAYER, src), "-o", str(out)], check=True, capture_output=True)
    for name, body in functions(out.read_text()).items():
        close = [c for c in close_products(body) if c[0] < 8]
        assert not close, (name, close[:3])
