"""Static checks of the kernels of pn_kv4_attn_shared, pn_residual_norm and
pn_logprobs on gfx950: the hazards around inline assembly that the attention
kernels' own checks cover, and one more.  A product writes its result some
eleven wait states after it was issued; of a result of which only one element
is used, the other registers are free for the compiler at once, and an
instruction from inline assembly that writes one of them is not kept apart
from the product.  So no inline assembly may write a product's result register
within those states, unless something has waited for the result meanwhile (an
instruction of the compiler's own that reads or writes it)."""
import os
import re
import shutil
import subprocess

import pytest

from test_isa_kv4 import HIPCC, ROOT, find, instructions, regs, writes

CSRC = os.path.join(ROOT, "bit_quantized_decode_pn3t_amd", "csrc")
STATES = 11  # 16x16x32: eight passes


def overwritten(asm):
    """Inline assembly that writes a result register of a product still at work, in straight-line code."""
    ins, bad = instructions(asm), []
    for i, (op, args, inside) in enumerate(ins):
        if not inside or not op.startswith("v_") or not args:
            continue
        left, ws = regs(args[0]), 0
        for o, a, ins2 in reversed(ins[max(0, i - 40):i]):
            if ws >= STATES or o.endswith(":") or not left:
                break
            if o == "s_nop":
                ws += int(a[0], 0) + 1
                continue
            if o.startswith("v_mfma"):
                if regs(a[0]) & left:
                    bad.append("asm over a product's result: %s %s after %s %s" % (op, args, o, a))
                    break
            elif not ins2 and o.startswith("v_"):
                left = left - set().union(*[regs(x) for x in a]) - writes(o, a)
            ws += 1
    return bad


def test_checker_flags_planted_overwrites():
    start, end = "\t;;#ASMSTART\n", "\t;;#ASMEND\n"
    write = start + "\tv_and_or_b32 v9, v1, s2, v3\n" + end
    mfma = "\tv_mfma_f32_16x16x32_f16 v[8:11], v[12:15], v[16:19], 0\n"
    assert len(overwritten(mfma + write)) == 1
    assert len(overwritten(mfma + "\ts_nop 7\n" + write)) == 1
    assert overwritten(mfma + "\ts_nop 10\n" + write) == []
    assert overwritten(mfma + "\tv_add_f32_e32 v1, v9, v1\n" + write) == []
    assert overwritten(mfma.replace("[8:11]", "[20:23]") + write) == []


def compiled(tmp_path, src):
    out = tmp_path / (src + ".s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "--cuda-device-only", "-S", "-Xclang",
                    "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-o",
                    str(out), os.path.join(CSRC, src)], check=True, capture_output=True)
    return out.read_text()


@pytest.mark.skipif(not os.path.exists(HIPCC) and shutil.which("hipcc") is None, reason="no hipcc")
@pytest.mark.parametrize("src,products", [("pn_kv4_shared.hip", 100), ("pn_kv4_attn.hip", 100), ("pn_norm.hip", 0),
                                          ("pn_logprobs.hip", 0)])
def test_assembly(tmp_path, src, products):
    asm = compiled(tmp_path, src)
    assert "s_endpgm" in asm
    assert re.findall(r"^\s*(?:v_pk_(?:add|mul|fma)_f32|buffer_wbl2|buffer_inv)\b.*$", asm, re.M) == []
    assert len(re.findall(r"^\s*v_mfma_f32_16x16x32_f16", asm, re.M)) >= products
    assert overwritten(asm) == []
    if products:
        assert find(asm) == []
