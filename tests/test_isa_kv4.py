"""Static checks of the attention kernels' instruction streams on gfx950.

The kernels take maxima and issue LDS loads from inline asm, which the
compiler's hazard recognizer does not look into.  gfx950 needs two wait states
between a VALU write of a VGPR and a v_permlane swap that reads it, and up to
19 between an MFMA's result and another instruction that reads it; five between
a VALU write of an SGPR and a buffer load that reads it; one between a write of
M0 and the LDS load that uses it.  M0 is set in that asm and must be the
compiler's nowhere else.  Checked in straight-line code (an s_nop n is n + 1
wait states)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "bit_quantized_decode_pn3t_amd", "csrc", "pn_kv4_attn.hip")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def instructions(asm):
    """(operation, operands, from inline asm) of every instruction and label."""
    inside, out = False, []
    for line in asm.splitlines():
        line = line.strip()
        if line.startswith((";;#ASMSTART", ";;#ASMEND")):
            inside = line.startswith(";;#ASMSTART")
            continue
        line = line.split(";")[0].strip()
        if not line or line.startswith("//") or (line.startswith(".") and not line.endswith(":")):
            continue
        op, _, rest = line.partition(" ")
        out.append((op, [a.strip() for a in rest.split(",")] if rest else [], inside))
    return out


def regs(operand):
    m = re.match(r"[-|]*([vsa])(?:\[(\d+):(\d+)\]|(\d+))", operand)
    if not m:
        return {operand} if operand == "m0" else set()
    lo, hi = (int(m[2]), int(m[3])) if m[2] else (int(m[4]), int(m[4]))
    return {(m[1], i) for i in range(lo, hi + 1)}


def writes(op, args):
    if not args or op.startswith(("s_cbranch", "s_branch", "s_wait", "s_nop", "s_cmp", "buffer_load_dword", "global_store", "ds_write")):
        return set()
    return regs(args[0]) | (regs(args[1]) if op.startswith("v_permlane") and "swap" in op else set())


def before(ins, i, read, need, writer):
    """Wait states since the last write of `read` by an instruction that `writer` picks, or None."""
    ws = 0
    for op, args, inside in reversed(ins[max(0, i - 40):i]):
        if ws >= need or op.endswith(":"):
            return None
        if op == "s_nop":
            ws += int(args[0], 0) + 1
            continue
        hit = writes(op, args) & read
        if hit and writer(op, inside):
            return ws
        read = read - hit
        ws += 1
    return None


def find(asm):
    ins, bad = instructions(asm), []
    for i, (op, args, inside) in enumerate(ins):
        if op.startswith("v_permlane"):
            read = regs(args[0]) | regs(args[1])
            if before(ins, i, read, 2, lambda o, a: a and o.startswith("v_")) is not None:
                bad.append("permlane after asm: %s %s" % (op, args))
        elif inside and op.startswith("v_"):
            read = set().union(*[regs(a) for a in args[1:]])
            if before(ins, i, read, 19, lambda o, a: o.startswith("v_mfma")) is not None:
                bad.append("asm after MFMA: %s %s" % (op, args))
        elif inside and op.startswith("buffer_load"):
            read = set().union(*[regs(a.split()[0]) for a in args if a])
            if before(ins, i, {r for r in read if r[0] == "s"}, 5, lambda o, a: o.startswith("v_")) is not None:
                bad.append("load after VALU write of its SGPR: %s %s" % (op, args))
            if before(ins, i, {"m0"}, 1, lambda o, a: o.startswith("s_mov")) is not None:
                bad.append("load after write of M0: %s %s" % (op, args))
        elif not inside and any("m0" == a for a in args):
            bad.append("M0 outside of asm: %s %s" % (op, args))
    return bad


def test_checker_flags_planted_hazards():
    start, end = "\t;;#ASMSTART\n", "\t;;#ASMEND\n"
    good = (start + "\tv_max_f32 v1, v2, v3\n" + end + "\ts_nop 1\n\tv_permlane32_swap_b32_e32 v1, v4\n"
            "\tv_mfma_f32_16x16x32_f16 v[8:11], v[12:15], v[16:19], 0\n\ts_nop 15\n\ts_nop 3\n" + start +
            "\tv_max3_f32 v1, v8, v9, v10\n" + end + "\tv_readfirstlane_b32 s9, v1\n" + start +
            "\ts_nop 4\n\ts_mov_b32 m0, s1\n\ts_nop 0\n\tbuffer_load_dwordx4 v1, s[8:11], s2 offen lds\n" + end)
    assert find(good) == []
    for a, b in (("\ts_nop 1\n", "\ts_nop 0\n"), ("\ts_nop 3\n", ""), ("\ts_nop 4\n", ""), ("\ts_nop 0\n", ""),
                 ("s9, v1\n", "s9, v1\n\ts_mov_b32 m0, s3\n")):
        assert a in good and len(find(good.replace(a, b, 1))) == 1, (a, find(good.replace(a, b, 1)))


@pytest.mark.skipif(not os.path.exists(HIPCC) and shutil.which("hipcc") is None, reason="no hipcc")
def test_attention_kernels(tmp_path):
    out = tmp_path / "attn.s"
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "--cuda-device-only", "-S", "-Xclang",
                    "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-o",
                    str(out), SRC], check=True, capture_output=True)
    asm = out.read_text()
    ins = instructions(asm)
    assert sum(a and op.startswith("buffer_load") for op, _, a in ins) > 100
    assert sum(op.startswith("v_permlane") for op, _, _ in ins) > 100
    assert find(asm) == []
