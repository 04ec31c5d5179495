"""Wait states around inline asm in the kernels' assembly.

The compiler inserts the wait states that gfx950 leaves to software, but it does
not look into asm blocks: what stands there must not depend on them.  Every
source with an instruction in an asm block is compiled to assembly, and each
function is read in program order for

* a vector register written by a vector instruction and read by an MFMA within
  two wait states;
* a scalar register written by a vector instruction and read by a vector memory
  instruction within five (a scalar copy between them interlocks);
* M0 written by the scalar unit right in front of an LDS-DMA load.
"""
import glob
import os
import re
import subprocess

import pytest

from fp4_routed_expert_amd import build

REG = re.compile(r"\b([vas])(?:\[(\d+):(\d+)\]|(\d+)\b)")


def with_asm():
    """Sources that issue instructions from asm blocks, their own or lds_dma.h's."""
    found = []
    for f in sorted(glob.glob(os.path.join(build.CSRC, "*.hip"))):
        text = re.sub(r"//[^\n]*", "", open(f).read())
        if "lds_dma.h" in text or re.search(r'asm\s+volatile\s*\(\s*"[a-z]', text):
            found.append(os.path.basename(f))
    return found


def registers(text):
    out = set()
    for kind, lo, hi, one in REG.findall(text):
        out |= {(kind, int(one))} if one else {(kind, i) for i in range(int(lo), int(hi) + 1)}
    return out


def hazards(assembly):
    """The findings of one file, as (rule, function, writer, reader)."""
    found, history, name = [], [], ""
    for line in assembly.splitlines():
        line = line.split(";")[0].strip()
        label = re.match(r"([_A-Za-z][\w.$]*):", line)
        if label and not line.startswith(".L"):
            name, history = label[1], []
        if not re.match(r"[a-z]\w*(\s|$)", line):
            continue
        op, _, rest = line.partition(" ") if " " in line else line.partition("\t")
        op, ops = op.strip(), [o.strip() for o in rest.split(",")]
        mfma = op.startswith("v_mfma")
        memory = op.startswith(("global_", "buffer_", "scratch_", "flat_"))
        reads = registers(",".join(ops[1:] if mfma else ops)) if mfma or memory else set()
        waits, interlocked = 0, set()
        for states, w_op, w_regs, w_line in reversed(history[-8:]):
            if mfma and waits < 2 and w_op.startswith("v_") and not w_op.startswith("v_mfma") and w_regs & reads:
                found.append(("vector write, MFMA", name, w_line, line))
            if memory and waits < 5:
                scalar = {r for r in reads if r[0] == "s"} - interlocked
                if w_op.startswith("v_") and w_regs & scalar:
                    found.append(("vector write of a scalar, load", name, w_line, line))
                if w_op.startswith("s_"):
                    interlocked |= w_regs
            if "_lds_" in op and memory and waits == 0 and re.match(r"s_\w+\s+m0\b", w_line):
                found.append(("M0, LDS-DMA", name, w_line, line))
            waits += states
        states = int(ops[0], 0) + 1 if op == "s_nop" else 1
        history.append((states, op, registers(ops[0]) if op.startswith(("v_", "s_")) else set(), line))
    return found


def test_the_reader_finds_each():
    text = """f:
	v_and_b32_e32 v5, 0xff, v1
	v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[8:15], v[16:23], a[0:3], v5, v6 op_sel_hi:[0,0,0]
	v_readfirstlane_b32 s4, v1
	s_nop 3
	global_load_lds_dword v2, s[4:5]
	s_mov_b32 m0, s9
	global_load_lds_dword v2, s[6:7]
"""
    assert [f[0] for f in hazards(text)] == ["vector write, MFMA", "vector write of a scalar, load", "M0, LDS-DMA"]
    text = """f:
	v_and_b32_e32 v5, 0xff, v1
	s_nop 1
	v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[8:15], v[16:23], a[0:3], v5, v6 op_sel_hi:[0,0,0]
	v_readfirstlane_b32 s4, v1
	s_nop 4
	global_load_lds_dword v2, s[4:5]
	v_readfirstlane_b32 s4, v1
	s_mov_b32 m0, s9
	s_mov_b64 s[10:11], s[4:5]
	global_load_lds_dword v2, s[10:11]
	v_readfirstlane_b32 s8, v1
	s_mov_b32 s8, s3
	global_load_dword v2, v3, s[8:9]
"""
    assert not hazards(text)


@pytest.mark.parametrize("source", with_asm())
def test_wait_states(source, tmp_path):
    out = str(tmp_path / "out.s")
    subprocess.check_call([build.HIPCC, *build.HIP_FLAGS, "-S", "--cuda-device-only", os.path.join(build.CSRC, source),
                           "-o", out], stderr=subprocess.DEVNULL)
    text = open(out).read()
    assert "v_mfma" in text or "_lds_" in text
    found = hazards(text)
    assert not found, f"{len(found)}: {found[:4]}"
