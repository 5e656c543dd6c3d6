"""The loads straight into LDS of mx.hip, in the code that is built from it.

Such a load takes its place in LDS from the scalar register M0, and the chip
does not wait by itself for a scalar write of M0 right before it: another
instruction has to stand between.  The compiler sees to that for its own
loads, but not inside an asm statement.  Nor does it see there that a scalar
register written by a vector instruction must not be an address within the
next five instructions."""

import os
import re
import subprocess

import pytest

from quantized_recurrent_state_gdnq_amd import build

M0_WRITE = re.compile(r"^s_\w+ m0,")
VECTOR_SGPR_WRITE = re.compile(r"^v_(?:readfirstlane|readlane|cmp)\w* (s\d+|s\[\d+:\d+\])")


def instructions(text):
    """The instructions in order, one text each; None at a label (a branch may come in there)."""
    out = []
    for line in text.splitlines():
        line = line.split(";")[0].split("//")[0].strip()
        if re.match(r"^[.\w$]+:", line):
            out.append(None)
        elif line and not line.startswith("."):
            out.append(re.sub(r"\s+", " ", line))
    return out


def scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m[1])} if m else set()


def faults(code):
    bad = []
    for i, ins in enumerate(code):
        if not ins or "load_lds" not in ins:
            continue
        if code[i - 1] is None or M0_WRITE.match(code[i - 1]):
            bad.append(f"no wait after the write of M0: {code[i - 1]}; {ins}")
        address = scalars(ins.split(", ")[-1].split(" ")[0])
        waited = 0
        for before in reversed(code[max(0, i - 6):i]):
            if waited >= 5 or before is None:
                break
            m = VECTOR_SGPR_WRITE.match(before)
            if m and scalars(m[1]) & address:
                bad.append(f"address written by a vector instruction: {before}; {ins}")
            nop = re.fullmatch(r"s_nop (\d+)", before)
            waited += 1 + (int(nop[1]) if nop else 0)
    return bad


def test_the_check_itself():
    good = "a:\ns_mov_b32 m0, s2\ns_nop 0\nglobal_load_lds_dwordx4 v1, s[4:5]\n"
    assert not faults(instructions(good))
    assert len(faults(instructions(good.replace("s_nop 0\n", "")))) == 1
    assert len(faults(instructions(good.replace("a:", "v_readfirstlane_b32 s5, v3")))) == 1
    assert not faults(instructions(good.replace("a:", "v_readfirstlane_b32 s5, v3\ns_nop 4")))
    assert len(faults(instructions(good.replace("a:\n", "v_readfirstlane_b32 s5, v3\nv_mov_b32 v1, v2\n")))) == 1
    assert not faults(instructions(good.replace("a:", "v_readfirstlane_b32 s6, v3")))


def test_loads_into_lds(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path / "mx.s"
    r = subprocess.run([build.HIPCC] + build.COMMON + build.GPU_FLAGS
                       + ["-w", "--offload-device-only", "-S", os.path.join(build.CSRC, "mx.hip"), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    code = instructions(out.read_text())
    loads = [i for i, ins in enumerate(code) if ins and "load_lds" in ins]
    assert len(loads) > 100
    bad = faults(code)
    assert not bad, f"{len(bad)} of {len(loads)}: {bad[0]}"
    # every use of M0 belongs to one of these loads: the compiler keeps nothing of its own there
    uses = [i for i, ins in enumerate(code) if ins and re.search(r"\bm0\b", ins)]
    assert len(uses) == len(loads) and all(M0_WRITE.match(code[i]) for i in uses)
