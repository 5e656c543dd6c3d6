"""The loads straight into LDS of the delta rule and the 8-bit product, in the
code that is built from them: as in mx.hip, an instruction has to stand between
the write of M0 and the load that takes its place in LDS from it."""

import os
import re
import subprocess

import pytest
from test_lds_loads_cpu import M0_WRITE, faults, instructions

from quantized_recurrent_state_gdnq_amd import build


@pytest.mark.parametrize("source", ["delta_rule.hip", "delta_rule_backward.hip", "int8.hip"])
def test_loads_into_lds(tmp_path, source):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path / "code.s"
    r = subprocess.run([build.HIPCC] + build.COMMON + build.GPU_FLAGS + build.SOURCE_FLAGS.get(source, [])
                       + ["-w", "--offload-device-only", "-S", os.path.join(build.CSRC, source), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    code = instructions(out.read_text())
    loads = [i for i, ins in enumerate(code) if ins and "load_lds" in ins]
    assert len(loads) > 50
    bad = faults(code)
    assert not bad, f"{len(bad)} of {len(loads)}: {bad[0]}"
    # no write of M0 but for these loads; one may serve several
    uses = [code[i] for i, ins in enumerate(code) if ins and re.search(r"\bm0\b", ins)]
    assert uses and all(M0_WRITE.match(u) for u in uses)
