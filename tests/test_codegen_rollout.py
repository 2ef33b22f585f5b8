"""What the compiler makes of the rollout operators' kernels: as for the serving
operators (test_codegen_serve.py), no register may be spilled, nor an
accumulation register written, while a branch of some lanes has the others
switched off."""
import os
import shutil
import subprocess

import pytest

from int4_weight_only_block_amd import build as q4build
from test_codegen_serve import functions, hazards


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="no hipcc")
@pytest.mark.parametrize("source", ["paged_attention_shared.hip", "verify_drafts.hip"])
def test_no_spill_with_lanes_switched_off(source, tmp_path):
    out = str(tmp_path / "kernels.s")
    flags = q4build.HIPCC_FLAGS + q4build.FILE_FLAGS.get(source, [])
    subprocess.run([q4build.hipcc(), *flags, "--cuda-device-only", "-S", os.path.join(q4build.CSRC, source), "-o", out],
                   check=True, capture_output=True, timeout=600)
    with open(out) as f:
        kernels = dict(functions(f.read()))
    results = {name: hazards(body) for name, body in kernels.items()}
    assert len(kernels) >= 4 and sum(n for _, n in results.values()) > 0  # it has been read
    bad = {name: found for name, (found, _) in results.items() if found}
    assert not bad, bad
