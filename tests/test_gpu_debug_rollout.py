"""The rollout operators in the debug build (Q4DEC_DEBUG=1): one child python
loads libq4dec_debug.so, runs every kernel of theirs and reports; no launch
check may fail, and what the build computes must still be right."""
import json
import os
import subprocess
import sys

import pytest

from int4_weight_only_block_amd import build as q4build

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(q4build.DEBUG_LIB_PATH),
                                 reason="libq4dec_debug.so not built (build(debug=True))")]


def test_rollout_operators_in_the_debug_build():
    env = dict(os.environ, Q4DEC_LIB=q4build.DEBUG_LIB_PATH,
               PYTHONPATH=os.pathsep.join(p for p in (ROOT, os.environ.get("PYTHONPATH")) if p))
    res = subprocess.run([sys.executable, "-u", os.path.join(HERE, "gpu_debug_rollout_child.py")], env=env,
                         capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-3000:]
    out = json.loads(res.stdout.strip().splitlines()[-1])
    assert out["lib"] == q4build.DEBUG_LIB_PATH
    assert out["start"] == [0, 0]
    assert out["after_calls"] == [0, 0], f"launch-contract bits set: {out['after_calls'][1]:#x}"
    assert out["close"]
