"""The serving operators in the debug build (Q4DEC_DEBUG=1): one child python
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


def test_serving_operators_in_the_debug_build():
    env = dict(os.environ, Q4DEC_LIB=q4build.DEBUG_LIB_PATH,
               PYTHONPATH=os.pathsep.join(p for p in (ROOT, os.environ.get("PYTHONPATH")) if p))
    res = subprocess.run([sys.executable, "-u", os.path.join(HERE, "gpu_debug_serve_child.py")], env=env,
                         capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-3000:]
    out = json.loads(res.stdout.strip().splitlines()[-1])
    assert out["lib"] == q4build.DEBUG_LIB_PATH
    assert out["start"] == [0, 0]
    assert out["after_calls"] == [0, 0], f"launch-contract bits set: {out['after_calls'][1]:#x}"
    assert out["close"]


SATURATED = """
import json, torch
import int4_weight_only_block_amd as q4
g = torch.Generator(device="cuda:0"); g.manual_seed(3)
for vocab in (50, 40009):
    z = 360 + 210 * torch.rand(4, vocab, generator=g, device="cuda:0")
    for heat in (1.3, 0.3, 0.01, 1e-6):
        print("case", vocab, heat, flush=True)
        full = lambda v, t=torch.float32: torch.full((4,), v, dtype=t, device="cuda:0")
        for kw in (dict(top_p=full(0.4)), dict(top_k=full(300, torch.int32))):
            q4.sample_logits(z, full(0.6), temperature=full(heat), **kw)
torch.cuda.synchronize()
print(json.dumps(dict(lib=q4.LIB_PATH, word=list(q4.debug_status()))))
"""


def test_sampling_steps_stay_in_the_histogram():
    """Rows whose logits are all 12 to 19 times the cap: no token's step lies outside the histogram."""
    env = dict(os.environ, Q4DEC_LIB=q4build.DEBUG_LIB_PATH,
               PYTHONPATH=os.pathsep.join(p for p in (ROOT, os.environ.get("PYTHONPATH")) if p))
    res = subprocess.run([sys.executable, "-u", "-c", SATURATED], env=env, capture_output=True, text=True, timeout=120,
                         cwd=ROOT)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-3000:]
    out = json.loads(res.stdout.strip().splitlines()[-1])
    assert out == dict(lib=q4build.DEBUG_LIB_PATH, word=[0, 0]), out
