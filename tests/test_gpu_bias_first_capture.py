"""GPU test: calls whose kernels this process has not run before, captured into
a graph: only a device's first attention call has to come before a capture, the
norms' none."""
import os
import subprocess
import sys

import pytest

from test_gpu_bias_attention import _cuda  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
import torch
import test_gpu_bias_attention as t
import test_gpu_bias_batches as l
import test_gpu_residual_norm as n
norms = [n.Problem(50, 8192, "f32", 1, gates=2), n.Problem(70, 768, "bf16", 2), n.Problem(9, 1027, "f32", 3, norm="rms")]
ps = [t.make("lists-500-32-bf16-3"), t.make("dense-1100-64-f32"), l.make("short-lists"), t.make("dense-300-64-bf16")]
torch.cuda.synchronize()

def capture(p):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = p.both()
    g.replay()
    torch.cuda.synchronize()
    want = p.both()
    for k in want:
        assert want[k] is None or torch.equal(want[k], out[k]), k

for p in norms:
    capture(p)
t.make("dense-33-64-bf16").forward()              # the first attention call
for p in ps:
    capture(p)
print("RESULT ok")
'''


def test_first_calls_in_a_capture():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "RESULT ok" in r.stdout
