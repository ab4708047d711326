"""GPU test of a process's first call, on a non-blocking stream beside a busy
default stream: a refused list is reported, not cleared by the status word's own
setting up."""
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
import resolution_block_sparse_b200 as mra
import test_gpu_bias_attention as t
p = t.Problem(1, 4, 200, 64, torch.bfloat16, 3, lists=t.rows(4))
p.lists[1, 0] = 49                                # past the last block
out = torch.empty_like(p.q)
side = torch.cuda.Stream()
x = torch.randn(8192, 8192, device="cuda")
torch.cuda.synchronize()
for _ in range(20):
    x @ x                                         # some tenths of a second on the default stream
mra.mra_blocksparse_attention_bias_fwd(p.q, p.k, p.v, None, p.table, p.bucket, out, block_idx=p.lists, stream=side)
side.synchronize()
assert mra.mra_get_device_status(side) & mra._binding.MRA_DEV_COUNT
assert mra.mra_get_device_status(side) == 0
print("RESULT ok")
'''


def test_status_of_the_first_call():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "RESULT ok" in r.stdout
