"""GPU test of the warp-level biased attention's way out of a wait that expires
(heads of 32, the backward of small batches): the host-set hook
MRA_TEST_EXPIRE_WAIT makes every block's first wait report expiry without
waiting.  The call returns, the status says so, the next call is clean."""
import os
import subprocess
import sys

import pytest

from test_gpu_bias_attention import _cuda  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import os, sys
sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
import bias_testlib as bt
import resolution_block_sparse_b200 as mra
from resolution_block_sparse_b200 import _binding as b
import test_gpu_bias_attention as t
for name in ("dense-1024-32-bf16", "dense-1056-32-bf16", "lists-500-32-bf16-3", "long-rows-d32", "dense-300-64-bf16",
             "lists-500-64-bf16-3"):
    p = t.make(name)
    want = p.want()
    lse = want["lse"][0].float()
    os.environ["MRA_TEST_EXPIRE_WAIT"] = "1"
    for call in (p.forward, lambda: p.backward(lse)):
        call()
        assert mra.mra_get_device_status() & b.MRA_DEV_TIMEOUT, name
    del os.environ["MRA_TEST_EXPIRE_WAIT"]
    bt.check(p.both(), want, name)
    assert mra.mra_get_device_status() == 0
print("RESULT ok")
'''


def test_warp_level_kernels():
    e = dict(os.environ)
    e.pop("MRA_TEST_EXPIRE_WAIT", None)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=e, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "RESULT ok" in r.stdout
