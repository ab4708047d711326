"""CPU test: the bucket map's generator, a C entry point, needs no memory of its
own, so that none of it can be missing (an exception must not leave a C entry)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes, os, resource, sys
sys.path.insert(0, sys.argv[1])
import numpy as np
import resolution_block_sparse_b200 as mra
fn = mra.load_library().mra_relative_buckets
cases = [(300, 32, 128, 1), (2000, 1024, 2048, 0), (65536, 1024, 1 << 30, 0), (65536, 1023, 511 << 12, 0)]      # distances on a border
outs = [np.zeros(2 * c[0] - 1, dtype=np.int32) for c in cases]
wants = [np.zeros(2 * c[0] - 1, dtype=np.int32) for c in cases]
args = [(*c, o.ctypes.data_as(ctypes.c_void_p)) for c, o in zip(cases, outs)]
for c, w in zip(cases, wants):
    assert fn(*c, w.ctypes.data_as(ctypes.c_void_p)) == 0
malloc = ctypes.CDLL(None).malloc
malloc.restype, malloc.argtypes = ctypes.c_void_p, [ctypes.c_size_t]
got = [0] * len(cases)
vm = int(open("/proc/self/statm").read().split()[0]) * os.sysconf("SC_PAGE_SIZE")
resource.setrlimit(resource.RLIMIT_AS, (vm, resource.RLIM_INFINITY))
size = 1 << 26
while size >= 32:                          # all that malloc still has
    while malloc(size):
        pass
    size >>= 1
for i in range(len(args)):
    got[i] = fn(*args[i])
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
assert got == [0] * len(cases), got
assert all(np.array_equal(o, w) for o, w in zip(outs, wants))
print("RESULT ok")
'''


def test_bucket_map_without_memory():
    e = dict(os.environ, MALLOC_ARENA_MAX="1")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=e, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-2000:], r.stderr[-3000:])
    assert "RESULT ok" in r.stdout
