"""GPU test of the residual norms called from several host threads at once with
different hidden sizes, which share kernel instances but not their needs of
shared memory."""
import threading

import pytest
import torch

import resolution_block_sparse_b200 as mra
from test_gpu_residual_norm import Problem, _cuda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,sizes", [("f32", (2304, 4096, 8192)), ("bf16", (4352, 5632, 8192)), ("f32", (2056, 3004, 4096)),
                                         ("bf16", (4099, 6001, 8191))])
def test_threads_of_different_sizes(dtype, sizes):
    ps = [Problem(2, n, dtype, n) for n in sizes]
    want = [p.both() for p in ps]
    torch.cuda.synchronize()
    got, errors = [None] * len(ps), []
    together = threading.Barrier(len(ps))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                together.wait()
                for _ in range(400):
                    got[i] = ps[i].both()
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # noqa: BLE001
            errors.append((sizes[i], e))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(ps))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errors, errors
    for a, b in zip(want, got):
        assert all(torch.equal(a[n], b[n]) for n in a if a[n] is not None)


@pytest.mark.parametrize("dtype,sizes", [("f32", (2564, 8192)), ("bf16", (5128, 8192)), ("f32", (4100, 8192)), ("f32", (2564, 4096))])
def test_c_calls_side_by_side(dtype, sizes):
    """The C entry points in tight loops, two threads a size: every call is taken."""
    lib = mra.load_library()
    kind = 1 if dtype == "f32" else 0
    bad, jobs = [], []
    for n in sizes * 2:
        p = Problem(1, n, dtype, n)
        stats, ws = torch.empty(4, 1, device="cuda"), torch.empty(lib.mra_residual_norm_workspace(1, n), dtype=torch.uint8, device="cuda")
        x_out, y, dx, dh = (torch.empty_like(p.x) for _ in range(4))
        stream = torch.cuda.Stream()
        keep = (p, stats, ws, x_out, y, dx, dh, stream)
        a = lambda *ts: [None if t is None else t.data_ptr() for t in ts]      # noqa: E731
        tail = [1, n, 0, 3, 1.0, 1e-5, kind]
        fwd = a(p.x, p.h, None) + [1] + a(None, None, None, None, x_out, y, stats) + tail + [stream.cuda_stream]
        bwd = (a(p.x, p.h, None) + [1] + a(None, None, None, None, stats, p.dx_out, p.dy, dx, dh) + [None] * 5 + tail
               + [ws.data_ptr(), ws.numel(), stream.cuda_stream])
        jobs.append((n, fwd, bwd, keep))
    torch.cuda.synchronize()
    together = threading.Barrier(len(jobs))

    def work(n, fwd, bwd, keep):
        together.wait()
        for i in range(4000):
            for name, args in (("fwd", fwd), ("bwd", bwd)):
                status = getattr(lib, "mra_residual_norm_" + name)(*args)
                if status:
                    bad.append((n, name, i, status))
        keep[-1].synchronize()

    ts = [threading.Thread(target=work, args=j) for j in jobs]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad, (len(bad), bad[:5])
