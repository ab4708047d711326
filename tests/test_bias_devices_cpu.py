"""CPU test: workspace sizes depend on the device's SM count, so the binding asks
for them with the tensors' device current and keeps them per device."""
import contextlib

import pytest
import torch

import resolution_block_sparse_b200 as mra
from resolution_block_sparse_b200 import _binding as b


class Stand:
    """What the checks read of a CUDA tensor."""
    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096


class Library:
    """Sizes by the current device; calls take their own device's size alone."""
    current = 0

    def mra_blocksparse_attention_bias_workspace(self, *args):
        return 1000 + self.current

    def mra_residual_norm_workspace(self, *args):
        return 2000 + self.current

    def mra_status_string(self, status):
        return b"status"

    def _take(self, size, want):
        return b.MRA_OK if size == want + self.current else b.MRA_ERR_TOO_LARGE

    def mra_blocksparse_attention_bias_fwd(self, *args):
        return self._take(args[-2], 1000)

    mra_blocksparse_attention_bias_bwd = mra_blocksparse_attention_bias_fwd

    def mra_residual_norm_bwd(self, *args):
        return self._take(args[-2], 2000)


@pytest.fixture
def library(monkeypatch):
    lib = Library()

    @contextlib.contextmanager
    def device(index):
        keep, lib.current = lib.current, index
        yield
        lib.current = keep

    def call_on(index, stream, size, call):
        with device(index):
            return call(4096, 0)

    monkeypatch.setattr(b, "load_library", lambda *a: lib)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(b, "_call_on", call_on)
    for f in (b._bias_workspace, b._norm_workspace):
        f.cache_clear()
    yield lib
    for f in (b._bias_workspace, b._norm_workspace):
        f.cache_clear()


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
def test_sizes_by_device(library, order):
    for i in order + order:
        q, lse = Stand((1, 2, 100, 64), torch.bfloat16, i), Stand((1, 2, 100), torch.float32, i)
        table, bucket = Stand((8, 2), torch.bfloat16, i), Stand((199,), torch.int32, i)
        mra.mra_blocksparse_attention_bias_fwd(q, q, q, None, table, bucket, q, lse=lse)
        mra.mra_blocksparse_attention_bias_bwd(q, q, q, None, table, bucket, lse, q, q, q, q, table)
        x, stats = Stand((10, 64), torch.float32, i), Stand((4, 10), torch.float32, i)
        mra.mra_residual_norm_bwd(x, x, stats, x, x, x, x)
