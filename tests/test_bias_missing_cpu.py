"""CPU test: a required tensor that is None is refused by name."""
import pytest
import torch

import resolution_block_sparse_b200 as mra
from test_bias_devices_cpu import Stand

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


@pytest.mark.parametrize("name", ["q", "k", "v", "bias_table", "bucket", "out"])
def test_forward(name):
    a = dict(q=Stand((1, 2, 100, 64), BF16, 0), key_mask=None, bias_table=Stand((8, 2), BF16, 0), bucket=Stand((199,), I32, 0))
    a.update(k=a["q"], v=a["q"], out=a["q"])
    a[name] = None
    with pytest.raises(ValueError, match=f"mra_blocksparse_attention_bias_fwd: {name} "):
        mra.mra_blocksparse_attention_bias_fwd(**a)


@pytest.mark.parametrize("name", ["q", "k", "v", "bias_table", "bucket", "lse", "dout", "dq", "dk", "dv", "dbias_table"])
def test_backward(name):
    q = Stand((1, 2, 100, 64), BF16, 0)
    a = dict(q=q, k=q, v=q, key_mask=None, bias_table=Stand((8, 2), BF16, 0), bucket=Stand((199,), I32, 0),
             lse=Stand((1, 2, 100), F32, 0), dout=q, dq=q, dk=q, dv=q, dbias_table=Stand((8, 2), BF16, 0))
    a[name] = None
    with pytest.raises(ValueError, match=f"mra_blocksparse_attention_bias_bwd: {name}[: ]"):
        mra.mra_blocksparse_attention_bias_bwd(**a)


def test_norms():
    x = Stand((10, 64), F32, 0)
    with pytest.raises(ValueError, match="mra_residual_norm_fwd: x "):
        mra.mra_residual_norm_fwd(None, x, x, x)
    with pytest.raises(ValueError, match="mra_residual_norm_bwd: x "):
        mra.mra_residual_norm_bwd(None, x, x, x, x, x, x)


def test_too_small_a_workspace_is_named():
    assert "workspace" in mra.mra_status_string(6)
