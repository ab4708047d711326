"""GPU test of the residual norms on batches without rows and with a gate, whose
gradient is then an empty sum."""
import pytest
import torch

import resolution_block_sparse_b200 as mra
from test_gpu_residual_norm import Problem, _cuda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0, 64), (0, 5, 64), (3, 0, 64)])
@pytest.mark.parametrize("gates", [0, 1, 3])
@pytest.mark.parametrize("own_stream", [False, True])
def test_no_rows_and_a_gate(shape, gates, own_stream):
    e = lambda: torch.empty(shape, dtype=torch.bfloat16, device="cuda")      # noqa: E731
    gate = torch.ones(gates, 64, dtype=torch.bfloat16, device="cuda")
    dgate, dw = torch.full_like(gate, 7.0), torch.full_like(gate[:1].reshape(-1) if gates else gate.new_empty(64), 7.0)
    stats = torch.empty(4, 0, device="cuda")
    stream = torch.cuda.Stream() if own_stream else None
    torch.cuda.synchronize()
    mra.mra_residual_norm_fwd(e(), e(), e(), e(), gate=gate, post_norm=True, stats=stats, stream=stream)
    mra.mra_residual_norm_bwd(e(), e(), stats, e(), e(), e(), e(), gate=gate, post_norm=True, dgate=dgate, dpre_w=dw,
                              stream=stream)
    torch.cuda.synchronize()
    assert float(dgate.abs().sum()) == 0.0 and float(dw.abs().sum()) == 0.0


def test_gates_that_do_not_divide_are_refused_still():
    p = Problem(12, 64, "bf16", 1)
    for gate in (p.x[:5], p.x[:0], p.x[0]):
        with pytest.raises(ValueError, match="gate must"):
            mra.mra_residual_norm_fwd(p.x, p.h, p.x, p.h, gate=gate.contiguous())
