"""GPU tests of how far the biased attention's bf16 results are from the exact
ones, norm against norm, in units of the error that the rounded exact result has.

The warp-level backward (heads of 32 at any size, heads of 64 in small batches)
takes its weights in two bf16 pieces: what is left beside the results' own
rounding are fp32 terms and 2^-8 of the weights' 2^-8, well below a tenth.
The forward and the tcgen05 backward round each weight once: an error of its own
of the same size, relative to terms whose sum has random signs, so sqrt(2) of the
rounding alone; 1.5 leaves 6 % for the spread of that sum.  The table's gradient
is an fp32 sum of fp32 terms and is held to a tenth everywhere; its few values
are rounded to bf16 once, and with 32 x 12 of them the two norms agree."""
import pytest
import torch

from test_gpu_bias_attention import Problem, _cuda, rows  # noqa: F401

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
WARP = {"heads-of-32": dict(B=8, H=12, N=512, D=32), "heads-of-32-lists": dict(B=2, H=12, N=1024, D=32, lists=rows(6, (3,), (0,))),
        "heads-of-32-odd": dict(B=1, H=3, N=1111, D=32, pad=[100]), "long-small-batch": dict(B=1, H=2, N=2048, D=64),
        "just-above-2-to-17": dict(B=1, H=5, N=420, D=64), "lists-small-batch": dict(B=1, H=4, N=1500, D=64, lists=rows(4))}
TC = {"train": dict(B=8, H=12, N=512, D=64, pad=[0, 100] + [0] * 6), "lists": dict(B=2, H=12, N=1500, D=64, lists=rows(20))}


def ratios(p):
    want, got = p.want(), p.both()
    r = {}
    for n in ("out", "dq", "dk", "dv", "dtable"):
        ref = want[n][0]
        r[n] = float((got[n].double() - ref).norm() / (ref.to(BF16).double() - ref).norm())
    return r


@pytest.mark.parametrize("name", list(WARP) + list(TC))
def test_error_norms(name):
    c = dict(WARP.get(name) or TC[name])
    p = Problem(c.pop("B"), c.pop("H"), c.pop("N"), c.pop("D"), BF16, 41, **c)
    r = ratios(p)
    top = 1.1 if name in WARP else 1.5
    assert r["out"] <= 1.5 and r["dtable"] <= 1.1, r
    assert max(r["dq"], r["dk"], r["dv"]) <= top, r
