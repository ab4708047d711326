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


@pytest.mark.parametrize("N", [2, 70, 1100])
@pytest.mark.parametrize("D,dtype,top,second", [(D, t, *x) for D in (64, 32) for t in (BF16, torch.float32)
                                                for x in ((30.0, 18.125), (1000.0, 991.6))
                                                if t != BF16 or x[0] == 30.0])      # (991.6 is no bf16 number)
def test_lse_of_large_scores(N, D, dtype, top, second):
    """A key of score `top` and neighbours of score `second`, whose small weights
    count: the scores are the table's values, exact in the type, so that the lse
    is off by its own rounding (half a step of `top`) and by a hundredth of it
    for the weights' and the logarithm's."""
    p = Problem(1, 2, N, D, dtype, 7, nb=4)
    p.q.zero_()
    p.table.fill_(0.0)
    p.table[0], p.table[1] = top, second
    p.bucket.fill_(-1)
    p.bucket[N - 1] = 0
    p.bucket[N - 2] = p.bucket[N] = 1
    got = p.forward()["lse"].double()
    n = torch.full((N,), 2.0, dtype=torch.float64, device="cuda")
    n[0] = n[-1] = 1.0
    want = top + torch.log1p(n * torch.exp(p.table[1, 0].double() - top))
    step = 2.0 ** (4 - 23) if top == 30.0 else 2.0 ** (9 - 23)
    assert float((got - want).abs().max()) <= 0.51 * step


@pytest.mark.parametrize("D,dtype", [(64, BF16), (32, BF16), (64, torch.float32)])
@pytest.mark.parametrize("spread", [1.0, 8.0, 60.0])
def test_rows_of_one_key_with_large_scores(D, dtype, spread):
    """The first rows of causal heads, with scores up to thousands: weight 1, no
    gradient of the scores, lse the score itself."""
    p = Problem(4, 8, 140, D, dtype, 19, causal=True, spread=spread)
    got = p.both()
    assert torch.equal(got["out"][:, :, 0], p.v[:, :, 0]) and float(got["dq"][:, :, 0].abs().max()) == 0.0
    s = (p.q[:, :, 0].double() * p.k[:, :, 0].double()).sum(-1) * p.scale + p.table[p.bucket[139].long()].double()
    size = (p.q[:, :, 0].double() * p.k[:, :, 0].double()).abs().sum(-1) * p.scale + 8.0
    assert bool(((got["lse"][:, :, 0].double() - s).abs() <= 2.0 ** -20 * size).all())
