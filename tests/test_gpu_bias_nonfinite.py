"""GPU tests of the biased attention with NaN and infinities in valid tokens: they
reach the block rows (columns) whose lists join them to the token's block, and
no others, although a kernel takes several block rows at once; padded rows and
columns stay without a gradient.

What a token in block J may reach: a NaN in V or K every query of the block rows
that list J (their delta, and with it all their dS), and by these the keys of
every block that those rows list; one in Q or dO its own row alone, and the
keys of the blocks that its block row lists.  Everything else is held to the
allowances of the clean problem."""
import math

import pytest
import torch

import bias_testlib as bt
import resolution_block_sparse_b200 as mra
from test_gpu_bias_attention import Problem, _cuda, rows  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# the kernels that each takes: tcgen05 forward and backward (a batch large
# enough for the latter)
TC = {"tc-lists": dict(B=8, H=8, N=1100, D=64, dtype=BF16, lists=rows(9, (1, 2), (0, 5)), pad=[0, 300] + [0] * 6),
      "tc-long-rows": dict(B=20, H=8, N=700, D=64, dtype=BF16, lists=rows(9, (), (0, 9))),
      "tc-causal": dict(B=20, H=16, N=161, D=64, dtype=BF16, causal=True)}
FP32 = {"f32-lists": dict(B=2, H=3, N=700, D=64, dtype=F32, lists=rows(6, (1, 2), (0, 5)), pad=[0, 200]),
        "f32-lists-d32": dict(B=2, H=2, N=500, D=32, dtype=F32, lists=rows(3, (1, 2), (0, 9)), pad=[100, 0]),
        "f32-causal": dict(B=2, H=2, N=161, D=64, dtype=F32, causal=True),
        "f32-causal-d32": dict(B=1, H=4, N=300, D=32, dtype=F32, causal=True)}
WARP = {"warp-lists-d32": dict(B=2, H=4, N=700, D=32, dtype=BF16, lists=rows(6, (1, 2), (0, 5)), pad=[0, 300]),
        "warp-half-listed-d32": dict(B=1, H=2, N=500, D=32, dtype=BF16, lists=rows(11, (1, 2), (0, 9)), pad=[100]),
        "warp-causal-d32": dict(B=2, H=2, N=161, D=32, dtype=BF16, causal=True),
        "warp-long-causal-d32": dict(B=1, H=1, N=1200, D=32, dtype=BF16, causal=True),
        "warp-padded-d32": dict(B=3, H=2, N=150, D=32, dtype=BF16, pad=[70, 0, 33]),
        "warp-backward": dict(B=2, H=2, N=400, D=64, dtype=BF16, lists=rows(3, (1,), (0, 5)), pad=[0, 150]),
        "warp-backward-causal": dict(B=1, H=2, N=300, D=64, dtype=BF16, causal=True, pad=[90])}
SPLIT = {"split-tc-causal": dict(B=3, H=4, N=1300, D=64, dtype=BF16, causal=True, pad=[0, 500, 1]),
         "split-forward-causal": dict(B=1, H=2, N=1200, D=64, dtype=BF16, causal=True),
         "split-f32-causal": dict(B=1, H=2, N=1200, D=32, dtype=F32, causal=True),
         "tc-short-causal": dict(B=8, H=8, N=600, D=64, dtype=BF16, causal=True, pad=[0, 90] + [0] * 6)}
CASES = {**TC, **FP32, **WARP, **SPLIT}


def make(name, seed=5):
    c = dict(CASES[name])
    return Problem(c.pop("B"), c.pop("H"), c.pop("N"), c.pop("D"), c.pop("dtype"), seed, **c)


def listed(p):
    """bool [BH, nbr, nbr]: the blocks that hold a pair."""
    B, H, N, _ = p.q.shape
    nbr = (N + 31) // 32
    on = torch.ones(B * H, nbr * nbr, dtype=torch.bool, device="cuda")
    if p.lists is not None:
        on = torch.zeros_like(on)
        for i in range(B * H):
            on[i, p.lists[i][p.lists[i] >= 0].long()] = True
    on = on.reshape(B * H, nbr, nbr)
    d = torch.arange(nbr, device="cuda")
    lo = (32 * (d[None, :] - d[:, None]) - 31 + N - 1).clamp(0, 2 * N - 2)
    hi = (32 * (d[None, :] - d[:, None]) + 31 + N - 1).clamp(0, 2 * N - 2)
    count = torch.cat([torch.zeros(1, device="cuda"), (p.bucket >= 0).cumsum(0)])
    return on & (count[hi + 1] > count[lo])


def tokens(blocks, N):
    return blocks.repeat_interleave(32, -1)[..., :N]


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("where,value", [("v", math.nan), ("v", math.inf), ("k", math.nan), ("q", math.nan), ("q", -math.inf),
                                         ("dout", math.nan), ("dout", math.inf)])
def test_reach(name, where, value):
    p = make(name)
    B, H, N, D = p.q.shape
    want, on = p.want(), listed(p)
    token = N // 2 + 3                              # in a valid token of every entry
    J = token // 32
    # one feature of the token: a NaN in V reaches one column of the output
    x = getattr(p, where)
    x[:, :, token, 5] = value
    got = p.both()
    nbr = on.shape[1]
    row_hit = on[:, :, J] if where in "vk" else torch.zeros(B * H, nbr, dtype=torch.bool, device="cuda")
    if where in "vk":
        col_hit = (row_hit[:, :, None] & on).any(1)
    else:
        col_hit = on[:, J]
    row_hit, col_hit = tokens(row_hit, N).reshape(B, H, N), tokens(col_hit, N).reshape(B, H, N)
    if where not in "vk":
        row_hit[:, :, token] = True
    none = torch.zeros_like(row_hit)
    hit = {"out": row_hit if where != "dout" else none, "lse": row_hit if where in "kq" else none, "dq": row_hit,
           "dk": col_hit, "dv": col_hit if where != "v" else none}
    live = torch.ones(B, N, dtype=torch.bool, device="cuda") if p.mask is None else p.mask > 0
    live = live[:, None].expand(B, H, N)
    for n, h in hit.items():
        h = h & live                                # padded tokens have no output and no gradient
        ref, allow = want[n]
        at = ~h
        bt.check({n: got[n][at]}, {n: (ref[at], allow[at])}, f"{name} {where} {value}")
    # and what it does reach is not hidden
    if where == "v":
        pairs = (with_pair(p, token) & live).nonzero(as_tuple=True)
        assert not bool(torch.isfinite(got["out"][pairs][:, 5]).any())
    if where == "dout" and value != value:
        i = on.reshape(B, H, nbr, nbr)[:, :, J]
        dv = got["dv"][..., 5].float().isnan()
        assert bool((dv.reshape(B, H, N) <= tokens(i, N)).all()) and bool(dv.any())


def with_pair(p, token):
    """bool [B, H, N]: the queries with a pair with this key."""
    B, H, N, _ = p.q.shape
    on = tokens(listed(p)[:, :, token // 32], N).reshape(B, H, N)
    d = token - torch.arange(N, device="cuda") + N - 1
    return on & (p.bucket[d] >= 0)[None, None]


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("where", ["q", "k", "table"])
def test_rows_with_a_nan_score_are_nan(name, where):
    """A query whose scores hold a NaN has pairs: its output and lse are NaN, not
    the 0 and -inf of a query without one, and so is its gradient."""
    p = make(name)
    B, H, N, D = p.q.shape
    token = N // 2 + 3
    live = torch.ones(B, N, dtype=torch.bool, device="cuda") if p.mask is None else p.mask > 0
    live = live[:, None].expand(B, H, N)
    any_pair = p.want()["lse"][0] > -math.inf
    if where == "q":
        hit = torch.zeros(B, H, N, dtype=torch.bool, device="cuda")
        hit[:, :, token] = True
    elif where == "k":
        hit = with_pair(p, token)
    else:
        # bucket 0: the query's own position
        on = listed(p).diagonal(dim1=1, dim2=2)
        hit = tokens(on, N).reshape(B, H, N)
    hit = hit & live & any_pair
    if where == "table":
        p.table[0] = math.nan
    else:
        getattr(p, where)[:, :, token, 3] = math.nan
    got = p.both()
    assert bool(hit.any())
    assert bool(got["out"][hit].isnan().all()) and bool(got["lse"][hit].isnan().all())
    assert bool(got["dq"][hit].isnan().all())
