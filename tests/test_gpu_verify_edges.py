"""kvc_verify_tree where a tree is not there, or not as it should be."""
import numpy as np
import pytest
import torch

import plain64
from test_gpu_verify import _case, _np, _run, _same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("root", [0, 3, 5, 99, -3, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("greedy", [False, True])
def test_a_root_with_a_parent_that_is_none(kvc, root, greedy):
    """Node 0's parent is -1, or -2 for no tree.  Anything else is flagged and
    counts as -2, as in the attention of the same tree."""
    p, q, tokens, parents, u, vv = _case(4, 3, 700, 11)
    q = None if greedy else q
    parents[0, 1] = root
    *got, st = _run(kvc, p, q, tokens, parents, u, vv)
    assert st == kvc.DEV_BAD_INDEX
    parents[0, 1] = -2
    _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))
    assert got[1][1] == 0 and got[2][1] == -1 and (got[0][1] == -1).all()
    assert (got[1][[0, 2]] > 0).all()
    *got, st = _run(kvc, p, q, tokens, parents, u, vv)  # and no tree at all is no error
    assert st == 0 and got[1][1] == 0


def test_the_attention_of_the_same_tree_agrees(kvc):
    """A sequence whose root has a parent that is none: absent in both calls."""
    from test_gpu_tree import Case
    parents = np.array([[-1, 0], [0, 0], [1, 1]])
    x = Case(kvc, 3, 2, 200, seed=3, parents=parents)
    assert x.call() == kvc.DEV_BAD_INDEX
    assert not x.out.t[:, 1].any() and bool((x.lse.t[:, 1] == -torch.inf).all())
    p, q, tokens, _, u, vv = _case(3, 2, 500, 12)
    *got, st = _run(kvc, p, q, tokens, parents.astype(np.int32), u, vv)
    assert st == kvc.DEV_BAD_INDEX and got[1][1] == 0 and got[1][0] > 0 and got[2][1] == -1


@pytest.mark.parametrize("greedy", [False, True])
def test_a_finished_sequence_may_hold_anything(kvc, greedy):
    """A padded batch: only the root of a finished sequence says so, its other
    nodes, tokens and rows are what was there before.  They raise no flag."""
    p, q, tokens, parents, u, vv = _case(5, 4, 900, 13)
    parents[0, 2] = -2
    tokens[1:, 2] = [-7, 900, 2 ** 31 - 1, 3]
    p[:, 2], q[:, 2] = float("nan"), float("inf")
    q = None if greedy else q
    *got, st = _run(kvc, p, q, tokens, parents, u, vv)
    assert st == 0
    _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))
    assert got[1][2] == 0 and got[2][2] == -1


def test_distribution_of_greedy_drafts(kvc):
    """Siblings chosen for certain, their tokens different: over many
    independent sequences the token behind the root is distributed as the
    target's row, each of 12 counts within 5 standard deviations of its
    expectation (the fp32 row's sum is within 10^-6 of 1)."""
    n, v, t = 40_000, 12, 4
    g = torch.Generator(device="cuda").manual_seed(6)
    row = torch.rand(v, generator=g, device="cuda") ** 2
    row /= row.sum()
    p = row.expand(t, n, v).contiguous()
    parents = torch.zeros(t, n, dtype=torch.int32, device="cuda")
    parents[0] = -1
    tokens = torch.tensor([0, 7, 2, 9], dtype=torch.int32, device="cuda")[:, None].repeat(1, n)
    u, vv = torch.rand(t, n, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    path = torch.empty(n, t, dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    kvc.verify_tree(p, None, tokens, parents, u, vv, path, n_path, nxt)
    second = path[:, 1].long()
    first = torch.where(second > 0, tokens[second.clamp_min(0), torch.arange(n, device="cuda")], nxt)
    count = torch.bincount(first.long(), minlength=v).double()
    sd = (n * row.double() * (1 - row.double())).sqrt()
    assert torch.all((count - n * row.double()).abs() <= 5 * sd)
    assert 0.02 < (n_path > 1).double().mean() < 1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("total", [0.5, 0.99, 1.01, 2.0])
def test_greedy_rows_whose_sum_is_not_one(kvc, dtype, total):
    """The mass is 1 less what was rejected, whatever the row's sum."""
    p, q, tokens, parents, u, vv = _case(6, 9, 400, 17, star=True)
    p = (total * p.float()).to(dtype)
    tokens[1:] = np.argsort(-_np(p)[0], -1)[:, :5].T
    *got, st = _run(kvc, p, None, tokens, parents, u, vv)
    assert st == 0
    _same(got, plain64.verify(_np(p), None, tokens, parents, u, vv))
