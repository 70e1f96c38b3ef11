"""kvc_tree_decode_attn: calls of many nodes against calls of few, and the
status word of calls without a fault.

Every result is checked with test_gpu_tree's bounds.  For the path of any
shape their logit term, 2^-24 (D / 8 + 16) max sum |q k| sm_scale, comes from
the order in which it adds: eight sums of D / 8 products each (one rounding a
product, inside its multiply-add), three additions of the eight, and the
product with the scale, D / 8 + 4 roundings; the scale itself is rounded once
more.  Its weights are fp32 and are added chunk by chunk, one rounding a key
in the sum and one in the output (N 2^-24 each, below the N 2^-23 there)."""
import numpy as np
import pytest
import torch

from test_gpu_tree import MLA, TINY, Case

pytestmark = pytest.mark.gpu


def _part(kvc, x, nodes, rows, **kw):
    """The call of x's first `nodes` nodes in the sequences `rows` alone."""
    y = Case(kvc, nodes, len(rows), x.cap, parents=x.parents[:nodes, rows].copy("C"), lengths=x.n[rows], **kw)
    y.rec, y.wl = x.rec[rows], x.wl
    y.topk = np.ascontiguousarray(x.topk[:nodes, rows])
    y.q, y.draft = x.q[:nodes, rows].contiguous(), x.draft[:nodes, rows].contiguous()
    y.win = x.win[rows].contiguous()
    return y


@pytest.mark.parametrize("shape", [MLA, TINY])
def test_many_nodes_as_in_smaller_calls(kvc, shape):
    """More nodes than fit on the device at once, and the same nodes in calls
    that split their keys among several CTAs (tensor cores) or do not.  The
    path of any shape gives the same bits; the other adds a node's parts in
    another order where it splits them, so each call is held to the formula."""
    kw = dict(shape, topk=128)
    x = Case(kvc, 16, 24, 300, seed=41, **kw)
    assert x.call() == 0
    x.check()
    whole = x.out.t.clone()
    for nodes, rows in ((16, [0, 1]), (16, [23]), (5, list(range(24))), (1, [7, 8, 9])):
        y = _part(kvc, x, nodes, rows, **kw)
        assert y.call() == 0
        y.check()
        if shape is TINY:
            assert torch.equal(y.out.t, whole[:nodes, rows])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.3e38])
@pytest.mark.parametrize("shape", [MLA, TINY, dict(MLA, heads=40), dict(MLA, act="f32")])
def test_rows_that_no_node_sees_raise_no_flag(kvc, shape, bad):
    """Window rows past the length and another branch's drafted row: neither
    path sets a bit for them, and what does not see them is unchanged."""
    x = Case(kvc, 4, 1, 200, seed=12, parents=np.array([-1, 0, 0, 1])[:, None],
             window_len=shape["window"], **dict(shape, topk=64))
    x.lens = [20]
    assert x.call() == 0
    want, lse = x.out.t.clone(), x.lse.t.clone()
    x.check()
    x.win[0, 20:] = bad
    x.draft[2] = bad  # the row of node 2, on no other node's path
    assert x.call() == 0
    keep = [0, 1, 3]
    assert torch.equal(x.out.t[keep], want[keep]) and torch.equal(x.lse.t[keep], lse[keep])


def test_repeats_of_a_call_give_the_same_bits(kvc):
    """Split keys, whole nodes and the path of any shape, warm and with the
    caches swept in between."""
    sweep = torch.empty(64 << 20, device="cuda")
    for nodes, batch, kw in ((4, 1, {}), (6, 8, {}), (8, 32, {}), (3, 2, TINY)):
        x = Case(kvc, nodes, batch, 700, seed=7, **kw)
        assert x.call() == 0
        out, lse = x.out.t.clone(), x.lse.t.clone()
        for i in range(12):
            if i % 2:
                sweep.fill_(float("nan"))
            x.out.t.fill_(float("nan"))
            kvc.tree_decode_attn(*x.args, **x.kw)
            assert torch.equal(x.out.t, out) and torch.equal(x.lse.t, lse)
