"""kvc_verify_tree against the rule followed one sequence at a time in fp64
(plain64.verify, which normalises the residual after every rejection).  All
outputs are whole numbers and must be equal: a border between two outcomes is
a real number that the two orders of summation place within 10^-15 of each
other, and no case's random number falls that close to one."""
import numpy as np
import pytest
import torch

import plain64
from helpers import Guarded

pytestmark = pytest.mark.gpu


def _run(kvc, p, q, tokens, parents, u, v, stream=None):
    t, b, _ = p.shape
    path, n_path, nxt = (Guarded(s, torch.int32, fill=-9) for s in ((b, t), (b,), (b,)))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = [None if x is None else torch.as_tensor(x).cuda() for x in (tokens, parents, u, v)]
    kvc.verify_tree(p, q, *dev, path.t, n_path.t, nxt.t, status=st, stream=stream)
    for g in (path, n_path, nxt):
        g.check()
    return path.t.cpu().numpy(), n_path.t.cpu().numpy(), nxt.t.cpu().numpy(), int(st.item())


def _np(x):
    return None if x is None else x.double().cpu().numpy()


def _same(got, want):
    for name, g, w in zip(("path", "n_path", "next_token"), got, want):
        assert np.array_equal(g, w), f"{name}: {np.argwhere(g != w)[:4].tolist()}"


def _case(t, b, v, seed, dtype=torch.float32, star=False, sharp=2.0, noise=0.7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = sharp * torch.randn(t, b, v, generator=g, device="cuda")
    p = logits.softmax(-1).to(dtype)
    q = (logits + noise * torch.randn(t, b, v, generator=g, device="cuda")).softmax(-1).to(dtype)
    rng = np.random.default_rng(seed)
    parents = np.full((t, b), -1, np.int32)
    for i in range(1, t):
        parents[i] = 0 if star else np.maximum(0, i - 1 - rng.integers(0, 3, b))
    tokens = rng.integers(0, v, (t, b)).astype(np.int32)
    for i in range(1, t):  # as a draft draws them
        for j in range(b):
            tokens[i, j] = int(torch.multinomial(q[parents[i, j], j].float(), 1, generator=g))
    u, vv = rng.random((t, b)).astype(np.float32), rng.random(b).astype(np.float32)
    return p, q, tokens, parents, u, vv


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,b,v", [(1, 1, 1), (1, 3, 5), (2, 1, 33), (4, 5, 1000), (8, 3, 4097),
                                   (5, 2, 50_001), (16, 40, 1024), (3, 1, 200_000), (6, 700, 96)])
def test_draft_probabilities(kvc, t, b, v, dtype):
    """One token to a large odd vocabulary, one sequence to more than fit at
    once; vectors and single loads."""
    for seed in (1, 2):
        p, q, tokens, parents, u, vv = _case(t, b, v, seed * 100 + t, dtype)
        *got, st = _run(kvc, p, q, tokens, parents, u, vv)
        assert st == 0
        _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))


@pytest.mark.parametrize("t,b,v", [(2, 4, 50), (7, 6, 3000), (33, 3, 20_011), (256, 2, 700)])
def test_many_rejections(kvc, t, b, v):
    """Stars: every sibling can be rejected, so the residual shrinks many
    times; drafts far from the target."""
    for greedy in (False, True):
        p, q, tokens, parents, u, vv = _case(t, b, v, 7 + t, star=True, noise=3.0)
        if greedy:  # siblings with different tokens, from the draft's best ones
            tokens[1:] = np.argsort(-_np(q)[0], -1)[:, :t - 1].T if v >= t else tokens[1:]
            u = np.maximum(u, np.float32(0.5))
        *got, st = _run(kvc, p, None if greedy else q, tokens, parents, u, vv)
        assert st == 0
        _same(got, plain64.verify(_np(p), None if greedy else _np(q), tokens, parents, u, vv))
        assert got[1].min() >= 1


def test_greedy_trees(kvc):
    p, q, tokens, parents, u, vv = _case(9, 12, 2500, 31)
    for j in range(12):
        seen = {}
        for i in range(1, 9):
            up = parents[i, j]
            order = np.argsort(-_np(q)[up, j])
            tokens[i, j] = order[seen.get(up, 0)]
            seen[up] = seen.get(up, 0) + 1
    *got, st = _run(kvc, p, None, tokens, parents, u, vv)
    assert st == 0
    _same(got, plain64.verify(_np(p), None, tokens, parents, u, vv))
    assert got[1].max() > 1


def test_equal_rows_accept_everything(kvc):
    """p = q: u q < p always, so every chain is accepted to its end; u just
    below 1 included."""
    p, _, tokens, parents, u, vv = _case(6, 4, 777, 41)
    parents[1:] = np.arange(5)[:, None]
    q = p.clone()
    tokens[1:] = _np(p)[:-1].argmax(-1)
    u[:] = np.nextafter(np.float32(1), np.float32(0))
    *got, _ = _run(kvc, p, q, tokens, parents, u, vv)
    assert np.array_equal(got[1], np.full(4, 6)) and np.array_equal(got[0][0], np.arange(6))
    _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))


def test_draws_at_the_borders(kvc):
    """Probabilities with exact sums: v = 0 takes the first token with mass, a
    border itself belongs to the next token, v just below 1 the last one."""
    v = 5000
    p = torch.zeros(1, 6, v, device="cuda")
    p[:, :, 1024] = 0.25
    p[:, :, 2047] = 0.25
    p[:, :, 2048] = 0.25
    p[:, :, 4999] = 0.25
    vv = np.array([0, 0.25, 0.5, 0.75, np.nextafter(np.float32(1), np.float32(0)),
                   np.nextafter(np.float32(0.25), np.float32(0))], np.float32)
    z = np.zeros((1, 6), np.int32)
    *got, _ = _run(kvc, p, None, z, z - 1, np.zeros((1, 6), np.float32), vv)
    assert got[2].tolist() == [1024, 2047, 2048, 4999, 4999, 1024]


def test_empty_residual_and_empty_rows(kvc):
    """A residual without mass gives way to the target's row (drafts above the
    target everywhere: p = q / 2); a row without mass gives -1 and a flag."""
    p, q, tokens, parents, u, vv = _case(3, 3, 300, 51, star=True)
    q[:] = 2 * p
    u[:] = 0.9
    *got, st = _run(kvc, p, q, tokens, parents, u, vv)
    assert st == 0 and got[1].tolist() == [1, 1, 1]
    _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))
    p[0, 1] = 0
    *got, st = _run(kvc, p, q, tokens, parents, u, vv)
    assert st == kvc.DEV_NONFINITE and got[2][1] == -1
    _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))


def test_absent_trees_bad_nodes_and_bad_probabilities(kvc):
    p, q, tokens, parents, u, vv = _case(7, 6, 600, 61)
    parents[:, 1] = -2                      # no tree
    parents[3:, 2] = -2                     # fewer nodes
    tokens[2, 3], tokens[4, 3] = -1, 600    # tokens outside the vocabulary
    parents[5, 4], parents[6, 4] = 5, 99    # no parent below the node
    p[:, 5, 17] = float("nan")
    p[:, 5, 18] = float("inf")
    p[:, 5, 19] = -1
    q[:, 5, 20] = float("nan")
    *got, st = _run(kvc, p, q, tokens, parents, u, vv)
    assert st & kvc.DEV_BAD_INDEX
    _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))
    assert got[1][1] == 0 and got[2][1] == -1 and (got[0][1] == -1).all()


def test_padded_rows_and_misaligned_rows(kvc):
    """Rows inside a wider, padded matrix, on every alignment of their start."""
    p0, q0, tokens, parents, u, vv = _case(4, 3, 1999, 71)
    want = plain64.verify(_np(p0), _np(q0), tokens, parents, u, vv)
    for lead, pad in ((0, 1), (1, 2), (3, 0), (4, 1), (8, 5)):
        wide = torch.full((2, 12 * (1999 + pad) + lead + 8), float("nan"), device="cuda")
        rows = []
        for x, w in ((p0, wide[0]), (q0, wide[1])):
            view = w[lead:lead + 12 * (1999 + pad)].view(4, 3, 1999 + pad)[..., :1999]
            view.copy_(x)
            rows.append(view)
        *got, st = _run(kvc, *rows, tokens, parents, u, vv)
        assert st == 0
        _same(got, want)


def test_distribution(kvc):
    """Over many independent sequences the token behind the root (the first
    accepted child's, or the next token) is distributed as the target's row:
    each of 12 counts within 5 standard deviations of its expectation."""
    n, v, t = 40_000, 12, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    row = torch.rand(v, generator=g, device="cuda") ** 2
    row /= row.sum()
    drf = torch.rand(v, generator=g, device="cuda") ** 2
    drf /= drf.sum()
    p = row.expand(t, n, v).contiguous()
    q = drf.expand(t, n, v).contiguous()
    parents = torch.zeros(t, n, dtype=torch.int32, device="cuda")
    parents[0] = -1
    tokens = torch.multinomial(drf, t * n, replacement=True, generator=g).view(t, n).int()
    u = torch.rand(t, n, generator=g, device="cuda")
    vv = torch.rand(n, generator=g, device="cuda")
    path = torch.empty(n, t, dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    kvc.verify_tree(p, q, tokens, parents, u, vv, path, n_path, nxt)
    second = path[:, 1].long()
    first = torch.where(second > 0, tokens[second.clamp_min(0), torch.arange(n, device="cuda")], nxt)
    count = torch.bincount(first.long(), minlength=v).double()
    sd = (n * row.double() * (1 - row.double())).sqrt()
    assert torch.all((count - n * row.double()).abs() <= 5 * sd)
    assert 0.2 < (n_path > 1).double().mean() < 1


def test_stream_graph_and_repeats(kvc):
    """On another stream, captured and replayed with new inputs in place; the
    same call twice gives the same bits."""
    p, q, tokens, parents, u, vv = _case(5, 8, 9000, 81)
    want = plain64.verify(_np(p), _np(q), tokens, parents, u, vv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            *got, _ = _run(kvc, p, q, tokens, parents, u, vv)
            _same(got, want)
    dev = [torch.as_tensor(x).cuda() for x in (tokens, parents, u, vv)]
    outs = [torch.empty(sh, dtype=torch.int32, device="cuda") for sh in ((8, 5), (8,), (8,))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.verify_tree(p, q, *dev, *outs)
    p2, q2, tokens2, parents2, u2, v2 = _case(5, 8, 9000, 82)
    for a, b in zip((p, q, *dev), (p2, q2, tokens2, parents2, u2, v2)):
        a.copy_(torch.as_tensor(b))
    graph.replay()
    torch.cuda.synchronize()
    _same([o.cpu().numpy() for o in outs],
          plain64.verify(_np(p2), _np(q2), tokens2, parents2, u2, v2))


def test_refused_calls(kvc):
    p, q, tokens, parents, u, vv = _case(3, 2, 64, 91)
    args = [torch.as_tensor(x).cuda() for x in (tokens, parents, u, vv)]
    outs = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((2, 3), (2,), (2,))]
    with pytest.raises(ValueError):
        kvc.verify_tree(p, q.bfloat16(), *args, *outs)
    with pytest.raises(ValueError):
        kvc.verify_tree(p.half(), None, *args, *outs)
    with pytest.raises(ValueError):
        kvc.verify_tree(p.transpose(0, 1), None, *args, *outs)
    with pytest.raises(ValueError):
        kvc.verify_tree(p, q, args[0].long(), *args[1:], *outs)


@pytest.mark.parametrize("t,b,v,dtype", [(2, 160, 140_000, torch.bfloat16),
                                         (3, 1, 1_200_003, torch.float32),
                                         (2, 1, 4_194_304, torch.float32)])
def test_largest_vocabularies(kvc, t, b, v, dtype):
    """Shares of a vocabulary in blocks of more than 128 entries."""
    p, q, tokens, parents, u, vv = _case(t, b, v, 101, dtype, star=True, noise=2.0)
    u = np.maximum(u, np.float32(0.8))
    *got, st = _run(kvc, p, q, tokens, parents, u, vv)
    assert st == 0
    _same(got, plain64.verify(_np(p), _np(q), tokens, parents, u, vv))


def test_small_probabilities(kvc):
    """Rows of subnormal fp32 numbers, and of single tokens next to them."""
    v = 3000
    g = torch.Generator(device="cuda").manual_seed(111)
    p = torch.rand(1, 4, v, generator=g, device="cuda") * 1e-40
    p[0, 1, 2999] = 1e-30
    p[0, 2] = 0
    p[0, 2, 1234] = 1.4e-45
    vv = np.array([0.5, 0.5, 0.999, 0.0], np.float32)
    z = np.zeros((1, 4), np.int32)
    *got, st = _run(kvc, p, None, z, z - 1, np.zeros((1, 4), np.float32), vv)
    assert st == 0
    _same(got, plain64.verify(_np(p), None, z, z - 1, np.zeros((1, 4), np.float32), vv))
