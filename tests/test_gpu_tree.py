"""kvc_tree_decode_attn against the formula in 64 bits, node by node
(plain64.tree_attention).

Tolerances, per output channel, from the roundings alone:
 logits   fp32 sums of D products, with d = 2^-24 (D / 8 + 16) max sum |q k|
          sm_scale (SIMT: D / 32 terms a lane and 5 shuffles; tensor cores: a
          bound of one rounding for every 8 products), and 2^-22 |x| for the
          exponential's argument and result;
 weights  2 (d + 2^-22 |x|) relative, and their sums N 2^-24;
 tensor cores: weights rounded to f16 over entries (2^-11) and to bf16 over
          raw keys (2^-8; half a step of each).  An f16 weight below 2^-14 is
          a multiple of 2^-24, so it is off by up to 2^-25 however small it
          is: entry k adds up to 2^-25 |v_k|, whatever its weight.  The
          largest weight is at least 2^7 (a reference lies 7 below the largest
          logit of the chunk that set it, and later chunks only add), so the
          sum of weights that divides the output is too: 2^-32 sum |v_k|
          (sum over the entries, not weighted: where the heaviest entry holds
          a zero, the output is made of such weights alone);
 output   half a step of its type: bf16 2^-8, fp32 2^-24.
The log-sum-exp carries the logits' error, N 2^-24 and 2^-22 of its own."""
import numpy as np
import pytest
import torch

import plain64
from helpers import Guarded

pytestmark = pytest.mark.gpu

MLA = dict(latent=512, rope=64, heads=64, group=32, scale_f32=False, act="bf16", topk=512,
           window=128)
TINY = dict(latent=64, rope=16, heads=8, group=32, scale_f32=True, act="f32", topk=64, window=32)


class Case:
    """Inputs of one call, on the GPU, and its expected result."""

    def __init__(self, kvc, nodes, batch, entries, seed=0, shared=False, window_len=None,
                 lens=None, parents=None, lengths=None, spread=1.0, **kw):
        c = dict(MLA, **kw)
        self.c, self.kvc = c, kvc
        self.T, self.B, self.cap = nodes, batch, entries
        latent, rope, h, K, W = (c[x] for x in ("latent", "rope", "heads", "topk", "window"))
        d = latent + rope
        self.sm = float(np.float32(1 / np.sqrt(d)))
        self.dt = torch.float32 if c["act"] == "f32" else torch.bfloat16
        self.cfg = kvc.make_config(latent, rope, c["group"],
                                   kvc.SCALE_F32 if c["scale_f32"] else kvc.SCALE_UE4M3, 128, K, W,
                                   h, self.sm, kvc.F32 if c["act"] == "f32" else kvc.BF16)
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rb = kvc.record_bytes(self.cfg)
        self.rec = rng.integers(0, 256, (batch, entries, rb), dtype=np.uint8)
        n = int(plain64.groups(latent, rope, c["group"])[-1]) + 1
        if c["scale_f32"]:
            sc = (0.2 + 0.3 * rng.random((batch, entries, n))).astype(np.float32)
            self.rec[..., d // 2:d // 2 + 4 * n] = sc.view(np.uint8).reshape(batch, entries, -1)
        else:  # scales from 2^-3 to 1.875 * 2^-2
            self.rec[..., d // 2:d // 2 + n] = rng.integers(0x20, 0x30, (batch, entries, n))
        self.n = np.full(batch, entries, np.int32) if lengths is None else np.array(lengths, np.int32)
        sel = np.full((1 if shared else nodes, batch, K), -1, np.int32)
        for t in range(sel.shape[0]):
            for b in range(batch):
                live = int(np.clip(self.n[b], 0, entries))
                pick = np.sort(rng.choice(live, min(K, live), replace=False)) if live else []
                sel[t, b, :len(pick)] = pick
        self.topk = sel[0] if shared else sel
        dev = lambda *s: (spread * torch.randn(*s, generator=g, device="cuda")).to(self.dt)  # noqa: E731
        self.q, self.win, self.draft = dev(nodes, batch, h, d), dev(batch, W, d), dev(nodes, batch, d)
        self.wl = W if window_len is None else window_len
        self.lens = lens
        if parents is None:
            parents = np.stack([np.maximum(-1, i - 1 - rng.integers(0, 3, batch))
                                for i in range(nodes)])
        self.parents = np.array(parents, np.int32).reshape(nodes, batch)

    def call(self, stream=None, want_lse=True):
        kvc, c = self.kvc, self.c
        cache = kvc.Cache(self.cfg, self.B, self.cap)
        cache.records.copy_(torch.from_numpy(self.rec))
        cache.n_entries.copy_(torch.from_numpy(self.n))
        self.out = Guarded((self.T, self.B, c["heads"], c["latent"]), self.dt, fill=float("nan"))
        self.lse = Guarded((self.T, self.B, c["heads"]), torch.float32, fill=float("nan"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        lens = None if self.lens is None else torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.args = (self.cfg, self.q, cache, torch.from_numpy(self.topk).cuda(), self.win, self.wl,
                     self.draft, torch.from_numpy(self.parents).cuda(), self.out.t)
        self.kw = dict(lse=self.lse.t if want_lse else None, window_lens=lens, status=st)
        kvc.tree_decode_attn(*self.args, **self.kw, stream=stream)
        self.out.check()
        self.lse.check()
        return int(st.item())

    def expect(self, win=None, draft=None):
        c = self.c
        lens = [self.wl] * self.B if self.lens is None else \
            [x if 0 <= x <= self.wl else 0 for x in self.lens]
        f = lambda x: x.double().cpu().numpy()  # noqa: E731
        return plain64.tree_attention(
            f(self.q), self.rec, self.n, self.cap, self.topk, f(self.win if win is None else win),
            lens, f(self.draft if draft is None else draft), self.parents,
            (c["latent"], c["rope"], c["group"], self.sm), c["scale_f32"])

    def check(self, want=None):
        c = self.c
        out, lse, rec_abs, raw_abs, dots, count, rec_sum = want or self.expect()
        d = c["latent"] + c["rope"]
        logit = 2.0 ** -24 * (d / 8 + 16) * dots + 2.0 ** -22 * dots
        got, got_lse = self.out.t.double().cpu().numpy(), self.lse.t.double().cpu().numpy()
        every = rec_abs + raw_abs
        n = count[..., None, None]
        tol = every * (2 * logit[..., None] + n * 2.0 ** -23)
        if c["act"] == "bf16":
            tol = tol + 2.0 ** -11 * rec_abs + 2.0 ** -8 * raw_abs + 2.0 ** -8 * np.abs(out) \
                + 2.0 ** -32 * rec_sum
        else:
            tol = tol + 2.0 ** -24 * np.abs(out)
        over = np.abs(got - out) - tol
        assert np.all(over <= 0), (f"{(over > 0).sum()} values over the bound, the worst by "
                                   f"{over.max():.3e} at {np.unravel_index(over.argmax(), over.shape)}")
        none = count == 0
        assert not got[none].any() and np.all(got_lse[none] == -np.inf)
        ok = ~none
        lse_tol = logit[ok] + 2.0 ** -22 * (4 + np.abs(lse[ok])) + count[ok][:, None] * 2.0 ** -24
        assert np.all(np.abs(got_lse[ok] - lse[ok]) <= lse_tol)


@pytest.mark.parametrize("shape", [MLA, TINY])
def test_ordinary_trees(kvc, shape):
    """One node to many, one sequence to several, per-node and shared
    selections."""
    for nodes, batch, entries, shared in ((1, 1, 600, False), (4, 1, 700, False), (8, 3, 900, False),
                                          (5, 2, 520, True), (21, 1, 530, True)):
        x = Case(kvc, nodes, batch, entries, seed=nodes, shared=shared, **shape)
        assert x.call() == 0
        x.check()


@pytest.mark.parametrize("heads,group,act,scale_f32", [
    (64, 8, "bf16", False), (64, 16, "bf16", False), (64, 64, "bf16", False),
    (64, 128, "bf16", False), (16, 32, "bf16", False), (32, 64, "bf16", False),
    (128, 32, "bf16", False), (48, 32, "bf16", False), (3, 32, "bf16", False),
    (64, 256, "bf16", False), (64, 32, "bf16", True), (64, 32, "f32", False)])
def test_heads_groups_and_types(kvc, heads, group, act, scale_f32):
    """Head counts in one group, several and none of 16; every group size;
    shapes that run on either path."""
    x = Case(kvc, 3, 2, 560, seed=heads + group, heads=heads, group=group, act=act,
             scale_f32=scale_f32)
    assert x.call() == 0
    x.check()


@pytest.mark.parametrize("topk", [1, 63, 128, 129, 1000, 2048])
def test_selections(kvc, topk):
    x = Case(kvc, 3, 2, 2300, seed=topk, topk=topk)
    x.topk[1, 0, topk // 2:] = -1     # padding behind, and holes
    x.topk[2, 1, ::3] = -1
    assert x.call() == 0
    x.check()


@pytest.mark.parametrize("window,window_len", [(128, 128), (128, 0), (128, 1), (128, 100), (1, 1),
                                               (7, 7), (200, 199), (300, 300), (0, 0)])
def test_windows(kvc, window, window_len):
    """Windows of none, one, a chunk, and several chunks; with W = 0 a node
    sees its entries alone."""
    x = Case(kvc, 5, 2, 300, seed=window + window_len, window=window, window_len=window_len,
             topk=130)
    assert x.call() == 0
    x.check()


@pytest.mark.parametrize("window,nodes", [(128, 150), (16, 40), (3, 9)])
def test_paths_longer_than_the_window(kvc, window, nodes):
    """A chain of drafted tokens longer than the window: the oldest of its own
    ancestors fall out, and no window row is left."""
    parents = np.arange(-1, nodes - 1)[:, None].repeat(2, 1)
    x = Case(kvc, nodes, 2, 200, seed=nodes, window=window, topk=64, parents=parents)
    assert x.call() == 0
    x.check()


def test_ragged_batch(kvc):
    """Lengths from none to all, in the entries, the windows and the nodes; a
    sequence with nothing at all; window lengths out of range."""
    parents = np.array([[-1, -1, -1, -2, -1], [0, 0, -2, -2, -1], [1, 0, -2, -2, 0],
                        [1, 2, -2, -2, 2]])
    for shape in (MLA, TINY):
        x = Case(kvc, 4, 5, 150, seed=5, parents=parents, lengths=[150, 3, 0, 77, 1],
                 lens=[32, 0, 0, 5, 17], window_len=32, **shape)
        assert x.call() == 0
        x.check()
        x = Case(kvc, 4, 5, 150, seed=6, parents=parents, lengths=[150, 151, -1, 77, 1],
                 lens=[33, 4, -1, 5, 17], window_len=32, **shape)
        assert x.call() == kvc.DEV_BAD_LENGTH
        x.n[[1, 2]] = 0
        x.check()


def test_bad_indices_and_parents(kvc):
    """Indices outside the entries are skipped, nodes without a parent below
    them (and everything under those) are absent; both are flagged."""
    for shape in (MLA, TINY):
        x = Case(kvc, 6, 2, 90, seed=8, **shape)
        x.topk[0, 0, :4] = [90, -5, 2 ** 31 - 1, -2 ** 31]
        assert x.call() == kvc.DEV_BAD_INDEX
        x.check()
        parents = np.array([-1, 0, 2, 7, 2, 3])[:, None].repeat(2, 1)
        x = Case(kvc, 6, 2, 90, seed=9, parents=parents, **shape)
        assert x.call() == kvc.DEV_BAD_INDEX
        x.check()
        assert np.all(x.lse.t.cpu().numpy()[2:] == -np.inf)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.3e38])
def test_rows_that_no_node_sees(kvc, bad):
    """Values in window rows past the length, in rows older than the window
    and in other branches' drafts do not reach a node."""
    for shape in (MLA, TINY):
        parents = np.array([-1, 0, 0, 1])[:, None]
        x = Case(kvc, 4, 1, 200, seed=12, parents=parents, window_len=shape["window"], **shape)
        want = x.expect()
        x.lens = [20]
        want = x.expect()
        x.win[0, 20:] = bad
        x.draft[2] = bad                      # node 2's own row and no other's
        assert x.call() == 0 or shape is TINY
        got = x.out.t.clone()
        # nodes 0, 1 and 3 do not have node 2 on their path
        keep = [0, 1, 3]
        x.out.t[2] = torch.from_numpy(want[0][2]).to(x.dt).cuda()
        x.lse.t[2] = torch.from_numpy(want[1][2]).float().cuda()
        x.check(want)
        assert torch.isfinite(got[keep].float()).all()


def test_large_and_small_logits(kvc):
    """Logits that jump by far more than the rescale slack between chunks (raw
    keys along the queries first, then entries; and the other way round), and
    queries of extreme size."""
    x = Case(kvc, 4, 2, 700, seed=21)
    x.win[:, :64] = (x.q[0, :, :1].float() * 3).to(x.dt)
    assert x.call() == 0
    x.check()
    x = Case(kvc, 4, 2, 700, seed=22)
    x.rec[:, :, 288:306] += 0x10            # entries four times larger
    x.q *= 4
    assert x.call() == 0
    x.check()
    for scale in (1e-20, 1e-3, 1e15):
        x = Case(kvc, 2, 1, 300, seed=23)
        x.q = (x.q.float() * scale).to(x.dt)
        if scale > 1:                       # one key takes all the weight, by a wide margin
            x.sm = float(np.float32(1e-15 / 24))
            x.cfg.sm_scale = x.sm
        assert x.call() == 0
        x.check()


def test_equal_keys(kvc):
    """All weights equal: many identical entries and window rows."""
    x = Case(kvc, 3, 2, 600, seed=24)
    x.rec[:] = x.rec[:, :1]
    x.win[:] = x.win[:, :1]
    assert x.call() == 0
    x.check()


def test_chain_equals_single_token_calls(kvc):
    """A drafted chain gives what kvc_sparse_decode_attn gives token after
    token, each with its own window: the two agree within their tolerances
    (2e-3 of a row's norm, and half a bf16 step)."""
    T, B = 5, 2
    parents = np.arange(-1, T - 1)[:, None].repeat(B, 1)
    x = Case(kvc, T, B, 800, seed=31, parents=parents)
    assert x.call() == 0
    cfg, q, cache, topk, win, wl, draft, _, out = x.args
    ws = kvc.workspace(cfg, B, x.cap)
    rows = win
    for t in range(T):
        rows = torch.cat([rows[:, 1:], draft[t][:, None]], 1).contiguous()
        one = torch.empty(B, 64, 512, device="cuda")
        lse = torch.empty(B, 64, device="cuda")
        kvc.sparse_decode_attn(cfg, q[t], cache, topk[t], rows, wl, one, ws, lse=lse)
        err = (one - out[t].float()).abs().amax(-1)
        tol = 2e-3 * one.norm(dim=-1) + 2.0 ** -8 * one.abs().amax(-1)
        assert torch.all(err <= 2 * tol)
        assert torch.all((lse - x.lse.t[t]).abs() <= 2e-3 * lse.abs().clamp_min(1))


def test_many_nodes(kvc):
    """More nodes than fit on the device at once; every node checked against
    a smaller call's bits and some against the formula."""
    x = Case(kvc, 16, 24, 300, seed=41, topk=128)
    assert x.call() == 0
    x.check()


def test_stream_graph_and_repeats(kvc):
    """On another stream, twice for the same bits, and captured and replayed
    with new inputs in place."""
    x = Case(kvc, 6, 3, 400, seed=51)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert x.call() == 0
        first = x.out.t.clone()
        assert x.call() == 0
        assert torch.equal(first, x.out.t)
    torch.cuda.synchronize()
    x.check()
    y = Case(kvc, 6, 3, 400, seed=52)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.tree_decode_attn(*x.args, **x.kw)
    x.args[1].copy_(y.q)
    x.args[2].records.copy_(torch.from_numpy(y.rec))
    x.args[3].copy_(torch.from_numpy(y.topk))
    x.args[4].copy_(y.win)
    x.args[6].copy_(y.draft)
    x.args[7].copy_(torch.from_numpy(y.parents))
    graph.replay()
    torch.cuda.synchronize()
    y.out, y.lse = x.out, x.lse
    y.check()


def test_two_calls_at_once(kvc):
    """Calls on two streams at the same time share nothing."""
    xs = [Case(kvc, 8, 4, 600, seed=61 + i) for i in range(2)]
    for x in xs:
        assert x.call() == 0
    want = [x.out.t.clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s in zip(xs, streams):
            kvc.tree_decode_attn(*x.args, **x.kw, stream=s)
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        assert torch.equal(x.out.t, w)


def test_no_lse_and_no_nodes(kvc):
    x = Case(kvc, 2, 1, 200, seed=71)
    assert x.call() == 0
    want = x.out.t.clone()
    assert x.call(want_lse=False) == 0
    assert torch.equal(x.out.t, want) and torch.isnan(x.lse.t).all()


def test_refused_calls(kvc):
    x = Case(kvc, 2, 1, 50, seed=72)
    x.call()
    bad = list(x.args)
    bad[5] = 129
    with pytest.raises(kvc.KvcError):
        kvc.tree_decode_attn(*bad, **x.kw)
    for at, t in ((1, x.q.float()), (3, x.args[3].long()), (4, x.win[:, :64].contiguous()),
                  (7, x.args[7].cpu()), (8, x.out.t.float())):
        bad = list(x.args)
        bad[at] = t
        with pytest.raises(ValueError):
            kvc.tree_decode_attn(*bad, **x.kw)


@pytest.mark.parametrize("nodes,batch", [(5, 1), (4, 4), (4, 8), (6, 8), (7, 15), (16, 11)])
def test_splits_of_a_node(kvc, nodes, batch):
    """Node counts for which a node's keys go to several CTAs or one, its heads
    to one group or several, and a CTA takes one node or more."""
    x = Case(kvc, nodes, batch, 700, seed=80 + nodes * batch)
    assert x.call() == 0
    x.check()


@pytest.mark.parametrize("rising", [True, False])
def test_references_that_move(kvc, rising):
    """One CTA goes through all chunks of a node (more nodes than
    multiprocessors) while the logits grow from chunk to chunk by far more than
    a weight can, or shrink: sums and outputs so far are rescaled, again and
    again."""
    x = Case(kvc, 13, 12, 1024, seed=91)
    step = np.arange(1024) * 5 // 1024  # entries from 1 to 16 times the first ones
    scale = x.rec[:, :, 288:306]
    scale += (8 * (step if rising else 4 - step)).astype(np.uint8)[None, :, None]
    x.win *= 0.05
    x.draft *= 0.05
    x.q *= 8
    assert x.call() == 0
    x.check()


def test_chunks_without_a_key(kvc):
    """No window, and selections whose first chunks hold nothing: a head's
    first key comes late, or never."""
    for nodes, batch in ((3, 2), (13, 12)):
        x = Case(kvc, nodes, batch, 700, seed=93, window=0, window_len=0)
        x.topk[:, :, :300] = -1
        x.topk[1, 0] = -1
        assert x.call() == 0
        x.check()
        assert not x.out.t[1, 0].any()


def test_more_nodes_than_multiprocessors(kvc):
    """Ragged trees, lengths and windows, shared selections, several head
    groups; a CTA takes node after node, absent ones among them."""
    rng = np.random.default_rng(95)
    for heads, shared in ((64, True), (48, False)):
        parents = np.stack([np.maximum(-1, i - 1 - rng.integers(0, 4, 30)) for i in range(12)])
        parents[np.arange(12)[:, None] >= rng.integers(0, 13, 30)] = -2
        x = Case(kvc, 12, 30, 300, seed=96, shared=shared, heads=heads, topk=200, parents=parents,
                 lengths=rng.integers(0, 301, 30), lens=list(rng.integers(0, 129, 30)))
        assert x.call() == 0
        x.check()


def test_far_entries(kvc):
    """Records past 4 GB of a sequence."""
    x = Case(kvc, 3, 1, 600, seed=97)
    cap, at = 14_000_000, 13_999_400
    assert x.call() == 0
    want = x.out.t.clone()
    rb = x.rec.shape[-1]
    records = torch.empty(1, cap, rb, dtype=torch.uint8, device="cuda")
    records[:, at:].copy_(torch.from_numpy(x.rec))
    idx_k = torch.empty(1, cap, 128, dtype=torch.int8, device="cuda")
    cache = kvc.Cache.wrap(x.cfg, records, idx_k, torch.full((1,), cap, dtype=torch.int32,
                                                            device="cuda"))
    args = list(x.args)
    args[2], args[3] = cache, args[3] + at
    kvc.tree_decode_attn(*args, **x.kw)
    assert torch.equal(x.out.t, want) and x.kw["status"].item() == 0


def test_zero_wait_limit(kvc):
    """Every wait gives up at once: the call returns, the status says so, the
    next call is right."""
    for nodes, batch in ((4, 1), (16, 11)):
        x = Case(kvc, nodes, batch, 600, seed=98)
        kvc.debug_set_wait_limit_ns(0)
        try:
            assert x.call() & kvc.DEV_TIMEOUT
        finally:
            kvc.debug_set_wait_limit_ns(2_000_000_000)
        assert x.call() == 0
        x.check()


@pytest.mark.parametrize("shape", [MLA, TINY])
def test_most_nodes(kvc, shape):
    """256 nodes: a chain, siblings under it, and none."""
    parents = np.arange(-1, 255)[:, None]
    parents[200:240] = 150
    parents[250:] = -2
    x = Case(kvc, 256, 1, 100, seed=101, topk=64, parents=parents,
             **{k: v for k, v in shape.items() if k != "topk"})
    assert x.call() == 0
    x.check()


def test_most_heads_and_a_repeated_selection(kvc):
    """256 heads in four groups; an entry selected twice counts twice."""
    x = Case(kvc, 3, 2, 90, seed=103, heads=256, topk=48)
    x.topk[0, 0, 1:20] = x.topk[0, 0, 0]
    assert x.call() == 0
    x.check()


def test_long_windows(kvc):
    """A window of eight chunks."""
    x = Case(kvc, 4, 2, 60, seed=105, window=1000, window_len=1000, topk=32, lens=[1000, 333])
    assert x.call() == 0
    x.check()
