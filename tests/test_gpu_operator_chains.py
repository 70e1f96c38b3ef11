"""Calls that follow one another on a stream with nothing between them, each
on the rows that the one before has just written: kvc_norm_rope or kvc_unpack,
then kvc_pack or an attention.  The results must be, bit for bit, those of the
same calls with a synchronisation after each; eager, and captured once and
replayed with other rows in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# batch, new tokens a sequence, tokens an entry, row type, indexer keys' format
APPENDS = [(64, 2, 2, "bf16", 0), (1, 2, 2, "f32", 0), (16, 512, 2, "bf16", 0),
           (5, 34, 2, "f32", 0), (64, 4, 4, "bf16", 0), (9, 36, 4, "f32", 0),
           (16, 8, 2, "bf16", 1), (2, 6000, 2, "bf16", 0)]


class Chain:
    """Raw rows, and the calls that turn them into records of two caches."""

    def __init__(self, kvc, batch, n_new, ratio, act, idx_fmt):
        self.kvc, self.dt = kvc, torch.float32 if act == "f32" else torch.bfloat16
        self.cfg = kvc.make_config(512, 64, 32, kvc.SCALE_UE4M3, 128, 512, 128, 64, 1 / 24,
                                   kvc.F32 if act == "f32" else kvc.BF16, ratio, idx_fmt)
        g = torch.Generator(device="cuda").manual_seed(batch + n_new)
        self.g, self.n = g, batch * n_new
        per = n_new // ratio
        self.raw = torch.empty(self.n, 576, dtype=self.dt, device="cuda")
        self.rows = torch.zeros(batch, n_new, 576, dtype=self.dt, device="cuda")
        self.pos = torch.arange(self.n, dtype=torch.int32, device="cuda")
        self.freq = (10_000.0 ** (-torch.arange(32, device="cuda") / 32.0)).float()
        self.gate = 0.1 * torch.randn(2, 576, generator=g, device="cuda")
        self.keys = torch.randint(-127, 128, (batch, per, 128), generator=g, device="cuda")
        self.keys = self.keys.to(self.dt if idx_fmt else torch.int8)
        self.caches = [kvc.Cache(self.cfg, batch, 2 * per) for _ in range(2)]
        self.fresh()

    def fresh(self):
        self.raw.copy_(torch.randn(self.n, 576, generator=self.g, device="cuda"))

    def clear(self):
        self.rows.zero_()
        for c in self.caches:
            c.records.zero_()
            c.idx_k.zero_()
            c.n_entries.zero_()
        torch.cuda.synchronize()

    def calls(self, between=lambda: None):
        """norm_rope, one pack behind it and another behind that one."""
        kvc, cfg = self.kvc, self.cfg
        kvc.norm_rope(cfg, None, self.raw, self.pos, self.freq, None,
                      self.rows.view(self.n, 576))
        between()
        for c in self.caches:
            kvc.pack(cfg, self.rows, self.gate, self.keys, c)
            between()

    def result(self):
        torch.cuda.synchronize()
        return [x.clone() for c in self.caches for x in (c.records, c.idx_k, c.n_entries)]


@pytest.mark.parametrize("append", APPENDS)
def test_norm_rope_then_pack(kvc, append):
    x = Chain(kvc, *append)
    graph = torch.cuda.CUDAGraph()
    x.calls(torch.cuda.synchronize)
    with torch.cuda.graph(graph):
        x.calls()
    for _ in range(6):
        x.fresh()
        x.clear()
        x.calls(torch.cuda.synchronize)
        want = x.result()
        assert want[0].any() and (want[2] > 0).all()
        for run in (x.calls, graph.replay):
            x.clear()
            run()
            assert all(torch.equal(a, b) for a, b in zip(x.result(), want))


@pytest.mark.parametrize("append", [APPENDS[0], APPENDS[2], APPENDS[4]])
def test_unpack_then_pack(kvc, append):
    """Entries read back as rows and packed again at once."""
    x = Chain(kvc, *append)
    batch, n_new = append[:2]
    src = kvc.Cache(x.cfg, batch, n_new)
    src.n_entries.fill_(n_new)
    rec = src.records.view(-1, src.records.shape[-1])

    def calls(between=lambda: None):
        kvc.unpack(x.cfg, src, x.rows)
        between()
        kvc.pack(x.cfg, x.rows, x.gate, x.keys, x.caches[0])
        between()

    for seed in range(6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rec[:, :288] = torch.randint(0, 256, (rec.shape[0], 288), generator=g, device="cuda",
                                     dtype=torch.uint8)
        rec[:, 288:306] = torch.randint(0x20, 0x30, (rec.shape[0], 18), generator=g, device="cuda",
                                        dtype=torch.uint8)
        x.clear()
        calls(torch.cuda.synchronize)
        want = x.result()
        assert want[0].any()
        x.clear()
        calls()
        assert all(torch.equal(a, b) for a, b in zip(x.result(), want))


@pytest.mark.parametrize("batch,layers", [(1, 2), (8, 4), (32, 2)])
def test_norm_rope_then_attention(kvc, batch, layers):
    """Queries and window rows of norm_rope taken at once by the attention of a
    tree, of single tokens and of a layer group, whose layers ask for their
    queries early."""
    cap, k, w = 700, 128, 32
    cfg = kvc.make_config(512, 64, 32, kvc.SCALE_UE4M3, 128, k, w, 64, 1 / 24, kvc.BF16)
    g = torch.Generator(device="cuda").manual_seed(batch)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    cache = kvc.Cache(cfg, batch, cap)
    cache.records[..., :288] = torch.randint(0, 256, (batch, cap, 288), generator=g, device="cuda",
                                             dtype=torch.uint8)
    cache.records[..., 288:306] = torch.randint(0x20, 0x30, (batch, cap, 18), generator=g,
                                                device="cuda", dtype=torch.uint8)
    cache.idx_k.copy_(torch.randint(-127, 128, cache.idx_k.shape, generator=g, device="cuda"))
    cache.n_entries.fill_(cap)
    n = layers * batch
    raw_q, raw_w = randn(n, 64, 576), randn(n * w, 576)
    q, win = torch.empty(layers, batch, 64, 576, device="cuda").bfloat16(), \
        torch.empty(layers, batch, w, 576, device="cuda").bfloat16()
    pos, wpos = (torch.arange(m, dtype=torch.int32, device="cuda") for m in (n, n * w))
    freq = (10_000.0 ** (-torch.arange(32, device="cuda") / 32.0)).float()
    iq = torch.randint(-127, 128, (layers, batch, 128), generator=g, device="cuda").to(torch.int8)
    topk = torch.empty(layers, batch, k, dtype=torch.int32, device="cuda")
    sel = torch.arange(k, dtype=torch.int32, device="cuda").expand(layers, batch, k).contiguous()
    par = torch.arange(-1, layers - 1, dtype=torch.int32, device="cuda")[:, None].repeat(1, batch)
    ws = kvc.workspace(cfg, batch, cap)
    out = torch.empty(layers, batch, 64, 512, device="cuda")
    tree = torch.empty(layers, batch, 64, 512, device="cuda").bfloat16()
    modes = [kvc.FULL] + [kvc.REUSE] * (layers - 1)

    def rows(between):
        kvc.norm_rope(cfg, None, raw_w, wpos, freq, None, win.view(-1, 576))
        between()
        kvc.norm_rope(cfg, raw_q, None, pos, freq, q.view(-1, 64, 576), None)
        between()

    def group(between=lambda: None):
        rows(between)
        kvc.layer_group_step(cfg, modes, q, iq, win, w, cache, out, topk, ws)

    def single(between=lambda: None):
        rows(between)
        kvc.sparse_decode_attn(cfg, q[0], cache, sel[0], win[0], w, out[0], ws)

    def drafted(between=lambda: None):
        rows(between)
        kvc.tree_decode_attn(cfg, q, cache, sel, win[0], w, draft, par, tree)

    draft = randn(layers, batch, 576)
    for run, res in ((group, out), (single, out), (drafted, tree)):
        graph = torch.cuda.CUDAGraph()
        run(torch.cuda.synchronize)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run()
        for _ in range(6):
            raw_q.copy_(randn(n, 64, 576))
            raw_w.copy_(randn(n * w, 576))
            q.zero_()
            win.zero_()
            res.zero_()
            torch.cuda.synchronize()
            run(torch.cuda.synchronize)
            torch.cuda.synchronize()
            want = res.clone()
            assert torch.isfinite(want).all() and want.any()
            for again in (run, graph.replay):
                q.zero_()
                win.zero_()
                res.zero_()
                torch.cuda.synchronize()
                again()
                torch.cuda.synchronize()
                assert torch.equal(res, want)
