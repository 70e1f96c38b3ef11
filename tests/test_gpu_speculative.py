"""One speculative decode step, the operators in the order of their use: raw
rows from norm_rope packed and kept in the window, selections of all drafted
tokens from the batched indexer, attention of the tree, verification, and the
accepted rows packed behind the context.  Each operator's result is checked
against the formula on what the one before it left on the device."""
import numpy as np
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu


def test_speculative_step(kvc):
    T, B, H, D, K, W, V = 6, 3, 64, 576, 512, 128, 4000
    sm = float(np.float32(1 / 24))
    cfg = kvc.make_config(512, 64, 32, kvc.SCALE_UE4M3, 128, K, W, H, sm, kvc.BF16)
    g = torch.Generator(device="cuda").manual_seed(7)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    np64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    freq = (10_000.0 ** (-torch.arange(32, device="cuda").double() / 32)).float()
    gain = 1 + 0.1 * randn(512)

    # the context: 1400 tokens a sequence, normalised, rotated, packed; the last 128 are the window
    n_ctx = 1400
    raw = randn(B, n_ctx, D).bfloat16()
    pos = torch.arange(n_ctx, device="cuda", dtype=torch.int32).repeat(B)
    rows = torch.empty_like(raw)
    kvc.norm_rope(cfg, None, raw.view(-1, D), pos, freq, None, rows.view(-1, D), k_gain=gain,
                  status=st)
    cache = kvc.Cache(cfg, B, 1000)
    gate = randn(2, D) * 0.1
    kvc.pack(cfg, rows, gate, torch.randint(-127, 128, (B, n_ctx // 2, 128), generator=g,
                                            device="cuda").to(torch.int8), cache, status=st)
    window = rows[:, -W:].contiguous()

    # the tree's rows and queries
    parents = torch.tensor([[-1] * B, [0] * B, [0] * B, [1] * B, [1, 2, -2], [3, 4, -2]],
                           dtype=torch.int32, device="cuda")
    depth = [0, 1, 1, 2, 2, 3]
    tpos = torch.tensor([n_ctx + d for d in depth], device="cuda", dtype=torch.int32)
    tpos = tpos[:, None].expand(T, B).contiguous().view(-1)
    proj = randn(T * B, (H + 1) * D + 64).bfloat16()  # queries and keys of one projection
    q, draft = torch.empty(T * B, H, D, device="cuda").bfloat16(), torch.empty(T * B, D, device="cuda").bfloat16()
    kvc.norm_rope(cfg, proj[:, :H * D].view(T * B, H, D), proj[:, H * D:(H + 1) * D], tpos, freq, q,
                  draft, k_gain=gain, q_norm=kvc.NORM_ROW, status=st)
    ref, mag = plain64.norm_rope(np64(proj[:, H * D:(H + 1) * D]), gain.cpu().numpy(), 512, 512,
                                 tpos.cpu().numpy(), freq.cpu().numpy(), False, float(np.float32(1e-6)))
    assert np.all(np.abs(np64(draft) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * mag)

    # selections of every node in one pass, then the tree's attention
    topk = torch.empty(T, B, K, dtype=torch.int32, device="cuda")
    iq = torch.randint(-127, 128, (T, B, 128), generator=g, device="cuda").to(torch.int8)
    kvc.index_topk_batched(cfg, iq, cache, topk, kvc.workspace_batched(cfg, T, B, 1000), status=st)
    out, lse = torch.empty(T, B, H, 512, device="cuda").bfloat16(), torch.empty(T, B, H, device="cuda")
    kvc.tree_decode_attn(cfg, q.view(T, B, H, D), cache, topk, window, W, draft.view(T, B, D),
                         parents, out, lse=lse, status=st)
    rec = cache.records.cpu().numpy()
    want, want_lse, rec_abs, raw_abs, dots, count, _ = plain64.tree_attention(
        np64(q.view(T, B, H, D)), rec, cache.n_entries.cpu().numpy(), 1000, topk.cpu().numpy(),
        np64(window), [W] * B, np64(draft.view(T, B, D)), parents.cpu().numpy(),
        (512, 64, 32, sm), False)
    # roundings of weights (entries 2^-11, raw keys 2^-8) and of the output
    # (2^-8); a logit's fp32 error, below 2^-16 of its sum |q k|, twice
    tol = 2.0 ** -11 * rec_abs + 2.0 ** -8 * (raw_abs + np.abs(want)) + \
        2.0 ** -15 * dots[..., None] * (rec_abs + raw_abs) + 1e-9
    assert np.all(np.abs(np64(out) - want) <= tol)
    live = count > 0
    assert np.all(np.abs(np64(lse)[live] - want_lse[live]) <=
                  2.0 ** -15 * (dots[live] + np.abs(want_lse[live])))

    # the selected entries read back are the values the attention saw
    back = torch.empty(B, K, D, device="cuda").bfloat16()
    kvc.unpack(cfg, cache, back, idx=topk[0].contiguous(), status=st)
    idx = topk[0].cpu().numpy()
    for b in range(B):
        assert np.array_equal(np64(back[b]), plain64.record_values(rec[b, idx[b]], 512, 64, 32, False))

    # verification; logits stand in for a model's output layer
    logits = 3 * out[..., 0, :].float() @ randn(512, V)
    p = logits.softmax(-1)
    dq = (logits + 0.5 * randn(T, B, V)).softmax(-1)
    tokens = torch.zeros(T, B, dtype=torch.int32, device="cuda")
    for t in range(1, T):
        up = parents[t].long().clamp_min(0)
        tokens[t] = torch.multinomial(dq[up, torch.arange(B, device="cuda")], 1, generator=g)[:, 0].int()
    u, v = torch.rand(T, B, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    path = torch.empty(B, T, dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    kvc.verify_tree(p, dq, tokens, parents, u, v, path, n_path, nxt, status=st)
    for got, ref in zip((path, n_path, nxt), plain64.verify(
            np64(p), np64(dq), tokens.cpu().numpy(), parents.cpu().numpy(), u.cpu().numpy(),
            v.cpu().numpy())):
        assert np.array_equal(got.cpu().numpy(), ref)

    # two tokens of every path (the root twice where it is alone) join the cache
    second = path[:, 1].clamp_min(0).long()
    pair = torch.stack([draft.view(T, B, D)[0], draft.view(T, B, D)[second, torch.arange(B, device="cuda")]], 1)
    kvc.pack(cfg, pair.contiguous(), gate, torch.zeros(B, 1, 128, dtype=torch.int8, device="cuda"),
             cache, status=st)
    assert cache.n_entries.tolist() == [n_ctx // 2 + 1] * B
    assert torch.equal(cache.records[:, :n_ctx // 2].cpu(), torch.from_numpy(rec[:, :n_ctx // 2]))
    assert st.item() == 0
