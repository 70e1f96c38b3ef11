"""Cases of the operators around one speculative decode step on a compressed
cache, their plain forms in elementary torch operations, and their values in
64 bits.

    norm_rope   norms of queries and keys for each head with the position
                rotation in the same pass: makes the query rows and raw key
                rows that the packing and the attention take
    unpack      reads packed records back as rows of values
    tree        attention of a tree of drafted tokens over the selected
                entries and each node's own sliding window
    verify      the drafted tree against the target's probabilities, from
                given random numbers

With ``own`` false ``run`` computes the plain form and nothing of this
repository's package is imported; with ``own`` true it makes the calls a user
makes.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# the two entry shapes of the repository's workloads: 512 latent + 64 RoPE
# channels shared by 64 heads in bf16, and the small fp32 one
_MLA = {"latent": 512, "rope": 64, "heads": 64, "act": "bf16", "scale_f32": False, "topk": 512,
        "window": 128}
_TINY = {"latent": 64, "rope": 16, "heads": 8, "act": "f32", "scale_f32": True, "topk": 64,
         "window": 32}


def listed():
    return [
        # the rows of one sequence's four drafted tokens, far into a 1M-token context
        {"name": "norm_rope 1x4", "op": "norm_rope", "n": 4, "first": 999_990, "pairs": False,
         "q_norm": "row", "k_norm": "latent", "fused": False, **_MLA},
        # a step's drafted tokens of 32 sequences, rows cut out of one projection's output
        {"name": "norm_rope 32x8", "op": "norm_rope", "n": 256, "first": 131_072, "pairs": False,
         "q_norm": "row", "k_norm": "latent", "fused": True, **_MLA},
        # a chunk of a prompt before it is packed
        {"name": "norm_rope prompt 8192", "op": "norm_rope", "n": 8192, "first": 0, "pairs": True,
         "q_norm": "latent", "k_norm": "latent", "fused": False, **_MLA},
        # a few entries of the small fp32 cache (odd count, padding among the indices)
        {"name": "unpack small f32", "op": "unpack", "batch": 3, "entries": 501, "n": 333,
         "gather": True, "group": 32, **_TINY},
        # the selected entries of 32 sequences, read back for a dense product
        {"name": "unpack 32x512 selected", "op": "unpack", "batch": 32, "entries": 65_536,
         "n": 512, "gather": True, "group": 64, **_MLA},
        # every entry of a 1M-token sequence, read back in order
        {"name": "unpack 1x500000", "op": "unpack", "batch": 1, "entries": 500_000, "n": 500_000,
         "gather": False, "group": 32, **_MLA},
        # one 1M-token sequence, four drafted tokens: latency
        {"name": "tree 1x4 1M", "op": "tree", "batch": 1, "nodes": 4, "entries": 500_000,
         "window_len": 128, "shared": False, "ragged": False, "group": 32, **_MLA},
        # the group of 8 sequences at 256K, six nodes each that share a selection; ragged lengths
        {"name": "tree 8x6 256K shared", "op": "tree", "batch": 8, "nodes": 6, "entries": 131_072,
         "window_len": 125, "shared": True, "ragged": True, "group": 32, **_MLA},
        # the wide batch at 128K, eight nodes each with a selection of its own
        {"name": "tree 32x8 128K", "op": "tree", "batch": 32, "nodes": 8, "entries": 65_536,
         "window_len": 128, "shared": False, "ragged": False, "group": 64, **_MLA},
        # one sequence, a drafted chain of three and an ordinary vocabulary
        {"name": "verify 1x4", "op": "verify", "batch": 1, "nodes": 4, "vocab": 32_000,
         "draft_q": True, "dtype": "f32"},
        # greedy drafts (no draft distribution), odd vocabulary, bf16 probabilities
        {"name": "verify 8x6 greedy odd", "op": "verify", "batch": 8, "nodes": 6,
         "vocab": 100_003, "draft_q": False, "dtype": "bf16"},
        # the wide batch, trees of eight nodes over a large vocabulary
        {"name": "verify 32x8", "op": "verify", "batch": 32, "nodes": 8, "vocab": 131_072,
         "draft_q": True, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "unpack", "tree", "verify"])
    small = rng.random() < 0.25
    shape = dict(_TINY if small else _MLA)
    if op == "norm_rope":
        if not small and rng.random() < 0.4:
            shape.update(latent=rng.choice([128, 256, 384]), rope=rng.choice([8, 32, 48, 128]),
                         heads=rng.choice([1, 6, 16, 40, 128]),
                         act=rng.choice(["f32", "bf16"]))
        wide = shape["latent"] + shape["rope"]
        most = 8192 * 65 * 576 // ((shape["heads"] + 1) * wide) // (2 if shape["act"] == "f32" else 1)
        return {"op": op, "n": _log(rng, 1, min(8192, most)), "first": rng.randrange(0, 1_000_000),
                "pairs": rng.random() < 0.5, "q_norm": rng.choice(["row", "latent", "none"]),
                "k_norm": rng.choice(["row", "latent"]), "fused": rng.random() < 0.5, **shape}
    if op == "unpack":
        batch = _log(rng, 1, 32)
        entries = _log(rng, 40, 400_000 // batch)
        gather = rng.random() < 0.5
        n = _log(rng, 1, min(entries, 2048)) if gather else _log(rng, 1, entries)
        return {"op": op, "batch": batch, "entries": entries, "n": n, "gather": gather,
                "group": 32 if small else rng.choice([16, 32, 64, 128]), **shape}
    if op == "tree":
        batch = _log(rng, 1, 32)
        return {"op": op, "batch": batch, "nodes": _log(rng, 1, min(16, 256 // batch)),
                "entries": _log(rng, 40, 2_000_000 // batch if batch > 8 else 200_000),
                "window_len": rng.randrange(0, shape["window"] + 1),
                "shared": rng.random() < 0.3, "ragged": rng.random() < 0.5,
                "group": 32 if small else rng.choice([16, 32, 64]), **shape}
    batch, nodes = _log(rng, 1, 32), _log(rng, 1, 8)
    return {"op": "verify", "batch": batch, "nodes": nodes, "vocab": _log(rng, 1000, 131_072),
            "draft_q": rng.random() < 0.6, "dtype": rng.choice(["f32", "f32", "bf16"])}


# ------------------------------------------------------------------- inputs
def _n_groups(c):
    return -(-c["latent"] // c["group"]) + -(-c["rope"] // c["group"])


def _record_bytes(c):
    d = c["latent"] + c["rope"]
    return -(-(d // 2 + _n_groups(c) * (4 if c["scale_f32"] else 1)) // 16) * 16


def _rows(gen, c, *shape):
    """Raw key rows: N(0, 1) with six channels of long tails."""
    d = c["latent"] + c["rope"]
    x = torch.randn(*shape, d, generator=gen, device="cuda")
    x[..., 5::max(1, d // 6)] *= 5.0
    return x.to(_DTYPES[c["act"]])


def _quantised(x, c):
    """fp32 rows [n][D] -> records [n][bytes]: E2M1 codes and group scales."""
    n = x.shape[0]
    codes, scales = [], []
    for seg in (x[:, :c["latent"]], x[:, c["latent"]:]):
        for g in seg.split(c["group"], dim=1) if seg.shape[1] % c["group"] else \
                [seg.reshape(n, -1, c["group"])]:
            g = g.reshape(n, -1, g.shape[-1])
            s = g.abs().amax(-1, keepdim=True) / 6
            if not c["scale_f32"]:
                s = s.to(torch.float8_e4m3fn)
            y = g / s.float().clamp_min(1e-30)
            edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
            m = torch.bucketize(y.abs(), edges).to(torch.uint8)
            codes.append((m | ((y < 0).to(torch.uint8) << 3)).reshape(n, -1))
            scales.append(s.reshape(n, -1).contiguous().view(torch.uint8))
    codes = torch.cat(codes, 1)
    rec = torch.zeros(n, _record_bytes(c), dtype=torch.uint8, device=x.device)
    half = codes.shape[1] // 2
    rec[:, :half] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    scales = torch.cat(scales, 1)
    rec[:, half:half + scales.shape[1]] = scales
    return rec


def _records(gen, c):
    rec = torch.empty(c["batch"], c["entries"], _record_bytes(c), dtype=torch.uint8, device="cuda")
    flat = rec.view(-1, rec.shape[-1])
    for i in range(0, flat.shape[0], 65_536):
        part = flat[i:i + 65_536]
        part.copy_(_quantised(_rows(gen, c, part.shape[0]).float(), c))
    return rec


def _lengths(gen, c, ragged):
    n = torch.full((c["batch"],), c["entries"], dtype=torch.int32, device="cuda")
    if ragged:
        n -= torch.randint(0, max(1, c["entries"] // 2), n.shape, generator=gen, device="cuda",
                           dtype=torch.int32)
    return n


def _selected(gen, n_entries, rows, entries, k):
    """[rows][batch][k] ascending indices below each length, -1 behind them;
    the rows of a sequence share most of what they select."""
    b = n_entries.shape[0]
    base = torch.rand(b, entries, generator=gen, device="cuda")
    base.masked_fill_(torch.arange(entries, device="cuda") >= n_entries[:, None], -1.0)
    out = torch.full((rows, b, k), -1, dtype=torch.int32, device="cuda")
    for r in range(rows):
        score = torch.where(base < 0, base, base + 0.01 *
                            torch.rand(b, entries, generator=gen, device="cuda"))
        top = score.topk(min(k, entries), dim=-1)
        idx = torch.where(top.values < 0, entries, top.indices).sort(-1).values
        out[r, :, :idx.shape[1]] = torch.where(idx == entries, -1, idx).to(torch.int32)
    return out


def _tree(gen, nodes, batch, ragged):
    """parents [nodes][batch]: -1 at the root, -2 where a sequence has fewer nodes."""
    par = torch.full((nodes, batch), -1, dtype=torch.int32, device="cuda")
    for t in range(1, nodes):
        back = torch.randint(0, min(t, 4), (batch,), generator=gen, device="cuda")
        chain = torch.rand(batch, generator=gen, device="cuda") < 0.6
        par[t] = torch.where(chain, t - 1, t - 1 - back).to(torch.int32)
    if ragged and nodes > 1:
        size = torch.randint(1, nodes + 1, (batch,), generator=gen, device="cuda")
        par.masked_fill_(torch.arange(nodes, device="cuda")[:, None] >= size, -2)
    return par


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"c": c}
    if c["op"] == "norm_rope":
        n, h, d = c["n"], c["heads"], c["latent"] + c["rope"]
        if c["fused"]:  # rows cut out of one wider matrix
            x = torch.randn(n, (h + 1) * d + 64, generator=gen, device="cuda")
            x = x.to(_DTYPES[c["act"]])
            s["q"], s["k"] = x[:, :h * d].view(n, h, d), x[:, h * d:(h + 1) * d]
        else:
            s["q"] = torch.randn(n, h, d, generator=gen, device="cuda").to(_DTYPES[c["act"]])
            s["k"] = torch.randn(n, d, generator=gen, device="cuda").to(_DTYPES[c["act"]])
        s["positions"] = (c["first"] + torch.arange(n, device="cuda")).to(torch.int32)
        half = c["rope"] // 2
        s["inv_freq"] = (10_000.0 ** (-torch.arange(half, device="cuda").double() / half)).float()
        for name in ("q", "k"):
            width = {"row": d, "latent": c["latent"], "none": 0}[c[name + "_norm"]]
            s[name + "_gain"] = (1 + 0.2 * torch.randn(width, generator=gen, device="cuda")
                                 if width else None)
    elif c["op"] == "unpack":
        s["records"] = _records(gen, c)
        s["n_entries"] = _lengths(gen, c, False)
        if c["gather"]:
            idx = torch.randint(0, c["entries"], (c["batch"], c["n"]), generator=gen,
                                device="cuda", dtype=torch.int32).sort(-1).values
            idx[:, c["n"] - c["n"] // 16:] = -1
            s["idx"] = idx
    elif c["op"] == "tree":
        t, b = c["nodes"], c["batch"]
        s["records"] = _records(gen, c)
        s["n_entries"] = _lengths(gen, c, c["ragged"])
        sel = _selected(gen, s["n_entries"], 1 if c["shared"] else t, c["entries"], c["topk"])
        s["topk"] = sel[0] if c["shared"] else sel
        s["q"] = torch.randn(t, b, c["heads"], c["latent"] + c["rope"], generator=gen,
                             device="cuda").to(_DTYPES[c["act"]])
        s["window"] = _rows(gen, c, b, c["window"])
        s["draft"] = _rows(gen, c, t, b)
        s["parents"] = _tree(gen, t, b, c["ragged"])
        if c["ragged"]:
            s["window_lens"] = torch.randint(0, c["window_len"] + 1, (b,), generator=gen,
                                             device="cuda", dtype=torch.int32)
    else:
        t, b, v = c["nodes"], c["batch"], c["vocab"]
        logits = 2.5 * torch.randn(t, b, v, generator=gen, device="cuda")
        p = logits.softmax(-1)
        logits += 0.8 * torch.randn(t, b, v, generator=gen, device="cuda")
        q = logits.softmax(-1)
        s["parents"] = _tree(gen, t, b, b > 1)
        tokens = torch.zeros(t, b, dtype=torch.int64, device="cuda")
        rows = torch.arange(b, device="cuda")
        rank = torch.zeros(t, b, dtype=torch.int64, device="cuda")
        for i in range(1, t):
            up = s["parents"][i].long().clamp_min(0)
            if c["draft_q"]:
                tokens[i] = torch.multinomial(q[up, rows], 1, generator=gen)[:, 0]
            else:  # greedy: a node's children are its draft's most likely tokens in order
                best = q[up, rows].topk(t, dim=-1).indices
                tokens[i] = best[rows, rank[up, rows]]
                rank[up, rows] += 1
        s["tokens"] = tokens.to(torch.int32)
        s["p"] = p.to(_DTYPES[c["dtype"]])
        s["q"] = q.to(_DTYPES[c["dtype"]]) if c["draft_q"] else None
        s["u"] = torch.rand(t, b, generator=gen, device="cuda")
        s["v"] = torch.rand(b, generator=gen, device="cuda")
    if own:  # the handles a user's program keeps: the configuration and the cache
        _handles(s)
    return s


# ----------------------------------------------------- the framework's calls
def _handles(s):
    from fp4_compressed_kv_b200 import kvc
    c = s["c"]
    s["kvc"] = kvc
    if c["op"] == "verify":
        return
    s["cfg"] = kvc.make_config(c["latent"], c["rope"], c.get("group", 32),
                               kvc.SCALE_F32 if c["scale_f32"] else kvc.SCALE_UE4M3, 128,
                               c["topk"], c["window"], c["heads"], _sm_scale(c),
                               kvc.F32 if c["act"] == "f32" else kvc.BF16)
    if "records" in s:
        idx_k = torch.zeros(c["batch"], c["entries"], 128, dtype=torch.int8, device="cuda")
        s["cache"] = kvc.Cache.wrap(s["cfg"], s["records"], idx_k, s["n_entries"])


def _own_norm_rope(s):
    kvc, c = s["kvc"], s["c"]
    q_out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    k_out = torch.empty(s["k"].shape, dtype=s["k"].dtype, device="cuda")
    norms = {"row": kvc.NORM_ROW, "latent": kvc.NORM_LATENT, "none": kvc.NORM_NONE}
    kvc.norm_rope(s["cfg"], s["q"], s["k"], s["positions"], s["inv_freq"], q_out, k_out,
                  q_gain=s["q_gain"], k_gain=s["k_gain"], q_norm=norms[c["q_norm"]],
                  k_norm=norms[c["k_norm"]], eps=1e-6,
                  layout=kvc.ROPE_PAIRS if c["pairs"] else kvc.ROPE_HALVES)
    return {"q": q_out, "k": k_out}


def _own_unpack(s):
    c = s["c"]
    out = torch.empty(c["batch"], c["n"], c["latent"] + c["rope"], dtype=_DTYPES[c["act"]],
                      device="cuda")
    s["kvc"].unpack(s["cfg"], s["cache"], out, idx=s.get("idx"))
    return {"rows": out}


def _own_tree(s):
    c = s["c"]
    t, b, h = c["nodes"], c["batch"], c["heads"]
    out = torch.empty(t, b, h, c["latent"], dtype=_DTYPES[c["act"]], device="cuda")
    lse = torch.empty(t, b, h, dtype=torch.float32, device="cuda")
    s["kvc"].tree_decode_attn(s["cfg"], s["q"], s["cache"], s["topk"], s["window"],
                              c["window_len"], s["draft"], s["parents"], out, lse=lse,
                              window_lens=s.get("window_lens"))
    return {"out": out, "lse": lse}


def _own_verify(s):
    c = s["c"]
    t, b = c["nodes"], c["batch"]
    path = torch.empty(b, t, dtype=torch.int32, device="cuda")
    n_path = torch.empty(b, dtype=torch.int32, device="cuda")
    token = torch.empty(b, dtype=torch.int32, device="cuda")
    s["kvc"].verify_tree(s["p"], s["q"], s["tokens"], s["parents"], s["u"], s["v"], path, n_path,
                         token)
    return {"path": path, "n_path": n_path, "token": token}


# ------------------------------------------------------------- plain forms
def _sm_scale(c):
    return 1.0 / math.sqrt(c["latent"] + c["rope"])


def _plain_norm(x, gain, width, eps):
    """x / sqrt(mean(x^2) + eps) * gain over the first `width` channels."""
    if not width:
        return x
    a = x[..., :width]
    a = a * (a.square().mean(-1, keepdim=True) + eps).rsqrt() * gain
    return torch.cat([a, x[..., width:]], -1)


def _plain_norm_rope(s):
    c = s["c"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    out = {}
    for name in ("q", "k"):
        width = {"row": c["latent"] + c["rope"], "latent": c["latent"], "none": 0}[c[name + "_norm"]]
        x = _plain_norm(s[name].float(), s[name + "_gain"], width, 1e-6)
        co, si = (cos[:, None], sin[:, None]) if name == "q" else (cos, sin)
        r = x[..., c["latent"]:]
        half = c["rope"] // 2
        a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :half], r[..., half:])
        a, b = a * co - b * si, a * si + b * co
        r = torch.stack([a, b], -1).flatten(-2) if c["pairs"] else torch.cat([a, b], -1)
        out[name] = torch.cat([x[..., :c["latent"]], r], -1).to(s[name].dtype)
    return out


def _plain_values(rec, c):
    """Records [..][bytes] -> fp32 values [..][D]."""
    d = c["latent"] + c["rope"]
    table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=rec.device)
    code = rec[..., :d // 2]
    x = table[torch.stack([code & 15, code >> 4], -1).flatten(-2).int()]
    n = _n_groups(c)
    if c["scale_f32"]:
        sc = rec[..., d // 2:d // 2 + 4 * n].contiguous().view(torch.float32)
    else:
        sc = rec[..., d // 2:d // 2 + n].contiguous().view(torch.float8_e4m3fn).float()
    first = -(-c["latent"] // c["group"])
    at = torch.cat([torch.arange(c["latent"], device=rec.device) // c["group"],
                    first + torch.arange(c["rope"], device=rec.device) // c["group"]])
    return x * sc[..., at]


def _plain_unpack(s):
    c = s["c"]
    if not c["gather"]:
        return {"rows": _plain_values(s["records"][:, :c["n"]], c).to(_DTYPES[c["act"]])}
    idx = s["idx"].long()
    b = torch.arange(c["batch"], device=idx.device)[:, None]
    x = _plain_values(s["records"][b, idx.clamp_min(0)], c)
    return {"rows": (x * (idx >= 0)[..., None]).to(_DTYPES[c["act"]])}


def _plain_masks(parents, lens, window):
    """Which window rows [T][B][W] and drafted rows [T][B][T] each node sees:
    the last `window` tokens of its own path."""
    t, b = parents.shape
    depth = torch.zeros(t, b, dtype=torch.int64, device=parents.device)
    gap = torch.full((t, b, t), -1, dtype=torch.int64, device=parents.device)  # steps up to a row
    rows = torch.arange(b, device=parents.device)
    for i in range(t):
        p = parents[i].long()
        up, live = p.clamp_min(0), p >= 0
        depth[i] = torch.where(live, depth[up, rows] + 1, (p == -1).long())
        gap[i] = torch.where(live[:, None] & (gap[up, rows] >= 0), gap[up, rows] + 1, -1)
        gap[i, :, i] = torch.where(p >= -1, 0, -1)
    w = torch.arange(window, device=parents.device)
    back = depth[..., None] + lens.long()[None, :, None] - 1 - w
    seen_w = (w < lens.long()[None, :, None]) & (back < window) & (depth > 0)[..., None]
    return seen_w, (gap >= 0) & (gap < window)


def _plain_tree(s):
    c = s["c"]
    t, b = c["nodes"], c["batch"]
    lens = s.get("window_lens")
    if lens is None:
        lens = torch.full((b,), c["window_len"], device="cuda", dtype=torch.int32)
    q = s["q"].float() * _sm_scale(c)
    win, draft = s["window"].float(), s["draft"].float()
    idx = s["topk"].long()
    rows = torch.arange(b, device=idx.device)[:, None]
    seen_w, seen_d = _plain_masks(s["parents"], lens, c["window"])
    live = (s["parents"] >= -1)[..., None]
    seen_r = (idx >= 0).expand(t, b, -1) & live
    key = _plain_values(s["records"][rows, idx.clamp_min(0)], c)  # [T][B][K][D] or [B][K][D]
    axes = "bkd" if c["shared"] else "tbkd"
    x = torch.cat([torch.einsum("tbhd,%s->tbhk" % axes, q, key),
                   torch.einsum("tbhd,bwd->tbhw", q, win),
                   torch.einsum("tbhd,sbd->tbhs", q, draft)], -1)
    seen = torch.cat([seen_r, seen_w, seen_d], -1)[:, :, None]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - m.clamp_min(-3e38)).exp()
    z = e.sum(-1, keepdim=True)
    e = e / z.clamp_min(1e-30)
    k, w, v = idx.shape[-1], win.shape[1], c["latent"]
    out = (torch.einsum("tbhk,%s->tbhd" % axes, e[..., :k], key[..., :v]) +
           torch.einsum("tbhw,bwd->tbhd", e[..., k:k + w], win[..., :v]) +
           torch.einsum("tbhs,sbd->tbhd", e[..., k + w:], draft[..., :v]))
    return {"out": out.to(s["q"].dtype), "lse": (m + z.log())[..., 0]}


def _plain_verify(s):
    """One pass over the nodes in order: a child of the deepest accepted node
    is accepted where u * mass * q(x) < max(p(x) - S q(x), 0)."""
    c = s["c"]
    t, b, v = c["nodes"], c["batch"], c["vocab"]
    p, q = s["p"], s["q"]
    rows = torch.arange(b, device=p.device)
    cur = torch.zeros(b, dtype=torch.int64, device=p.device)
    shift = torch.zeros(b, dtype=torch.float64, device=p.device)
    mass = torch.ones(b, dtype=torch.float64, device=p.device)
    gone = torch.zeros(b, v, dtype=torch.bool, device=p.device)
    over = torch.zeros(b, dtype=torch.bool, device=p.device)
    path = torch.full((b, t), -1, dtype=torch.int32, device=p.device)
    path[:, 0] = 0
    n_path = torch.ones(b, dtype=torch.int64, device=p.device)
    for i in range(1, t):
        x = s["tokens"][i].long()
        child = (s["parents"][i] == cur) & ~over
        px = p[cur, rows, x].double()
        if q is None:
            rx = torch.where(gone[rows, x], 0.0, px)
            take = child & (s["u"][i].double() * mass < rx)
        else:
            qx = q[cur, rows, x].double()
            rx = (px - shift * qx).clamp_min(0)
            take = child & (s["u"][i].double() * mass * qx < rx)
        left = child & ~take
        if q is None:
            gone[rows, x] |= left
            mass = torch.where(left, (mass - rx).clamp_min(0), mass)
        else:
            shift = torch.where(left, shift + mass, shift)
            rest = (p[cur, rows].double() - shift[:, None] * q[cur, rows].double()).clamp_min(0)
            mass = torch.where(left, rest.sum(-1), mass)
            over = over | (left & (mass <= 0))
        path[rows, n_path.clamp_max(t - 1)] = torch.where(
            take, i, path[rows, n_path.clamp_max(t - 1)]).to(torch.int32)
        n_path = n_path + take
        cur = torch.where(take, i, cur)
        shift, mass = torch.where(take, 0.0, shift), torch.where(take, 1.0, mass)
        gone &= ~take[:, None]
    row = p[cur, rows].double()
    r = row.masked_fill(gone, 0.0) if q is None else \
        (row - shift[:, None] * q[cur, rows].double()).clamp_min(0)
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, row)
    run_sum = r.cumsum(-1)
    hit = run_sum > s["v"].double()[:, None] * r.sum(-1, keepdim=True)
    last = v - 1 - (r > 0).flip(-1).int().argmax(-1)
    token = torch.where(hit.any(-1), hit.int().argmax(-1), last)
    return {"path": path, "n_path": n_path.to(torch.int32), "token": token.to(torch.int32)}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "unpack": _own_unpack, "tree": _own_tree,
                "verify": _own_verify}[op](state)
    return {"norm_rope": _plain_norm_rope, "unpack": _plain_unpack, "tree": _plain_tree,
            "verify": _plain_verify}[op](state)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    size = 4 if (c.get("act") or c.get("dtype")) == "f32" else 2
    if c["op"] == "verify":
        # every sequence reads the row it samples from, and its draft row
        rows = c["batch"] * (2 if c["draft_q"] else 1)
        return {"bytes": rows * c["vocab"] * size + c["nodes"] * c["batch"] * 16,
                "flops": 4 * rows * c["vocab"]}
    d = c["latent"] + c["rope"]
    if c["op"] == "norm_rope":
        rows = c["n"] * (c["heads"] + 1)
        return {"bytes": 2 * rows * d * size, "flops": 6 * rows * d}
    rec = d // 2 + _n_groups(c) * (4 if c["scale_f32"] else 1)
    if c["op"] == "unpack":
        rows = c["batch"] * c["n"]
        return {"bytes": rows * (rec + d * size), "flops": rows * d}
    t, b = c["nodes"], c["batch"]
    picked = b * (1 if c["shared"] else t) * min(c["topk"], c["entries"])
    keys = min(c["topk"], c["entries"]) + min(c["window"], c["window_len"] + t)
    return {"bytes": picked * (rec + 4) + b * (c["window_len"] + t) * d * size +
            t * b * c["heads"] * (d + c["latent"]) * size,
            "flops": 2 * t * b * c["heads"] * keys * (d + c["latent"])}


# ------------------------------------------------------- values in 64 bits
def _exact_record(rec, c):
    """Sign, exponent and mantissa of each code and scale, in fp64."""
    d = c["latent"] + c["rope"]
    b = rec[..., :d // 2].long()
    code = torch.empty(*b.shape[:-1], d, dtype=torch.int64, device=rec.device)
    code[..., 0::2], code[..., 1::2] = b % 16, b // 16
    e, m = (code // 2) % 4, code % 2
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    val = torch.where(code >= 8, -mag, mag).double()
    n = _n_groups(c)
    if c["scale_f32"]:
        raw = rec[..., d // 2:d // 2 + 4 * n].cpu().numpy()
        scale = torch.from_numpy(np.ascontiguousarray(raw).view(np.float32).astype(np.float64))
        scale = scale.to(rec.device)
    else:
        y = rec[..., d // 2:d // 2 + n].long()
        ye, ym = (y // 8) % 16, y % 8
        scale = torch.where(ye == 0, ym * 2.0 ** -9,
                            (8 + ym) * torch.pow(2.0, (ye - 10).double())).double()
    parts, at = [], 0
    for lo, hi in ((0, c["latent"]), (c["latent"], d)):
        for g in range(lo, hi, c["group"]):
            parts.append(val[..., g:min(g + c["group"], hi)] * scale[..., at:at + 1])
            at += 1
    return torch.cat(parts, -1)


def _exact_unpack(s):
    c = s["c"]
    out = torch.zeros(c["batch"], c["n"], c["latent"] + c["rope"], dtype=torch.float64)
    for b in range(c["batch"]):
        for i in range(0, c["n"], 100_000):
            if c["gather"]:
                idx = s["idx"][b, i:i + 100_000]
                ok = (idx >= 0).nonzero()[:, 0]
                rows = _exact_record(s["records"][b, idx[ok].long()], c)
                out[b, i + ok.cpu()] = rows.cpu()
            else:
                hi = min(i + 100_000, c["n"])
                out[b, i:hi] = _exact_record(s["records"][b, i:hi], c).cpu()
    return {"rows": out}


def _exact_norm_rope(s):
    c = s["c"]
    lat, half = c["latent"], c["rope"] // 2
    turn = s["positions"].cpu().numpy().astype(np.float64)[:, None] * \
        s["inv_freq"].cpu().numpy().astype(np.float64)
    z = torch.from_numpy(np.exp(1j * turn)).to("cuda")
    out = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        width = {"row": lat + c["rope"], "latent": lat, "none": 0}[c[name + "_norm"]]
        if width:
            ms = torch.einsum("...d,...d->...", x[..., :width], x[..., :width]) / width
            x[..., :width] *= s[name + "_gain"].double() / torch.sqrt(ms + 1e-6)[..., None]
        first = slice(lat, None, 2) if c["pairs"] else slice(lat, lat + half)
        second = slice(lat + 1, None, 2) if c["pairs"] else slice(lat + half, None)
        y = torch.complex(x[..., first], x[..., second]) * (z[:, None] if name == "q" else z)
        x[..., first], x[..., second] = y.real, y.imag
        out[name] = x
    return out


def _exact_tree(s):
    """Each node's own list of keys, one softmax at a time."""
    c = s["c"]
    t, b, v = c["nodes"], c["batch"], c["latent"]
    out = torch.zeros(t, b, c["heads"], v, dtype=torch.float64, device="cuda")
    lse = torch.full((t, b, c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    parents = s["parents"].tolist()
    lens = s["window_lens"].tolist() if "window_lens" in s else [c["window_len"]] * b
    for j in range(b):
        for i in range(t):
            if parents[i][j] < -1:
                continue
            path, at = [], i
            while at >= 0:
                path.append(at)
                at = parents[at][j]
            raw = torch.cat([s["window"][j, :lens[j]], s["draft"][path[::-1], j]])
            raw = raw[max(0, raw.shape[0] - c["window"]):].double()
            idx = (s["topk"] if c["shared"] else s["topk"][i])[j].long()
            keys = torch.cat([_exact_record(s["records"][j, idx[idx >= 0]], c), raw])
            if not keys.shape[0]:
                continue
            x = s["q"][i, j].double() @ keys.T / math.sqrt(c["latent"] + c["rope"])
            lse[i, j] = torch.logsumexp(x, -1)
            out[i, j] = torch.exp(x - lse[i, j][:, None]) @ keys[:, :v]
    return {"out": out, "lse": lse}


def _exact_verify(s):
    """Each sequence by itself, normalising the residual after every rejection."""
    c = s["c"]
    t, b = c["nodes"], c["batch"]
    parents, tokens = s["parents"].tolist(), s["tokens"].tolist()
    u, v = s["u"].double().tolist(), s["v"].double().tolist()
    path = np.full((b, t), -1, np.int32)
    n_path, token = np.zeros(b, np.int32), np.zeros(b, np.int32)
    for j in range(b):
        row = lambda a, i: a[i, j].double().cpu().numpy()  # noqa: E731
        cur, n = 0, 1
        path[j, 0] = 0
        res = row(s["p"], 0)
        scale, i = 1.0, 1  # the residual's mass; the first is taken as 1
        while i < t:
            if parents[i][j] == cur:
                x = tokens[i][j]
                dq = row(s["q"], cur) if s["q"] is not None else None
                if u[i][j] * scale * (1.0 if dq is None else dq[x]) < res[x]:
                    cur, path[j, n], n = i, i, n + 1
                    res, scale = row(s["p"], i), 1.0
                elif dq is None:
                    scale = max(scale - res[x], 0.0)
                    res[x] = 0.0
                else:
                    res = np.maximum(res - scale * dq, 0.0)
                    scale = math.fsum(res)
                    if scale <= 0:
                        break
            i += 1
        if not res.sum() > 0:
            res = row(s["p"], cur)
        total = np.cumsum(res)
        hit = np.flatnonzero(total > v[j] * total[-1])
        token[j] = hit[0] if hit.size else np.flatnonzero(res > 0)[-1]
        n_path[j] = n
    return {"path": path, "n_path": n_path, "token": token}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "unpack": _exact_unpack, "tree": _exact_tree,
            "verify": _exact_verify}[case["op"]](s)
