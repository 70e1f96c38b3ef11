"""The operators around a speculative decode step restated in numpy, in 64
bits, one row at a time: what the GPU tests compare with.  Shares no code with
the library or its binding."""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3(byte):
    """Value of an E4M3 byte (sign in bit 7)."""
    b = np.asarray(byte).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b & 128, -v, v)


def groups(latent, rope, group):
    """Group of every channel: latent and RoPE channels are grouped apart."""
    first = -(-latent // group)
    return np.concatenate([np.arange(latent) // group, first + np.arange(rope) // group])


def record_values(rec, latent, rope, group, scale_f32):
    """Records [..][bytes] uint8 -> fp64 values [..][D]."""
    d = latent + rope
    code = rec[..., :d // 2]
    nib = np.stack([code & 15, code >> 4], -1).reshape(*rec.shape[:-1], d)
    val = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    n = int(groups(latent, rope, group)[-1]) + 1
    if scale_f32:
        sc = np.ascontiguousarray(rec[..., d // 2:d // 2 + 4 * n]).view(np.float32).astype(np.float64)
    else:
        sc = e4m3(rec[..., d // 2:d // 2 + n] & 127)
    return val * sc[..., groups(latent, rope, group)]


def norm_rope(x, gain, width, latent, positions, inv_freq, pairs, eps):
    """x [n][..][D] fp64; one norm and one rotation a row."""
    y = np.array(x, np.float64)
    if width:
        ms = (y[..., :width] ** 2).mean(-1, keepdims=True)
        y[..., :width] /= np.sqrt(ms + eps)
        if gain is not None:
            y[..., :width] *= gain.astype(np.float64)
    rope = x.shape[-1] - latent
    half = rope // 2
    ang = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)[None]
    ang = ang.reshape(len(positions), *([1] * (x.ndim - 2)), half)
    c, s = np.cos(ang), np.sin(ang)
    r = y[..., latent:]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :half], r[..., half:])
    p, q = a * c - b * s, a * s + b * c
    out = y.copy()
    if pairs:
        out[..., latent::2], out[..., latent + 1::2] = p, q
    else:
        out[..., latent:latent + half], out[..., latent + half:] = p, q
    mag = np.abs(y)  # what the errors of a channel are measured by
    if rope:
        both = np.abs(a) + np.abs(b)
        mag[..., latent:] = np.repeat(both, 2, -1) if pairs else np.concatenate([both, both], -1)
    return out, mag


def path_of(parents, t):
    """Nodes from the first ancestor of t down to t, or None for an absent node."""
    path = []
    at = t
    while True:
        path.append(at)
        p = int(parents[at])
        if p == -1:
            return path[::-1]
        if p < -1 or p >= at:
            return None
        at = p


def tree_attention(q, records, n_entries, capacity, topk, window, lens, draft, parents, cfg,
                   scale_f32):
    """cfg: (latent, rope, group, sm_scale).  Returns out, lse and the bounds'
    ingredients: sum p |v| over entries and over raw keys, the largest
    sum |q k| of a logit, the number of keys, and sum |v| over entries."""
    latent, rope, group, sm = cfg
    T, B, H, D = q.shape
    W = window.shape[1]
    out = np.zeros((T, B, H, latent))
    lse = np.full((T, B, H), -np.inf)
    rec_abs, raw_abs = np.zeros_like(out), np.zeros_like(out)
    dots, count = np.zeros((T, B, H)), np.zeros((T, B), int)
    rec_sum = np.zeros((T, B, 1, latent))
    for b in range(B):
        for t in range(T):
            path = path_of(parents[:, b], t)
            if path is None:
                continue
            raw = np.concatenate([window[b, :lens[b]].astype(np.float64),
                                  draft[path, b].astype(np.float64)])
            raw = raw[max(0, len(raw) - W):]
            idx = topk[b] if topk.ndim == 2 else topk[t, b]
            n = n_entries[b] if 0 <= n_entries[b] <= capacity else 0
            idx = idx[(idx >= 0) & (idx < n)]
            ent = record_values(records[b, idx], latent, rope, group, scale_f32)
            keys = np.concatenate([ent, raw]) if len(idx) or len(raw) else np.zeros((0, D))
            count[t, b] = len(keys)
            if not len(keys):
                continue
            x = sm * (q[t, b].astype(np.float64) @ keys.T)
            dots[t, b] = sm * (np.abs(q[t, b].astype(np.float64)) @ np.abs(keys).T).max(-1)
            m = x.max(-1, keepdims=True)
            e = np.exp(x - m)
            z = e.sum(-1, keepdims=True)
            lse[t, b] = (m + np.log(z))[:, 0]
            p = e / z
            out[t, b] = p @ keys[:, :latent]
            rec_abs[t, b] = p[:, :len(idx)] @ np.abs(ent[:, :latent])
            raw_abs[t, b] = p[:, len(idx):] @ np.abs(raw[:, :latent])
            rec_sum[t, b, 0] = np.abs(ent[:, :latent]).sum(0)
    return out, lse, rec_abs, raw_abs, dots, count, rec_sum


def clean(row):
    row = np.asarray(row, np.float64)
    return np.where((row >= 0) & (row < np.inf), row, 0.0)


def verify(p, q, tokens, parents, u, v):
    """p, q [T][B][V] (q None: greedy drafts) -> path, n_path, next token."""
    T, B, V = p.shape
    path = np.full((B, T), -1, np.int32)
    n_path, token = np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        if parents[0, b] == -2:
            continue
        cur, taken = 0, [0]
        res, mass = clean(p[0, b]), 1.0
        for t in range(1, T):
            x = int(tokens[t, b])
            if parents[t, b] != cur or not 0 <= x < V:
                continue
            draft = None if q is None else clean(q[cur, b])
            if float(u[t, b]) * mass * (1.0 if draft is None else draft[x]) < res[x]:
                cur = t
                taken.append(t)
                res, mass = clean(p[t, b]), 1.0
            elif draft is None:
                mass = max(mass - res[x], 0.0)
                res[x] = 0.0
            else:
                res = np.maximum(res - mass * draft, 0.0)
                mass = math.fsum(res)
                if not mass > 0:
                    break
        if not res.sum() > 0:
            res = clean(p[cur, b])
        path[b, :len(taken)] = taken
        n_path[b] = len(taken)
        run = np.cumsum(res)
        if run[-1] > 0:
            hit = np.flatnonzero(run > float(v[b]) * run[-1])
            token[b] = hit[0] if hit.size else np.flatnonzero(res > 0)[-1]
    return path, n_path, token
