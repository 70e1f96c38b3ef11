"""kvc_norm_rope against the formula in 64 bits.

Tolerance, per channel: the kernel's sums and products are fp32.  A lane adds
at most 16 x 8 + 8 x (rope / 64) squares one after another, then three partial
sums: with w <= 1024 channels at most 160 roundings of a sum of positive
terms, halved by the square root, and 8 more for the root, the divisions, the
gain and the rotation; the angle is off by 2^-25 turns and its functions by
2^-22.  Together below 128 x 2^-24 of |x| + |y| of the pair.  On top half a
step of the row's type (bf16: 2^-8 of the value)."""
import numpy as np
import pytest
import torch

import plain64
from helpers import Guarded

pytestmark = pytest.mark.gpu

MLA = (512, 64, 64, "bf16")
TINY = (64, 16, 8, "f32")


def _cfg(kvc, shape):
    latent, rope, heads, act = shape
    return kvc.make_config(latent, rope, 8, kvc.SCALE_UE4M3, 128, 64, 128, heads, 0.05,
                           kvc.F32 if act == "f32" else kvc.BF16)


def _check(got, ref, mag, dtype):
    got = got.double().cpu().numpy()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    tol = half * np.abs(ref) + 128 * 2.0 ** -24 * mag + 1e-38
    worst = np.max(np.abs(got - ref) - tol)
    assert worst <= 0, f"over the bound by {worst:.3e}"


def _inputs(shape, n, seed, fused=False, scale=1.0):
    latent, rope, h, act = shape
    d = latent + rope
    dt = torch.float32 if act == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = (scale * torch.randn(n, (h + 1) * d + 24, generator=g, device="cuda")).to(dt)
        q, k = x[:, 8:8 + h * d].view(n, h, d), x[:, 8 + h * d:8 + (h + 1) * d]
        if act == "bf16" and (x.stride(0) * 2) % 16:
            raise AssertionError("the row stride must keep 16-byte rows")
    else:
        q = (scale * torch.randn(n, h, d, generator=g, device="cuda")).to(dt)
        k = (scale * torch.randn(n, d, generator=g, device="cuda")).to(dt)
    half = rope // 2
    freq = (10_000.0 ** (-torch.arange(half, device="cuda").double() / max(half, 1))).float()
    gains = [1 + 0.3 * torch.randn(w, generator=g, device="cuda") for w in (latent, d)]
    return q, k, freq, gains


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("shape", [
    MLA, TINY, (8, 8, 1, "bf16"), (8, 8, 3, "f32"), (72, 24, 5, "bf16"), (128, 48, 2, "f32"),
    (256, 128, 7, "bf16"), (384, 32, 16, "f32"), (520, 504, 2, "bf16"), (1016, 8, 3, "f32"),
    (16, 1008, 2, "f32"), (1024, 0, 2, "bf16"), (64, 0, 4, "f32")])
def test_shapes(kvc, shape, pairs):
    """Every piece count a lane can hold, RoPE widths from none to nearly all
    channels, one head and odd numbers of them; both norms."""
    latent, rope, h, _ = shape
    d = latent + rope
    for n, qn, kn in ((1, kvc.NORM_ROW, kvc.NORM_LATENT), (37, kvc.NORM_LATENT, kvc.NORM_ROW),
                      (5, kvc.NORM_NONE, kvc.NORM_NONE)):
        q, k, freq, gains = _inputs(shape, n, seed=n)
        gain = {kvc.NORM_NONE: None, kvc.NORM_LATENT: gains[0], kvc.NORM_ROW: gains[1]}
        width = {kvc.NORM_NONE: 0, kvc.NORM_LATENT: latent, kvc.NORM_ROW: d}
        pos = torch.arange(n, device="cuda", dtype=torch.int32) * 977 + 3
        qo = Guarded(q.shape, q.dtype, fill=float("nan"))
        ko = Guarded(k.shape, k.dtype, fill=float("nan"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvc.norm_rope(_cfg(kvc, shape), q, k, pos, freq if rope else None, qo.t, ko.t,
                      q_gain=gain[qn], k_gain=gain[kn], q_norm=qn, k_norm=kn, eps=1e-5,
                      layout=kvc.ROPE_PAIRS if pairs else kvc.ROPE_HALVES, status=st)
        qo.check()
        ko.check()
        assert st.item() == 0
        for x, o, norm in ((q, qo.t, qn), (k, ko.t, kn)):
            g = None if gain[norm] is None else gain[norm].cpu().numpy()
            ref, mag = plain64.norm_rope(x.double().cpu().numpy(), g, width[norm], latent,
                                         pos.cpu().numpy(), freq.cpu().numpy(), pairs,
                                         float(np.float32(1e-5)))
            _check(o, ref, mag, x.dtype)


def test_far_and_negative_positions(kvc):
    """Angles of 2^31 turns' worth of radians keep their precision: formed and
    reduced in 64 bits."""
    q, k, freq, _ = _inputs(TINY, 6, seed=3)
    pos = torch.tensor([0, 1_000_000, -7, 2 ** 31 - 1, -2 ** 31, 123_456_789], dtype=torch.int32,
                       device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    for pairs in (0, 1):
        kvc.norm_rope(_cfg(kvc, TINY), q, k, pos, freq, qo, ko, layout=pairs, eps=0.0)
        for x, o, w in ((q, qo, 80), (k, ko, 64)):
            ref, mag = plain64.norm_rope(x.double().cpu().numpy(), None, w, 64, pos.cpu().numpy(),
                                         freq.cpu().numpy(), bool(pairs), 0.0)
            # 2^31 x freq in fp64 is off by 2^-22, the turns after it by 2^-21 radians
            _check(o, ref, 4 * mag, x.dtype)


def test_strided_rows_in_place_and_alone(kvc):
    """Rows cut out of a wider matrix (its other columns stay), queries or keys
    alone, rotation in place, no gain."""
    shape = MLA
    cfg = _cfg(kvc, shape)
    n = 70
    q, k, freq, gains = _inputs(shape, n, seed=5, fused=True)
    pos = torch.randint(0, 100_000, (n,), device="cuda", dtype=torch.int32)
    qo, ko = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k))
    kvc.norm_rope(cfg, q, k, pos, freq, qo, ko, q_gain=gains[1], k_gain=gains[0])
    q2, k2 = torch.full_like(qo, 7), torch.full_like(ko, 7)
    kvc.norm_rope(cfg, q.contiguous(), None, pos, freq, q2, None, q_gain=gains[1])
    kvc.norm_rope(cfg, None, k, pos, freq, None, k2, k_gain=gains[0])
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    q3, k3 = q.contiguous(), k.contiguous()
    kvc.norm_rope(cfg, q3, k3, pos, freq, q3, k3, q_gain=gains[1], k_gain=gains[0])
    assert torch.equal(q3, qo) and torch.equal(k3, ko)
    for x, o, w, g in ((q, qo, 576, gains[1]), (k, ko, 512, gains[0])):
        ref, mag = plain64.norm_rope(x.double().cpu().numpy(), g.cpu().numpy(), w, 512,
                                     pos.cpu().numpy(), freq.cpu().numpy(), False,
                                     float(np.float32(1e-6)))
        _check(o, ref, mag, x.dtype)


def test_many_rows_of_a_group(kvc):
    """Enough rows that a lane group takes several heads of a token."""
    for shape, n in ((MLA, 1500), (TINY, 9000)):
        q, k, freq, gains = _inputs(shape, n, seed=9)
        latent, d = shape[0], shape[0] + shape[1]
        pos = torch.arange(n, device="cuda", dtype=torch.int32).flip(0).contiguous()
        qo, ko = Guarded(q.shape, q.dtype), Guarded(k.shape, k.dtype)
        kvc.norm_rope(_cfg(kvc, shape), q, k, pos, freq, qo.t, ko.t, q_gain=gains[1],
                      k_gain=gains[0])
        qo.check()
        ko.check()
        pick = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")
        for x, o, w, g in ((q, qo.t, d, gains[1]), (k, ko.t, latent, gains[0])):
            ref, mag = plain64.norm_rope(x[pick].double().cpu().numpy(), g.cpu().numpy(), w, latent,
                                         pos[pick].cpu().numpy(), freq.cpu().numpy(), False,
                                         float(np.float32(1e-6)))
            _check(o[pick], ref, mag, x.dtype)
        # the same rows in smaller calls give the same bits
        q2, k2 = torch.empty_like(qo.t[:3]), torch.empty_like(ko.t[:3])
        kvc.norm_rope(_cfg(kvc, shape), q[5:8].contiguous(), k[5:8].contiguous(),
                      pos[5:8].contiguous(), freq, q2, k2, q_gain=gains[1], k_gain=gains[0])
        assert torch.equal(q2, qo.t[5:8]) and torch.equal(k2, ko.t[5:8])


def test_nonfinite_rows_are_flagged_and_alone(kvc):
    q, k, freq, _ = _inputs(MLA, 4, seed=11)
    q[1, 3, 100] = float("nan")
    k[2, 5] = float("inf")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    kvc.norm_rope(_cfg(kvc, MLA), q, k, pos, freq, qo, ko, status=st)
    assert st.item() == kvc.DEV_NONFINITE
    bad = ~torch.isfinite(qo.float()).all(-1)
    assert bad.sum() == 1 and bad[1, 3]
    bad = ~torch.isfinite(ko.float()).all(-1)
    assert bad.sum() == 1 and bad[2]


def test_zero_rows_and_zero_row(kvc):
    """No rows: nothing happens; a row of zeros stays zeros with eps > 0."""
    cfg = _cfg(kvc, TINY)
    q, k, freq, _ = _inputs(TINY, 2, seed=13)
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    kvc.norm_rope(cfg, q[:0], k[:0], empty, freq, q[:0].clone(), k[:0].clone())
    q[0] = 0
    qo = torch.empty_like(q)
    pos = torch.arange(2, device="cuda", dtype=torch.int32)
    kvc.norm_rope(cfg, q, None, pos, freq, qo, None)
    assert not qo[0].any() and torch.isfinite(qo).all()


def test_refused_calls(kvc):
    cfg = _cfg(kvc, TINY)
    q, k, freq, gains = _inputs(TINY, 3, seed=17)
    pos = torch.arange(3, device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    for kw in (dict(layout=2), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(kvc.KvcError):
            kvc.norm_rope(cfg, q, k, pos, freq, qo, ko, **kw)
    with pytest.raises(ValueError):  # gain of the wrong width
        kvc.norm_rope(cfg, q, k, pos, freq, qo, ko, q_gain=gains[0])
    with pytest.raises(ValueError):
        kvc.norm_rope(cfg, q.bfloat16(), k, pos, freq, qo, ko)
    with pytest.raises(ValueError):
        kvc.norm_rope(cfg, q, k, pos.cpu(), freq, qo, ko)
    wide = torch.randn(3, 8 * 80 + 2, device="cuda")
    with pytest.raises(kvc.KvcError):  # rows that do not start on 16 bytes
        kvc.norm_rope(cfg, wide[:, :640].view(3, 8, 80), None, pos, freq, qo, None)
    wide = torch.randn(3, 8 * 80 + 4, device="cuda")
    with pytest.raises(ValueError):  # a strided output
        kvc.norm_rope(cfg, q, None, pos, freq, wide[:, :640].view(3, 8, 80), None)


def test_longest_runs_of_a_warp(kvc):
    """So many rows that a warp goes through several fours of them, odd counts
    of heads and rows, in place: the same bits as in small calls."""
    for shape, n in (((8, 8, 41, "f32"), 7501), ((64, 64, 64, "bf16"), 5003)):
        q, k, freq, gains = _inputs(shape, n, seed=19)
        pos = torch.arange(n, device="cuda", dtype=torch.int32)
        cfg = _cfg(kvc, shape)
        kw = dict(q_gain=gains[1], k_gain=gains[0])
        want_q, want_k = torch.empty_like(q), torch.empty_like(k)
        for i in range(0, n, 400):
            part = slice(i, min(n, i + 400))
            kvc.norm_rope(cfg, q[part], k[part], pos[part], freq, want_q[part], want_k[part], **kw)
        kvc.norm_rope(cfg, q, k, pos, freq, q, k, **kw)
        assert torch.equal(q, want_q) and torch.equal(k, want_k)


def test_stream_and_graph(kvc):
    """On another stream, and captured and replayed with other rows in place."""
    cfg = _cfg(kvc, MLA)
    q, k, freq, gains = _inputs(MLA, 9, seed=23)
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    kw = dict(q_gain=gains[1], k_gain=gains[0])
    qo, ko, q1, k1 = (torch.empty_like(x) for x in (q, k, q, k))
    kvc.norm_rope(cfg, q, k, pos, freq, qo, ko, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kvc.norm_rope(cfg, q, k, pos, freq, q1, k1, stream=s, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.norm_rope(cfg, q, k, pos, freq, q1, k1, **kw)
    q2, k2, _, _ = _inputs(MLA, 9, seed=24)
    q.copy_(q2)
    k.copy_(k2)
    pos += 77
    graph.replay()
    kvc.norm_rope(cfg, q2, k2, pos, freq, qo, ko, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
