"""kvc_unpack and kvc_unpack_window_fp8: records and FP8 window rows read
back.  A code times a UE4M3 scale is exact in bf16 and fp32; with an fp32
scale the product of 2 and 24 significant bits is rounded once to fp32 (the
numpy fp32 rounding of the fp64 product is the same), and once more to bf16
where the rows are bf16 (2^-8 and 2^-24 of the value)."""
import numpy as np
import pytest
import torch

import plain64
from helpers import Guarded

pytestmark = pytest.mark.gpu


def _cache(kvc, shape, batch, cap, seed):
    latent, rope, group, scale_f32, act = shape
    cfg = kvc.make_config(latent, rope, group, kvc.SCALE_F32 if scale_f32 else kvc.SCALE_UE4M3,
                          128, 64, 32, 8, 0.1, kvc.F32 if act == "f32" else kvc.BF16)
    cache = kvc.Cache(cfg, batch, cap)
    rng = np.random.default_rng(seed)
    rec = rng.integers(0, 256, cache.records.shape, dtype=np.uint8)
    d = latent + rope
    n = plain64.groups(latent, rope, group)[-1] + 1
    if scale_f32:
        sc = (rng.standard_normal((batch, cap, n)) ** 2 + 1e-3).astype(np.float32)
        rec[..., d // 2:d // 2 + 4 * n] = sc.view(np.uint8).reshape(batch, cap, -1)
    else:
        rec[..., d // 2:d // 2 + n] &= 127
        rec[..., d // 2:d // 2 + n] %= 127  # 0x7F is the format's NaN
    cache.records.copy_(torch.from_numpy(rec))
    cache.n_entries.fill_(cap)
    return cfg, cache, plain64.record_values(rec, latent, rope, group, scale_f32)


SHAPES = [(512, 64, 32, False, "bf16"), (512, 64, 64, False, "bf16"), (512, 64, 16, False, "f32"),
          (512, 64, 128, False, "bf16"), (64, 16, 32, True, "f32"), (64, 16, 8, True, "bf16"),
          (256, 0, 256, False, "bf16"), (8, 8, 8, False, "f32"), (960, 64, 64, True, "f32")]


def _equal(got, want, scale_f32, act):
    got = got.double().cpu().numpy()
    if scale_f32 and act == "bf16":
        assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want))
    else:
        assert np.array_equal(got, want.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("shape", SHAPES)
def test_range_and_gather(kvc, shape):
    cfg, cache, want = _cache(kvc, shape, 3, 130, seed=1)
    d, dt = shape[0] + shape[1], torch.float32 if shape[4] == "f32" else torch.bfloat16
    for first, n in ((0, 130), (5, 1), (129, 1), (64, 33)):
        out = Guarded((3, n, d), dt, fill=float("nan"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvc.unpack(cfg, cache, out.t, first=first, status=st)
        out.check()
        assert st.item() == 0
        _equal(out.t, want[:, first:first + n], shape[3], shape[4])
    rng = np.random.default_rng(2)
    for n in (1, 17, 100):  # any order, repeats, padding
        idx = rng.integers(-1, 130, (3, n)).astype(np.int32)
        idx[:, 0] = 129
        out = Guarded((3, n, d), dt, fill=float("nan"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvc.unpack(cfg, cache, out.t, idx=torch.from_numpy(idx).cuda(), status=st)
        out.check()
        assert st.item() == 0
        ref = np.stack([np.where(idx[b][:, None] >= 0, want[b, idx[b]], 0.0) for b in range(3)])
        _equal(out.t, ref, shape[3], shape[4])


def test_entries_that_are_not_there(kvc):
    """Ragged lengths: rows behind a sequence's last entry are zeros; indices
    out of range are flagged and zero; a bad length empties its sequence."""
    cfg, cache, want = _cache(kvc, SHAPES[0], 4, 40, seed=3)
    cache.n_entries.copy_(torch.tensor([40, 0, 7, 41], dtype=torch.int32))
    out = torch.full((4, 40, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.unpack(cfg, cache, out, status=st)
    assert st.item() == kvc.DEV_BAD_LENGTH
    live = np.arange(40)[None] < np.array([40, 0, 7, 0])[:, None]
    _equal(out, want * live[..., None], False, "bf16")
    idx = torch.tensor([[0, 39, 40, -2, -1, 2 ** 31 - 1]] * 4, dtype=torch.int32, device="cuda")
    cache.n_entries[3] = 40
    out = torch.full((4, 6, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    st.zero_()
    kvc.unpack(cfg, cache, out, idx=idx, status=st)
    assert st.item() == kvc.DEV_BAD_INDEX
    ok = np.zeros((4, 6, 1))
    ok[0, :2] = ok[3, :2] = ok[2, 0] = 1
    _equal(out, want[:, [0, 39, 0, 0, 0, 0]] * ok, False, "bf16")


def test_reads_back_what_pack_writes(kvc, orc):
    """pack -> unpack equals the oracle's entries, dequantised."""
    from fp4_compressed_kv_b200 import synth
    from helpers import oracle_cfg, oracle_pack
    for name in ("tiny", "mla32k"):
        w = synth.WORKLOADS[name].scaled(context=2 * 75, batch=2)
        inp = synth.make_inputs(w)
        cfg = kvc.config_for(w)
        cache = kvc.Cache(cfg, 2, 80)
        kvc.pack(cfg, inp["tokens"].cuda(), inp["gate"].cuda(), inp["idx_k"].cuda(), cache)
        out = torch.empty(2, 75, w.dim, dtype=w.torch_dtype, device="cuda")
        kvc.unpack(cfg, cache, out, first=0)
        rec, _, _, _ = oracle_pack(w, inp["tokens"], inp["gate"], inp["idx_k"])
        ocfg = oracle_cfg(w)
        for b in range(2):
            for j in range(75):
                want = torch.from_numpy(orc.dequantize_entry(ocfg, rec[b, j])).to(w.torch_dtype)
                assert torch.equal(out[b, j].cpu(), want)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 128, 5000])
def test_window_fp8(kvc, act, n):
    cfg = kvc.make_config(512, 64, 32, kvc.SCALE_UE4M3, 128, 64, 32, 8, 0.1,
                          kvc.F32 if act == "f32" else kvc.BF16)
    dt = torch.float32 if act == "f32" else torch.bfloat16
    rng = np.random.default_rng(n)
    codes = rng.integers(0, 256, (n, 576), dtype=np.uint8)
    codes[(codes & 127) == 127] = 3  # the format's NaN is never written
    scales = np.abs(rng.standard_normal(n)).astype(np.float32)
    scales[0] = 0
    out = Guarded((n, 576), dt, fill=float("nan"))
    kvc.unpack_window_fp8(cfg, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), out.t)
    out.check()
    want = plain64.e4m3(codes) * scales[:, None].astype(np.float64)
    _equal(out.t, want, True, act)
    # and what pack_window_fp8 wrote comes back within half a step of E4M3 (2^-4)
    x = torch.randn(n, 576, device="cuda").to(dt)
    c = torch.empty(n, 576, dtype=torch.uint8, device="cuda")
    s = torch.empty(n, dtype=torch.float32, device="cuda")
    kvc.pack_window_fp8(cfg, x, c, s)
    kvc.unpack_window_fp8(cfg, c, s, out.t)
    # (subnormal codes: half a step is 2^-10 of the scale)
    err = (out.t.double() - x.double()).abs()
    assert torch.all(err <= (2.0 ** -4 + 2.0 ** -8) * x.double().abs() + 2.0 ** -10 * s[:, None].double())


def test_far_entries(kvc):
    """Byte offsets past 2^32 in one sequence's records."""
    cfg = kvc.make_config(512, 64, 32, kvc.SCALE_UE4M3, 128, 64, 32, 8, 0.1, kvc.BF16)
    cap = 14_000_000  # 320 bytes each: 4.48e9
    rec = torch.zeros(1, cap, 320, dtype=torch.uint8, device="cuda")
    idx_k = torch.zeros(1, 1, 128, dtype=torch.int8, device="cuda").expand(1, cap, 128)
    far = torch.randint(0, 256, (3, 320), dtype=torch.uint8, device="cuda")
    far[:, 288:306] &= 63
    at = [cap - 1, 13_421_773, 2]
    rec[0, at] = far
    n = torch.tensor([cap], dtype=torch.int32, device="cuda")
    cache = kvc.Cache.__new__(kvc.Cache)  # (no 1.8 GB of indexer keys: unpack reads none)
    cache.cfg, cache.batch, cache.capacity = cfg, 1, cap
    cache.records, cache.idx_k, cache.n_entries = rec, idx_k, n
    want = plain64.record_values(far.cpu().numpy(), 512, 64, 32, False)
    out = torch.empty(1, 3, 576, dtype=torch.bfloat16, device="cuda")
    kvc.unpack(cfg, cache, out, idx=torch.tensor([at], dtype=torch.int32, device="cuda"))
    _equal(out[0], want, False, "bf16")
    one = torch.empty(1, 1, 576, dtype=torch.bfloat16, device="cuda")
    kvc.unpack(cfg, cache, one, first=cap - 1)
    _equal(one[0], want[:1], False, "bf16")


def test_refused_calls(kvc):
    cfg, cache, _ = _cache(kvc, SHAPES[0], 2, 10, seed=5)
    out = torch.empty(2, 4, 576, dtype=torch.bfloat16, device="cuda")
    for first in (-1, 7, 2 ** 31 - 3):
        with pytest.raises(kvc.KvcError):
            kvc.unpack(cfg, cache, out, first=first)
    with pytest.raises(ValueError):
        kvc.unpack(cfg, cache, out, idx=torch.zeros(2, 5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kvc.unpack(cfg, cache, out.float())
    kvc.unpack(cfg, cache, out[:, :0].contiguous())  # nothing to read


def test_long_ranges(kvc):
    """More rows than one round of the grid: the same bits as in small calls,
    some of them against the formula."""
    shape = SHAPES[0]
    cfg, cache, want = _cache(kvc, shape, 2, 30_011, seed=9)
    out = Guarded((2, 30_011, 576), torch.bfloat16, fill=float("nan"))
    kvc.unpack(cfg, cache, out.t)
    out.check()
    pick = np.r_[0:50, 15_000:15_050, 29_950:30_011]
    _equal(out.t[:, pick], want[:, pick], shape[3], shape[4])
    for first in range(0, 30_011, 5_000):
        n = min(5_000, 30_011 - first)
        part = torch.empty(2, n, 576, dtype=torch.bfloat16, device="cuda")
        kvc.unpack(cfg, cache, part, first=first)
        assert torch.equal(part, out.t[:, first:first + n])


def test_stream_and_graph(kvc):
    """On another stream, and captured and replayed with other indices and
    lengths in place."""
    cfg, cache, want = _cache(kvc, SHAPES[0], 2, 64, seed=21)
    idx = torch.randint(0, 64, (2, 10), device="cuda", dtype=torch.int32)
    out = torch.empty(2, 10, 576, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kvc.unpack(cfg, cache, out, idx=idx, stream=s)
    torch.cuda.synchronize()
    _equal(out, np.stack([want[b, idx[b].cpu().numpy()] for b in range(2)]), False, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.unpack(cfg, cache, out, idx=idx)
    idx.copy_(idx.flip(1))
    idx[0, 3] = 50
    cache.n_entries.copy_(torch.tensor([50, 64], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    i = idx.cpu().numpy()
    ref = np.stack([want[b, i[b]] for b in range(2)])
    ref[0, i[0] >= 50] = 0
    _equal(out, ref, False, "bf16")
