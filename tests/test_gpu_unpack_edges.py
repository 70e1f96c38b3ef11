"""kvc_unpack of so many rows that the grid fills the device several times over
(bf16 rows then go two rounds a tile, fp32 rows one): the same bits as in calls
of a few rows, which are held to the formula elsewhere."""
import pytest
import torch

from helpers import Guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["f32", "ue4m3"])
@pytest.mark.parametrize("batch,cap,gather", [(1, 40_003, False), (3, 11_111, False), (2, 20_011, True)])
def test_long_calls(kvc, act, fmt, batch, cap, gather):
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    cfg = kvc.make_config(512, 64, 64, kvc.SCALE_F32 if fmt == "f32" else kvc.SCALE_UE4M3, 128, 64, 32,
                          8, 0.1, kvc.BF16 if act == "bf16" else kvc.F32)
    cache = kvc.Cache(cfg, batch, cap)
    g = torch.Generator(device="cuda").manual_seed(cap)
    cache.records[..., :288] = torch.randint(0, 256, (batch, cap, 288), generator=g, device="cuda",
                                             dtype=torch.uint8)
    if fmt == "f32":
        sc = torch.rand(batch, cap, 9, generator=g, device="cuda") + 0.1
        cache.records[..., 288:324] = sc.view(torch.uint8)
    else:
        cache.records[..., 288:297] = torch.randint(1, 127, (batch, cap, 9), generator=g,
                                                    device="cuda", dtype=torch.uint8)
    cache.n_entries.copy_(torch.tensor([cap, cap - 5, 0][:batch], dtype=torch.int32))
    idx = torch.randint(0, cap - 5, (batch, cap), generator=g, device="cuda",
                        dtype=torch.int32) if gather else None
    out = Guarded((batch, cap, 576), dt, fill=float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.unpack(cfg, cache, out.t, idx=idx, status=st)
    out.check()
    assert st.item() == 0
    for lo in range(0, cap, 4000):
        n = min(4000, cap - lo)
        part = torch.full((batch, n, 576), float("nan"), dtype=dt, device="cuda")
        for i in range(0, n, 250):  # small calls: one round a tile for both types
            m = min(250, n - i)
            few = torch.empty(batch, m, 576, dtype=dt, device="cuda")
            if gather:
                kvc.unpack(cfg, cache, few, idx=idx[:, lo + i:lo + i + m].contiguous())
            else:
                kvc.unpack(cfg, cache, few, first=lo + i)
            part[:, i:i + m] = few
        assert torch.equal(out.t[:, lo:lo + n], part)
    if batch == 3:
        assert not out.t[2].any() and not out.t[1, cap - 5:].any() and out.t[1, cap - 6].any()
