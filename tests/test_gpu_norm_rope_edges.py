"""kvc_norm_rope at the ends of fp32's range: rows without a finite factor are
flagged, rows next to them are not and hold the formula's values.  The bound is
that of the ordinary rows (128 x 2^-24 of |x| + |y| of a pair, half a step of
fp32): the factor is a square root and a quotient of normal numbers there."""
import numpy as np
import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu


def _run(kvc, k, eps, norm):
    cfg = kvc.make_config(64, 16, 8, kvc.SCALE_UE4M3, 128, 64, 128, 8, 0.05, kvc.F32)
    n = k.shape[0]
    out, st = torch.empty_like(k), torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freq = torch.linspace(1, 0.01, 8, device="cuda")
    kvc.norm_rope(cfg, None, k, pos, freq, None, out, k_norm=norm, eps=eps, status=st)
    return out, int(st.item()), pos, freq


def _rows(scale, n=5):
    g = torch.Generator(device="cuda").manual_seed(3)
    return scale * torch.randn(n, 80, generator=g, device="cuda")


@pytest.mark.parametrize("norm", [1, 2])
@pytest.mark.parametrize("scale,eps", [(1e18, 0.0), (1e18, 1e-6), (1e-15, 0.0), (1e-12, 1e-30),
                                       (1e-30, 1e-6), (0.0, 1e-6), (0.0, 1e-38)])
def test_rows_with_a_factor(kvc, norm, scale, eps):
    """Squares up to 10^38 and down to 10^-30; smaller ones under an eps."""
    k = _rows(scale)
    out, st, pos, freq = _run(kvc, k, eps, norm)
    assert st == 0
    ref, mag = plain64.norm_rope(k.double().cpu().numpy(), None,
                                 {kvc.NORM_LATENT: 64, kvc.NORM_ROW: 80}[norm], 64,
                                 pos.cpu().numpy(), freq.cpu().numpy(), False, float(np.float32(eps)))
    got = out.double().cpu().numpy()
    # (an eps of 1e-38 is normal; products below 2^-126 round to multiples of 2^-149)
    tol = 2.0 ** -24 * np.abs(ref) + 128 * 2.0 ** -24 * mag + 2.0 ** -149
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("norm", [1, 2])
@pytest.mark.parametrize("row,eps", [(0.0, 0.0), (1e-24, 0.0), (1e-40, 0.0), (3e19, 1e-6), (3e38, 0.0),
                                     (float("inf"), 1e-6), (float("nan"), 1e-6)])
def test_rows_without_one(kvc, norm, row, eps):
    """Squares that vanish with nothing beside them, or overflow: flagged, and
    the other rows as ever."""
    k = _rows(1.0)
    want, st, _, _ = _run(kvc, k, eps, norm)
    assert st == 0
    k[2] = row
    out, st, _, _ = _run(kvc, k, eps, norm)
    assert st == kvc.DEV_NONFINITE
    keep = [0, 1, 3, 4]
    assert torch.equal(out[keep], want[keep])
