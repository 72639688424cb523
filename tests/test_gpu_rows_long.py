"""The weights' gradients of long rows: the dot products of a pair, with a bound that follows the row's length.

A CTA of 256 threads takes the dot of a row of more than 1024 vectors: each thread adds ceil(vectors / 256) vectors of V products by
fused multiply-adds (one rounding each), then follow five exchanges in the warp and eight additions of the warps' sums."""
import numpy as np
import pytest
import torch

from oracle import rows as ro

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def _roundings(H, dt):
    V = 128 // torch.finfo(dt).bits
    V = V if H % V == 0 else 1
    assert H // V > 1024
    return -(-(H // V) // 256) * V + 5 + 8


@pytest.mark.parametrize("T,H,k", [(3, 16400, 1), (2, 16385, 2), (2, 65544, 3), (1, 131072, 6), (2, 50001, 9), (1, 1 << 20, 2)])
@pytest.mark.parametrize("dt", list(DT))
def test_dots_and_rows(moe, cuda_device, T, H, k, dt):
    dt = DT[dt]
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn((T, H), generator=g, device="cuda").to(dt)
    rows = torch.randn((T * k, H), generator=g, device="cuda").to(dt)
    w = torch.rand(T * k, generator=g, device="cuda")
    row = torch.randperm(T * k, generator=g, device="cuda").int()
    if k > 2:
        row[1] = -1
    r = moe.Routing(None, w, None, None, row, None)
    f = lambda t: t.double().cpu().numpy()
    rn = row.cpu().numpy()
    rf, xf, wf = f(rows), f(x), f(w)
    dots, mag = ro.pair_dots(rf, xf, rn, k), ro.pair_dots(np.abs(rf), np.abs(xf), rn, k)
    dx, dw = moe.moe_sort_rows_bwd(rows, r, T, k, x=x, weighted=True)
    dr, dv = moe.moe_unsort_rows_bwd(x, r, k, rows=rows, d_rows=torch.full_like(rows, float("nan")))
    for d in (dw, dv):
        assert (np.abs(f(d) - dots) <= _roundings(H, dt) * U * mag).all(), float((np.abs(f(d) - dots) / np.maximum(mag, 1e-30)).max() / U)
    half = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 1e-44
    ref = ro.unsort_rows(rf, wf, rn, T, k)
    lim = half * np.abs(ref) + (k + 1) * U * ro.unsort_rows(np.abs(rf), wf, rn, T, k) + tiny
    assert (np.abs(f(dx) - ref) <= lim).all()
    ref = ro.sort_rows(xf, wf, rn, k, np.full((T * k, H), np.nan))
    got, kept = f(dr), ~np.isnan(ref)
    assert np.isnan(got[~kept]).all()
    assert (np.abs(got[kept] - ref[kept]) <= (half + U) * np.abs(ref[kept]) + tiny).all()
