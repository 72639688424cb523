"""The norms' gradient with an eps so small that 1 / eps is past fp32's largest number: r^3 <z, w dh> stays what the formula says."""
import numpy as np
import pytest
import torch

from oracle import block_norm as bn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [64, 1024, 1001, 9216])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -80])
def test_rows_of_zeros_and_tiny_rows(moe, cuda_device, H, scale):
    """eps = 1e-40: r = 1e20.  A row of zeros has r^3 z <z, w dh> = 0; of elements near 2^-80 (squares below fp32's smallest number) the
    term is far below r w dh.  Bound: 2 C = 128 roundings of 2^-24 (as in test_gpu_block_norm.py) of the largest value."""
    eps = float(np.float32(1e-40))
    g = torch.Generator().manual_seed(H)
    rn = lambda *s: torch.randn(s, generator=g)
    T = 3
    z, y, dz, dh = rn(T, H) * scale, rn(T, H) * scale, rn(T, H), rn(T, H)
    wp, wn = 1 + 0.2 * rn(H), 1 + 0.2 * rn(H)
    got = moe.moe_block_norm_bwd(z.cuda(), dz.cuda(), dh.cuda(), y=y.cuda(), w_post=wp.cuda(), w_next=wn.cuda(), alpha=2.0 ** -60, eps=eps)
    f = lambda t: t.double().numpy()
    ref = bn.block_norm_bwd(f(z), f(dz), f(dh), f(y), f(wp), None, False, 2.0 ** -60, f(wn), eps)
    for n in ("dx", "dy", "dw_post", "dw_next"):
        v = getattr(got, n).double().cpu().numpy()
        assert np.isfinite(v).all(), n
        lim = 128 * 2.0 ** -24 * np.abs(ref[n]).max() + 1e-44
        assert (np.abs(v - ref[n]) <= lim).all(), (n, float(np.abs(v - ref[n]).max() / np.abs(ref[n]).max()))
