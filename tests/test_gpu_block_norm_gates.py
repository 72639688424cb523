"""The sigmoid gates of the block norms far from zero, where e^v is small: against float64, with bounds from the arithmetic.

With u = 2^-24 (one fp32 rounding): e = expf(-|v|) is off by at most 2 units in the last place (4 u), s = 1 / (1 + e) by the
rounding of the sum (u), a quotient of 2 units (4 u) and e's own error; e s adds a rounding, alpha a another: 4 + 1 + 4 + 4 + 2 = 15 u,
16 taken.  Below 2^-126 a value is rounded to a multiple of 2^-149, e and e s half a unit each.

On its way into a z of 16 bits an elementwise gate's exponential may be off by 2^-22 and 1.3 |v| u (the product v log2(e) is rounded,
and so is the constant: 1.22 u of an exponent of |v| / ln 2), and below 2^-126 the sigmoid may be 0, as moe.h says."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U, LAST = 2.0 ** -24, 2.0 ** -149


def _f64(t):
    return t.double().cpu().numpy()


def _sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))  # float64: no overflow for |v| < 700


def _values(dt, n, lo=-103.0, hi=20.0):
    return torch.linspace(lo, hi, n).to(dt).cuda()


@pytest.mark.parametrize("alpha", [1.0, 2.0 ** 96])
@pytest.mark.parametrize("per", ["token", "element"])
@pytest.mark.parametrize("dt", list(DT))
def test_forward(moe, cuda_device, dt, per, alpha):
    """z = alpha sigmoid(gate), with x = 0 and y = 1."""
    T, H, dt = (512, 64, DT[dt]) if per == "token" else (8, 1024, DT[dt])
    hi = 20.0 if dt != torch.float16 or alpha == 1.0 else -65.0  # 2^96 e^-65 is below 2^3, far from fp16's largest
    gate = _values(torch.float32, T, hi=hi) if per == "token" else _values(dt, T * H, hi=hi).view(T, H)
    x, y = torch.zeros((T, H), dtype=dt, device="cuda"), torch.ones((T, H), dtype=dt, device="cuda")
    z, _ = moe.moe_block_norm(x, y, gate=gate, gate_sigmoid=True, alpha=alpha)
    g = _f64(gate)
    ref = alpha * _sigmoid(g[:, None] if g.ndim == 1 else g) * np.ones((T, H))
    half = torch.finfo(dt).eps / 2 if dt != torch.float32 else 0.0
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: LAST / 2}[dt]  # half the smallest step
    lim = 16 * U * ref + 1.5 * LAST * alpha
    if per == "element" and dt != torch.float32:
        lim = (16 + 1.3 * np.abs(g)) * U * ref + 2.0 ** -126 * alpha
    lim = lim + half * (ref + lim) + tiny
    err = np.abs(_f64(z) - ref)
    assert (err <= lim).all(), (float((err / lim).max()), float(g.reshape(-1)[np.argmax((err / lim).max(1) if g.ndim == 1 else err / lim)]))


@pytest.mark.parametrize("H", [1024, 7168, 1001])
@pytest.mark.parametrize("dt", list(DT))
def test_weight_gradient_of_an_elementwise_gate(moe, cuda_device, dt, H):
    """dw_post = alpha a dz y q in fp32, whatever the gate's type: with one token, y = dz = 1 and q = 1 / sqrt(1 + eps) the error is
    a's (16 u), q's (the mean of H ones is exact; eps rounded and added, rsqrt off by 2 units: 6 u) and four products."""
    dt = DT[dt]
    gate = _values(dt, H, lo=-80.0).view(1, H)
    one = torch.ones((1, H), dtype=dt, device="cuda")
    g = moe.moe_block_norm_bwd(one, one, None, y=one, w_post=one[0], gate=gate, gate_sigmoid=True, alpha=0.5, eps=1e-6)
    ref = 0.5 * _sigmoid(_f64(gate))[0] / np.sqrt(1 + 1e-6)
    err = np.abs(_f64(g.dw_post) - ref)
    assert (err <= 26 * U * ref).all(), float((err / ref).max() / U)


@pytest.mark.parametrize("dt", list(DT))
def test_infinite_gates(moe, cuda_device, dt):
    dt = DT[dt]
    inf = float("inf")
    gate = torch.tensor([[inf, -inf, 0.0, 1.0]], dtype=dt).cuda()
    one = torch.ones((1, 4), dtype=dt, device="cuda")
    z, _ = moe.moe_block_norm(torch.zeros_like(one), one, gate=gate, gate_sigmoid=True)
    assert z[0, :3].tolist() == [1.0, 0.0, 0.5]
    z, _ = moe.moe_block_norm(torch.zeros_like(one).expand(2, 4).contiguous(), one.expand(2, 4).contiguous(), gate_sigmoid=True,
                              gate=torch.tensor([inf, -inf]).cuda())
    assert bool((z[0] == 1).all()) and bool((z[1] == 0).all())
