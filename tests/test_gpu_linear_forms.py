"""Every form of the product with one 4-bit matrix on mma.sync, each at several chunks of K: token tiles, warps and CTAs on
different parts of K, scales read singly and as vectors, ragged rows, partial last chunks.  Bounds as in test_gpu_linear.py (half
a step of the output, and n 2^-24 of sum_k |x_k w_k| with n = 272 + groups + 16), the reference in float64."""
import numpy as np
import pytest
import torch

from oracle.quant import dequant_nvfp4, dequant_w4g128

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _form(T, N, K, fmt):
    """(token tiles, warps on K, CTAs on K, vector scales) the library takes; None: the tcgen05 kernel."""
    up = lambda a, b: -(-a // b)
    tiles, G, passes = up(N, 16), K // 128, up(T, 16)
    if T > 16 and passes * tiles * G > 30000:
        return None
    NT = 1 if T <= 8 else 2
    blocks = lambda kw: up(tiles, 8 // kw) * passes
    kw = s = 1
    if G <= 16:
        while kw < (8 if NT == 1 else 4) and blocks(kw) < 100 and kw * 2 <= G:
            kw *= 2
        while s < 8 and blocks(kw) * s < 100 and kw * s * 4 <= G:
            s *= 2
    else:
        while kw < (8 if NT == 1 else 4) and blocks(kw) * 4 < 100:
            kw *= 2
        while s < 4 and blocks(kw) * s * 2 <= (444 if NT == 1 else 148):
            s *= 2
    return NT, kw, s, fmt == 0 and kw == 1 and G % ((8 if NT == 1 else 4) * s) == 0


def _weights(lin):
    """The matrix in float64, on the GPU."""
    N, K = lin.shape()
    if lin.fmt == 0:
        u = (lin.w.unsqueeze(-1) >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15
        return ((u.double() - 8.0).view(N, K // 128, 128) * lin.scale.double().unsqueeze(-1)).view(N, K)
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
    code = torch.stack([lin.w & 15, lin.w >> 4], -1).view(N, K // 16, 16).long()
    return (table[code] * lin.scale.view(torch.float8_e4m3fn).double().unsqueeze(-1)).view(N, K) * lin.gscale.double()


def _matrix(moe, fmt, N, K, seed):
    """Groups of very different sizes, so that a scale of another group or row shows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn((N, K), generator=g, device="cuda") * 0.02
    size = torch.exp2(torch.randint(-3, 4, (N, K // 128, 1), generator=g, device="cuda").float())
    return moe.quantize_linear(fmt, (w.view(N, K // 128, 128) * size).view(N, K).bfloat16())


def _check(got, x, w, swiglu=False, residual=None):
    xf = x.double()
    y, mag = xf @ w.t(), xf.abs() @ w.abs().t()
    n = 272 + w.shape[1] // 128 + 16
    e = n * U * mag
    if swiglu:
        h = w.shape[0] // 2
        a, b, ea, eb = y[:, :h], y[:, h:], e[:, :h], e[:, h:]
        s = a * torch.sigmoid(a)
        y, e = s * b, 1.1 * ea * b.abs() + s.abs() * eb + 1.1 * ea * eb + 16 * U * (s * b).abs()
    if residual is not None:
        y = y + residual.double()
        e = e + 2 * U * (y.abs() + residual.double().abs())
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    lim = e + (half + U) * (y.abs() + e) + (2.0 ** -25 if got.dtype == torch.float16 else 1e-44)
    err = (got.double() - y).abs()
    assert bool((err <= lim).all()), float((err - lim).max())


def test_the_reference_matrix_is_the_oracles(moe, cuda_device):
    for fmt in (0, 2):
        lin = _matrix(moe, fmt, 40, 384, 1)
        if fmt == 0:
            ref = dequant_w4g128(lin.w.cpu().numpy().view(np.uint32), lin.scale.view(torch.int16).cpu().numpy().view(np.uint16))
        else:
            ref = dequant_nvfp4(lin.w.cpu().numpy()[None], lin.scale.cpu().numpy()[None], lin.gscale.cpu().numpy())[0]
        assert np.allclose(_weights(lin).cpu().numpy(), ref, rtol=1e-15, atol=0)


SHAPES = [  # T, N, K, the form with W4 (NVFP4: the same without vector scales)
    (1, 3300, 4096, (1, 1, 4, True)), (8, 3401, 8192, (1, 1, 4, True)), (8, 4096, 7168, (1, 1, 4, False)), (8, 3301, 2432, (1, 1, 4, False)),
    (2, 14500, 4096, (1, 1, 2, True)), (3, 14400, 2432, (1, 1, 2, False)), (1, 12701, 2048, (1, 1, 1, True)),
    (5, 28501, 5120, (1, 1, 1, True)), (7, 12703, 1920, (1, 1, 1, False)), (1, 28500, 2176, (1, 1, 1, False)),
    (4, 1700, 2176, (1, 2, 4, False)), (3, 7171, 2048, (1, 2, 1, False)), (6, 1000, 4096, (1, 4, 4, False)), (7, 90, 8064, (1, 8, 4, False)),
    (16, 12701, 2048, (2, 1, 1, True)), (16, 13003, 7168, (2, 1, 1, True)), (48, 4300, 2048, (2, 1, 1, True)),
    (9, 12705, 1920, (2, 1, 1, False)), (13, 13001, 2432, (2, 1, 1, False)), (33, 4305, 2176, (2, 1, 1, False)),
    (15, 7000, 4096, (2, 1, 2, True)), (10, 7001, 2304, (2, 1, 2, False)), (9, 3300, 4096, (2, 1, 4, True)),
    (16, 3299, 7168, (2, 1, 4, False)), (12, 3201, 2432, (2, 1, 4, False)), (11, 2601, 2560, (2, 2, 2, False)),
    (14, 1700, 4224, (2, 2, 4, False)), (16, 300, 2304, (2, 4, 4, False))]


@pytest.mark.parametrize("T,N,K,form", SHAPES)
@pytest.mark.parametrize("fmt", [0, 2])
def test_product(moe, cuda_device, T, N, K, form, fmt):
    assert _form(T, N, K, fmt) == form[:3] + (form[3] and fmt == 0,)
    lin = _matrix(moe, fmt, N, K, N + K)
    w = _weights(lin)
    for xt, yt in (("bf16", "bf16"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32")):
        x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(DT[xt]).cuda()
        got = moe.moe_linear_w4(x, lin, out_dtype=DT[yt])
        _check(got, x, w)
        assert torch.equal(got, moe.moe_linear_w4(x, lin, out_dtype=DT[yt]))  # the same bits twice


@pytest.mark.parametrize("T,N,K,form", [s for s in SHAPES if s[0] in (2, 3, 8, 9, 16, 48) and s[1] < 15000])
@pytest.mark.parametrize("fmt", [0, 2])
def test_swiglu_residual_and_strides(moe, cuda_device, T, N, K, form, fmt):
    N += N % 2
    assert _form(T, N, K, fmt) == form[:3] + (form[3] and fmt == 0,)
    lin = _matrix(moe, fmt, N, K, N * 3 + K)
    w = _weights(lin)
    g = torch.Generator().manual_seed(T + N)
    wide = torch.randn((T, K + 24), generator=g).bfloat16().cuda()
    x = wide[:, 8:8 + K]
    for act, M in ((moe.ACT_SWIGLU, N // 2), (moe.ACT_NONE, N)):
        res = torch.randn((T, M), generator=g).bfloat16().cuda()
        buf = torch.full((T + 1, M + 13), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_linear_w4(x, lin, act=act, residual=res, out=buf[:T, 5:5 + M])
        _check(buf[:T, 5:5 + M], x, w, act == moe.ACT_SWIGLU, res)
        assert bool((buf[:, :5] == 7).all()) and bool((buf[:, 5 + M:] == 7).all()) and bool((buf[T] == 7).all())


def test_every_form_is_among_them():
    """Over a sweep of sizes, no form turns up that the shapes above leave out (those of a single group or of few rows are
    test_gpu_linear.py's)."""
    seen = {s[3] for s in SHAPES} | {(1, 1, 1, False), (1, 2, 1, False), (1, 4, 1, False), (1, 8, 1, False), (2, 2, 1, False),
                                     (2, 4, 1, False), (2, 4, 2, False)}
    for T in (1, 8, 9, 16, 17, 40, 64, 200):
        for N in list(range(1, 600, 37)) + list(range(600, 60000, 333)):
            for G in range(1, 70):
                form = _form(T, N, 128 * G, 0)
                assert form is None or form in seen, (T, N, G, form)
