"""The product with one 4-bit matrix on the GPU against the float64 oracle.

Tolerance: half a step of the output type, plus n 2^-24 of sum_k |x_k w_k|: a group of 128 is 8 MMA steps of 16
products, each addition off by at most one unit (two half units, truncation) of the running sum's last place,
2 * 17 * 8 = 272; then one rounded addition per group and 16 for the joins.  SwiGLU carries both errors: the
slope of silu is below 1.1, and silu(g) u adds its own few roundings."""
import numpy as np
import pytest
import torch

from layer_inputs import as_u32, host_bits
from oracle.linear import linear, silu
from oracle.quant import dequant_nvfp4, dequant_w4g128

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def _f64(t):
    return t.double().cpu().numpy()


def _matrix(moe, fmt, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    lin = moe.quantize_linear(fmt, (torch.randn((N, K), generator=g) * 0.02).bfloat16().cuda())
    if fmt == moe.FMT_W4G128:
        return lin, dequant_w4g128(as_u32(lin.w), host_bits(lin.scale))
    return lin, dequant_nvfp4(lin.w.cpu().numpy()[None], lin.scale.cpu().numpy()[None], lin.gscale.cpu().numpy())[0]


def _check(got, x, w, swiglu, residual):
    xf = _f64(x)
    ref = linear(xf, w, swiglu, residual)
    n = 272 + w.shape[1] // 128 + 16
    e = n * U * (np.abs(xf) @ np.abs(w).T)
    if swiglu:
        h = w.shape[0] // 2
        y = xf @ w.T
        e = 1.1 * e[:, :h] * np.abs(y[:, h:]) + np.abs(silu(y[:, :h])) * e[:, h:] + 16 * U * np.abs(silu(y[:, :h]) * y[:, h:])
        e = e + 1.1 * n * n * U * U * (np.abs(xf) @ np.abs(w[:h]).T) * (np.abs(xf) @ np.abs(w[h:]).T)
    if residual is not None:
        e = e + 2 * U * (np.abs(ref) + np.abs(residual))
    dt = got.dtype
    half = 0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2
    lim = e + (half + U) * (np.abs(ref) + e) + (2.0 ** -25 if dt == torch.float16 else 1e-44)
    err = np.abs(_f64(got) - ref)
    assert (err <= lim).all(), float((err - lim).max())


# every token-tile count, both ends of each; one row, ragged and odd rows; one group to many, odd group counts
SHAPES = [(1, 1, 128), (1, 16, 256), (1, 2048, 2048), (2, 17, 384), (7, 83, 1920), (8, 200, 128), (9, 33, 2048), (16, 515, 7168),
          (17, 16, 640), (32, 100, 1152), (33, 31, 256), (64, 264, 2176), (65, 40, 512), (130, 7, 1024), (1, 5000, 128),
          (5, 2, 12288), (3, 130, 128 * 257)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("fmt", [0, 2])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_product(moe, cuda_device, T, N, K, fmt, xt, yt):
    lin, w = _matrix(moe, fmt, N, K, N + K)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(DT[xt]).cuda()
    got = moe.moe_linear_w4(x, lin, out_dtype=DT[yt])
    assert got.shape == (T, N) and got.dtype == DT[yt]
    _check(got, x, w, False, None)
    assert torch.equal(got, moe.moe_linear_w4(x, lin, out_dtype=DT[yt]))  # the same bits twice


@pytest.mark.parametrize("T,N,K", [(1, 2, 128), (3, 34, 384), (8, 4096, 2048), (20, 514, 640), (64, 48, 1024), (70, 1026, 256)])
@pytest.mark.parametrize("fmt", [0, 2])
@pytest.mark.parametrize("residual", [None, "rows", "bias"])
def test_swiglu_and_residual(moe, cuda_device, T, N, K, fmt, residual):
    lin, w = _matrix(moe, fmt, N, K, N * 3 + K)
    g = torch.Generator().manual_seed(T + N)
    x = torch.randn((T, K), generator=g).bfloat16().cuda()
    for act, M in ((moe.ACT_SWIGLU, N // 2), (moe.ACT_NONE, N)):
        res = None if residual is None else torch.randn((M,) if residual == "bias" else (T, M), generator=g).bfloat16().cuda()
        got = moe.moe_linear_w4(x, lin, act=act, residual=res)
        assert got.shape == (T, M)
        _check(got, x, w, act == moe.ACT_SWIGLU, None if res is None else _f64(res))


# More than 16 tokens and more than 30000 units of 16 rows x 128 k x 16 tokens: the tcgen05 kernel.  One pass of 32 or 64
# tokens and several, ragged ends of each; K in 1, 2, 4, 6 and 8 parts; one, two and odd numbers of groups
LARGE = [(17, 4100, 7680), (32, 15500, 2048), (33, 5411, 3968), (64, 17000, 1024), (65, 33000, 384), (130, 27001, 256), (300, 515, 7168),
         (1000, 7700, 128), (4100, 34, 5248), (64, 2048, 7680), (64, 1152, 13568)]


def _is_large(T, N, K):
    return T > 16 and -(-T // 16) * -(-N // 16) * (K // 128) > 30000


@pytest.mark.parametrize("T,N,K", LARGE)
@pytest.mark.parametrize("fmt,xt,yt", [(0, "bf16", "bf16"), (0, "f16", "f32"), (2, "bf16", "f32"), (2, "f16", "f16")])
def test_product_of_larger_ones(moe, cuda_device, T, N, K, fmt, xt, yt):
    assert _is_large(T, N, K)
    lin, w = _matrix(moe, fmt, N, K, N + K)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(DT[xt]).cuda()
    got = moe.moe_linear_w4(x, lin, out_dtype=DT[yt])
    _check(got, x, w, False, None)
    assert torch.equal(got, moe.moe_linear_w4(x, lin, out_dtype=DT[yt]))
    moe.moe_check_device_errors()


@pytest.mark.parametrize("T,N,K", [(20, 7778, 4096), (33, 5402, 3968), (200, 1026, 4736), (4100, 34, 5248)])
@pytest.mark.parametrize("fmt", [0, 2])
@pytest.mark.parametrize("residual", [None, "rows", "bias"])
def test_swiglu_and_residual_of_larger_ones(moe, cuda_device, T, N, K, fmt, residual):
    assert _is_large(T, N, K)
    test_swiglu_and_residual(moe, cuda_device, T, N, K, fmt, residual)


@pytest.mark.parametrize("T,N,K", [(40, 50, 256), (40, 6001, 3584)])  # passes of 16 tokens, and tcgen05
def test_strided_rows_of_many_tokens(moe, cuda_device, T, N, K):
    assert _is_large(T, N, K) == (N > 1000)
    lin, _ = _matrix(moe, 0, N, K, 1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn((T, K + 24), generator=g).bfloat16().cuda()[:, 8:8 + K]
    res = torch.randn((T, N), generator=g).bfloat16().cuda()
    ref = moe.moe_linear_w4(x.contiguous(), lin, residual=res)
    buf = torch.full((T + 1, N + 13), 7.0, dtype=torch.bfloat16, device="cuda")
    got = moe.moe_linear_w4(x, lin, residual=res, out=buf[:T, 5:5 + N])
    assert torch.equal(got, ref)
    assert bool((buf[:, :5] == 7).all()) and bool((buf[:, 5 + N:] == 7).all()) and bool((buf[T] == 7).all())
    assert torch.equal(moe.moe_linear_w4(x, lin, residual=res, out=res), ref)  # in place


def test_strided_rows_and_in_place_residual(moe, cuda_device):
    """Rows inside wider buffers; what lies between them is not touched."""
    T, N, K = 6, 50, 256
    lin, w = _matrix(moe, 0, N, K, 1)
    g = torch.Generator().manual_seed(2)
    wide = torch.randn((T, K + 24), generator=g).bfloat16().cuda()
    x = wide[:, 8:8 + K]
    ref = moe.moe_linear_w4(x.contiguous(), lin)
    buf = torch.full((T, N + 13), 7.0, dtype=torch.bfloat16, device="cuda")
    got = moe.moe_linear_w4(x, lin, out=buf[:, 5:5 + N])
    assert torch.equal(got, ref)
    assert bool((buf[:, :5] == 7).all()) and bool((buf[:, 5 + N:] == 7).all())
    res = torch.randn((T, N), generator=g).bfloat16().cuda()
    ref = moe.moe_linear_w4(x, lin, residual=res)
    got = moe.moe_linear_w4(x, lin, residual=res, out=res)
    assert got.data_ptr() == res.data_ptr() and torch.equal(got, ref)


def test_large_and_tiny_tokens(moe, cuda_device):
    """bf16's whole range meets the weights unscaled."""
    lin, w = _matrix(moe, 0, 40, 512, 5)
    x = torch.randn((4, 512), generator=torch.Generator().manual_seed(6))
    x[0] *= 1e30
    x[1] *= 1e-30
    x = x.bfloat16().cuda()
    _check(moe.moe_linear_w4(x, lin), x, w, False, None)


@pytest.mark.parametrize("T,N,K", [(3, 70, 256), (12, 70, 256), (40, 70, 256), (330, 1500, 2048)])
def test_infinities_and_nan_stay_in_their_token(moe, cuda_device, T, N, K):
    lin, w = _matrix(moe, 2, N, K, 7)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    ref = moe.moe_linear_w4(x, lin)
    x[1, 3], x[2, 100] = float("nan"), float("inf")
    got = moe.moe_linear_w4(x, lin)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(got[keep], ref[keep])
    assert bool(torch.isnan(got[1]).all()) and not bool(torch.isfinite(got[2]).any())


def test_zero_groups_and_extreme_codes(moe, cuda_device):
    """Rows of zeros (scale 0), and every code with every sign."""
    N, K = 24, 256
    w = torch.zeros((N, K))
    w[1] = torch.linspace(-8, 7, 16).repeat(16)
    w[2, 128:] = -1e-30
    w[3] = 1e30
    for fmt in (0, 2):
        src = w.clone()
        if fmt == 2:
            src[2:4] = 0.0  # one scale for the tensor: values of these sizes would all round to zero
        lin = moe.quantize_linear(fmt, src.bfloat16().cuda())
        dq = (dequant_w4g128(as_u32(lin.w), host_bits(lin.scale)) if fmt == 0 else
              dequant_nvfp4(lin.w.cpu().numpy()[None], lin.scale.cpu().numpy()[None], lin.gscale.cpu().numpy())[0])
        x = torch.randn((2, K), generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
        _check(moe.moe_linear_w4(x, lin, out_dtype=torch.float32), x, dq, False, None)


def test_every_nvfp4_code_and_scale(moe, cuda_device):
    """All E2M1 codes under all finite E4M3 scales, negative and subnormal ones among them."""
    K, scales = 128, [b for b in range(256) if b & 0x7F != 0x7F]
    N = (len(scales) + 7) // 8
    codes = np.tile(np.arange(16, dtype=np.uint8), N * K // 16).reshape(N, K)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    sb = np.resize(np.array(scales, np.uint8), N * 8).reshape(N, 8)
    lin = moe.Linear(moe.FMT_NVFP4, torch.from_numpy(packed).cuda(), torch.from_numpy(sb).cuda(), torch.tensor([0.37]).cuda())
    w = dequant_nvfp4(packed[None], sb[None], np.array([0.37], np.float32))[0]
    for dt in (torch.bfloat16, torch.float16):
        x = torch.randn((5, K), generator=torch.Generator().manual_seed(10)).to(dt).cuda()
        _check(moe.moe_linear_w4(x, lin, out_dtype=torch.float32), x, w, False, None)


def test_no_tokens(moe, cuda_device):
    lin, _ = _matrix(moe, 0, 10, 128, 3)
    assert moe.moe_linear_w4(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), lin).shape == (0, 10)


def test_captured_and_replayed(moe, cuda_device):
    lin, _ = _matrix(moe, 0, 96, 1024, 11)
    x = torch.randn((12, 1024), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    moe.moe_linear_w4(x, lin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = moe.moe_linear_w4(x, lin)
    x.copy_(torch.randn((12, 1024), generator=torch.Generator().manual_seed(2)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, moe.moe_linear_w4(x, lin))


def test_on_a_given_stream(moe, cuda_device):
    lin, _ = _matrix(moe, 2, 64, 512, 12)
    x = torch.randn((3, 512), generator=torch.Generator().manual_seed(3)).half().cuda()
    ref = moe.moe_linear_w4(x, lin)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = moe.moe_linear_w4(x, lin, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)


@pytest.mark.parametrize("fmt", [0, 2])
def test_layer_with_a_shared_expert(moe, cuda_device, fmt):
    """Routed experts plus a shared one added on the way, in the experts' format; the shared expert alone
    agrees with the grouped FFN of a single expert."""
    T, H, I, E, k = 9, 512, 256, 8, 2
    g = torch.Generator().manual_seed(fmt)
    rn = lambda *s: (torch.randn(s, generator=g) * 0.05).bfloat16().cuda()
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    ex = moe.quantize_experts(fmt, rn(E, 2 * I, H), rn(E, H, I))
    s13, s2 = rn(2 * I, H), rn(H, I)
    up, down = moe.quantize_linear(fmt, s13), moe.quantize_linear(fmt, s2)
    r = moe.moe_route_topk(x, rn(E, H), None, k)
    routed = moe.moe_combine(moe.moe_grouped_ffn(x, r, ex, I, E, k), r, T, k)
    h = moe.moe_linear_w4(x, up, act=moe.ACT_SWIGLU)
    out = moe.moe_linear_w4(h, down, residual=routed)
    alone = moe.moe_linear_w4(h, down)
    one = moe.quantize_experts(fmt, s13[None], s2[None])
    r1 = moe.moe_permute(torch.zeros(T, dtype=torch.int32, device="cuda"), T, 1, 1)
    ref = moe.moe_grouped_ffn(x, r1, one, I, 1, 1)
    moe.moe_check_device_errors()
    fa, fb = _f64(alone), _f64(ref)
    assert np.linalg.norm(fa - fb) <= 1e-2 * np.linalg.norm(fb) and np.abs(fa - fb).max() <= 2e-2  # the FFN's tolerance
    y32 = _f64(moe.moe_linear_w4(h, down, out_dtype=torch.float32)) + _f64(routed)
    assert (np.abs(_f64(out) - y32) <= 1.01 * 2.0 ** -8 * np.abs(y32) + 1e-6).all()
