"""The product with one 4-bit matrix at the ends of the tokens' range that moe.h states: |x| < 2^118 with W4G128, K |x| < 2^124 with
NVFP4 keep every partial sum finite, in the form for few tokens and in the one for many."""
import numpy as np
import pytest
import torch

from test_gpu_linear_forms import _check as _check_product
from test_gpu_linear_forms import _matrix, _weights

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SHAPES = [(3, 40, 3968), (14, 300, 3968), (20, 64, 3968), (33, 5411, 3968), (64, 5411, 3968)]


def _is_large(T, N, K):
    return T > 16 and -(-T // 16) * -(-N // 16) * (K // 128) > 30000


def _check(got, ref, mag, K):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= (272 + K // 128 + 16 + 1) * U * mag).all(), float((err / mag).max() / U)


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_nvfp4(moe, cuda_device, T, N, K):
    """The largest code, 6, under the largest block scale, 448: with all tokens of one sign the sum before the per-tensor scale is
    2688 K |x|, here 2^134.4; rows of alternating signs beside them."""
    assert _is_large(T, N, K) == (N > 1000)
    code = torch.full((N, K // 2), 0x77, dtype=torch.uint8, device="cuda")  # two codes of 6
    code[1::2] = 0xF7                                                       # 6, -6
    scale = torch.full((N, K // 16), 0x7E, dtype=torch.uint8, device="cuda")
    lin = moe.Linear(moe.FMT_NVFP4, code, scale, torch.tensor([2.0 ** -24], device="cuda"))
    x = torch.full((T, K), 2.0 ** 111, device="cuda")
    x[:, 0] = 2.0 ** 110
    got = moe.moe_linear_w4(x.bfloat16(), lin, out_dtype=torch.float32)
    w = 2688.0 * 2.0 ** -24
    mag = w * (K - 0.5) * 2.0 ** 111
    ref = np.where(np.arange(N) % 2 == 0, mag, -w * 2.0 ** 110)
    assert bool(torch.isfinite(got).all())
    _check(got, ref[None], mag, K)
    moe.moe_check_device_errors()


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_w4(moe, cuda_device, T, N, K):
    """The largest code, -8, under scales that leave the result below 2^122."""
    assert _is_large(T, N, K) == (N > 1000)
    word = torch.zeros((N, K // 8), dtype=torch.int32, device="cuda")  # u = 0: q = -8
    lin = moe.Linear(moe.FMT_W4G128, word, torch.full((N, K // 128), 2.0 ** -12, device="cuda").bfloat16())
    top = 2.0 ** 118 * (1 - 2.0 ** -8)  # bf16's last value below 2^118
    x = torch.full((T, K), top, device="cuda").bfloat16()
    got = moe.moe_linear_w4(x, lin, out_dtype=torch.float32)
    assert bool(torch.isfinite(got).all())
    _check(got, -8.0 * 2.0 ** -12 * top * K, 8.0 * 2.0 ** -12 * top * K, K)


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_tiny_tokens(moe, cuda_device, T, N, K):
    """Tokens far below one keep their products, although the weights meet them times 2^-8."""
    lin = _matrix(moe, moe.FMT_NVFP4, N, K, N)
    x = (torch.randn((T, K), generator=torch.Generator().manual_seed(N)) * 2.0 ** -90).bfloat16().cuda()
    _check_product(moe.moe_linear_w4(x, lin, out_dtype=torch.float32), x, _weights(lin))
