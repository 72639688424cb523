"""Buffers of more than 2^31 elements: what stands at their end equals a call on the end alone (the last rows' arithmetic does not
depend on how many rows come before them, as long as the same kernel takes both)."""
import pytest
import torch

from test_gpu_linear_forms import _check, _matrix, _weights

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _rand(g, *shape):
    return torch.empty(shape, dtype=BF16, device="cuda").normal_(generator=g)


@pytest.mark.parametrize("T,H", [(270001, 8192), (1 << 21, 1025)])  # wide vectors, single elements
def test_norms(moe, cuda_device, T, H):
    assert T * H > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(H)
    x, y, w, gate = _rand(g, T, H), _rand(g, T, H), _rand(g, H), torch.randn(T, generator=g, device="cuda")
    end = slice(T - 4096, T)
    kw = dict(w_post=w, gate_sigmoid=True, alpha=0.5, w_next=w)
    z, h = moe.moe_block_norm(x, y, gate=gate, **kw)
    ze, he = moe.moe_block_norm(x[end], y[end], gate=gate[end], **kw)
    assert torch.equal(z[end], ze) and torch.equal(h[end], he)
    b = moe.moe_block_norm_bwd(z, x, h, y=y, gate=gate, **kw)
    e = moe.moe_block_norm_bwd(ze, x[end], he, y=y[end], gate=gate[end], **kw)
    for n in ("dx", "dy", "dgate"):
        assert torch.equal(getattr(b, n)[end], getattr(e, n)), n
    assert bool(torch.isfinite(b.dw_post).all()) and bool(torch.isfinite(b.dw_next).all())


def test_norm_of_routed_rows(moe, cuda_device):
    T, H, k = 45001, 8192, 6
    assert T * k * H > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x, rows, w = _rand(g, T, H), _rand(g, T * k, H), _rand(g, H)
    row = torch.arange(T * k, device="cuda", dtype=torch.int32)
    tw = torch.rand(T * k, generator=g, device="cuda")
    z, h = moe.moe_block_norm(x, rows, routing=moe.Routing(None, tw, None, None, row, None), k=k, w_post=w, w_next=w)
    n = 300
    r = moe.Routing(None, tw[-n * k:].contiguous(), None, None, row[:n * k].contiguous(), None)
    ze, he = moe.moe_block_norm(x[-n:], rows[-n * k:], routing=r, k=k, w_post=w, w_next=w)
    assert torch.equal(z[-n:], ze) and torch.equal(h[-n:], he)


@pytest.mark.parametrize("T,H", [(45001, 8192), (360001, 1021)])
def test_rows(moe, cuda_device, T, H):
    k, n = 6, 200
    assert T * k * H > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(2)
    x, rows = _rand(g, T, H), _rand(g, T * k, H)
    row = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k).flip(1).reshape(-1).contiguous()
    tw = torch.rand(T * k, generator=g, device="cuda")
    full = moe.Routing(None, tw, None, None, row, None)
    part = moe.Routing(None, tw[-n * k:].contiguous(), None, None, row[:n * k].contiguous(), None)
    xe, re = x[-n:], rows[-n * k:]
    assert torch.equal(moe.moe_unsort_rows(rows, full, T, k, residual=x)[-n:], moe.moe_unsort_rows(re, part, n, k, residual=xe))
    assert torch.equal(moe.moe_sort_rows(x, full, k, True)[-n * k:], moe.moe_sort_rows(xe, part, k, True))
    a, b = moe.moe_sort_rows_bwd(rows, full, T, k, x=x, weighted=True), moe.moe_sort_rows_bwd(re, part, n, k, x=xe, weighted=True)
    assert torch.equal(a[0][-n:], b[0]) and torch.equal(a[1][-n * k:], b[1])
    a, b = moe.moe_unsort_rows_bwd(x, full, k, rows=rows), moe.moe_unsort_rows_bwd(xe, part, k, rows=re)
    assert torch.equal(a[0][-n * k:], b[0]) and torch.equal(a[1][-n * k:], b[1])


@pytest.mark.parametrize("T", [70, 16])  # the tcgen05 form, and the other: outputs or weights past 2^31
@pytest.mark.parametrize("fmt", [0, 2])
def test_linear(moe, cuda_device, T, fmt):
    N, K = (31000007, 128) if T > 16 else (2100003, 2176)
    assert T * N > 1 << 31 or N * K > 1 << 32
    n = 257
    tail = _matrix(moe, fmt, n, K, 3)  # the last rows of a matrix that repeats them
    reps = -(-N // n)
    rep = lambda t: t.repeat(reps, 1)[-N:].clone()  # a copy starts on 16 bytes, the slice need not
    big = moe.Linear(fmt, rep(tail.w), rep(tail.scale), tail.gscale)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    y = moe.moe_linear_w4(x, big)
    _check(y[:, -n:].contiguous(), x, _weights(tail))
    mid = N // n // 2 * n  # the same rows in the middle of the matrix
    assert torch.equal(y[:, N - mid - n:N - mid], y[:, N - n:])
    moe.moe_check_device_errors()
