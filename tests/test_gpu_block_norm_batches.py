"""The forward kernels of the block norms that batches take: two, four, eight and sixteen vectors per thread, two and three CTAs
per SM, plain and over routed rows.  References and bounds are test_gpu_block_norm.py's: C = 64 roundings for a row sum and what
is formed with it; the longest chain here is 32 additions of a thread (16-bit rows of 16384) and a tree of 10."""
import numpy as np
import pytest
import torch

from test_gpu_block_norm import DT, EPS, _check_forward, _f64, _inputs

pytestmark = pytest.mark.gpu


def _form(T, H, dt, routed):
    """(elements per vector, vectors per thread, CTAs asked for per SM) of the forward kernel."""
    V = 16 // (4 if dt == "f32" else 2)
    V = V if H % V == 0 else 1
    nv = H // V
    if nv <= 1024 and (T < 296 or nv <= 64):
        return V, 1, 1
    if nv <= 1024:
        return V, 2, 3 if nv > 768 and not routed else 2
    if nv <= 4096:
        return V, 4, 1
    return V, 8 if nv <= 8192 else 16, 1


CASES = [  # T, H, type, gate, sigmoid, post, next, form
    (300, 2048, "bf16", "token", True, True, True, (8, 2, 2)), (296, 520, "f16", "full", False, True, True, (8, 2, 2)),
    (301, 7168, "bf16", "full", True, True, True, (8, 2, 3)), (300, 6152, "f16", None, False, True, True, (8, 2, 3)),
    (297, 8192, "bf16", "token", False, False, True, (8, 2, 3)), (300, 1001, "bf16", "full", True, True, True, (1, 2, 3)),
    (300, 767, "f16", "token", True, True, True, (1, 2, 2)), (300, 1023, "f32", "full", True, True, True, (1, 2, 3)),
    (310, 2048, "f32", "full", True, True, False, (4, 2, 2)), (300, 4096, "f32", "token", True, True, True, (4, 2, 3)),
    (300, 9216, "bf16", "full", True, True, True, (8, 4, 1)), (40, 16384, "f16", "token", True, True, True, (8, 4, 1)),
    (300, 8192, "f32", "full", False, True, True, (4, 4, 1)), (30, 16384, "f32", None, False, True, True, (4, 4, 1)),
    (300, 2051, "bf16", "full", True, True, True, (1, 4, 1)), (150, 5001, "bf16", "token", True, True, True, (1, 8, 1)),
    (90, 8191, "f32", "full", True, True, True, (1, 8, 1)), (150, 9001, "f16", "full", True, True, True, (1, 16, 1)),
    (20, 16383, "f32", "token", False, False, True, (1, 16, 1))]


@pytest.mark.parametrize("T,H,dt,gate,sigmoid,post,nxt,form", CASES)
def test_batches(moe, cuda_device, T, H, dt, gate, sigmoid, post, nxt, form):
    assert _form(T, H, dt, False) == form
    d = _inputs(T * 3 + H, T, H, DT[dt], gate, post, nxt)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_sigmoid=sigmoid, alpha=0.5, w_next=d["w_next"], eps=EPS)
    z, h = moe.moe_block_norm(d["x"], d["y"], **kw)
    y = _f64(d["y"])
    _check_forward(z, h, d, y, np.abs(y), sigmoid, 0.5, DT[dt])
    x = d["x"].clone()
    z2, h2 = moe.moe_block_norm(x, d["y"], z=x, **kw)  # in place, and the same bits
    assert z2.data_ptr() == x.data_ptr() and torch.equal(z, z2) and (h is None or torch.equal(h, h2))


@pytest.mark.parametrize("T,H,dt", [(300, 2048, "bf16"), (300, 8192, "f16"), (300, 1001, "f32"), (33, 9216, "bf16"), (17, 9001, "bf16")])
def test_batches_without_a_block(moe, cuda_device, T, H, dt):
    d = _inputs(T + H, T, H, DT[dt], None, False, True)
    _, h = moe.moe_block_norm(d["x"], w_next=d["w_next"], eps=EPS)
    _check_forward(None, h, d, None, None, False, 1.0, DT[dt])


@pytest.mark.parametrize("T,H,k,dt,form", [
    (300, 2048, 3, "bf16", (8, 2, 2)), (300, 7168, 8, "bf16", (8, 2, 2)), (300, 7168, 9, "f16", (8, 2, 2)), (296, 4096, 3, "f32", (4, 2, 2)),
    (300, 1001, 9, "bf16", (1, 2, 2)), (60, 9216, 3, "bf16", (8, 4, 1)), (20, 16384, 9, "f16", (8, 4, 1)), (60, 8192, 9, "f32", (4, 4, 1)),
    (60, 3001, 3, "f16", (1, 4, 1)), (30, 5001, 9, "bf16", (1, 8, 1)), (30, 5001, 3, "f32", (1, 8, 1)), (30, 9001, 3, "bf16", (1, 16, 1)),
    (9, 16383, 17, "f32", (1, 16, 1))])
def test_batches_of_routed_rows(moe, cuda_device, T, H, k, dt, form):
    """y combined from its routed rows, a third of the pairs and one whole token without any (those rows hold NaN).  Two error
    sources meet in y: the sum over the slots (k + 1 roundings, within C) and what is formed from it."""
    assert _form(T, H, dt, True) == form
    d = _inputs(T + H + k, T, H, DT[dt], "token", True, True, k)
    P = T * k
    row = torch.randperm(P, generator=torch.Generator().manual_seed(k)).int()
    row[::3] = -1
    row[2 * k:3 * k] = -1
    w = torch.rand(P, generator=torch.Generator().manual_seed(T))
    rows = d["y"].clone()
    used = torch.zeros(P, dtype=torch.bool)
    used[row[row >= 0].long()] = True
    rows[~used.cuda()] = float("nan")
    r = moe.Routing(None, w.cuda(), None, None, row.cuda(), None)
    z, h = moe.moe_block_norm(d["x"], rows, routing=r, k=k, w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, alpha=1.0,
                              w_next=d["w_next"], eps=EPS)
    src = torch.nan_to_num(rows.double())[row.clamp(min=0).long().cuda()] * (w.double() * (row >= 0)).cuda().unsqueeze(1)
    y = _f64(src.view(T, k, H).sum(1))
    ymag = _f64(src.abs().view(T, k, H).sum(1))
    ss = np.sum(y * y, 1, keepdims=True)  # an error of y also moves the mean square it is divided by
    ymag = ymag + np.abs(y) * (1 + np.sum(np.abs(y) * ymag, 1, keepdims=True) / np.where(ss > 0, ss, 1.0))
    _check_forward(z, h, d, y, ymag, True, 1.0, DT[dt])


def test_every_form_is_among_them():
    seen = {c[-1] for c in CASES} | {(8, 1, 1), (4, 1, 1), (1, 1, 1)}
    for H in range(1, 16385):
        for dt in ("bf16", "f32"):
            for T in (1, 295, 296, 4096):
                assert _form(T, H, dt, False) in seen, (T, H, dt)
