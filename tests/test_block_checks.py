"""Refusals of the operators around the expert layer, on the CPU: the C entry points reject invalid
arguments before any CUDA call, and the binding rejects buffers of the wrong type, size or device."""
import ctypes

import pytest
import torch

import bit_mixed_precision_router_b200 as moe
from bit_mixed_precision_router_b200 import BlockNormGradsT, BlockNormT, RoutingT

OK, INVALID, SHAPE, WS, CUDA, MISALIGNED = 0, 1, 2, 3, 4, 5
A = 0x10000  # a fake, 16-byte aligned device address: validation only inspects the number
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from bit_mixed_precision_router_b200 import build
    build.build()
    return moe.load()


def test_permutation(lib):
    r = RoutingT(None, None, A, A, A, A)
    call = lambda T=4, k=2, E=8, cap=0, ids=A: lib.moe_permute_capacity(ids, T, k, E, cap, ctypes.byref(r), None)
    assert call(cap=-1) == INVALID
    assert call(T=-1) == INVALID
    assert call(E=1025) == SHAPE
    assert call(E=0) == SHAPE
    assert call(k=33) == SHAPE
    assert call(T=1 << 31) == SHAPE
    assert call(ids=None) == INVALID
    assert call(ids=A + 2) == MISALIGNED
    assert call(T=0, ids=None) == OK
    r.expert_list = None
    assert call() == INVALID


def test_rows(lib):
    r = RoutingT(None, A, None, None, A, None)
    sort = lambda x=A, dt=BF16, w=1, T=4, H=64, k=2, rows=A: lib.moe_sort_rows(x, dt, ctypes.byref(r), w, T, H, k, rows, None)
    back = lambda x=A, dt=BF16, w=1, res=None, T=4, H=64, k=2, out=A: lib.moe_unsort_rows(
        x, dt, ctypes.byref(r), w, res, T, H, k, out, None)
    for f in (sort, back):
        assert f(dt=3) == INVALID
        assert f(T=-1) == INVALID
        assert f(k=0) == INVALID
        assert f(H=0) == INVALID
        assert f(k=33) == SHAPE
        assert f(H=(1 << 20) + 1) == SHAPE
        assert f(T=1 << 30, k=4) == SHAPE
        assert f(x=None) == INVALID
        assert f(x=A + 1) == MISALIGNED
        assert f(x=A + 2, dt=F32) == MISALIGNED
        assert f(T=0, x=None) == OK
    assert back(res=A + 1) == MISALIGNED
    r.topk_w = None
    assert sort() == INVALID
    r.pair_to_row = None
    assert sort(w=0) == INVALID
    r = RoutingT(None, A, None, None, A + 2, None)
    assert lib.moe_sort_rows(A, BF16, ctypes.byref(r), 1, 4, 64, 2, A, None) == MISALIGNED
    assert lib.moe_sort_rows(A, BF16, None, 1, 4, 64, 2, A, None) == INVALID


def test_row_gradients(lib):
    r = RoutingT(None, A, None, None, A, None)
    for f in (lib.moe_sort_rows_bwd, lib.moe_unsort_rows_bwd):
        call = lambda other=A, dw=A, w=1: f(A, BF16, ctypes.byref(r), w, other, 4, 64, 2, A, dw, None)
        assert call(other=None) == INVALID      # dw without what it is a product with
        assert call(dw=None) == INVALID
        assert call(w=0) == INVALID             # no weights, no gradient of them
        assert call(dw=A + 2) == MISALIGNED
    r = RoutingT(A, A, None, None, None, None)
    call = lambda dw=A, T=4, E=8, k=2, out=A: lib.moe_route_topk_bwd(dw, ctypes.byref(r), T, E, k, out, None)
    assert call(dw=None) == INVALID
    assert call(out=A + 1) == MISALIGNED
    assert call(E=2000) == SHAPE
    assert call(k=33) == SHAPE
    assert call(T=0, dw=None) == OK
    r.topk_ids = None
    assert call() == INVALID


def _step(**kw):
    d = dict(y=A, pair_to_row=None, topk_w=None, k=0, w_post=A, gate_mode=0, gate=None, gate_sigmoid=0, alpha=1.0,
             w_next=A, eps=1e-6)
    d.update(kw)
    return BlockNormT(*[d[n] for n, _ in BlockNormT._fields_])


def test_block_norm(lib):
    def call(x=A, dt=BF16, T=4, H=64, z=A, h=A, **kw):
        s = _step(**kw)
        return lib.moe_block_norm(ctypes.byref(s), x, dt, T, H, z, h, None)

    assert call(dt=7) == INVALID
    assert call(T=-1) == INVALID
    assert call(H=0) == INVALID
    assert call(H=16385) == SHAPE
    assert call(T=(1 << 30) + 1) == SHAPE
    assert call(eps=0.0) == INVALID
    assert call(eps=float("nan")) == INVALID
    assert call(alpha=float("inf")) == INVALID
    assert call(gate_mode=3) == INVALID
    assert call(gate_mode=1) == INVALID                 # a mode without a gate
    assert call(gate=A) == INVALID                      # a gate without a mode
    assert call(gate_mode=1, gate=A + 2) == MISALIGNED
    assert call(gate_mode=2, gate=A + 1) == MISALIGNED
    assert call(y=None, z=None) == INVALID              # a norm behind a block that is not there
    assert call(y=None, w_post=None) == INVALID         # z without a block
    assert call(z=None) == INVALID
    assert call(h=None) == INVALID
    assert call(w_next=None) == INVALID
    assert call(y=None, w_post=None, w_next=None, z=None, h=None) == INVALID
    assert call(pair_to_row=A) == INVALID               # k
    assert call(pair_to_row=A, k=33) == SHAPE
    assert call(pair_to_row=A + 2, k=2) == MISALIGNED
    assert call(x=None) == INVALID
    assert call(x=A + 1) == MISALIGNED
    assert call(h=A + 2, dt=F32) == MISALIGNED
    assert call(T=0, x=None) == OK
    assert lib.moe_block_norm(None, A, BF16, 4, 64, A, A, None) == INVALID


def test_block_norm_gradient(lib):
    need = lib.moe_block_norm_bwd_workspace_bytes(4, 64)
    assert need > 0 and lib.moe_block_norm_bwd_workspace_bytes(-1, 64) == 0

    def call(z=A, dz=A, dh=A, dt=BF16, T=4, H=64, dx=A, dy=A, dgate=None, dwp=A, dwn=A, ws=A, wsb=need, **kw):
        s, g = _step(**kw), BlockNormGradsT(dx, dy, dgate, dwp, dwn)
        return lib.moe_block_norm_bwd(ctypes.byref(s), z, dz, dh, dt, T, H, ctypes.byref(g), ws, wsb, None)

    assert call(dz=None, dh=None, dwn=None) == INVALID
    assert call(z=None) == INVALID
    assert call(w_next=None) == INVALID                 # dh without its norm
    assert call(dh=None) == INVALID                     # dw_next without dh
    assert call(y=None, w_post=None, dwp=None) == INVALID  # dy without y
    assert call(dgate=A) == INVALID
    assert call(w_post=None) == INVALID                 # dw_post without w_post
    assert call(pair_to_row=A, k=2) == INVALID          # the combined y is needed
    assert call(ws=None) == WS
    assert call(wsb=need - 1) == WS
    assert call(ws=A + 8) == MISALIGNED
    assert call(dx=A + 1) == MISALIGNED
    assert call(dwp=A + 2) == MISALIGNED
    assert call(H=20000) == SHAPE


def _routing(P):
    return moe.Routing(torch.zeros(P, dtype=torch.int32), torch.zeros(P), None, None, torch.zeros(P, dtype=torch.int32), None)


def test_binding_rows():
    x, rows, r = torch.zeros((4, 64)), torch.zeros((8, 64)), _routing(8)
    with pytest.raises(ValueError, match="rows"):
        moe.moe_sort_rows(x, r, 2, rows=torch.zeros((7, 64)))
    with pytest.raises(TypeError, match="rows"):
        moe.moe_sort_rows(x, r, 2, rows=rows.half())
    with pytest.raises(TypeError, match="x"):
        moe.moe_sort_rows(x.double(), r, 2)
    with pytest.raises(ValueError, match="x"):
        moe.moe_sort_rows(x[0], r, 2)
    with pytest.raises(ValueError, match="pair_to_row"):
        moe.moe_sort_rows(x, _routing(7), 2)
    with pytest.raises(ValueError, match="residual"):
        moe.moe_unsort_rows(rows, r, 4, 2, residual=torch.zeros((4, 63)))
    with pytest.raises(ValueError, match="rows"):
        moe.moe_unsort_rows(rows, _routing(10), 5, 2)
    with pytest.raises(ValueError, match="unweighted"):
        moe.moe_sort_rows_bwd(rows, r, 4, 2, x=x, weighted=False)
    with pytest.raises(ValueError, match="dw needs rows"):
        moe.moe_unsort_rows_bwd(x, r, 2, dw=torch.zeros(8))
    with pytest.raises(ValueError, match="dw"):
        moe.moe_unsort_rows_bwd(x, r, 2, rows=rows, dw=torch.zeros(7))
    with pytest.raises(ValueError, match="k >= 1"):
        moe.moe_unsort_rows(rows, r, 4, 0)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_sort_rows(x, r, 2)
    with pytest.raises(TypeError, match="ids"):
        moe.moe_permute_capacity(torch.zeros(8, dtype=torch.int64), 4, 2, 4)
    with pytest.raises(ValueError, match="ids"):
        moe.moe_permute_capacity(torch.zeros(7, dtype=torch.int32), 4, 2, 4)
    with pytest.raises(ValueError, match="d_logits"):
        moe.moe_route_topk_bwd(torch.zeros(8), r, 4, 4, 2, d_logits=torch.zeros((4, 5)))


def test_binding_norms():
    x = torch.zeros((4, 64))
    w = torch.ones(64)
    with pytest.raises(ValueError, match="w_post"):
        moe.moe_block_norm(x, x, w_post=torch.ones(63))
    with pytest.raises(TypeError, match="w_next"):
        moe.moe_block_norm(x, x, w_next=w.half())
    with pytest.raises(ValueError, match="need y"):
        moe.moe_block_norm(x, w_post=w)
    with pytest.raises(ValueError, match="gate"):
        moe.moe_block_norm(x, x, gate=torch.zeros(3))
    with pytest.raises(ValueError, match="gate"):
        moe.moe_block_norm(x, x, gate=torch.zeros(5))
    with pytest.raises(ValueError, match="gate"):
        moe.moe_block_norm(x, x, gate=torch.zeros((4, 1)))
    with pytest.raises(TypeError, match="gate"):
        moe.moe_block_norm(x.half(), x.half(), gate=torch.zeros(4).half())
    with pytest.raises(TypeError, match="gate"):
        moe.moe_block_norm(x.half(), x.half(), gate=torch.zeros((4, 64)))
    with pytest.raises(ValueError, match="y"):
        moe.moe_block_norm(x, x, routing=_routing(8), k=2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_block_norm(x, x, w_next=w)
    with pytest.raises(ValueError, match="dz or dh"):
        moe.moe_block_norm_bwd(x.cuda() if torch.cuda.is_available() else x, y=None)


def test_linear(lib):
    w = moe.LinearT(0, A, A, None)

    def call(x=A, ldx=256, xt=BF16, T=4, N=32, K=256, act=0, res=None, ldr=0, y=A, ldy=32, yt=BF16):
        return lib.moe_linear_w4(x, ldx, xt, ctypes.byref(w), T, N, K, act, res, ldr, y, ldy, yt, None)

    assert call(xt=F32) == INVALID
    assert call(yt=3) == INVALID
    assert call(act=2) == INVALID
    assert call(T=-1) == INVALID
    assert call(N=0) == INVALID
    assert call(K=200, ldx=200) == SHAPE
    assert call(K=(1 << 20) + 128, ldx=1 << 21) == SHAPE
    assert call(N=(1 << 30) + 1, ldy=1 << 31) == SHAPE
    assert call(N=31, act=1) == SHAPE
    assert call(T=65535 * 64 + 1) == SHAPE
    assert call(ldx=248) == INVALID
    assert call(ldx=260) == MISALIGNED
    assert call(ldy=31) == INVALID
    assert call(res=A, ldr=31) == INVALID
    assert call(res=A + 1, ldr=32) == MISALIGNED
    assert call(x=A + 8) == MISALIGNED
    assert call(y=A + 2, yt=F32) == MISALIGNED
    assert call(x=None) == INVALID
    assert call(T=0, x=None) == OK
    w.fmt = 1
    assert call() == INVALID
    w.fmt = 2
    assert call() == INVALID  # NVFP4 without its per-tensor scale
    w.scale = A + 8
    w.gscale = A
    assert call() == MISALIGNED


def test_binding_linear():
    w4 = moe.Linear(moe.FMT_W4G128, torch.zeros((32, 32), dtype=torch.int32), torch.zeros((32, 2), dtype=torch.bfloat16))
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="columns"):
        moe.moe_linear_w4(x[:, :128], w4)
    with pytest.raises(TypeError, match="x"):
        moe.moe_linear_w4(x.float(), w4)
    with pytest.raises(ValueError, match="scale"):
        moe.moe_linear_w4(x, moe.Linear(0, w4.w, w4.scale[:, :1]))
    with pytest.raises(TypeError, match="w:"):
        moe.moe_linear_w4(x, moe.Linear(2, w4.w, w4.scale))
    with pytest.raises(ValueError, match="per-tensor"):
        moe.moe_linear_w4(x, moe.Linear(2, torch.zeros((32, 128), dtype=torch.uint8), torch.zeros((32, 16), dtype=torch.uint8)))
    with pytest.raises(ValueError, match="format"):
        moe.moe_linear_w4(x, moe.Linear(1, w4.w, w4.scale))
    with pytest.raises(ValueError, match="residual"):
        moe.moe_linear_w4(x, w4, residual=torch.zeros((4, 31), dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="residual"):
        moe.moe_linear_w4(x, w4, residual=torch.zeros((4, 32)))
    with pytest.raises(ValueError, match="out"):
        moe.moe_linear_w4(x, w4, act=moe.ACT_SWIGLU, out=torch.zeros((4, 32), dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="out"):
        moe.moe_linear_w4(x, w4, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="adjacent"):
        moe.moe_linear_w4(torch.zeros((256, 4), dtype=torch.bfloat16).t(), w4)
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_linear_w4(x, w4, out=torch.zeros((1, 32), dtype=torch.bfloat16).expand(4, 32))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_linear_w4(x, w4)
