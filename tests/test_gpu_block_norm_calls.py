"""Calls of the block norms that moe.h allows beside the usual one: some of the gradients only, dx in place of dz, a given stream, two
streams at once, two captured graphs with a workspace each."""
import ctypes

import pytest
import torch

from oracle import block_norm as bn
from test_gpu_block_norm import DT, EPS, C, U, _check_backward, _close, _f64, _inputs

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dy", "dgate", "dw_post", "dw_next")


def _raw(moe, d, z, want, dt, dz=None, dx=None):
    """moe_block_norm_bwd of the C library for the gradients in `want` alone; outputs start as NaN."""
    T, H = z.shape
    gate, f32 = d["gate"], torch.float32
    full = lambda shape, t: torch.full(shape, float("nan"), dtype=t, device="cuda")
    out = {"dx": full((T, H), dt) if dx is None else dx, "dy": full((T, H), dt), "dw_post": full((H,), f32), "dw_next": full((H,), f32),
           "dgate": full(gate.shape, gate.dtype)}
    p = lambda t: t.data_ptr()
    step = moe.BlockNormT(p(d["y"]), None, None, 0, p(d["w_post"]), 1 if gate.dim() == 1 else 2, p(gate), 1, 0.5, p(d["w_next"]), EPS)
    g = moe.BlockNormGradsT(*[p(out[n]) if n in want else None for n in NAMES])
    need = moe.moe_block_norm_bwd_workspace_bytes(T, H)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = moe.load().moe_block_norm_bwd(ctypes.byref(step), p(z), p(d["dz"] if dz is None else dz), p(d["dh"]), moe.DTYPES[dt], T, H,
                                       ctypes.byref(g), p(ws), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("T,H,dt", [(5, 2048, "bf16"), (300, 7168, "bf16"), (40, 1001, "f16"), (200, 9216, "bf16"), (33, 12288, "f32")])
@pytest.mark.parametrize("gate", ["token", "full"])
def test_some_gradients_only(moe, cuda_device, T, H, dt, gate):
    dt = DT[dt]
    d = _inputs(T + H, T, H, dt, gate, True, True)
    z, _ = moe.moe_block_norm(d["x"], d["y"], w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, alpha=0.5, w_next=d["w_next"], eps=EPS)
    whole = moe.BlockNormGrads(**_raw(moe, d, z, NAMES, dt))
    _check_backward(whole, d, _f64(z), _f64(d["y"]), True, 0.5, dt)
    for want in [(n,) for n in NAMES] + [("dx", "dw_next"), ("dy", "dgate"), ("dw_post", "dw_next")]:
        some = _raw(moe, d, z, want, dt)
        for n in NAMES:
            if n not in want:
                assert bool(torch.isnan(some[n]).all()), (want, n)  # not written
            some.setdefault(n, None)
        mixed = moe.BlockNormGrads(**{n: some[n] if n in want else getattr(whole, n) for n in NAMES})
        _check_backward(mixed, d, _f64(z), _f64(d["y"]), True, 0.5, dt)


@pytest.mark.parametrize("T,H,dt", [(5, 2048, "bf16"), (500, 7168, "bf16"), (400, 1001, "f16"), (320, 9216, "bf16"), (310, 12288, "f32")])
def test_dx_in_place_of_dz(moe, cuda_device, T, H, dt):
    dt = DT[dt]
    d = _inputs(T * 2 + H, T, H, dt, "token", True, True)
    z, _ = moe.moe_block_norm(d["x"], d["y"], w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, alpha=0.5, w_next=d["w_next"], eps=EPS)
    ref = _raw(moe, d, z, NAMES, dt)
    dz = d["dz"].clone()
    got = _raw(moe, d, z, NAMES, dt, dz=dz, dx=dz)
    for n in NAMES:
        assert torch.equal(got[n], ref[n]), n


def _step(moe, d, ws=None, stream=None):
    z, h = moe.moe_block_norm(d["x"], d["y"], w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, w_next=d["w_next"], stream=stream)
    g = moe.moe_block_norm_bwd(z, d["dz"], d["dh"], y=d["y"], w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, w_next=d["w_next"],
                               workspace=ws, stream=stream)
    return [z, h] + [getattr(g, n) for n in NAMES]


def test_two_streams_at_once(moe, cuda_device):
    cases = [_inputs(s, 700, 2048, torch.bfloat16, "token", True, True) for s in (1, 2)]
    ref = [_step(moe, d) for d in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [_step(moe, d, stream=s) for d, s in zip(cases, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(got, ref):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_graphs_in_turn_on_one_workspace(moe, cuda_device):
    """Graphs that share a workspace and run one after the other (at the same time they would race, as moe.h says); inputs change in
    place between the replays."""
    T, H = 500, 1024
    ws = torch.empty(moe.moe_block_norm_bwd_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    cases = [_inputs(s, T, H, torch.bfloat16, "token", True, True) for s in (3, 4)]
    graphs, outs = [], []
    for d in cases:
        _step(moe, d, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_step(moe, d, ws))
        graphs.append(g)
    for seed in (5, 6):
        for d in cases:
            e = _inputs(seed + int(d is cases[0]), T, H, torch.bfloat16, "token", True, True)
            for n in ("x", "y", "gate", "dz", "dh"):
                d[n].copy_(e[n])
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        got = [[o.clone() for o in out] for out in outs]
        for a, d in zip(got, cases):
            assert all(torch.equal(p, q) for p, q in zip(a, _step(moe, d)))


def test_back_in_place_of_its_residual(moe, cuda_device):
    T, H, k = 40, 1000, 3
    g = torch.Generator().manual_seed(1)
    rows, res = torch.randn((T * k, H), generator=g).half().cuda(), torch.randn((T, H), generator=g).half().cuda()
    row = torch.randperm(T * k, generator=g).int()
    row[::4] = -1
    r = moe.Routing(None, torch.rand(T * k, generator=g).cuda(), None, None, row.cuda(), None)
    ref = moe.moe_unsort_rows(rows, r, T, k, residual=res)
    got = moe.moe_unsort_rows(rows, r, T, k, residual=res, out=res)
    assert got.data_ptr() == res.data_ptr() and torch.equal(got, ref)
