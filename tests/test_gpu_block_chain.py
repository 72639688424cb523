"""The operators around the expert layer run together, as a model's stack uses them: a serving step with a
shared expert, captured and replayed; and a training step whose gradients, chained through every backward
call, agree with automatic differentiation in float64."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _rms(v, w, eps=1e-6):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w


def test_training_step_gradients(moe, cuda_device):
    """norm -> router -> sort (capacity, so some pairs are dropped) -> experts -> back -> gate, norm, add, norm.
    Every value is fp32: each call is off by at most 64 u of its terms' magnitudes (see the calls' own tests), the
    chain back to x passes seven of them, and cancellation in the norms' gradients at most doubles that:
    7 * 2 * 64 u = 5.4e-5 in relative L2."""
    T, H, E, k, cap = 48, 96, 5, 2, 14  # 96 pairs for 70 places
    g = torch.Generator().manual_seed(7)
    rn = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    leaves = {"x": rn(T, H), "w_in": 1 + 0.2 * rn(H), "w_post": 1 + 0.2 * rn(H), "w_next": 1 + 0.2 * rn(H),
              "router": 0.3 * rn(E, H), "experts": rn(E, H, H) / H ** 0.5, "gate": rn(T)}
    leaves = {n: v.float().double().requires_grad_() for n, v in leaves.items()}
    a, b = rn(T, H).float().double(), rn(T, H).float().double()

    d = {n: v.detach().float().cuda() for n, v in leaves.items()}
    _, h = moe.moe_block_norm(d["x"], w_next=d["w_in"])
    logits = h @ d["router"].t()
    top, ids = logits.topk(k, dim=1)
    r = moe.moe_permute_capacity(ids.int().reshape(-1).contiguous(), T, k, E, cap)
    r.topk_w = torch.softmax(top, 1).reshape(-1).contiguous()
    off = r.expert_offsets.tolist()
    rows = moe.moe_sort_rows(h, r, k, rows=torch.zeros((T * k, H), device="cuda"))
    out = torch.zeros_like(rows)
    for e in range(E):
        out[off[e]:off[e + 1]] = rows[off[e]:off[e + 1]] @ d["experts"][e].t()
    y = moe.moe_unsort_rows(out, r, T, k)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, alpha=0.5, w_next=d["w_next"])
    z, nxt = moe.moe_block_norm(d["x"], y, **kw)

    # and back: the loss is <z, a> + <nxt, b>
    n2 = moe.moe_block_norm_bwd(z, a.float().cuda(), b.float().cuda(), y=y, **kw)
    d_out, dw = moe.moe_unsort_rows_bwd(n2.dy, r, k, rows=out, d_rows=torch.zeros_like(out))
    d_rows = torch.zeros_like(rows)
    got = {"experts": torch.zeros_like(d["experts"])}
    for e in range(E):
        s = slice(off[e], off[e + 1])
        d_rows[s] = d_out[s] @ d["experts"][e]
        got["experts"][e] = d_out[s].t() @ rows[s]
    dh, _ = moe.moe_sort_rows_bwd(d_rows, r, T, k)
    dl = moe.moe_route_topk_bwd(dw, moe.Routing(r.topk_ids, r.topk_w, None, None, None, None), T, E, k)
    n1 = moe.moe_block_norm_bwd(d["x"], None, dh + dl @ d["router"], w_next=d["w_in"])
    got |= {"x": n2.dx + n1.dx, "w_in": n1.dw_next, "w_post": n2.dw_post, "w_next": n2.dw_next, "gate": n2.dgate,
            "router": dl.t() @ h}
    moe.moe_check_device_errors()

    # the same step in float64 on the CPU, with the same choices and the same dropped pairs
    h64 = _rms(leaves["x"], leaves["w_in"])
    idc, kept = ids.cpu(), (r.pair_to_row >= 0).cpu().view(T, k)
    assert 0 < int((~kept).sum()) < T * k
    w64 = torch.softmax(torch.gather(h64 @ leaves["router"].t(), 1, idc), 1)
    per = torch.einsum("th,eoh->teo", h64, leaves["experts"])
    per = torch.gather(per, 1, idc.unsqueeze(-1).expand(T, k, H))
    y64 = (per * (w64 * kept).unsqueeze(-1)).sum(1)
    z64 = leaves["x"] + 0.5 * torch.sigmoid(leaves["gate"]).unsqueeze(1) * _rms(y64, leaves["w_post"])
    ((z64 * a).sum() + (_rms(z64, leaves["w_next"]) * b).sum()).backward()
    for n, v in leaves.items():
        ref, err = v.grad, got[n].double().cpu() - v.grad
        assert float(err.norm()) <= 7 * 2 * 64 * U * float(ref.norm()), (n, float(err.norm() / ref.norm()))


def _serving_inputs(T, H, seed):
    return torch.randn((T, H), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("T", [1, 12, 24])
def test_serving_step_captured(moe, cuda_device, T):
    """norm -> route -> experts, shared expert beside them, combined and normed: a replay on new tokens equals the same
    step run directly, bit for bit, and equals the step put together from the separate calls."""
    H, I, E, k = 512, 256, 8, 2
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: (torch.randn(s, generator=g) * 0.05).bfloat16().cuda()
    experts = moe.quantize_experts(moe.FMT_W4G128, rn(E, 2 * I, H), rn(E, H, I))
    up, down = moe.quantize_linear(moe.FMT_W4G128, rn(2 * I, H)), moe.quantize_linear(moe.FMT_NVFP4, rn(H, I))
    w_router, w = rn(E, H), [(1 + rn(H)).contiguous() for _ in range(3)]
    x = _serving_inputs(T, H, 1)

    def step():
        _, h = moe.moe_block_norm(x, w_next=w[0])
        r = moe.moe_route_topk(h, w_router, None, k)
        rows = moe.moe_grouped_ffn(h, r, experts, I, E, k)
        s = moe.moe_linear_w4(moe.moe_linear_w4(h, up, act=moe.ACT_SWIGLU), down, residual=x)
        return moe.moe_block_norm(s, rows, routing=r, k=k, w_post=w[1], w_next=w[2]) + (rows, s, r.pair_to_row, r.topk_w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (5, 6):
        x.copy_(_serving_inputs(T, H, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for p, q in zip(got, step()):
            assert torch.equal(p, q)
    moe.moe_check_device_errors()
    z, h, rows, s, row, tw = got
    y = torch.zeros((T, H), dtype=torch.float64)
    for p in range(T * k):
        y[p // k] += tw[p].double().cpu() * rows[row[p]].double().cpu()
    ref = s.double().cpu() + _rms(y, w[1].double().cpu())
    nxt = _rms(ref, w[2].double().cpu())
    for got_, ref_ in ((z, ref), (h, nxt)):  # half a step of bf16, and fp32 arithmetic far below it
        assert bool(((got_.double().cpu() - ref_).abs() <= 1.01 * 2.0 ** -8 * ref_.abs() + 1e-5).all())
