"""The block norms and their gradients on the GPU against the float64 oracle.

Tolerances, with u = 2^-24 (one fp32 rounding) and eps/2 the rounding to the element type (fp16: plus
half its smallest subnormal, 2^-25): a row sum of magnitudes is off by at most C u relative, C = 64
covering the longest chain of a thread (16) and its tree (10) for H <= 16384, the 2-ulp rsqrt and the
handful of products around it; a value built from such sums and products is off by C u times the sum of
the magnitudes of its terms; two dependent sums make 2 C, and with a gate's derivative 3 C; a sum over T tokens adds T u."""
import numpy as np
import pytest
import torch

from oracle import block_norm as bn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U, C = 2.0 ** -24, 64.0
EPS = 1e-6


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, ref, mag, n, dt, what):
    rel, tiny = 0.0, 0.0
    if dt is not None:
        rel, tiny = torch.finfo(dt).eps / 2, (2.0 ** -25 if dt == torch.float16 else 1e-44)
    err = np.abs(_f64(got) - ref)
    lim = rel * np.abs(ref) + n * U * mag + tiny
    assert (err <= lim).all(), (what, float((err - lim).max()), float(err.max()))


def _inputs(seed, T, H, dt, gate, post, nxt, k=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g).to(dt).cuda()
    d = dict(x=rn(T, H), y=rn(max(T * k, 1) if k else T, H))
    d["w_post"] = (1 + 0.2 * torch.randn(H, generator=g)).to(dt).cuda() if post else None
    d["w_next"] = (1 + 0.2 * torch.randn(H, generator=g)).to(dt).cuda() if nxt else None
    d["gate"] = {None: None, "token": torch.randn(T, generator=g).cuda(), "full": rn(T, H)}[gate]
    d["dz"], d["dh"] = rn(T, H), rn(T, H)
    return d


def _factor(d, y, sigmoid, alpha):
    """|alpha a w q|: what multiplies y on its way into z."""
    a = np.abs(bn._gate(_f64(d["gate"]), sigmoid)[0])
    if d["w_post"] is None:
        return np.abs(alpha) * a * np.ones_like(y)
    return np.abs(alpha) * a * np.abs(_f64(d["w_post"])) * bn._inv_rms(y, EPS)


def _check_forward(z, h, d, y, ymag, sigmoid, alpha, dt):
    x = _f64(d["x"])
    rz, rh = bn.block_norm(x, y, _f64(d["w_post"]), _f64(d["gate"]), sigmoid, alpha, _f64(d["w_next"]), EPS)
    zmag = np.abs(x) + (0 if y is None else _factor(d, y, sigmoid, alpha) * ymag)
    if y is not None:
        _close(z, rz, zmag, C, dt, "z")
    if rh is not None:
        r = bn._inv_rms(rz, EPS)
        spread = np.sum(np.abs(rz) * zmag, 1, keepdims=True) / np.maximum(np.sum(rz * rz, 1, keepdims=True), 1e-300)
        _close(h, rh, r * np.abs(_f64(d["w_next"])) * zmag + np.abs(rh) * (1 + spread), C, dt, "h")


def _check_backward(g, d, z, y, sigmoid, alpha, dt, use_dz=True, use_dh=True):
    T, H = z.shape
    dz, dh = (_f64(d["dz"]) if use_dz else None), (_f64(d["dh"]) if use_dh else None)
    wp, wn, gate = _f64(d["w_post"]), _f64(d["w_next"]), _f64(d["gate"])
    ref = bn.block_norm_bwd(z, dz, dh, y, wp, gate, sigmoid, alpha, wn, EPS)
    dm = np.zeros((T, H)) if dz is None else np.abs(dz)
    if dh is not None:
        r, v = bn._inv_rms(z, EPS), np.abs(wn * dh)
        dm = dm + r * v + np.abs(z) * r ** 3 * np.sum(np.abs(z) * v, 1, keepdims=True) / H
        _close(g.dw_next, ref["dw_next"], np.sum(np.abs(dh * z * r), 0), T + C, None, "dw_next")
    _close(g.dx, ref["dx"], dm, C, dt, "dx")
    if y is None:
        return
    a, da = bn._gate(gate, sigmoid)
    q = bn._inv_rms(y, EPS)
    n = np.abs(y if wp is None else y * q * wp)
    if gate is not None:
        m = np.abs(alpha * da) * dm * n
        if gate.ndim == 1:
            _close(g.dgate, ref["dgate"], np.sum(m, 1), 3 * C, None, "dgate")
        else:
            _close(g.dgate, ref["dgate"], m, 3 * C, dt, "dgate")
    am = np.abs(alpha * a) * dm
    if wp is None:
        _close(g.dy, ref["dy"], am, 2 * C, dt, "dy")
        return
    _close(g.dw_post, ref["dw_post"], np.sum(am * np.abs(y) * q, 0), T + 2 * C, None, "dw_post")
    v = np.abs(wp) * am
    _close(g.dy, ref["dy"], q * v + np.abs(y) * q ** 3 * np.sum(np.abs(y) * v, 1, keepdims=True) / H, 2 * C, dt, "dy")


CASES = [  # T, H, gate, sigmoid, post, next, alpha
    (1, 2048, "token", True, True, True, 1.0), (3, 1, None, False, True, True, 0.5), (7, 37, "full", True, True, True, 0.5),
    (300, 64, "full", False, False, True, 0.22), (5, 2047, "token", False, False, True, -1.0),
    (2, 7168, "full", True, True, True, 1.0), (9, 8200, None, False, True, False, 0.5), (3, 16384, "token", True, True, True, 1.0),
    (2, 16383, "full", True, True, True, 1.0), (160, 264, "token", True, False, False, 0.5), (4, 1028, None, False, False, True, 2.0)]


@pytest.mark.parametrize("T,H,gate,sigmoid,post,nxt,alpha", CASES)
@pytest.mark.parametrize("dt", list(DT))
def test_step_and_gradient(moe, cuda_device, T, H, gate, sigmoid, post, nxt, alpha, dt):
    dt = DT[dt]
    d = _inputs(T * 7 + H, T, H, dt, gate, post, nxt)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_sigmoid=sigmoid, alpha=alpha, w_next=d["w_next"], eps=EPS)
    alpha = float(np.float32(alpha))
    z, h = moe.moe_block_norm(d["x"], d["y"], **kw)
    assert (h is None) == (not nxt)
    y = _f64(d["y"])
    _check_forward(z, h, d, y, np.abs(y), sigmoid, alpha, dt)
    zf = _f64(z)
    g = moe.moe_block_norm_bwd(z, d["dz"], d["dh"] if nxt else None, y=d["y"], **kw)
    _check_backward(g, d, zf, y, sigmoid, alpha, dt, True, nxt)
    again = moe.moe_block_norm_bwd(z, d["dz"], d["dh"] if nxt else None, y=d["y"], **kw)
    for f in ("dx", "dy", "dgate", "dw_post", "dw_next"):  # the same bits twice
        a, b = getattr(g, f), getattr(again, f)
        assert (a is None and b is None) or torch.equal(a, b), f
    if nxt:  # without a gradient of the residual stream
        g = moe.moe_block_norm_bwd(z, None, d["dh"], y=d["y"], **kw)
        _check_backward(g, d, zf, y, sigmoid, alpha, dt, False, True)


# several rows per CTA of every form of the backward kernel: single elements (one, four, eight and sixteen to a thread),
# vectors (one, two and four), staged and read directly, with and without the elementwise gate's array
@pytest.mark.parametrize("T,H,gate,dt", [
    (2000, 101, "token", "bf16"), (1000, 203, "full", "f16"), (2001, 401, "token", "f16"), (1000, 777, "full", "bf16"),
    (470, 1501, "token", "f32"), (470, 1999, "full", "bf16"), (450, 3001, "full", "f32"), (450, 3003, "token", "bf16"),
    (400, 5001, "full", "bf16"), (400, 5001, "token", "f32"), (300, 9001, "token", "f16"), (1000, 2048, "token", "bf16"),
    (450, 4096, "full", "f16"), (450, 5504, "token", "bf16"), (450, 5504, "full", "bf16"), (450, 5504, "token", "f32"),
    (450, 7168, "token", "f32"), (320, 7168, "full", "f32"), (320, 8192, None, "f32"), (320, 9216, "token", "bf16"),
    (320, 9216, "full", "f16"), (300, 12288, "token", "f32")])
def test_gradient_of_many_rows(moe, cuda_device, T, H, gate, dt):
    dt = DT[dt]
    d = _inputs(T + H, T, H, dt, gate, True, True)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, alpha=0.5, w_next=d["w_next"], eps=EPS)
    z, _ = moe.moe_block_norm(d["x"], d["y"], **kw)
    g = moe.moe_block_norm_bwd(z, d["dz"], d["dh"], y=d["y"], **kw)
    _check_backward(g, d, _f64(z), _f64(d["y"]), True, 0.5, dt)
    again = moe.moe_block_norm_bwd(z, d["dz"], d["dh"], y=d["y"], **kw)
    for f in ("dx", "dy", "dgate", "dw_post", "dw_next"):
        a, b = getattr(g, f), getattr(again, f)
        assert (a is None and b is None) or torch.equal(a, b), f


@pytest.mark.parametrize("T,H,dt", [(1, 2048, "bf16"), (130, 513, "f32"), (6, 64, "f16"), (700, 128, "bf16")])
def test_norm_alone(moe, cuda_device, T, H, dt):
    dt = DT[dt]
    d = _inputs(T, T, H, dt, None, False, True)
    z, h = moe.moe_block_norm(d["x"], w_next=d["w_next"], eps=EPS)
    assert z is None
    _check_forward(None, h, d, None, None, False, 1.0, dt)
    g = moe.moe_block_norm_bwd(d["x"], None, d["dh"], w_next=d["w_next"], eps=EPS)
    assert g.dy is None and g.dgate is None and g.dw_post is None
    _check_backward(g, d, _f64(d["x"]), None, False, 1.0, dt, False, True)


@pytest.mark.parametrize("T,H,k,dt", [(1, 2048, 8, "bf16"), (5, 77, 3, "f16"), (17, 1024, 32, "bf16"), (40, 260, 2, "f32")])
@pytest.mark.parametrize("weighted", [True, False])
def test_with_routed_rows(moe, cuda_device, T, H, k, dt, weighted):
    """y combined on the way from its routed rows, some of them dropped (their rows hold NaN)."""
    dt = DT[dt]
    d = _inputs(T + k, T, H, dt, "token", True, True, k)
    P = T * k
    row = torch.randperm(P, generator=torch.Generator().manual_seed(k)).int()
    row[::3] = -1
    if T > 2:
        row[2 * k:3 * k] = -1  # a token without any row
    w = torch.rand(P, generator=torch.Generator().manual_seed(T))
    rows = d["y"].clone()
    free = sorted(set(range(P)) - set(row[row >= 0].tolist()))
    rows[free] = float("nan")
    r = moe.Routing(None, w.cuda() if weighted else None, None, None, row.cuda(), None)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, alpha=1.0, w_next=d["w_next"], eps=EPS)
    z, h = moe.moe_block_norm(d["x"], rows, routing=r, k=k, **kw)
    rf, wf = np.nan_to_num(_f64(rows)), (_f64(w) if weighted else np.ones(P))
    y, ymag = np.zeros((T, H)), np.zeros((T, H))
    for p in range(P):
        if row[p] >= 0:
            y[p // k] += wf[p] * rf[row[p]]
            ymag[p // k] += np.abs(wf[p] * rf[row[p]])
    # an error of y also moves the mean square it is divided by: the sum of magnitudes over the row, relative
    ss = np.sum(y * y, 1, keepdims=True)
    ymag = ymag + np.abs(y) * (1 + np.sum(np.abs(y) * ymag, 1, keepdims=True) / np.where(ss > 0, ss, 1.0))
    _check_forward(z, h, d, y, ymag, True, 1.0, dt)


def test_rows_of_zeros_and_in_place(moe, cuda_device):
    T, H = 4, 256
    x = torch.zeros((T, H), device="cuda")
    y = torch.zeros((T, H), device="cuda")
    w = torch.ones(H, device="cuda")
    z, h = moe.moe_block_norm(x, y, w_post=w, w_next=w)
    assert bool((z == 0).all()) and bool((h == 0).all())
    g = moe.moe_block_norm_bwd(z, y, torch.ones_like(x), y=y, w_post=w, w_next=w, eps=1e-6)
    assert bool(torch.isfinite(g.dx).all()) and bool((g.dw_next == 0).all())
    x, y = torch.randn((T, H), device="cuda"), torch.randn((T, H), device="cuda")
    z, h = moe.moe_block_norm(x, y, w_post=w, w_next=w)
    x2 = x.clone()
    z2, h2 = moe.moe_block_norm(x2, y, w_post=w, w_next=w, z=x2)
    assert z2.data_ptr() == x2.data_ptr() and torch.equal(z, z2) and torch.equal(h, h2)


def test_no_tokens(moe, cuda_device):
    x, w = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    z, h = moe.moe_block_norm(x, x, w_post=w, w_next=w)
    assert z.shape == h.shape == (0, 64)
    g = moe.moe_block_norm_bwd(x, x, x, y=x, w_post=w, w_next=w)
    assert bool((g.dw_post == 0).all()) and bool((g.dw_next == 0).all())


def test_infinities_stay_in_their_token(moe, cuda_device):
    T, H = 5, 128
    d = _inputs(1, T, H, torch.bfloat16, "full", True, True)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, w_next=d["w_next"])
    z, h = moe.moe_block_norm(d["x"], d["y"], **kw)
    y = d["y"].clone()
    y[2, 5] = float("inf")
    z2, h2 = moe.moe_block_norm(d["x"], y, **kw)
    keep = [0, 1, 3, 4]
    assert torch.equal(z[keep], z2[keep]) and torch.equal(h[keep], h2[keep])


def test_captured_and_replayed(moe, cuda_device):
    T, H = 200, 512
    d = _inputs(2, T, H, torch.bfloat16, "token", True, True)
    kw = dict(w_post=d["w_post"], gate=d["gate"], gate_sigmoid=True, w_next=d["w_next"])

    def step():
        z, h = moe.moe_block_norm(d["x"], d["y"], **kw)
        g = moe.moe_block_norm_bwd(z, d["dz"], d["dh"], y=d["y"], **kw)
        return z, h, g.dx, g.dy, g.dgate, g.dw_post, g.dw_next

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    e = _inputs(3, T, H, torch.bfloat16, "token", True, True)
    for n in ("x", "y", "gate", "dz", "dh"):
        d[n].copy_(e[n])
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


def test_a_step_between_two_layers(moe, cuda_device):
    """norm -> route -> grouped FFN -> combined, normed, added and normed for the next layer, against
    the same step from the combined output of moe_unsort_rows."""
    T, H, I, E, k = 12, 256, 128, 8, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    w = [(1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda() for _ in range(3)]
    ex = moe.quantize_experts(moe.FMT_W4G128, (torch.randn((E, 2 * I, H), generator=g) * 0.05).bfloat16().cuda(),
                              (torch.randn((E, H, I), generator=g) * 0.05).bfloat16().cuda())
    wr = (torch.randn((E, H), generator=g) * 0.05).bfloat16().cuda()
    _, h = moe.moe_block_norm(x, w_next=w[0])
    r = moe.moe_route_topk(h, wr, None, k)
    rows = moe.moe_grouped_ffn(h, r, ex, I, E, k)
    z, nxt = moe.moe_block_norm(x, rows, routing=r, k=k, w_post=w[1], w_next=w[2])
    y = moe.moe_unsort_rows(rows.float(), r, T, k)
    ref, rnxt = bn.block_norm(_f64(x), _f64(y), _f64(w[1]), None, False, 1.0, _f64(w[2]), 1e-6)
    # y differs by fp32 rounding only (both sums run in fp32 in slot order), far below bf16's half step
    assert (np.abs(_f64(z) - ref) <= 1.01 * 2.0 ** -8 * np.abs(ref) + 1e-5).all()
    assert (np.abs(_f64(nxt) - rnxt) <= 1.01 * 2.0 ** -8 * np.abs(rnxt) + 1e-5).all()
