"""The operators around the routed-expert layer, as cases that can be timed and compared.

Three operators:
  linear     matrix-vector products with 4-bit weights (INT4 group 128, or NVFP4) for a few tokens,
             with the SwiGLU epilogue of a shared expert or a residual;
  sort/back  tokens sorted by expert and brought back with their routing weights, and the gradients
             of both and of the routing softmax ("sort", "sort_bwd", "back", "back_bwd");
  norm       the norm behind a block, its gate and residual scale, the residual add and the norm in
             front of the next block in one pass ("norm"), and its gradient ("norm_bwd").

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, by the
calls of the library; `exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # one token through a projection of the small layer: the latency of a single call
        {"name": "linear-t1-h2048", "op": "linear", "fmt": "w4", "T": 1, "N": 2048, "K": 2048, "x": "bf16", "y": "bf16",
         "act": "none", "residual": False},
        # a decode batch through the gate and up matrices of a shared expert of the large layer
        {"name": "linear-t8-swiglu-h7168", "op": "linear", "fmt": "w4", "T": 8, "N": 4096, "K": 7168, "x": "bf16",
         "y": "bf16", "act": "swiglu", "residual": False},
        # three tokens through an NVFP4 matrix with an odd number of rows, added to the residual stream
        {"name": "linear-t3-nvfp4-odd", "op": "linear", "fmt": "nvfp4", "T": 3, "N": 7171, "K": 2048, "x": "f16", "y": "f16",
         "act": "none", "residual": True},
        # sixteen tokens through an output head: the largest matrix a decode step reads, logits in 32 bits
        {"name": "linear-t16-head", "op": "linear", "fmt": "w4", "T": 16, "N": 50304, "K": 7168, "x": "bf16", "y": "f32",
         "act": "none", "residual": False},
        # a decode batch sorted by expert
        {"name": "sort-t16-h2048", "op": "sort", "T": 16, "H": 2048, "E": 64, "k": 8, "cap": 0, "drop": False,
         "dt": "bf16", "weighted": False},
        # a training batch of the large layer, each expert taking at most its capacity
        {"name": "sort-t4096-h7168-cap", "op": "sort", "T": 4096, "H": 7168, "E": 256, "k": 8, "cap": 160, "drop": False,
         "dt": "bf16", "weighted": True},
        # the gradient of the weighted sort
        {"name": "sort-bwd-t2048-h2048", "op": "sort_bwd", "T": 2048, "H": 2048, "E": 128, "k": 8, "cap": 0,
         "drop": False, "dt": "f16", "weighted": True},
        # expert outputs brought back on one of several ranks (pairs of other ranks' experts are dropped), odd row length
        {"name": "back-t777-odd-drop", "op": "back", "T": 777, "H": 2047, "E": 64, "k": 6, "cap": 0, "drop": True,
         "dt": "bf16", "weighted": True, "residual": True},
        # the gradient of the weighted return, down to the router's logits
        {"name": "back-bwd-t4096-h2048", "op": "back_bwd", "T": 4096, "H": 2048, "E": 64, "k": 8, "cap": 0,
         "drop": False, "dt": "bf16", "weighted": True},
        # one token between two blocks: its expert outputs combined, normed, added and normed again
        {"name": "norm-t1-k8-h2048", "op": "norm", "T": 1, "H": 2048, "k": 8, "dt": "bf16", "gate": "token",
         "sigmoid": True, "post": True, "next": True, "alpha": 1.0},
        # a prefill batch with an elementwise gate
        {"name": "norm-t2048-h7168-gate", "op": "norm", "T": 2048, "H": 7168, "k": 0, "dt": "bf16", "gate": "full",
         "sigmoid": True, "post": True, "next": True, "alpha": 0.5},
        # the gradient of the same step over a training batch with a gate per token
        {"name": "norm-bwd-t4096-h7168", "op": "norm_bwd", "T": 4096, "H": 7168, "dt": "bf16", "gate": "token",
         "sigmoid": True, "post": True, "next": True, "alpha": 0.5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "sort", "sort_bwd", "back", "back_bwd", "norm", "norm", "norm_bwd"])
    if op == "linear":
        K = 128 * _log(rng, 2, 96)
        act = rng.choice(["none", "none", "swiglu"])
        N = _log(rng, 64, min(60000, 50304 * 7168 // K))
        N += N % 2 if act == "swiglu" else 0
        T = _log(rng, 1, 64)
        while T * N * K > 16 * 50304 * 7168:
            T = (T + 1) // 2
        x = rng.choice(["bf16", "bf16", "f16"])
        return {"op": op, "fmt": rng.choice(["w4", "w4", "nvfp4"]), "T": T, "N": N, "K": K, "x": x,
                "y": rng.choice([x, x, "f32"]), "act": act, "residual": rng.random() < 0.3}
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    H = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        H = 64 * max(1, round(H / 64))
    if op in ("norm", "norm_bwd"):
        T = _log(rng, 1, 4096)
        post = rng.random() < 0.7
        c = {"op": op, "T": T, "H": H, "dt": dt, "gate": rng.choice(["none", "token", "full"]), "sigmoid": rng.random() < 0.5,
             "post": post, "next": rng.random() < 0.8, "alpha": rng.choice([1.0, 0.5, 0.22])}
        if op == "norm":
            c["k"] = rng.choice([0, 0, 1, 4, 8])
        return c
    E = _log(rng, 4, 256)
    k = min(E, _log(rng, 1, 12))
    T = _log(rng, 1, 4096)
    while T * k * H * SIZES[dt] > 4096 * 8 * 7168 * 2:
        T = (T + 1) // 2
    cap = rng.choice([0, 0, 1]) * max(1, round(1.25 * T * k / E))
    c = {"op": op, "T": T, "H": H, "E": E, "k": k, "cap": cap, "drop": rng.random() < 0.25, "dt": dt,
         "weighted": rng.random() < 0.7}
    if op == "back":
        c["residual"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs
def _randn(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dt)


def _routing(ids, T, k, E, cap):
    """The stable order of the kept pairs by expert: (expert_offsets, sorted_pair, pair_to_row, expert_list); the
    dropped pairs (an expert outside 0..E-1, or past the expert's capacity) follow the last row in order and have
    no row."""
    P = T * k
    dev = ids.device
    ok = (ids >= 0) & (ids < E)
    key = torch.where(ok, ids, torch.full_like(ids, E)).long()
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)
    if cap:  # the pairs past their expert's capacity join the dropped ones
        start = torch.cumsum(counts, 0) - counts
        place = torch.empty(P, dtype=torch.long, device=dev)
        place[order] = torch.arange(P, device=dev)
        ok = ok & (place - start[key] < cap)
        key = torch.where(ok, key, torch.full_like(key, E))
        order = torch.argsort(key, stable=True)
        counts = torch.bincount(key, minlength=E + 1)
    off = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(counts[:E], 0)])
    row = torch.empty(P, dtype=torch.long, device=dev)
    row[order] = torch.arange(P, device=dev)
    row = torch.where(ok, row, torch.full_like(row, -1))
    used = counts[:E] > 0
    e = torch.arange(E, device=dev)
    first = torch.argsort(torch.where(used, e, e + E))
    lst = torch.cat([used.sum()[None], torch.where(e < used.sum(), first, torch.zeros_like(e))])
    return off.int(), order.int(), row.int(), lst.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c = dict(case)
    s = {"case": c}
    if c["op"] == "linear":
        T, N, K, xt = c["T"], c["N"], c["K"], DTYPES[c["x"]]
        s["x"] = _randn(g, (T, K), xt)
        if c["fmt"] == "w4":
            # codes of normally distributed weights whose largest of 128 is coded 7: u = q + 8, eight to a word
            u = (torch.randn((N, K // 8, 8), generator=g, device="cuda") * 2.6).round_().clamp_(-8, 7).add_(8).int()
            s["scale"] = (0.0077 * (0.7 + 0.6 * torch.rand((N, K // 128), generator=g, device="cuda"))).bfloat16()
            w = u[..., 7].clone()
            for i in range(6, -1, -1):
                w = (w << 4) | u[..., i]
            s["w"] = w.contiguous()
        else:
            s["w"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            e4m3 = (32.0 + 400.0 * torch.rand((N, K // 16), generator=g, device="cuda")).to(torch.float8_e4m3fn)
            s["scale"] = e4m3.view(torch.uint8)
            s["gscale"] = torch.full((1,), 0.05 / 2688.0, device="cuda")
        M = N // 2 if c["act"] == "swiglu" else N
        s["residual"] = _randn(g, (T, M), DTYPES[c["y"]]) if c["residual"] else None
        return s
    dt, T, H = DTYPES[c["dt"]], c["T"], c["H"]
    if c["op"] in ("norm", "norm_bwd"):
        s["x"] = _randn(g, (T, H), dt)
        s["w_post"] = _randn(g, (H,), dt, 0.1).add_(1.0) if c["post"] else None
        s["w_next"] = _randn(g, (H,), dt, 0.1).add_(1.0) if c["next"] else None
        s["gate"] = {"none": None, "token": _randn(g, (T,), torch.float32), "full": _randn(g, (T, H), dt)}[c["gate"]]
        if c["op"] == "norm":
            k = c["k"]
            s["y"] = _randn(g, (T * max(k, 1), H), dt)
            if k:
                s["w"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1).reshape(-1)
                s["row"] = torch.randperm(T * k, generator=g, device="cuda").int()
        else:
            s["y"], s["dz"] = _randn(g, (T, H), dt), _randn(g, (T, H), dt)
            s["dh"] = _randn(g, (T, H), dt) if c["next"] else None
        return s
    E, k = c["E"], c["k"]
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    ids = ids.int().reshape(-1)
    if c["drop"]:  # the experts of this rank, counted from its first one
        ids = ids - E // 4
        ids = torch.where((ids >= 0) & (ids < E // 2), ids, torch.full_like(ids, -1))
    s["E"] = E // 2 if c["drop"] and E >= 2 else E
    s["ids"] = ids.contiguous()
    s["w"] = torch.softmax(top, 1).reshape(-1).contiguous()
    if c["op"] == "sort":
        s["x"] = _randn(g, (T, H), dt)
        s["rows"] = torch.zeros((T * k, H), dtype=dt, device="cuda")
        return s
    s["off"], s["pair"], s["row"], s["list"] = _routing(s["ids"], T, k, s["E"], c["cap"])
    if c["op"] in ("sort_bwd", "back"):
        s["rows"] = _randn(g, (T * k, H), dt)
        s["x"] = _randn(g, (T, H), dt)
    else:
        s["rows"] = _randn(g, (T * k, H), dt)
        s["x"] = _randn(g, (T, H), dt)
        s["drows"] = torch.zeros((T * k, H), dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _library(state)
    return _PLAIN[state["case"]["op"]](state, state["case"])


def _plain_linear(s, c):
    T, N, K = c["T"], c["N"], c["K"]
    nib = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    if c["fmt"] == "w4":
        q = ((s["w"].unsqueeze(-1) >> nib) & 15) - 8
        w = (q.view(N, K // 128, 128).float() * s["scale"].float().unsqueeze(-1)).view(N, K)
    else:
        code = torch.stack([s["w"] & 15, s["w"] >> 4], -1).view(N, K).int()
        levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
        sc = s["scale"].view(torch.float8_e4m3fn).float()
        w = (levels[code].view(N, K // 16, 16) * sc.unsqueeze(-1)).view(N, K) * s["gscale"]
    y = s["x"].float() @ w.t()
    if c["act"] == "swiglu":
        gate, up = y[:, : N // 2], y[:, N // 2:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["y"]])


def _plain_sort(s, c):
    T, k, H = c["T"], c["k"], c["H"]
    off, pair, row, lst = _routing(s["ids"], T, k, s["E"], c["cap"])
    rows = s["x"].float()[(pair // k).long()]
    if c["weighted"]:
        rows = rows * s["w"][pair.long()].unsqueeze(-1)
    kept = (torch.arange(T * k, device="cuda") < off[-1]).unsqueeze(-1)
    rows = torch.where(kept, rows, torch.zeros_like(rows)).to(DTYPES[c["dt"]])
    return {"rows": rows, "off": off, "pair": pair, "row": row}


def _back32(s, c):
    """sum_j (w) rows[row], per token in slot order, in 32 bits, and each pair's row (zero where it has none)."""
    T, k, H = c["T"], c["k"], c["H"]
    row = s["row"].long()
    has = (row >= 0).unsqueeze(-1)
    r = torch.where(has, s["rows"][row.clamp(min=0)].float(), torch.zeros((), device="cuda"))
    r = r.view(T, k, H)
    return (r * s["w"].view(T, k, 1) if c["weighted"] else r).sum(1), r


def _plain_sort_bwd(s, c):
    dx, r = _back32(s, c)
    dx = dx.to(DTYPES[c["dt"]])
    if not c["weighted"]:
        return {"dx": dx}
    return {"dx": dx, "dw": (r * s["x"].float().unsqueeze(1)).sum(-1).view(-1)}


def _plain_back(s, c):
    out, _ = _back32(s, c)
    if c["residual"]:
        out = out + s["x"].float()
    return out.to(DTYPES[c["dt"]])


def _plain_back_bwd(s, c):
    T, k, H = c["T"], c["k"], c["H"]
    dout, row = s["x"].float().unsqueeze(1), s["row"].long()
    kept = row >= 0
    d = dout.expand(T, k, H)
    d = (d * s["w"].view(T, k, 1) if c["weighted"] else d).reshape(T * k, H).to(DTYPES[c["dt"]])
    drows = torch.zeros((T * k, H), dtype=d.dtype, device="cuda")
    kept_rows = (torch.arange(T * k, device="cuda") < s["off"][-1]).unsqueeze(-1)
    drows = torch.where(kept_rows, d[s["pair"].long()], drows)
    if not c["weighted"]:
        return {"drows": drows}
    _, r = _back32(s, {**c, "weighted": False})
    dw = (r * dout).sum(-1)
    w = s["w"].view(T, k)
    dl = w * (dw - (w * dw).sum(1, keepdim=True))
    ids = s["ids"].view(T, k).long()
    ok = (ids >= 0) & (ids < s["E"])
    dlogits = torch.zeros((T, s["E"] + 1), device="cuda")
    dlogits.scatter_(1, torch.where(ok, ids, torch.full_like(ids, s["E"])), dl)
    return {"drows": drows, "dw": dw.view(-1), "dlogits": dlogits[:, : s["E"]].contiguous()}


def _plain_norm(s, c):
    dt = DTYPES[c["dt"]]
    x, y = s["x"].float(), s["y"].float()
    if c["k"]:
        y = (y[s["row"].long()] * s["w"].unsqueeze(-1)).view(c["T"], c["k"], c["H"]).sum(1)
    if c["post"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        a = s["gate"].float()
        a = 1.0 / (1.0 + torch.exp(-a)) if c["sigmoid"] else a
        y = y * (a.unsqueeze(-1) if c["gate"] == "token" else a)
    z = x + c["alpha"] * y
    if not c["next"]:
        return {"z": z.to(dt)}
    h = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s["w_next"].float()
    return {"z": z.to(dt), "h": h.to(dt)}


def _plain_norm_bwd(s, c):
    dt = DTYPES[c["dt"]]
    z, y, d = s["x"].float(), s["y"].float(), s["dz"].float()
    out = {}
    if c["next"]:
        dh, wn = s["dh"].float(), s["w_next"].float()
        r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
        v = wn * dh
        d = d + r * v - z * (r * r * r) * (z * v).mean(-1, keepdim=True)
        out["dw_next"] = (dh * z * r).double().sum(0).float()
    out["dx"] = d.to(dt)
    a = torch.ones((), device="cuda")
    if s["gate"] is not None:
        a = s["gate"].float() if c["gate"] == "full" else s["gate"].unsqueeze(-1)
        a, da = (1.0 / (1.0 + torch.exp(-a)), None) if c["sigmoid"] else (a, torch.ones_like(a))
        da = a * (1.0 - a) if da is None else da
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) if c["post"] else None
    n = y * ry * s["w_post"].float() if c["post"] else y
    if s["gate"] is not None:
        dg = c["alpha"] * da * d * n
        out["dgate"] = dg.to(dt) if c["gate"] == "full" else dg.sum(-1)
    dn = c["alpha"] * a * d
    if c["post"]:
        out["dw_post"] = (dn * y * ry).double().sum(0).float()
        v = dn * s["w_post"].float()
        dn = ry * v - y * (ry * ry * ry) * (y * v).mean(-1, keepdim=True)
    out["dy"] = dn.to(dt)
    return out


_PLAIN = {"linear": _plain_linear, "sort": _plain_sort, "sort_bwd": _plain_sort_bwd, "back": _plain_back,
          "back_bwd": _plain_back_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


def _library(s):
    import bit_mixed_precision_router_b200 as moe
    c = s["case"]
    op = c["op"]
    if op == "linear":
        w = moe.Linear(moe.FMT_W4G128 if c["fmt"] == "w4" else moe.FMT_NVFP4, s["w"], s["scale"], s.get("gscale"))
        return moe.moe_linear_w4(s["x"], w, act=moe.ACT_SWIGLU if c["act"] == "swiglu" else moe.ACT_NONE,
                                 residual=s["residual"], out_dtype=DTYPES[c["y"]])
    if op == "norm":
        routing = moe.Routing(None, s["w"], None, None, s["row"], None) if c["k"] else None
        z, h = moe.moe_block_norm(s["x"], s["y"], routing=routing, k=c["k"], w_post=s["w_post"], gate=s["gate"],
                                  gate_sigmoid=c["sigmoid"], alpha=c["alpha"], w_next=s["w_next"], eps=EPS)
        return {"z": z, "h": h} if c["next"] else {"z": z}
    if op == "norm_bwd":
        g = moe.moe_block_norm_bwd(s["x"], s["dz"], s["dh"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                                   gate_sigmoid=c["sigmoid"], alpha=c["alpha"], w_next=s["w_next"], eps=EPS)
        return {n: v for n, v in (("dx", g.dx), ("dy", g.dy), ("dgate", g.dgate), ("dw_post", g.dw_post),
                                  ("dw_next", g.dw_next)) if v is not None}
    T, k, E = c["T"], c["k"], s["E"]
    if op == "sort":
        r = moe.moe_permute_capacity(s["ids"], T, k, E, capacity=c["cap"])
        r.topk_w = s["w"]
        rows = moe.moe_sort_rows(s["x"], r, k, weighted=c["weighted"], rows=s["rows"])
        return {"rows": rows, "off": r.expert_offsets, "pair": r.sorted_pair, "row": r.pair_to_row}
    r = moe.Routing(s["ids"], s["w"], s["off"], s["pair"], s["row"], s["list"])
    if op == "sort_bwd":
        dx, dw = moe.moe_sort_rows_bwd(s["rows"], r, T, k, x=s["x"] if c["weighted"] else None, weighted=c["weighted"])
        return {"dx": dx, "dw": dw} if c["weighted"] else {"dx": dx}
    if op == "back":
        return moe.moe_unsort_rows(s["rows"], r, T, k, weighted=c["weighted"], residual=s["x"] if c["residual"] else None)
    drows, dw = moe.moe_unsort_rows_bwd(s["x"], r, k, rows=s["rows"] if c["weighted"] else None, weighted=c["weighted"],
                                        d_rows=s["drows"])
    if not c["weighted"]:
        return {"drows": drows}
    return {"drows": drows, "dw": dw, "dlogits": moe.moe_route_topk_bwd(dw, r, T, E, k)}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        M = N // 2 if c["act"] == "swiglu" else N
        b = N * K / 2 + (N * K / 64 if c["fmt"] == "w4" else N * K / 16) + T * K * 2
        return {"bytes": b + T * M * SIZES[c["y"]] * (2 if c["residual"] else 1), "flops": 2.0 * T * N * K}
    T, H, e = c["T"], c["H"], SIZES[c["dt"]]
    if c["op"] in ("norm", "norm_bwd"):
        gate = {"none": 0, "token": 4 * T, "full": T * H * e}[c["gate"]]
        weights = H * e * (int(c["post"]) + int(c["next"]))
        if c["op"] == "norm":
            k = max(c["k"], 1)
            return {"bytes": T * H * e * (2 + k + int(c["next"])) + gate + weights + 8 * T * c["k"],
                    "flops": 1.0 * T * H * (2 * k + 12)}
        return {"bytes": T * H * e * (5 + int(c["next"])) + 2 * gate + weights + 4 * H * (int(c["post"]) + int(c["next"])),
                "flops": 25.0 * T * H}
    k, E = c["k"], c["E"]
    share = 0.5 if c["drop"] else 1.0
    P = T * k * share
    if c["cap"]:
        P = min(P, E * c["cap"])
    index = T * k * 8 + (4 * T * k if c["weighted"] else 0)
    if c["op"] == "sort":
        return {"bytes": (T + P) * H * e + index + 4 * T * k, "flops": P * H if c["weighted"] else 0.0}
    if c["op"] == "sort_bwd":
        return {"bytes": ((2 if c["weighted"] else 1) * T + P) * H * e + index, "flops": (4.0 if c["weighted"] else 1.0) * P * H}
    if c["op"] == "back":
        return {"bytes": ((2 if c["residual"] else 1) * T + P) * H * e + index, "flops": 2.0 * P * H}
    rows = 2 if c["weighted"] else 1
    return {"bytes": (T + rows * P) * H * e + index + (4 * T * E * share if c["weighted"] else 0), "flops": 3.0 * P * H}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f = torch.float64
    if c["op"] == "linear":
        return _exact_linear(s, c)
    if c["op"] == "norm":
        x, y = s["x"].to(f), s["y"].to(f)
        T, H = x.shape
        if c["k"]:
            src, y = y, torch.zeros((T, H), dtype=f, device="cuda")
            for j in range(c["k"]):
                y += s["w"].to(f).view(T, -1)[:, j:j + 1] * src.index_select(0, s["row"].long().view(T, -1)[:, j])
        if c["post"]:
            y = s["w_post"].to(f) * (y / torch.sqrt(torch.linalg.vecdot(y, y).unsqueeze(1) / H + EPS))
        z = x + c["alpha"] * _exact_gate(s, c)[0] * y
        out = {"z": z}
        if c["next"]:
            out["h"] = s["w_next"].to(f) * (z / torch.sqrt(torch.linalg.vecdot(z, z).unsqueeze(1) / H + EPS))
        return out
    if c["op"] == "norm_bwd":
        return _exact_norm_bwd(s, c)
    T, k, H = c["T"], c["k"], c["H"]
    w = s["w"].to(f) if c["weighted"] else torch.ones(T * k, dtype=f, device="cuda")
    if c["op"] == "sort":
        off, pair, row, _ = _routing(s["ids"], T, k, s["E"], c["cap"])
        rows = torch.zeros((T * k, H), dtype=f, device="cuda")
        for j in range(k):  # slot j of every token
            r = row.view(T, k)[:, j].long()
            m = r >= 0
            rows[r[m]] = w.view(T, k)[m, j].unsqueeze(1) * s["x"][m].to(f)
        return {"rows": rows, "off": None, "pair": None, "row": None}
    row = s["row"].long().view(T, k)
    if c["op"] in ("sort_bwd", "back"):
        total, dw = torch.zeros((T, H), dtype=f, device="cuda"), torch.zeros((T, k), dtype=f, device="cuda")
        for j in range(k):
            m = row[:, j] >= 0
            r = s["rows"][row[m, j]].to(f)
            total[m] += w.view(T, k)[m, j].unsqueeze(1) * r
            dw[m, j] = torch.linalg.vecdot(r, s["x"][m].to(f))
        if c["op"] == "back":
            return total + s["x"].to(f) if c["residual"] else total
        return {"dx": total, "dw": dw.view(-1)} if c["weighted"] else {"dx": total}
    d = torch.zeros((T * k, H), dtype=f, device="cuda")
    dw = torch.zeros((T, k), dtype=f, device="cuda")
    for j in range(k):
        m = row[:, j] >= 0
        d[row[m, j]] = w.view(T, k)[m, j].unsqueeze(1) * s["x"][m].to(f)
        dw[m, j] = torch.linalg.vecdot(s["rows"][row[m, j]].to(f), s["x"][m].to(f))
    if not c["weighted"]:
        return {"drows": d}
    w = w.view(T, k)
    jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
    dl = torch.einsum("tij,tj->ti", jac, dw)
    dlogits = torch.zeros((T, s["E"]), dtype=f, device="cuda")
    ids = s["ids"].view(T, k).long()
    for j in range(k):
        m = (ids[:, j] >= 0) & (ids[:, j] < s["E"])
        dlogits[m, ids[m, j]] += dl[m, j]
    return {"drows": d, "dw": dw.reshape(-1), "dlogits": dlogits}


def _exact_linear(s, c):
    f = torch.float64
    T, N, K = c["T"], c["N"], c["K"]
    x, y = s["x"].to(f), torch.empty((T, N), dtype=f, device="cuda")
    step = max(1, (1 << 26) // K)
    e2m1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    table = torch.tensor(e2m1 + [-v for v in e2m1], dtype=f, device="cuda")
    for n in range(0, N, step):
        p = s["w"][n:n + step]
        w = torch.empty((p.shape[0], K), dtype=f, device="cuda")
        if c["fmt"] == "w4":
            for i in range(8):
                w[:, i::8] = (torch.bitwise_right_shift(p, 4 * i) & 15).to(f) - 8.0
            w *= torch.repeat_interleave(s["scale"][n:n + step].to(f), 128, dim=1)
        else:
            w[:, 0::2] = table[(p & 15).long()]
            w[:, 1::2] = table[(p >> 4).long()]
            sc = s["scale"][n:n + step].view(torch.float8_e4m3fn).to(f)
            w *= torch.repeat_interleave(sc, 16, dim=1) * s["gscale"].to(f)
        y[:, n:n + step] = torch.matmul(x, w.t())
    if c["act"] == "swiglu":
        y = y[:, : N // 2] * torch.sigmoid(y[:, : N // 2]) * y[:, N // 2:]
    return y if s["residual"] is None else y + s["residual"].to(f)


def _exact_gate(s, c):
    """(a(gate), a'(gate)) broadcast over the rows."""
    if s["gate"] is None:
        one = torch.ones((), dtype=torch.float64, device="cuda")
        return one, one
    v = s["gate"].double()
    v = v[:, None] if c["gate"] == "token" else v
    if not c["sigmoid"]:
        return v, torch.ones_like(v)
    a = torch.sigmoid(v)
    return a, a * (1 - a)


def _exact_norm_bwd(s, c):
    f = torch.float64
    H = c["H"]
    z, y, dx = s["x"].to(f), s["y"].to(f), s["dz"].to(f)
    out = {}
    if c["next"]:
        rms = torch.sqrt(torch.linalg.vecdot(z, z).unsqueeze(1) / H + EPS)
        unit = z / rms
        out["dw_next"] = torch.einsum("th,th->h", s["dh"].to(f), unit)
        u = s["dh"].to(f) * s["w_next"].to(f)
        dx = dx + (u - unit * (torch.linalg.vecdot(unit, u).unsqueeze(1) / H)) / rms
    out["dx"] = dx
    a, da = _exact_gate(s, c)
    unit, w = y, None
    if c["post"]:
        rms = torch.sqrt(torch.linalg.vecdot(y, y).unsqueeze(1) / H + EPS)
        unit, w = y / rms, s["w_post"].to(f)
    if s["gate"] is not None:
        d = c["alpha"] * da * dx * (unit if w is None else unit * w)
        out["dgate"] = d.sum(1) if c["gate"] == "token" else d
    d = c["alpha"] * a * dx
    if c["post"]:
        out["dw_post"] = torch.einsum("th,th->h", d, unit)
        d = d * w
        d = (d - unit * (torch.linalg.vecdot(unit, d).unsqueeze(1) / H)) / rms
    out["dy"] = d
    return out
