"""The row operators on the GPU against their float64 oracle: the permutation with dropped pairs
(exact), sorting and bringing back with weights, the gradients, and the whole path around the
grouped FFN.

Tolerances: a product rounded once to the element type is off by half a step, eps/2 relative (plus
half of fp16's smallest subnormal, 2^-25); an fp32 sum of n terms adds n 2^-24 times the sum of the
terms' magnitudes; the dots' longest chain is 8 * ceil(H / 2048) sequential additions per thread and
a tree of 10, so 64 covers H <= 8192."""
import numpy as np
import pytest
import torch

from oracle import rows as ro

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def _half_step(dt):
    return torch.finfo(dt).eps / 2, (2.0 ** -25 if dt == torch.float16 else 1e-44)


def _close(got, ref, mag, n, dt, what):
    rel, tiny = _half_step(dt) if dt is not None else (0.0, 0.0)
    err = np.abs(got.double().cpu().numpy() - ref)
    lim = rel * np.abs(ref) + n * U * mag + tiny
    assert (err <= lim).all(), (what, float((err - lim).max()))


def _case(seed, T, H, E, k, dt, lo=0, hi=None):
    """Random rows of the type, weights, ids in lo..hi-1 (distinct per token where there are enough)."""
    rng = np.random.default_rng(seed)
    hi = E if hi is None else hi
    if hi - lo >= k:
        ids = np.stack([rng.permutation(np.arange(lo, hi))[:k] for _ in range(T)]) if T else np.zeros((0, k))
    else:
        ids = rng.integers(lo, hi, (T, k))
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).to(dt).cuda()
    rows = torch.randn((max(T * k, 1), H), generator=g).to(dt).cuda()
    w = torch.rand(max(T * k, 1), generator=g).cuda()
    return torch.from_numpy(ids.astype(np.int32).reshape(-1)).cuda(), x, rows, w


def _f64(t):
    return t.double().cpu().numpy()


def _sentinel(moe, P, E):
    i32 = dict(dtype=torch.int32, device="cuda")
    return moe.Routing(None, None, torch.full((E + 1,), -77, **i32), torch.full((max(P, 1),), -77, **i32),
                       torch.full((max(P, 1),), -77, **i32), torch.full((E + 1,), -77, **i32))


# small, one bin, many bins, several CTAs, odd counts, no pair kept, all pairs of one expert
@pytest.mark.parametrize("T,k,E,cap,lo,hi", [
    (1, 1, 1, 0, 0, 1), (16, 8, 64, 0, 0, 64), (7, 3, 1024, 0, 0, 1024), (129, 2, 4, 3, -2, 6), (33, 32, 40, 5, 0, 40),
    (5, 4, 3, 0, 7, 9), (64, 2, 1, 7, 0, 1), (1500, 8, 64, 100, -8, 70), (4099, 2, 1024, 0, 0, 1024),
    (2049, 8, 256, 80, 0, 256), (900, 5, 3, 1, 0, 3), (4096, 1, 8, 0, 0, 1)])
def test_permutation(moe, cuda_device, T, k, E, cap, lo, hi):
    rng = np.random.default_rng(T)
    ids = rng.integers(lo, hi, T * k).astype(np.int32)
    r = moe.moe_permute_capacity(torch.from_numpy(ids).cuda(), T, k, E, cap, out=_sentinel(moe, T * k, E))
    off, pair, row, lst = ro.permute_capacity(ids, E, cap)
    assert np.array_equal(r.expert_offsets.cpu().numpy(), off)
    assert np.array_equal(r.sorted_pair.cpu().numpy(), pair)
    assert np.array_equal(r.pair_to_row.cpu().numpy(), row)
    n = 1 + lst[0]
    assert np.array_equal(r.expert_list.cpu().numpy()[:n], lst[:n])


def test_permutation_without_drops_equals_moe_permute(moe, cuda_device):
    T, k, E = 600, 4, 96
    ids = torch.randint(0, E, (T * k,), dtype=torch.int32, device="cuda")
    a, b = moe.moe_permute(ids, T, k, E), moe.moe_permute_capacity(ids, T, k, E)
    n = 1 + int(a.expert_list[0])
    for f in ("expert_offsets", "sorted_pair", "pair_to_row"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f
    assert torch.equal(a.expert_list[:n], b.expert_list[:n])


SHAPES = [  # T, H, E, k, capacity, first id, end of ids
    (1, 2048, 8, 1, 0, 0, 8), (3, 1, 4, 2, 0, 0, 4), (16, 2048, 64, 8, 0, 0, 64), (5, 37, 6, 3, 2, -2, 8),
    (9, 257, 40, 32, 0, 0, 40), (40, 264, 12, 9, 10, -3, 12), (2, 7168, 256, 8, 0, 0, 256), (6, 64, 4, 2, 0, 5, 9),
    (31, 4104, 16, 4, 3, 0, 16),
    # several vectors or single elements to a thread, and several rounds of them
    (5, 2047, 8, 4, 0, 0, 8), (4, 9001, 4, 2, 0, 0, 4), (3, 16400, 4, 1, 0, 0, 4), (6, 8200, 6, 3, 0, -1, 6), (3, 8191, 16, 8, 0, -4, 16),
    (7, 5000, 9, 6, 0, 0, 9), (9, 1024, 4, 2, 3, 0, 4), (4, 4099, 20, 13, 0, 0, 20)]


@pytest.mark.parametrize("T,H,E,k,cap,lo,hi", SHAPES)
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("weighted", [False, True])
def test_rows_and_gradients(moe, cuda_device, T, H, E, k, cap, lo, hi, dt, weighted):
    dt = DT[dt]
    ids, x, rows, w = _case(T + H, T, H, E, k, dt, lo, hi)
    r = moe.moe_permute_capacity(ids, T, k, E, cap)
    r.topk_w = w
    row = r.pair_to_row.cpu().numpy()
    wn = _f64(w)[:T * k] if weighted else None
    mag_w = np.ones(T * k) if wn is None else np.abs(wn)
    free = sorted(set(range(T * k)) - set(row[row >= 0]))

    # to the rows; the rows of no pair keep what they held (NaN), and are never read
    held = torch.full_like(rows, float("nan"))
    got = moe.moe_sort_rows(x, r, k, weighted=weighted, rows=held)
    ref = ro.sort_rows(_f64(x), wn, row, k, np.zeros((T * k, H)))
    used = row[row >= 0]
    _close(got[used], ref[used], np.abs(ref[used]), 1, dt, "sort")
    assert bool(torch.isnan(got[free]).all())
    rows = rows.clone()
    rows[free] = float("nan")

    # and back, without and with a residual
    rf = np.nan_to_num(_f64(rows))
    mag = ro.unsort_rows(np.abs(rf), mag_w, row, T, k)
    got = moe.moe_unsort_rows(rows, r, T, k, weighted=weighted)
    _close(got, ro.unsort_rows(rf, wn, row, T, k), mag, k + 1, dt, "back")
    got = moe.moe_unsort_rows(rows, r, T, k, weighted=weighted, residual=x)
    _close(got, ro.unsort_rows(rf, wn, row, T, k, _f64(x)), mag + np.abs(_f64(x)), k + 2, dt, "back + residual")

    # gradients: of the sort (rows as the gradient of the rows), of the way back (x as that of the output)
    dots = ro.pair_dots(rf, _f64(x), row, k)
    dmag = ro.pair_dots(np.abs(rf), np.abs(_f64(x)), row, k)
    dx, dw = moe.moe_sort_rows_bwd(rows, r, T, k, x=x if weighted else None, weighted=weighted)
    _close(dx, ro.unsort_rows(rf, wn, row, T, k), mag, k + 1, dt, "d sort")
    held = torch.full_like(rows, float("nan"))
    dr, dv = moe.moe_unsort_rows_bwd(x, r, k, rows=rows if weighted else None, weighted=weighted, d_rows=held)
    _close(dr[used], ref[used], np.abs(ref[used]), 1, dt, "d back")
    assert bool(torch.isnan(dr[free]).all())
    if weighted:
        for d in (dw, dv):
            _close(d, dots, dmag, 64, None, "dw")
            assert bool((d.cpu()[row < 0] == 0).all())
    else:
        assert dw is None and dv is None
    if weighted:  # weights that are constants: no dw
        dx2, none = moe.moe_sort_rows_bwd(rows, r, T, k, weighted=True)
        assert none is None and torch.equal(dx2, dx)


def test_back_equals_combine_bit_for_bit(moe, cuda_device):
    T, H, E, k = 50, 256, 16, 4
    ids, x, rows, w = _case(5, T, H, E, k, torch.bfloat16)
    r = moe.moe_permute(ids, T, k, E)
    r.topk_w, r.topk_ids = w, ids
    a = moe.moe_combine(rows, r, T, k, residual=x)
    b = moe.moe_unsort_rows(rows, r, T, k, residual=x)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_combine_skips_dropped_pairs(moe, cuda_device):
    T, H, E, k = 20, 64, 6, 3
    ids, x, rows, w = _case(6, T, H, E, k, torch.bfloat16, -2, 6)
    full = moe.moe_permute_capacity(ids, T, k, E, 4)
    full.topk_w = w
    a = moe.moe_combine(rows, full, T, k, residual=x)
    b = moe.moe_unsort_rows(rows, full, T, k, residual=x)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("offset", [1, 3])
def test_rows_that_start_on_odd_elements(moe, cuda_device, offset):
    """Row buffers aligned to their element only: the same numbers as aligned ones."""
    T, H, E, k = 11, 64, 5, 2
    ids, x, rows, w = _case(9, T, H, E, k, torch.bfloat16)
    r = moe.moe_permute_capacity(ids, T, k, E)
    r.topk_w = w

    def moved(t):
        buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")
        v = buf[offset:].view(t.shape)
        v.copy_(t)
        return v

    assert torch.equal(moe.moe_sort_rows(moved(x), r, k, True), moe.moe_sort_rows(x, r, k, True))
    assert torch.equal(moe.moe_unsort_rows(moved(rows), r, T, k), moe.moe_unsort_rows(rows, r, T, k))
    a, b = moe.moe_sort_rows_bwd(moved(rows), r, T, k, x=x, weighted=True), moe.moe_sort_rows_bwd(rows, r, T, k, x=x, weighted=True)
    assert torch.equal(a[0], b[0]) and torch.allclose(a[1], b[1], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 64, 8), (3, 1024, 32), (67, 7, 3)])
def test_router_softmax_gradient(moe, cuda_device, T, E, k):
    rng = np.random.default_rng(E)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    top, ids = logits.topk(k, dim=1)
    w = torch.softmax(top, 1).reshape(-1).contiguous()
    dw = torch.from_numpy(rng.standard_normal(T * k).astype(np.float32))
    ids = ids.int().reshape(-1).contiguous()
    ids[:: 5] = torch.where(torch.arange(ids[::5].numel()) % 2 == 0, ids[::5], torch.full_like(ids[::5], -1))
    r = moe.Routing(ids.cuda(), w.cuda(), None, None, None, None)
    got = moe.moe_route_topk_bwd(dw.cuda(), r, T, E, k, d_logits=torch.full((T, E), float("nan"), device="cuda"))
    ref = ro.route_topk_bwd(_f64(dw), _f64(w), ids.numpy(), T, E, k)
    mag = ro.route_topk_bwd(np.abs(_f64(dw)), -np.abs(_f64(w)), ids.numpy(), T, E, k)  # w (|dw| + sum w |dw|), negated
    _close(got, ref, np.abs(mag), 16, None, "d logits")


def test_an_expert_chosen_twice_gets_both_parts(moe, cuda_device):
    ids = torch.tensor([2, 2, 0], dtype=torch.int32).cuda()
    w, dw = torch.tensor([0.5, 0.3, 0.2]).cuda(), torch.tensor([1.0, -2.0, 0.5]).cuda()
    got = moe.moe_route_topk_bwd(dw, moe.Routing(ids, w, None, None, None, None), 1, 4, 3)
    ref = ro.route_topk_bwd(_f64(dw), _f64(w), ids.cpu().numpy(), 1, 4, 3)
    assert np.abs(_f64(got) - ref).max() <= 16 * U


def test_no_tokens(moe, cuda_device):
    E, k, H = 4, 2, 64
    r = moe.moe_permute_capacity(torch.empty(0, dtype=torch.int32, device="cuda"), 0, k, E)
    r.topk_w = torch.empty(0, device="cuda")
    x = torch.empty((0, H), device="cuda")
    assert moe.moe_unsort_rows(torch.zeros((1, H), device="cuda"), r, 0, k).shape == (0, H)
    moe.moe_sort_rows(x, r, k, True)
    assert moe.moe_route_topk_bwd(torch.empty(0, device="cuda"), r, 0, E, k).shape == (0, E)
    moe.moe_check_device_errors()


def test_captured_and_replayed_on_new_inputs(moe, cuda_device):
    """The whole chain in a graph on a side stream; replays follow inputs changed in place."""
    T, H, E, k = 64, 256, 16, 4
    ids, x, rows, w = _case(3, T, H, E, k, torch.bfloat16, -2, 16)

    def chain():
        r = moe.moe_permute_capacity(ids, T, k, E, 20)
        r.topk_w = w
        s = moe.moe_sort_rows(x, r, k, True, rows=torch.zeros_like(rows))
        out = moe.moe_unsort_rows(s, r, T, k, residual=x)
        dr, dw = moe.moe_unsort_rows_bwd(x, r, k, rows=s, d_rows=torch.zeros_like(rows))
        dx, _ = moe.moe_sort_rows_bwd(dr, r, T, k, x=x, weighted=True)
        return out, dr, dw, dx, moe.moe_route_topk_bwd(dw, r, T, E, k)

    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = chain()
    for seed in (11, 12):
        ids2, x2, _, w2 = _case(seed, T, H, E, k, torch.bfloat16, -2, 16)
        ids.copy_(ids2), x.copy_(x2), w.copy_(w2)
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, chain()):
            assert torch.equal(a, b)


def test_on_a_given_stream(moe, cuda_device):
    T, H, E, k = 33, 128, 8, 2
    ids, x, rows, w = _case(4, T, H, E, k, torch.float16)
    r = moe.moe_permute_capacity(ids, T, k, E)
    r.topk_w = w
    ref = moe.moe_unsort_rows(rows, r, T, k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r2 = moe.moe_permute_capacity(ids, T, k, E, stream=side)
    r2.topk_w = w
    got = moe.moe_unsort_rows(rows, r2, T, k, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)


@pytest.mark.parametrize("T", [6, 200])  # the weight-streaming path, the tensor-core path
def test_around_the_grouped_ffn(moe, cuda_device, T):
    """Rows of kept pairs come out of the grouped FFN as without drops, and the layer's output is the
    weighted sum of those rows alone."""
    H, I, E, k = 256, 128, 8, 2
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    ex = moe.quantize_experts(moe.FMT_W4G128, (torch.randn((E, 2 * I, H), generator=g) * 0.05).bfloat16().cuda(),
                              (torch.randn((E, H, I), generator=g) * 0.05).bfloat16().cuda())
    wr = (torch.randn((E, H), generator=g) * 0.05).bfloat16().cuda()
    r = moe.moe_route_topk(x, wr, None, k)
    full = moe.moe_grouped_ffn(x, r, ex, I, E, k)
    cap = max(1, T * k // E)
    d = moe.moe_permute_capacity(r.topk_ids, T, k, E, cap)
    d.topk_w = r.topk_w
    rows = moe.moe_grouped_ffn(x, d, ex, I, E, k)
    moe.moe_check_device_errors()
    a, b = r.pair_to_row.cpu().numpy(), d.pair_to_row.cpu().numpy()
    kept = b >= 0
    assert 0 < kept.sum() < T * k
    fa, fb = _f64(full)[a[kept]], _f64(rows)[b[kept]]
    # 1e-2 relative L2 and 2e-2 absolute: the FFN's tolerance (an expert may take the other path)
    assert np.linalg.norm(fa - fb) <= 1e-2 * np.linalg.norm(fa) and np.abs(fa - fb).max() <= 2e-2
    out = moe.moe_unsort_rows(rows, d, T, k, residual=x)
    rf = np.nan_to_num(_f64(rows))
    ref = ro.unsort_rows(rf, _f64(r.topk_w), b, T, k, _f64(x))
    _close(out, ref, ro.unsort_rows(np.abs(rf), _f64(r.topk_w), b, T, k, np.abs(_f64(x))), k + 2, torch.bfloat16, "layer")


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_every_pair_dropped(moe, cuda_device, T, fmt):
    """A rank none of whose experts were chosen: the grouped FFN computes nothing, every token keeps its residual, and the
    gradients of the weights are zero."""
    H, I, E, k = 256, 128, 4, 2
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    ex = moe.quantize_experts(fmt, torch.ones((E, 2 * I, H), dtype=torch.bfloat16, device="cuda"),
                              torch.ones((E, H, I), dtype=torch.bfloat16, device="cuda"))
    r = moe.moe_permute_capacity(torch.full((T * k,), E, dtype=torch.int32, device="cuda"), T, k, E)
    r.topk_w = torch.ones(T * k, device="cuda")
    assert int(r.expert_offsets[E]) == 0 and int(r.expert_list[0]) == 0
    held = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = moe.moe_grouped_ffn(x, r, ex, I, E, k, bits=torch.full((T * k,), 4, dtype=torch.uint8, device="cuda"), y_rows=held)
    moe.moe_check_device_errors()
    assert bool((rows == 7).all())
    rows.fill_(float("nan"))
    assert torch.equal(moe.moe_unsort_rows(rows, r, T, k, residual=x), x)
    assert bool((moe.moe_unsort_rows(rows, r, T, k) == 0).all())
    dr, dw = moe.moe_unsort_rows_bwd(x, r, k, rows=rows, d_rows=torch.full_like(rows, 3.0))
    assert bool((dr == 3).all()) and bool((dw == 0).all())
    z, _ = moe.moe_block_norm(x, rows, routing=r, k=k, w_post=torch.ones(H, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(z, x)


def test_two_streams_at_once(moe, cuda_device):
    """Calls without a workspace on two streams at the same time."""
    T, H, E, k = 512, 1024, 32, 4
    cases = [_case(s, T, H, E, k, torch.bfloat16, -2, 32) for s in (21, 22)]

    def chain(c, stream):
        ids, x, rows, w = c
        r = moe.moe_permute_capacity(ids, T, k, E, 70, stream=stream)
        r.topk_w = w
        out = moe.moe_unsort_rows(rows, r, T, k, residual=x, stream=stream)
        return out, moe.moe_sort_rows_bwd(rows, r, T, k, x=x, weighted=True, stream=stream)

    ref = [chain(c, None) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [chain(c, s) for c, s in zip(cases, streams)]
        for s in streams:
            s.synchronize()
        for (a, (b, c)), (p, (q, r)) in zip(got, ref):
            assert torch.equal(a, p) and torch.equal(b, q) and torch.equal(c, r)
