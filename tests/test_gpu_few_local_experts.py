"""A rank that holds fewer experts than a token chooses: the permutation drops the other ranks' pairs, and the grouped FFN and the
combine take the routing it leaves.  Reference: the same experts one at a time, by calls of one expert with k = 1."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _experts(moe, fmt, E, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: (torch.randn(s, generator=g) * 0.05).bfloat16().cuda()
    return rn(E, 2 * I, H), rn(E, H, I)


def _alone(moe, fmt, w13, w2, x, e, bits):
    """x through expert e alone: [T][H] in float64."""
    T, H = x.shape
    r = moe.moe_permute(torch.zeros(T, dtype=torch.int32, device="cuda"), T, 1, 1)
    ex = moe.quantize_experts(fmt, w13[e:e + 1].contiguous(), w2[e:e + 1].contiguous())
    b = torch.full((T,), bits, dtype=torch.uint8, device="cuda")
    return moe.moe_grouped_ffn(x, r, ex, w2.shape[2], 1, 1, bits=b).double().cpu().numpy()


@pytest.mark.parametrize("T", [1, 6, 200])  # the weight-streaming path, the tensor-core path
@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("ids", ["other ranks", "one expert twice"])
def test_more_choices_than_experts(moe, cuda_device, T, fmt, ids):
    H, I, E, k, bits = 256, 128, 2, 4, 6
    w13, w2 = _experts(moe, fmt, E, H, I, T)
    ex = moe.quantize_experts(fmt, w13, w2)
    rng = np.random.default_rng(T)
    if ids == "other ranks":  # four of eight experts each; this rank holds numbers 3 and 4
        pick = np.stack([rng.permutation(8)[:k] for _ in range(T)]) - 3
    else:
        pick = rng.integers(0, E, (T, k))
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(T + 1)).bfloat16().cuda()
    r = moe.moe_permute_capacity(torch.from_numpy(pick.astype(np.int32).reshape(-1)).cuda(), T, k, E)
    r.topk_w = torch.rand(T * k, generator=torch.Generator().manual_seed(T)).cuda()
    held = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = moe.moe_grouped_ffn(x, r, ex, I, E, k, bits=torch.full((T * k,), bits, dtype=torch.uint8, device="cuda"), y_rows=held)
    moe.moe_check_device_errors()
    alone = [_alone(moe, fmt, w13, w2, x, e, bits) for e in range(E)]
    row, got, n = r.pair_to_row.cpu().numpy(), rows.double().cpu().numpy(), int(r.expert_offsets[E])
    kept = [p for p in range(T * k) if 0 <= pick.reshape(-1)[p] < E]
    assert len(kept) == n and (got[n:] == 7).all()  # rows of no pair are left as they were
    w, out = r.topk_w.double().cpu().numpy(), np.zeros((T, H))
    for p in kept:
        out[p // k] += w[p] * got[row[p]]
    if kept:
        ref = np.stack([alone[pick.reshape(-1)[p]][p // k] for p in kept])
        err = got[row[kept]] - ref
        # the FFN's tolerance: 1e-2 relative L2, 2e-2 absolute (an expert may take the other path)
        assert np.linalg.norm(err) <= 1e-2 * np.linalg.norm(ref) and np.abs(err).max() <= 2e-2
    got = moe.moe_combine(rows, r, T, k).double().cpu().numpy()
    assert (np.abs(got - out) <= 2.0 ** -8 * np.abs(out) + 1e-5).all()
