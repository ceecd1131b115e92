"""paged_index_scores_fp8 against float64 dot products of the dequantised keys,
and block_topk (bit-exact) against a sorted enumeration.

Tolerance of a score: products of a bf16 query and an E4M3 code are exact; the
tensor cores add d of them in fp32, each addition off by at most one unit of
the last place of the running magnitude, 2^-23 of the sum of magnitudes; the
scale of the key, the query's power of two and idx_scale are three more fp32
roundings.  Sequences with 512 rows and more multiply with the query as two E4M3
terms, the largest element of a row scaled into [224, 448]: their sum is the
query but for elements below 2^-10 of the largest, which are off by half of
E4M3's smallest step, 2^-10, at most: 2^-10 / 224 of the row's largest for each
element of the key."""
from __future__ import annotations

import pytest
import torch

from tests.chunk_util import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_gqa_idx_b200 as msa

    return msa


def reference(c: Cache, q, scale):
    """(scores, tolerances) in float64, -inf where no score is due."""
    T, H, d = q.shape
    ref = torch.full((T, H, c.max_pages), -float("inf"), dtype=torch.float64)
    tol = torch.zeros_like(ref)
    for s in range(c.S):
        keys = c.dense[s, "i"]
        for i in range(c.new[s]):
            t = int(c.cu[s]) + i
            own = (c.have[s] + i) // c.B_k
            if own == 0:
                continue
            k = keys[: own * c.B_k]
            x = q[t].double() @ k.T
            mag = q[t].double().abs() @ k.abs().T
            split = 2.0**-10 / 224 * q[t].double().abs().amax(-1, keepdim=True) * k.abs().sum(-1)
            split = split if c.new[s] * H >= 512 else 0.0
            ref[t, :, :own] = scale * x.view(H, own, c.B_k).amax(-1)
            tol[t, :, :own] = scale * (mag * (d * 2.0**-23 + 2.0**-21) + split).view(H, own, c.B_k).amax(-1)
    return ref, tol


CASES = [  # new, have, B_k, H_kv, d_idx, pad
    ([1], [0], 128, 4, 64, 0),
    ([1], [5000], 128, 4, 64, 0),
    ([1, 1, 1], [127, 128, 1000], 64, 1, 128, 3),
    ([1, 0, 1, 1], [700, 3, 129, 64], 128, 8, 64, 1),
    ([6, 1, 0, 40], [300, 500, 0, 90], 64, 3, 64, 2),
    ([33, 130], [1000, 65], 64, 2, 128, 0),
    ([300, 5, 129], [20, 900, 0], 128, 4, 64, 7),
    ([600], [1300], 128, 4, 128, 0),
    ([3], [1000], 128, 4, 64, 200),  # one sequence, whose rows are few, and much padding
    ([100], [700], 64, 2, 128, 300),
    ([257, 400], [64, 2000], 64, 8, 64, 5),
    ([700, 1], [0, 3000], 128, 1, 64, 0),
    ([100, 1, 90], [3000, 700, 0], 64, 3, 64, 4),
    ([1] * 40 + [50] * 4, [260] * 44, 128, 5, 128, 0),
    ([4, 4, 60, 300, 2], [5000, 128, 127, 64, 1], 128, 8, 128, 9),
    ([300, 1], [1000, 1000], 64, 2, 128, 0),
    ([2, 1] * 300 + [0] * 20 + [150, 3, 140], [70] * 623, 64, 4, 64, 3),
]


@pytest.mark.parametrize("new,have,B_k,H_kv,d_idx,pad", CASES)
@pytest.mark.parametrize("scale", [0.0, 3.5])
def test_scores(msa, new, have, B_k, H_kv, d_idx, pad, scale):
    c = Cache(new, have, B_k, H_kv, 64, d_idx, seed=sum(new) + H_kv, pad=pad)
    q = torch.randn(c.T, H_kv, d_idx, generator=c.g).bfloat16()
    q[0] *= 2.0**40   # queries of any magnitude keep their digits
    q[-1] *= 2.0**-60
    d = c.gpu(c.appended())
    mark = torch.full((c.T, H_kv, c.max_pages), 5.0, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = msa.paged_index_scores_fp8(q.cuda(), d["ip"], d["is"], d["table"], d["cu"], d["len"], idx_scale=scale,
                                     scores=mark, workspace=ws).cpu()
    assert msa.device_status(ws) == (0, 0)
    ref, tol = reference(c, q, scale or d_idx**-0.5)
    live = c.positions() >= 0
    assert bool((got[~live] == 5.0).all())
    got, ref, tol = got[live].double(), ref[live], tol[live]
    none = ref == -float("inf")
    assert torch.equal(got == -float("inf"), none)
    assert bool(((got - ref).abs()[~none] <= tol[~none]).all())


@pytest.mark.parametrize("new,have", [([1, 1], [400, 400]), ([30, 20], [400, 300]), ([90, 50], [400, 300])])
def test_bad_pages_score_nothing(msa, new, have):
    c = Cache(new, have, 64, 4, 64, 64, seed=5)
    d = c.gpu(c.appended())
    d["table"][0, 2] = c.n_pages
    d["table"][1, 0] = -1
    q = torch.randn(c.T, 4, 64, generator=c.g).bfloat16()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = msa.paged_index_scores_fp8(q.cuda(), d["ip"], d["is"], d["table"], d["cu"], d["len"], workspace=ws).cpu()
    assert msa.device_status(ws)[0] == 2
    ref, tol = reference(c, q, 64**-0.5)
    ref[: new[0], :, 2] = -float("inf")
    ref[new[0]:, :, 0] = -float("inf")
    none = ref == -float("inf")
    assert torch.equal(got == -float("inf"), none)
    assert bool(((got.double() - ref).abs()[~none] <= tol[~none]).all())
    # a sequence that does not fit its pages is skipped whole
    d["len"][1] = c.max_pages * 64 - new[1] + 1
    mark = torch.full((c.T, 4, c.max_pages), 5.0, device="cuda")
    got = msa.paged_index_scores_fp8(q.cuda(), d["ip"], d["is"], d["table"], d["cu"], d["len"], scores=mark,
                                     workspace=ws)
    assert bool((got[new[0]:] == 5.0).all()) and msa.device_status(ws)[0] in (2, 3)
    for cu in ([0, -4, 2**31 - 1], [7, 5, 3], [-(2**31), 2**31 - 1, 4], [9, 9, 9]):
        msa.paged_index_scores_fp8(q.cuda(), d["ip"], d["is"], d["table"],
                                   torch.tensor(cu, dtype=torch.int32).cuda(), d["len"])
        torch.cuda.synchronize()


def brute(x, pos, B_k, k):
    T, H, n = x.shape
    out = torch.full((T, H, k), -1, dtype=torch.int32)
    for t in range(T):
        own = int(pos[t]) // B_k
        if pos[t] < 0:
            continue
        for h in range(H):
            row = x[t, h, : min(own, n)].tolist()
            best = sorted((b for b, v in enumerate(row) if v > -float("inf")), key=lambda b: (-row[b], b))
            got = sorted(best[: k - 1] + [own])
            out[t, h, : len(got)] = torch.tensor(got, dtype=torch.int32)
    return out


@pytest.mark.parametrize("T,H,n,B_k,k", [
    (1, 1, 1, 128, 1), (1, 4, 257, 128, 16), (7, 3, 33, 64, 32), (5, 2, 1025, 128, 32), (40, 4, 300, 64, 16),
    (3, 1, 5000, 128, 20), (9, 8, 64, 64, 2), (6, 2, 31, 64, 8), (130, 1, 256, 128, 31), (2, 2, 2048, 64, 1),
])
@pytest.mark.parametrize("kind", ["normal", "ties", "holes"])
def test_topk(msa, T, H, n, B_k, k, kind):
    g = torch.Generator().manual_seed(T * 1000 + n + k)
    x = torch.randn(T, H, n, generator=g)
    if kind == "ties":
        x = torch.randint(0, 3, (T, H, n), generator=g).float()
    if kind == "holes":
        pick = torch.randint(0, 4, (T, H, n), generator=g)
        x = torch.where(pick == 0, float("nan"), torch.where(pick == 1, -float("inf"), x))
        x[0, 0] = -float("inf")
        x[-1, -1, ::5] = float("inf")
    pos = torch.randint(0, n * B_k, (T,), generator=g, dtype=torch.int32)
    pos[-1] = n * B_k - 1
    if T > 4:
        pos[1], pos[2], pos[3] = -1, 0, B_k
    mark = torch.full((T, H, k), -9, dtype=torch.int32, device="cuda")
    got = msa.block_topk(x.cuda(), pos.cuda(), B_k, k, idx_out=mark).cpu()
    ref = brute(x, pos, B_k, k)
    ref[pos < 0] = -9
    assert torch.equal(got, ref)


def test_scores_then_topk_is_the_prefill_selection(msa):
    """A prompt scored chunk by chunk on the cache selects what one prefill call selects from the
    same (dequantised) keys, but where two blocks are nearly equal."""
    from tests import compare
    from tests.gpu_util import to_host_bits

    N, H, d, B_k, k = 3000, 4, 64, 128, 8
    c = Cache([N], [0], B_k, H, 64, d, seed=77)
    # powers of two as scales: the dequantised keys are bf16 values, so both paths see the same ones
    pool = c.appended()
    pool["i"][1] = torch.exp2(torch.round(torch.log2(pool["i"][1].abs().nan_to_num(1.0, 1.0, 1.0).clamp(min=1e-4))))
    page, slot = c.where(0, torch.arange(N))
    from tests.chunk_util import e4m3
    keys = (e4m3(pool["i"][0][page, slot]) * pool["i"][1][page, slot].double()[:, None]).bfloat16()
    q = torch.randn(N, H, d, generator=c.g).bfloat16()
    ref = msa.index_topk(q.cuda(), keys.cuda(), B_k, k).cpu()
    dev = c.gpu(pool)
    parts = []
    for a, b in ((0, 1), (1, 700), (700, 2999), (2999, N)):
        cu = torch.tensor([0, b - a], dtype=torch.int32).cuda()
        ln = torch.tensor([a], dtype=torch.int32).cuda()
        x = msa.paged_index_scores_fp8(q[a:b].cuda(), dev["ip"], dev["is"], dev["table"], cu, ln)
        parts.append(msa.block_topk(x, msa.chunk_positions(cu, ln, b - a), B_k, k).cpu())
    got = torch.cat(parts)
    rows = (got != ref).any(-1).nonzero()
    for t, h in rows.tolist():  # a differing row: the blocks it swaps score the same to fp32
        x = q[t, h].double() @ keys[: t + 1].double().T
        m = {b: float(x[b * B_k: (b + 1) * B_k].max()) for b in set(got[t, h].tolist()) ^ set(ref[t, h].tolist())}
        assert max(m.values()) - min(m.values()) <= 1e-5 * max(abs(v) for v in m.values())
    assert len(rows) <= 3


def test_refusals_and_graph(msa):
    c = Cache([3, 40], [200, 300], 64, 2, 64, 64, seed=2)
    d = c.gpu(c.appended())
    q = torch.randn(c.T, 2, 64, generator=c.g).bfloat16().cuda()
    args = [q, d["ip"], d["is"], d["table"], d["cu"], d["len"]]
    for at, bad in ((0, q.float()), (0, q[:, :, :32]), (1, d["ip"][:, ::2]), (2, d["is"][:, :5]), (3, d["table"][0]),
                    (4, d["cu"].cpu()), (5, d["len"].long())):
        a = list(args)
        a[at] = bad
        with pytest.raises((TypeError, ValueError)):
            msa.paged_index_scores_fp8(*a)
    x = msa.paged_index_scores_fp8(*args)
    pos = msa.chunk_positions(d["cu"], d["len"], c.T)
    for k in (0, 33):
        with pytest.raises(msa.MSAError):
            msa.block_topk(x, pos, 64, k)
    with pytest.raises(msa.MSAError):
        msa.block_topk(x, pos, 32, 4)
    with pytest.raises(ValueError):
        msa.block_topk(x, pos[:-1], 64, 4)
    assert msa.block_topk(x[:0], pos[:0], 64, 4).shape == (0, 2, 4)
    idx = msa.block_topk(x, pos, 64, 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = msa.paged_index_scores_fp8(*args)
        i = msa.block_topk(y, msa.chunk_positions(d["cu"], d["len"], c.T), 64, 4)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, x) and torch.equal(i, idx)
    side = torch.cuda.Stream()
    y = msa.paged_index_scores_fp8(*args, stream=side)
    i = msa.block_topk(y, pos, 64, 4, stream=side)
    side.synchronize()
    assert torch.equal(y, x) and torch.equal(i, idx)
