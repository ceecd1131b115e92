"""paged_append_fp8, paged_gather_fp8 and chunk_positions: bit-exact against
the append rule and the E4M3 definition, bytes that no token owns untouched."""
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


CASES = [  # new, have, B_k, H_kv, d_h, d_idx, pad
    ([1], [0], 128, 1, 128, 64, 0),
    ([1, 1, 1], [127, 128, 129], 128, 4, 128, 64, 2),
    ([5, 0, 200, 1, 63], [63, 10, 0, 64, 1], 64, 2, 64, 128, 5),
    ([0, 300, 0], [5, 1000, 0], 128, 8, 64, 64, 0),
    ([130, 7], [400, 3], 64, 5, 128, 128, 1),
]


def same(a, b):
    """Bit equality (NaN scales in stale memory included)."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("new,have,B_k,H_kv,d_h,d_idx,pad", CASES)
def test_append_and_gather(msa, new, have, B_k, H_kv, d_h, d_idx, pad):
    c = Cache(new, have, B_k, H_kv, d_h, d_idx, seed=len(new), pad=pad)
    c.rows["k"][0, 0] = 0.0                      # a zero row: scale 1
    c.rows["v"][0, 0, :2] = torch.tensor([3e38, -3e38]).bfloat16()
    d = c.gpu()
    assert same(msa.chunk_positions(d["cu"], d["len"], c.T).cpu(), c.positions())
    ws = torch.full((256,), 77, dtype=torch.uint8, device="cuda")
    msa.paged_append_fp8(d["new_k"], d["new_v"], d["new_i"], *c.pools(d), d["table"], d["cu"],
                         d["len"], workspace=ws)
    assert msa.device_status(ws) == (0, 0)
    want = c.appended()
    for n in "kvi":
        assert same(d[n + "p"].cpu(), want[n][0]), f"codes of {n}"
        assert same(d[n + "s"].cpu(), want[n][1]), f"scales of {n}"
    assert d["len"].cpu().tolist() == have
    # the rows read back, at the chunk's own positions; the padding stays as it was
    out = [torch.full_like(d["new_" + n], 9.0) for n in "kvi"]
    got = msa.paged_gather_fp8(*c.pools(d), d["table"], d["cu"], d["len"], c.T, out=out)
    live = c.positions() >= 0
    for n, y in zip("kvi", got):
        rows = c.rows[n].float()
        from tests.chunk_util import e4m3, quantise
        codes, scale = quantise(c.rows[n])
        ref = (e4m3(codes).float() * scale[..., None]).bfloat16()
        assert torch.equal(y.cpu()[live], ref[live]) and bool((y.cpu()[~live] == 9.0).all())
        # and they are the rows that went in, to half a step of E4M3 (or of its
        # smallest: 2^-10 of the scale), the quotient's and bf16's roundings
        err = (y.cpu().float() - rows)[live].abs()
        tol = rows.abs() * (2.0**-4 + 2.0**-7) + scale[..., None] * 2.0**-9
        assert bool((err <= tol[live]).all())


def test_gather_of_a_prefix(msa):
    """Any range of positions, rows of several sequences, empty ranges among them."""
    c = Cache([4, 9, 1], [500, 64, 200], 64, 3, 64, 64, seed=8)
    d = c.gpu()
    start, rows = [37, 0, 199], [300, 0, 1]
    cu = torch.tensor([0, 300, 300, 301], dtype=torch.int32).cuda()
    k, v, ki = msa.paged_gather_fp8(*c.pools(d), d["table"], cu,
                                    torch.tensor(start, dtype=torch.int32).cuda(), 301)
    for n, y in (("k", k), ("v", v), ("i", ki)):
        ref = torch.cat([c.dense[s, n][a: a + r] for s, (a, r) in enumerate(zip(start, rows))])
        err = (y.cpu().double() - ref).abs()
        # one rounding to fp32 (the product) and one to bf16
        assert bool((err <= ref.abs() * (2.0**-8 + 2.0**-23)).all())


def test_skipped_rows_are_recorded(msa):
    """A sequence that does not fit, a page outside the pool, broken offsets: nothing is
    written for them, the others are served."""
    c = Cache([3, 3, 3], [62, 62, 62], 64, 2, 64, 64, seed=4)
    d = c.gpu()
    before = {k: v.clone() for k, v in d.items()}
    d["len"][0] = c.max_pages * 64 - 2           # one token too many
    d["table"][1, 0] = c.n_pages                 # outside
    d["table"][1, 1] = -1
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (d["new_k"], d["new_v"], d["new_i"], *c.pools(d), d["table"], d["cu"], d["len"])
    msa.paged_append_fp8(*args, workspace=ws)
    assert msa.device_status(ws)[0] in (2, 3)
    want = c.appended()
    for n in "kvi":
        mine, old = d[n + "p"].cpu(), before[n + "p"].cpu()
        p2, s2 = c.where(2, torch.arange(62, 65))
        assert same(mine[p2, s2], want[n][0][p2, s2])
        mine[p2, s2] = old[p2, s2]
        assert same(mine, old)
    assert msa.chunk_positions(d["cu"], d["len"], c.T, max_len=c.max_pages * 64).cpu().tolist()[:3] == [-1] * 3
    out = [torch.full_like(d["new_" + n], 9.0) for n in "kvi"]
    msa.paged_gather_fp8(*c.pools(d), d["table"], d["cu"], d["len"], c.T, out=out)
    assert all(bool((y[:6] == 9.0).all()) for y in out)
    for cu in ([0, -4, 5, 2**31 - 1], [7, 5, 3, 1], [-(2**31), 2**31 - 1, 0, 4], [9, 9, 9, 9]):
        bad = torch.tensor(cu, dtype=torch.int32).cuda()
        msa.paged_append_fp8(*args[:-2], bad, d["len"], workspace=ws)
        msa.chunk_positions(bad, d["len"], c.T)
        torch.cuda.synchronize()


def test_append_then_decode_continues(msa):
    """A cache filled by chunks serves the framework's own decode step: the same result as
    with the cache filled by quantize_fp8_rows."""
    S, H_kv, G, d_h, d_idx, B_k, kk, L = 3, 4, 8, 128, 64, 128, 4, 600
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    k, v, ki = r(S, L, H_kv, d_h), r(S, L, H_kv, d_h), r(S, L, d_idx)
    max_pages = 5
    table = torch.arange(S * max_pages, device="cuda", dtype=torch.int32).view(S, max_pages)
    outs = []
    for how in range(2):
        P = S * max_pages
        pools = [torch.zeros(P, B_k, H_kv, d_h, dtype=torch.uint8, device="cuda"),
                 torch.ones(P, B_k, H_kv, device="cuda"),
                 torch.zeros(P, B_k, H_kv, d_h, dtype=torch.uint8, device="cuda"),
                 torch.ones(P, B_k, H_kv, device="cuda"),
                 torch.zeros(P, B_k, d_idx, dtype=torch.uint8, device="cuda"),
                 torch.ones(P, B_k, device="cuda")]
        seq_len = torch.zeros(S, dtype=torch.int32, device="cuda")
        if how == 0:
            for a, b in ((0, 250), (250, 251), (251, L)):  # three chunks
                n = b - a
                cu = torch.arange(S + 1, device="cuda", dtype=torch.int32) * n
                rows = [t[:, a:b].reshape(S * n, *t.shape[2:]).contiguous() for t in (k, v, ki)]
                msa.paged_append_fp8(*rows, *pools,
                                     table, cu, seq_len)
                seq_len += n
        else:
            for x, p, sc in ((k, 0, 1), (v, 2, 3), (ki, 4, 5)):
                codes, scale = msa.quantize_fp8_rows(x)
                pools[p].view(S, max_pages * B_k, *x.shape[2:])[:, :L] = codes
                pools[sc].view(S, max_pages * B_k, *x.shape[2:-1])[:, :L] = scale
            seq_len += L
        gg = torch.Generator("cuda").manual_seed(9)
        rr = lambda *s: torch.randn(*s, generator=gg, device="cuda").bfloat16()  # noqa: E731
        idx = torch.empty(S, H_kv, kk, dtype=torch.int32, device="cuda")
        o, _ = msa.paged_decode_fp8(rr(S, H_kv * G, d_h), rr(S, H_kv, d_idx), rr(S, H_kv, d_h), rr(S, H_kv, d_h),
                                    rr(S, d_idx), *pools, table, seq_len, B_k, kk, idx_out=idx)
        outs.append((o, idx, seq_len, *pools))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_refusals_streams_and_graph(msa):
    c = Cache([2, 70], [60, 3], 64, 2, 64, 64, seed=6)
    d = c.gpu()
    args = [d["new_k"], d["new_v"], d["new_i"], *c.pools(d), d["table"], d["cu"], d["len"]]
    for at, bad in ((0, d["new_k"].float()), (0, d["new_k"].cpu()), (2, d["new_i"][:, :32]),
                    (3, d["kp"][:, ::2]), (4, d["ks"].double()), (7, d["ip"][1:]), (9, d["table"].long()),
                    (10, d["cu"][:2]), (11, d["len"][:1])):
        a = list(args)
        a[at] = bad
        with pytest.raises((TypeError, ValueError)):
            msa.paged_append_fp8(*a)
    with pytest.raises(ValueError):
        msa.paged_append_fp8(*args, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(msa.MSAError):  # 32-token pages
        p = [t[:, :32].contiguous() for t in c.pools(d)]
        msa.paged_append_fp8(*args[:3], *p, *args[9:])
    none = [t[:0] for t in args[:3]]
    msa.paged_append_fp8(*none, *args[3:])  # no rows: no work
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    msa.paged_append_fp8(*args, stream=side)
    side.synchronize()
    want = c.appended()
    assert all(same(d[n + "p"].cpu(), want[n][0]) for n in "kvi")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.paged_append_fp8(*args)
        out = msa.paged_gather_fp8(*c.pools(d), d["table"], d["cu"], d["len"], c.T)
    d["new_k"].neg_()
    graph.replay()
    got = out[0].clone()
    d["new_k"].neg_()
    graph.replay()
    assert torch.equal(got, -out[0])
