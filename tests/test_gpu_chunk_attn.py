"""paged_sparse_attn_fp8 against float64 attention over the dequantised cache
(tests/chunk_util.py derives the tolerances)."""
from __future__ import annotations

import pytest
import torch

from tests.chunk_util import Cache, attention, refresh, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_gqa_idx_b200 as msa

    return msa


def call(msa, c, d, q, idx, **kw):
    return msa.paged_sparse_attn_fp8(q.cuda(), idx.cuda(), d["kp"], d["ks"], d["vp"], d["vs"], d["table"], d["cu"],
                                     d["len"], **kw)


def check(c, o, lse, ref, live=None):
    ro, rl, otol, ltol = ref
    live = c.positions() >= 0 if live is None else live
    o, lse, ro, rl, otol, ltol = o.double().cpu()[live], lse.double().cpu()[live], ro[live], rl[live], otol[live], ltol[live]
    none = rl == -float("inf")
    assert torch.equal(lse == -float("inf"), none)
    assert bool((o[none] == 0).all())
    bad = (o - ro).abs() / otol.clamp(min=1e-300)
    assert bool(torch.isfinite(o).all()) and float(bad[~none].max() if bad[~none].numel() else 0) <= 1.0
    assert bool(((lse - rl).abs()[~none] <= ltol[~none]).all())


CASES = [  # new, have, B_k, H_kv, G, d_h, k, pad
    ([1], [0], 128, 1, 1, 128, 1, 0),
    ([1], [2000], 128, 4, 8, 128, 16, 0),
    ([1, 1, 1, 0], [15, 16, 1000, 3], 64, 2, 4, 64, 5, 2),
    ([3, 1, 40], [126, 700, 5], 128, 4, 8, 128, 4, 1),
    ([2, 90], [63, 300], 64, 3, 5, 128, 32, 0),
    ([33], [400], 128, 2, 16, 64, 3, 0),
    ([17, 5], [100, 900], 64, 1, 12, 128, 7, 3),
    ([130, 1, 20], [0, 2000, 64], 128, 8, 2, 64, 6, 0),
    ([257], [10], 64, 4, 8, 64, 4, 5),
    ([300, 20], [500, 300], 128, 2, 8, 128, 5, 2),
    # enough rows x selected keys for the KV-outer form
    # (meant to be; some are too small for it, or have too few rows a sequence: which form a
    # case takes is asserted in test_gpu_chunk_forms.py)
    ([300, 20], [500, 300], 128, 4, 8, 128, 8, 2),
    ([530], [10], 64, 8, 1, 64, 8, 0),
    ([257, 0, 9], [1000, 5, 64], 128, 4, 16, 64, 16, 3),
    ([200, 100, 1], [64, 2000, 700], 64, 8, 2, 128, 16, 0),
    ([290], [0], 128, 2, 4, 128, 32, 1),
    ([1] * 90 + [60] * 5, [130] * 95, 128, 4, 8, 128, 6, 0),
    ([520, 60], [500, 300], 128, 4, 8, 128, 8, 2),
    ([1100], [10], 64, 8, 1, 64, 8, 0),
    ([1030, 0, 9], [1000, 5, 64], 64, 4, 16, 64, 16, 3),
    ([1] * 90 + [130] * 5, [130] * 95, 128, 4, 8, 128, 6, 0),
    # every number of heads per group with either head size
    # (16 heads with d_h = 128: test_gpu_chunk_forms.py)
    ([1030], [10], 64, 8, 1, 128, 8, 2),
    ([1100, 3], [10, 700], 64, 8, 2, 64, 8, 0),
    ([600], [500], 128, 4, 4, 64, 16, 1),
]


@pytest.mark.parametrize("new,have,B_k,H_kv,G,d_h,k,pad", CASES)
@pytest.mark.parametrize("holes", [False, True])
def test_against_float64(msa, new, have, B_k, H_kv, G, d_h, k, pad, holes):
    c = Cache(new, have, B_k, H_kv, d_h, 64, seed=sum(new) + G, pad=pad)
    q = torch.randn(c.T, H_kv * G, d_h, generator=c.g).bfloat16()
    idx = selection(c, k, holes)
    d = c.gpu(c.appended())
    o = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    d_ = msa.chunk_dims(c.S, c.T, c.max_pages, c.n_pages, H_kv * G, H_kv, d_h, 64, B_k, k)
    ws = torch.empty(msa.paged_sparse_attn_fp8_workspace_size(d_), dtype=torch.uint8, device="cuda")
    call(msa, c, d, q, idx, o=o, lse=lse, workspace=ws)
    assert msa.device_status(ws) == (0, 0)
    check(c, o, lse, attention(c, q, idx, d_h**-0.5))
    dead = c.positions() < 0
    assert bool((o.cpu()[dead] == 3.0).all()) and bool((lse.cpu()[dead] == 3.0).all())
    again, _ = call(msa, c, d, q, idx, want_lse=False)
    live = (~dead).cuda()
    assert torch.equal(again[live], o[live])


@pytest.mark.parametrize("new,have", [([1, 1], [700, 300]), ([200, 30], [300, 500]), ([700, 30], [300, 500]),
                                      ([1500, 30], [300, 500])])
def test_scales_of_any_size(msa, new, have):
    """Value rows from 1e-20 to 1e15, a peaked softmax, large and tiny queries."""
    c = Cache(new, have, 64, 2 if sum(new) < 700 else 4, 64, 64, seed=21)
    q = torch.randn(c.T, 4 * c.H_kv, 64, generator=c.g).bfloat16()
    q[:, 1] *= 30.0
    q[:, 2] *= 2.0**-30
    mag = 10.0 ** torch.randint(-20, 16, (c.T,), generator=c.g).float()
    c.rows["v"] = (c.rows["v"].float() * mag[:, None, None]).bfloat16()
    refresh(c)
    # and the cached tokens' scales
    p, s = c.where(0, torch.arange(have[0]))
    f = 10.0 ** torch.randint(-20, 16, (have[0],), generator=c.g).float()
    c.pool["v"][1][p, s] *= f[:, None]
    from tests.chunk_util import e4m3
    c.dense[0, "v"][: have[0]] = e4m3(c.pool["v"][0][p, s]) * c.pool["v"][1][p, s].double()[..., None]
    idx = selection(c, 6 if sum(new) < 700 else 12)
    d = c.gpu(c.appended())
    o, lse = call(msa, c, d, q, idx, attn_scale=0.3)
    check(c, o, lse, attention(c, q, idx, 0.3))


@pytest.mark.parametrize("new,have,k", [([3, 1], [100, 64], 3), ([140, 70], [100, 40], 3), ([440, 70], [900, 40], 17),
                                        ([900, 70], [900, 40], 17)])
def test_later_tokens_never_reach_a_row(msa, new, have, k):
    """NaN and infinite rows of later tokens of the same chunk, and stale pages, leave earlier rows alone."""
    c = Cache(new, have, 64, 2, 128, 64, seed=31)
    q = torch.randn(c.T, 16, 128, generator=c.g).bfloat16()
    cut = new[0] - 1
    for n in "kv":
        c.rows[n][cut] = float("nan")
        c.rows[n][cut, 0, :3] = float("inf")
    idx = selection(c, k)
    d = c.gpu(c.appended())
    for x in "kv":
        c.rows[x][cut] = 0.0  # the reference of the other rows does not see it
    refresh(c)
    o, lse = call(msa, c, d, q, idx)
    live = torch.ones(c.T, dtype=torch.bool)
    live[cut] = False
    check(c, o, lse, attention(c, q, idx, 128**-0.5), live)
    assert bool(torch.isnan(o[cut]).all()) and bool(torch.isnan(lse[cut]).all())


@pytest.mark.parametrize("new,have,H_kv,k", [([1, 1], [400, 300], 2, 5), ([150, 80], [400, 300], 2, 5),
                                             ([250, 80], [400, 300], 8, 13), ([560, 80], [400, 300], 8, 13)])
def test_bad_pages_and_entries(msa, new, have, H_kv, k):
    c = Cache(new, have, 64, H_kv, 64, 64, seed=41)
    q = torch.randn(c.T, 8 * H_kv, 64, generator=c.g).bfloat16()
    idx = selection(c, k)
    idx[:, 0, 0] = 1
    idx[:, 0, 1:3] = torch.tensor([0, 2], dtype=torch.int32)
    idx[:, 0, 3:] = -1
    d = c.gpu(c.appended())
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda")
    ref = attention(c, q, idx, 0.125)
    wrong = idx.clone()
    wrong[:, 0, 3] = c.max_pages       # outside: ignored, recorded
    wrong[:, 0, 4] = -7
    o, lse = call(msa, c, d, q, wrong, workspace=ws)
    assert msa.device_status(ws)[0] == 2
    check(c, o, lse, ref)
    d["table"][0, 1] = c.n_pages       # the page of a selected block
    d["table"][1, 1] = -3
    gone = idx.clone()
    gone[gone == 1] = -1
    o, lse = call(msa, c, d, q, idx, workspace=ws)
    assert msa.device_status(ws)[0] == 2
    check(c, o, lse, attention(c, q, gone, 0.125))
    d["len"][1] = c.max_pages * 64     # a sequence that does not fit is skipped whole
    mark = torch.full_like(o, 9.0)
    call(msa, c, d, q, idx, o=mark, workspace=ws)
    assert bool((mark[new[0]:] == 9.0).all()) and bool((mark[: new[0]] != 9.0).any())
    for cu in ([0, -4, 2**31 - 1], [7, 5, 3], [-(2**31), 2**31 - 1, 4], [9, 9, 9]):
        d["cu"] = torch.tensor(cu, dtype=torch.int32).cuda()
        call(msa, c, d, q, idx, workspace=ws)
        torch.cuda.synchronize()


def test_equals_the_decode_step(msa):
    """Single tokens: the framework's decode step on the same cache, and this operator on its selection."""
    c = Cache([1, 1, 1], [500, 1300, 127], 128, 4, 128, 64, seed=51)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16()
    qi = torch.randn(c.T, 4, 64, generator=c.g).bfloat16()
    d = c.gpu()
    idx = torch.empty(3, 4, 6, dtype=torch.int32, device="cuda")
    table = d["table"].clamp(0, c.n_pages - 1)
    o, _ = msa.paged_decode_fp8(q.cuda(), qi.cuda(), d["new_k"], d["new_v"], d["new_i"], *c.pools(d), table,
                                d["len"].clone(), 128, 6, idx_out=idx)
    x = msa.paged_index_scores_fp8(qi.cuda(), d["ip"], d["is"], table, d["cu"], d["len"])
    mine = msa.block_topk(x, msa.chunk_positions(d["cu"], d["len"], 3), 128, 6)
    assert torch.equal(mine, idx)
    got, _ = call(msa, c, d, q, idx)
    # both are within their roundings of the same value: bf16 weights there (2^-8)
    ref = attention(c, q, idx.cpu(), 128**-0.5)
    assert bool(((got.double() - o.double()).abs().cpu() <= 2 * ref[2] + 2.0**-8 * ref[0].abs() + 0.01).all())
    check(c, got, call(msa, c, d, q, idx)[1], ref)


@pytest.mark.parametrize("new,have,k", [([1, 1], [400, 300], 5), ([150, 80], [400, 300], 5), ([650, 80], [400, 1300], 24),
                                        ([1300, 80], [400, 1300], 24)])
def test_refusals_streams_and_graphs(msa, new, have, k):
    c = Cache(new, have, 64, 2, 64, 64, seed=61)
    q = torch.randn(c.T, 16, 64, generator=c.g).bfloat16()
    idx = selection(c, k)
    d = c.gpu(c.appended())
    args = [q.cuda(), idx.cuda(), d["kp"], d["ks"], d["vp"], d["vs"], d["table"], d["cu"], d["len"]]
    for at, bad in ((0, q), (0, q.cuda().float()), (0, args[0][:, :15]), (1, args[1].long()), (1, args[1][:-1]),
                    (2, d["kp"][:, :, ::2]), (3, d["ks"][1:]), (6, d["table"].T), (7, d["cu"][1:])):
        a = list(args)
        a[at] = bad
        with pytest.raises((TypeError, ValueError, msa.MSAError)):
            msa.paged_sparse_attn_fp8(*a)
    with pytest.raises(msa.MSAError):
        msa.paged_sparse_attn_fp8(*args, attn_scale=-1.0)
    assert msa.paged_sparse_attn_fp8(args[0][:0], args[1][:0], *args[2:])[0].shape == (0, 16, 64)
    ref = msa.paged_sparse_attn_fp8(*args)
    torch.cuda.synchronize()
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [msa.paged_sparse_attn_fp8(*args, stream=s) for _ in range(4) for s in streams]
    for s in streams:
        s.synchronize()
    assert all(torch.equal(a, b) for got in outs for a, b in zip(got, ref))
    # two captured calls that share the caller's workspace, replayed in turn
    d_ = msa.chunk_dims(c.S, c.T, c.max_pages, c.n_pages, 16, 2, 64, 64, 64, k)
    ws = torch.empty(msa.paged_sparse_attn_fp8_workspace_size(d_), dtype=torch.uint8, device="cuda")
    q2 = (args[0] * 0.5).contiguous()
    ref2 = msa.paged_sparse_attn_fp8(q2, *args[1:])
    graphs, got = [], []
    for x in (args[0], q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(msa.paged_sparse_attn_fp8(x, *args[1:], workspace=ws))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, (ref, ref2)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("k", [8, 12])
def test_wide_page_tables(msa, k):
    """More (group, block) keys than one CTA scans: the same result as with a narrow table."""
    c = Cache([300, 20, 40], [500, 300, 0], 128, 4, 128, 64, seed=91, wide=4096)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16()
    idx = selection(c, k)
    d = c.gpu(c.appended())
    o, lse = call(msa, c, d, q, idx)
    check(c, o, lse, attention(c, q, idx, 128**-0.5))
    d["table"] = d["table"][:, :8].contiguous()
    again, lse2 = call(msa, c, d, q, idx)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


def test_more_rows_than_a_window(msa):
    """A chunk longer than the window of rows whose partial results are held at once: what two calls give."""
    T, cut, ctx = 131072 + 700, 131072 - 300, 1000
    g = torch.Generator("cuda").manual_seed(5)
    n_pages = (ctx + T + 63) // 64
    kp, vp = (torch.randint(0, 120, (n_pages, 64, 1, 64), generator=g, device="cuda", dtype=torch.uint8) for _ in "kv")
    ks, vs = (torch.rand(n_pages, 64, 1, generator=g, device="cuda") * 0.01 + 0.01 for _ in "kv")
    q = torch.randn(T, 8, 64, generator=g, device="cuda").bfloat16()
    pos = torch.arange(T, device="cuda") + ctx
    own = pos // 64
    early = (torch.rand(T, generator=g, device="cuda") * own).long()
    idx = torch.stack([torch.minimum(early, own), torch.where(early < own, own, -1)], -1)[:, None].to(torch.int32).contiguous()
    table = torch.arange(n_pages, device="cuda", dtype=torch.int32)[None]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse = msa.paged_sparse_attn_fp8(q, idx, kp, ks, vp, vs, table, i32(0, T), i32(ctx))
    parts = [msa.paged_sparse_attn_fp8(q[a:b].contiguous(), idx[a:b].contiguous(), kp, ks, vp, vs, table, i32(0, b - a),
                                       i32(ctx + a)) for a, b in ((0, cut), (cut, T))]
    assert bool(torch.isfinite(lse).all())
    assert torch.equal(lse, torch.cat([p[1] for p in parts])) or float((lse - torch.cat([p[1] for p in parts])).abs().max()) < 1e-4
    ref = torch.cat([p[0] for p in parts]).float()
    assert float((o.float() - ref).abs().max()) <= 2.0**-7 * float(ref.abs().max())
