"""The chunk operators in a run together, as a server uses them: projections,
norm and rotation, prompts written and attended chunk by chunk on the paged FP8
cache, then single tokens by the decode step."""
from __future__ import annotations

import pytest
import torch

from tests.chunk_util import Cache, attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_gqa_idx_b200 as msa

    return msa


@pytest.mark.parametrize("new,have,pad", [([1, 1, 1], [500, 128, 127], 1), ([150, 0, 33, 1], [300, 40, 0, 700], 6)])
def test_step_is_its_parts(msa, new, have, pad):
    c = Cache(new, have, 64, 4, 128, 64, seed=81, pad=pad)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16()
    qi = torch.randn(c.T, 4, 64, generator=c.g).bfloat16()
    k = 5
    a, b = c.gpu(), c.gpu()
    msa.paged_append_fp8(a["new_k"], a["new_v"], a["new_i"], *c.pools(a), a["table"], a["cu"], a["len"])
    pos = msa.chunk_positions(a["cu"], a["len"], c.T)
    x = msa.paged_index_scores_fp8(qi.cuda(), a["ip"], a["is"], a["table"], a["cu"], a["len"])
    idx = msa.block_topk(x, pos, 64, k)
    o, lse = msa.paged_sparse_attn_fp8(q.cuda(), idx, *c.pools(a)[:4], a["table"], a["cu"], a["len"])
    d = msa.chunk_dims(c.S, c.T, c.max_pages, c.n_pages, 32, 4, 128, 64, 64, k)
    ws = torch.empty(msa.paged_chunk_fp8_workspace_size(d), dtype=torch.uint8, device="cuda")
    mark = [torch.full_like(o, 7.0), torch.full_like(lse, 7.0), torch.full_like(idx, 7)]
    got = msa.paged_chunk_fp8(q.cuda(), qi.cuda(), b["new_k"], b["new_v"], b["new_i"], *c.pools(b), b["table"], b["cu"],
                              b["len"], k, o=mark[0], lse=mark[1], idx_out=mark[2], workspace=ws)
    assert msa.device_status(ws) == (0, 0)
    live = c.positions() >= 0
    for m, r in zip(got, (o, lse, idx)):
        assert torch.equal(m.cpu()[live], r.cpu()[live]) and bool((m.cpu()[~live] == 7).all())
    for n in ("kp", "vp", "ip"):
        assert torch.equal(a[n], b[n])
    assert b["len"].cpu().tolist() == [n + h for n, h in zip(new, have)]
    ref = attention(c, q, idx.cpu(), 128**-0.5)
    assert bool(((o.cpu().double() - ref[0]).abs() <= ref[2])[live].all())


def test_step_skips_what_does_not_fit(msa):
    c = Cache([3, 4], [60, 60], 64, 2, 64, 64, seed=83)
    q, qi = torch.randn(7, 4, 64, generator=c.g).bfloat16().cuda(), torch.randn(7, 2, 64, generator=c.g).bfloat16().cuda()
    d = c.gpu()
    d["len"][0] = c.max_pages * 64 - 2
    full = [int(d["len"][0]), 64]
    mark = torch.full((7, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    msa.paged_chunk_fp8(q, qi, d["new_k"], d["new_v"], d["new_i"], *c.pools(d), d["table"], d["cu"], d["len"], 3,
                        o=mark, workspace=ws)
    assert msa.device_status(ws)[0] == 3
    assert d["len"].cpu().tolist() == full
    assert bool((mark[:3] == 7.0).all()) and bool(torch.isfinite(mark[3:]).all())


def test_prompts_in_chunks_then_decode(msa):
    """Two prompts through project -> qk_norm_rope -> paged_chunk_fp8 in chunks of different
    sizes give what one chunk gives, and the decode step continues on the cache."""
    S, d_model, H_q, H_kv, d_h, d_idx, B_k, kk = 2, 256, 16, 2, 64, 64, 64, 4
    lens = [330, 201]
    g = torch.Generator("cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = [(r(d_model, n) * d_model**-0.5).bfloat16() for n in
         (H_q * d_h, H_kv * d_h, H_kv * d_h, H_kv * d_idx, d_idx)]
    nw = [(1 + 0.1 * r(d_h)).bfloat16() for _ in range(2)] + [(1 + 0.1 * r(d_idx)).bfloat16() for _ in range(2)]
    x = [r(n, d_model).bfloat16() for n in lens]
    max_pages = 7

    def pools():
        P = S * max_pages
        u = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device="cuda")  # noqa: E731  NaN codes
        f = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
        return [u(P, B_k, H_kv, d_h), f(P, B_k, H_kv), u(P, B_k, H_kv, d_h), f(P, B_k, H_kv), u(P, B_k, d_idx), f(P, B_k)]

    def rows(rows_of, cu, seq_len):
        tokens = torch.cat(rows_of)
        p = msa.project(tokens, *w, H_q, H_kv)
        pos = msa.chunk_positions(cu, seq_len, tokens.shape[0])
        q, k = msa.qk_norm_rope(p["q"], p["k"], nw[0], nw[1], pos, theta=1e6)
        qi, ki = msa.qk_norm_rope(p["q_idx"], p["k_idx"][:, None, :], nw[2], nw[3], pos, theta=1e6)
        return q, qi, k, p["v"], ki[:, 0].contiguous()

    outs = []
    for plan in ([(330, 201)], [(1, 64), (100, 1), (0, 130), (229, 6)]):
        table = torch.randperm(S * max_pages, generator=torch.Generator().manual_seed(1)).view(S, max_pages).int().cuda()
        pool, seq_len = pools(), torch.zeros(S, dtype=torch.int32, device="cuda")
        at, parts = [0, 0], [[], []]
        for n in plan:
            cu = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32).cuda()
            args = rows([x[s][at[s]: at[s] + n[s]] for s in range(S)], cu, seq_len)
            o, lse, idx = msa.paged_chunk_fp8(*args, *pool, table, cu, seq_len, kk)
            for s, (a, b) in enumerate(((0, n[0]), (n[0], n[0] + n[1]))):
                parts[s].append((o[a:b], lse[a:b], idx[a:b]))
                at[s] += n[s]
        assert seq_len.cpu().tolist() == lens
        whole = [torch.cat([torch.cat([p[j] for p in parts[s]]) for s in range(S)]) for j in range(3)]
        cu = torch.arange(S + 1, dtype=torch.int32).cuda()
        args = rows([x[s][:1] * 0.5 for s in range(S)], cu, seq_len)
        dec, _ = msa.paged_decode_fp8(*args, *pool, table, seq_len, B_k, kk)
        outs.append((*whole, dec, *[p.clone() for p in pool]))
    # the projections' products may differ in their last bits with the number of rows: the cache
    # and the results agree to the formats' steps, not bit for bit
    (o0, l0, i0, d0, *_), (o1, l1, i1, d1, *_) = outs
    same = (i0 == i1).all(-1).all(-1)
    assert float(same.float().mean()) > 0.9
    assert bool(torch.isfinite(o0).all()) and bool(torch.isfinite(d0).all())
    assert float((o0 - o1)[same].float().abs().max()) <= 2.0**-3 * float(o0.float().abs().max())
    assert float((l0 - l1)[same].abs().max()) <= 0.1
    assert float((d0 - d1).float().norm()) <= 0.2 * float(d0.float().norm())


def test_captured_step_serves_growing_sequences(msa):
    """One captured step, replayed as the sequences grow (the offsets are read on the device)."""
    c = Cache([1, 2, 0], [62, 5, 9], 64, 2, 64, 64, seed=85)
    q, qi = torch.randn(3, 8, 64, generator=c.g).bfloat16().cuda(), torch.randn(3, 2, 64, generator=c.g).bfloat16().cuda()
    a, b = c.gpu(), c.gpu()
    args = lambda d: (q, qi, d["new_k"], d["new_v"], d["new_i"], *c.pools(d), d["table"], d["cu"], d["len"], 2)  # noqa: E731
    a["table"].clamp_(0, c.n_pages - 1)
    b["table"].clamp_(0, c.n_pages - 1)
    msa.paged_chunk_fp8(*args(c.gpu()))  # first call of the process outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse, idx = msa.paged_chunk_fp8(*args(a))
    for step in range(5):
        graph.replay()
        ref = msa.paged_chunk_fp8(*args(b))
        torch.cuda.synchronize()
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1]) and torch.equal(idx, ref[2])
        assert a["len"].cpu().tolist() == [63 + step, 7 + 2 * step, 9]


@pytest.mark.parametrize("T,H_kv,k", [(0, 2, 3), (5, 2, 3), (700, 8, 16)])
def test_nothing_but_padding(msa, T, H_kv, k):
    """No rows at all, or only rows that no sequence holds (few, and as many as the forms for long
    chunks take): nothing is read, and what the caller handed in stays as it was."""
    c = Cache([0, 0], [300, 5], 128, H_kv, 128, 64, seed=87, pad=T)
    d = c.gpu()
    before = [p.clone() for p in c.pools(d)]
    q, qi = torch.randn(T, 8 * H_kv, 128).bfloat16().cuda(), torch.randn(T, H_kv, 64).bfloat16().cuda()
    o = torch.full_like(q, 3.0)
    lse = torch.full((T, 8 * H_kv), 4.0, device="cuda")
    scores = torch.full((T, H_kv, c.max_pages), 5.0, device="cuda")
    idx = torch.full((T, H_kv, k), 6, dtype=torch.int32, device="cuda")
    where = (d["table"], d["cu"], d["len"])
    assert bool((msa.chunk_positions(d["cu"], d["len"], T) == -1).all())
    msa.paged_append_fp8(d["new_k"], d["new_v"], d["new_i"], *c.pools(d), *where)
    rows = msa.paged_gather_fp8(*c.pools(d), *where, T, out=tuple(t.fill_(2.0) for t in (
        torch.empty_like(d["new_k"]), torch.empty_like(d["new_v"]), torch.empty_like(d["new_i"]))))
    msa.paged_index_scores_fp8(qi, *c.pools(d)[4:], *where, scores=scores)
    msa.block_topk(scores, torch.full((T,), -1, dtype=torch.int32, device="cuda"), 128, k, idx_out=idx)
    msa.paged_sparse_attn_fp8(q, idx, *c.pools(d)[:4], *where, o=o, lse=lse)
    msa.paged_chunk_fp8(q, qi, d["new_k"], d["new_v"], d["new_i"], *c.pools(d), *where, k, o=o, lse=lse, idx_out=idx)
    torch.cuda.synchronize()
    for got, mark in ((o, 3.0), (lse, 4.0), (scores, 5.0), (idx, 6), *((r, 2.0) for r in rows)):
        assert bool((got == mark).all())
    for a, b in zip(c.pools(d), before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert d["len"].cpu().tolist() == [300, 5]


@pytest.mark.parametrize("new,have", [([1, 2], [300, 127]), ([560, 40], [300, 900])])
def test_pages_beyond_four_gigabytes(msa, new, have):
    """Pages whose byte offsets pass 32 bits give what the same pages give in a small pool."""
    c = Cache(new, have, 128, 8, 128, 64, seed=41)
    q, qi = torch.randn(c.T, 16, 128, generator=c.g).bfloat16().cuda(), torch.randn(c.T, 8, 64, generator=c.g).bfloat16().cuda()
    small = c.gpu()
    at = (1 << 32) // (128 * 8 * 128) + 3  # the first page of the sequences in the large pool
    big = dict(small, len=small["len"].clone(), table=small["table"] + at)
    for n in ("kp", "ks", "vp", "vs", "ip", "is"):
        big[n] = torch.empty(at + c.n_pages, *small[n].shape[1:], dtype=small[n].dtype, device="cuda")
        big[n][at:] = small[n]
    assert big["kp"][at:].data_ptr() - big["kp"].data_ptr() > 1 << 32
    got = []
    for d in (small, big):
        got.append(msa.paged_chunk_fp8(q, qi, d["new_k"], d["new_v"], d["new_i"], *c.pools(d), d["table"], d["cu"],
                                       d["len"], 6))
        cu = torch.tensor([0, 200, 320], dtype=torch.int32).cuda()
        got[-1] += msa.paged_gather_fp8(*c.pools(d), d["table"], cu, torch.zeros(2, dtype=torch.int32).cuda(), 320)
    for a, b in zip(*got):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)
