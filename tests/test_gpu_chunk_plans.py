"""A prompt served in chunks is the same prompt: whatever the cuts, the cache's
bytes and the selections are equal, and every row is within the attention's
derived tolerance of float64 (tests/chunk_util.py).

For selections to be equal, block scores must be exact, since the form that
computes them depends on how many rows a call has: index queries and keys are
whole numbers up to 7 in magnitude, and every key has a 7, so that its scale is
7 / 448 = 2^-6, its codes are exact (64 .. 448 in steps of 64) and a score is a
whole number below 2^24 times powers of two.  Ties go to the lower block."""
from __future__ import annotations

import pytest
import torch

from tests.chunk_util import Cache, attention, refresh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_gqa_idx_b200 as msa

    return msa


def whole_numbers(g, *shape):
    x = torch.randint(-7, 8, shape, generator=g).float()
    x.view(-1, shape[-1])[torch.arange(x.numel() // shape[-1]), torch.randint(0, shape[-1], (x.numel() // shape[-1],),
                                                                                  generator=g)] = 7.0
    return x.bfloat16()


PLANS = [  # lengths, B_k, k, the cuts: few rows a call, and calls of either form of the attention
    ([330, 201], 64, 4, [(1, 64), (100, 1), (0, 130), (229, 6)]),
    ([700, 500], 64, 16, [(1, 64), (100, 1), (0, 430), (599, 5)]),
    ([640, 3], 128, 10, [(128, 0), (127, 3), (385, 0)]),
]


@pytest.mark.parametrize("lens,B_k,kk,cuts", PLANS)
def test_cuts_do_not_matter(msa, lens, B_k, kk, cuts):
    S, d_model, H_q, H_kv, d_h, d_idx = 2, 256, 32, 4, 128, 64
    c = Cache(lens, [0, 0], B_k, H_kv, d_h, d_idx, seed=sum(lens), wide=14)
    g = torch.Generator("cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = [(r(d_model, n) * d_model**-0.5).bfloat16() for n in
         (H_q * d_h, H_kv * d_h, H_kv * d_h, H_kv * d_idx, d_idx)]
    nw = [(1 + 0.1 * r(d_h)).bfloat16() for _ in range(2)]
    # projected, normalised and rotated once, so that both plans get the same rows
    p = msa.project(r(c.T, d_model).bfloat16(), *w, H_q, H_kv)
    pos = msa.chunk_positions(c.cu.cuda(), c.len.cuda(), c.T)
    assert torch.equal(pos.cpu(), c.positions())
    q, k = msa.qk_norm_rope(p["q"], p["k"], nw[0], nw[1], pos, theta=1e6)
    c.rows["k"], c.rows["v"], c.rows["i"] = k.cpu(), p["v"].cpu(), whole_numbers(c.g, c.T, d_idx)
    refresh(c)
    qi = whole_numbers(c.g, c.T, H_kv, d_idx).cuda()
    last = [t.cuda() for t in (torch.randn(S, H_q, d_h, generator=c.g).bfloat16(), whole_numbers(c.g, S, H_kv, d_idx),
                               *(torch.randn(S, H_kv, d_h, generator=c.g).bfloat16() for _ in "kv"),
                               whole_numbers(c.g, S, d_idx))]
    outs = []
    for plan in ([tuple(lens)], cuts):
        assert [sum(n[s] for n in plan) for s in range(S)] == lens
        d = c.gpu()
        # the decode step's token has its page too
        d["table"].clamp_(0, c.n_pages - 1)
        at = [0, 0]
        o, lse = torch.zeros_like(q), torch.zeros(c.T, H_q, device="cuda")
        idx = torch.zeros(c.T, H_kv, kk, dtype=torch.int32, device="cuda")
        for n in plan:
            rows = torch.cat([torch.arange(n[s]) + int(c.cu[s]) + at[s] for s in range(S)]).cuda()
            take = lambda t: t[rows].contiguous()  # noqa: E731
            cu = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32).cuda()
            assert d["len"].cpu().tolist() == at
            o[rows], lse[rows], idx[rows] = msa.paged_chunk_fp8(
                take(q), take(qi), take(d["new_k"]), take(d["new_v"]), take(d["new_i"]), *c.pools(d), d["table"], cu,
                d["len"], kk)
            at = [a + b for a, b in zip(at, n)]
        live = []
        for s in range(S):
            page, slot = c.where(s, torch.arange(lens[s]))
            live += [t[page.cuda(), slot.cuda()] for t in c.pools(d)]
        dec = None
        if all(n % B_k for n in lens):  # the next token is in a page of its sequence
            dec, _ = msa.paged_decode_fp8(*last, *c.pools(d), d["table"], d["len"], B_k, kk)
        outs.append((o, lse, idx, live, dec))
    (o0, l0, i0, p0, d0), (o1, l1, i1, p1, d1) = outs
    assert torch.equal(i0, i1)
    for a, b, name in zip(p0, p1, "k ks v vs i is".split() * S):
        assert torch.equal(a, b), name
    for s in range(S):  # and they are the append rule's bytes
        assert torch.equal(p0[6 * s + 5].cpu(), torch.full((lens[s],), 2.0**-6))
    assert d0 is None or (torch.equal(d0, d1) and bool(torch.isfinite(d0).all()))
    ref = attention(c, q.cpu(), i0.cpu(), d_h**-0.5)
    for o, lse in ((o0, l0), (o1, l1)):
        assert bool(((o.cpu().double() - ref[0]).abs() <= ref[2]).all())
        assert bool(((lse.cpu().double() - ref[1]).abs() <= ref[3]).all())
    # the tolerance is tight enough to miss no key: with each row's own key left out, rows fail
    c.positions = lambda: torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]) - 1
    off = attention(c, q.cpu(), i0.cpu(), d_h**-0.5)
    wrong = ((ref[0] - off[0]).abs() > 2 * ref[2]).flatten(1).any(1)
    assert float(wrong.float().mean()) > 0.9


def test_step_is_its_parts_with_many_rows(msa):
    """The whole step and its parts, bit for bit, where the attention is KV-outer, with padding."""
    c = Cache([600, 0, 40], [300, 40, 700], 64, 4, 128, 64, seed=82, pad=40)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16()
    qi = torch.randn(c.T, 4, 64, generator=c.g).bfloat16()
    k = 16
    a, b = c.gpu(), c.gpu()
    msa.paged_append_fp8(a["new_k"], a["new_v"], a["new_i"], *c.pools(a), a["table"], a["cu"], a["len"])
    x = msa.paged_index_scores_fp8(qi.cuda(), a["ip"], a["is"], a["table"], a["cu"], a["len"])
    idx = msa.block_topk(x, msa.chunk_positions(a["cu"], a["len"], c.T), 64, k)
    o, lse = msa.paged_sparse_attn_fp8(q.cuda(), idx, *c.pools(a)[:4], a["table"], a["cu"], a["len"])
    d = msa.chunk_dims(c.S, c.T, c.max_pages, c.n_pages, 32, 4, 128, 64, 64, k)
    ws = torch.empty(msa.paged_chunk_fp8_workspace_size(d), dtype=torch.uint8, device="cuda")
    mark = [torch.full_like(o, 7.0), torch.full_like(lse, 7.0), torch.full_like(idx, 70000)]
    msa.profile_enable(True)
    try:
        got = msa.paged_chunk_fp8(q.cuda(), qi.cuda(), b["new_k"], b["new_v"], b["new_i"], *c.pools(b), b["table"],
                                  b["cu"], b["len"], k, o=mark[0], lse=mark[1], idx_out=mark[2], workspace=ws)
        assert "chunk_tile" in msa.profile_read()
    finally:
        msa.profile_enable(False)
    assert msa.device_status(ws) == (0, 0)
    live = c.positions() >= 0
    for m, r, fill in zip(got, (o, lse, idx), (7, 7, 70000)):
        assert torch.equal(m.cpu()[live], r.cpu()[live]) and bool((m.cpu()[~live] == fill).all())
    for n in ("kp", "ks", "vp", "vs", "ip", "is"):
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8))
    assert b["len"].cpu().tolist() == [900, 40, 740]
    ref = attention(c, q, idx.cpu(), 128**-0.5)
    assert bool(((o.cpu().double() - ref[0]).abs() <= ref[2])[live].all())
    assert bool(((lse.cpu().double() - ref[1]).abs() <= ref[3])[live].all())
