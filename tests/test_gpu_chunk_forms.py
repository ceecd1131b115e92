"""Which form of the chunk attention a call takes (by the names of the kernels
that it launches), and its results there (tests/chunk_util.py derives the
tolerances)."""
from __future__ import annotations

import pytest
import torch

from tests.chunk_util import Cache, attention, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_gqa_idx_b200 as msa

    return msa


KV_OUTER = [  # new, have, B_k, H_kv, G, d_h, k, pad: rows x selected keys x d_h of 2^28 and more
    ([300], [1000], 128, 4, 16, 128, 16, 2),
    ([530], [700], 64, 4, 16, 128, 16, 0),
    ([130] * 5 + [1] * 20, [130] * 25, 128, 4, 8, 128, 8, 0),
    ([300], [500], 128, 8, 1, 128, 8, 1),
    ([700, 0, 3], [10, 5, 700], 64, 8, 2, 64, 12, 0),
    ([300], [1000], 128, 4, 4, 128, 16, 0),
    ([600], [800], 128, 8, 2, 64, 8, 0),
    ([260], [500], 128, 4, 8, 128, 16, 0),
    ([530], [300], 64, 4, 16, 64, 32, 0),
]
QUERY_OUTER = [
    ([1] * 256, [200] * 256, 128, 4, 8, 128, 16, 0),           # a decode step: no two rows share a page
    ([1] * 128, [200] * 128, 128, 8, 4, 128, 16, 0),
    ([20] * 13 + [1] * 40, [130] * 53, 128, 4, 8, 128, 16, 0),  # few rows a sequence
    ([300], [500], 128, 4, 12, 128, 16, 0),                     # heads that do not divide 16
    ([250], [500], 128, 4, 8, 128, 16, 0),                      # too little work
]


@pytest.mark.parametrize("form,new,have,B_k,H_kv,G,d_h,k,pad", [("chunk_tile", *c) for c in KV_OUTER] +
                         [("chunk_attend", *c) for c in QUERY_OUTER])
def test_form_and_result(msa, form, new, have, B_k, H_kv, G, d_h, k, pad):
    c = Cache(new, have, B_k, H_kv, d_h, 64, seed=sum(new) + 3 * G, pad=pad)
    q = torch.randn(c.T, H_kv * G, d_h, generator=c.g).bfloat16()
    idx = selection(c, k, holes=True)
    d = c.gpu(c.appended())
    d_ = msa.chunk_dims(c.S, c.T, c.max_pages, c.n_pages, H_kv * G, H_kv, d_h, 64, B_k, k)
    ws = torch.empty(msa.paged_sparse_attn_fp8_workspace_size(d_), dtype=torch.uint8, device="cuda")
    msa.profile_enable(True)
    try:
        o, lse = msa.paged_sparse_attn_fp8(q.cuda(), idx.cuda(), *c.pools(d)[:4], d["table"], d["cu"], d["len"],
                                           workspace=ws)
        ran = set(msa.profile_read())
    finally:
        msa.profile_enable(False)
    assert {"chunk_tile", "chunk_attend"} & ran == {form}
    assert msa.device_status(ws) == (0, 0)
    live = c.positions() >= 0
    o, lse = o.double().cpu()[live], lse.double().cpu()[live]
    ro, rl, otol, ltol = (t[live] for t in attention(c, q, idx, d_h**-0.5))
    none = rl == -float("inf")
    assert torch.equal(lse == -float("inf"), none) and bool((o[none] == 0).all())
    assert bool(((o - ro).abs() <= otol)[~none].all()) and bool(((lse - rl).abs() <= ltol)[~none].all())


@pytest.mark.parametrize("wide", [4200, 9000])
def test_wide_tables_of_many_rows(msa, wide):
    """Page tables of more (group, block) pairs than one CTA scans (33600), and than a CTA counts in shared
    memory (72000): the KV-outer form gives what it gives with a narrow table, bit for bit."""
    c = Cache([700, 30], [500, 64], 64, 4, 128, 64, seed=93, wide=wide)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16()
    idx = selection(c, 16, holes=True)
    d = c.gpu(c.appended())
    narrow = d["table"][:, :24].contiguous()
    got = []
    for table in (d["table"], narrow):
        msa.profile_enable(True)
        try:
            got.append(msa.paged_sparse_attn_fp8(q.cuda(), idx.cuda(), *c.pools(d)[:4], table, d["cu"], d["len"]))
            ran = set(msa.profile_read())
        finally:
            msa.profile_enable(False)
        assert "chunk_tile" in ran and ("inv_count" in ran) == (table is not narrow)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    o, lse = (t.double().cpu() for t in got[0])
    ro, rl, otol, ltol = attention(c, q, idx, 128**-0.5)
    none = rl == -float("inf")
    assert bool(((o - ro).abs() <= otol)[~none].all()) and bool(((lse - rl).abs() <= ltol)[~none].all())
