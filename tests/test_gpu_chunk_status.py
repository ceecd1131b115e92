"""What the chunk operators record in the status word, and what they leave out
of it: rows that a call skips have no entries to report."""
from __future__ import annotations

import time

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


# few rows (query-outer), and as many as the KV-outer form takes, with a narrow page table and with
# tables of so many (group, block) pairs that the inverse index counts them over several CTAs
SHAPES = [([5, 1], [300, 90], 0), ([1030, 9], [1000, 64], 0), ([1030, 9], [1000, 64], 4200)]


@pytest.mark.parametrize("new,have,wide", SHAPES)
@pytest.mark.parametrize("left", [2**31 - 1, -7, 1 << 20])
def test_entries_of_padding_rows_are_not_read(msa, new, have, wide, left):
    """Whatever lies in the selection of a padding row, nothing is recorded and nothing is written."""
    c = Cache(new, have, 64, 4, 128, 64, seed=95, pad=70, wide=wide)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16()
    idx = selection(c, 16)
    live = c.positions() >= 0
    idx[~live] = left
    d = c.gpu(c.appended())
    o = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    d_ = msa.chunk_dims(c.S, c.T, c.max_pages, c.n_pages, 32, 4, 128, 64, 64, 16)
    ws = torch.empty(msa.paged_sparse_attn_fp8_workspace_size(d_), dtype=torch.uint8, device="cuda")
    msa.paged_sparse_attn_fp8(q.cuda(), idx.cuda(), *c.pools(d)[:4], d["table"], d["cu"], d["len"], o=o, lse=lse,
                              workspace=ws)
    assert msa.device_status(ws) == (0, 0)
    assert bool((o.cpu()[~live] == 3.0).all()) and bool((lse.cpu()[~live] == 3.0).all())
    ref = attention(c, q, idx, 128**-0.5)
    assert bool(((o.cpu().double() - ref[0]).abs() <= ref[2])[live].all())


@pytest.mark.parametrize("new,have,wide", SHAPES)
def test_entries_of_a_sequence_that_does_not_fit_are_not_read(msa, new, have, wide):
    """Its rows are skipped: the status is that of the full cache, wherever the sequence stands."""
    c = Cache(new, have, 64, 4, 128, 64, seed=96, wide=wide)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16()
    idx = selection(c, 16)
    idx[new[0]:] = 2**31 - 1
    d = c.gpu(c.appended())
    d["len"][1] = c.max_pages * 64
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    o = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    msa.paged_sparse_attn_fp8(q.cuda(), idx.cuda(), *c.pools(d)[:4], d["table"], d["cu"], d["len"], o=o, workspace=ws)
    assert msa.device_status(ws)[0] == 3
    assert bool((o.cpu()[new[0]:] == 3.0).all()) and bool((o.cpu()[: new[0]] != 3.0).any())


@pytest.mark.parametrize("new,have,wide", SHAPES)
def test_step_with_padding_records_nothing(msa, new, have, wide):
    """The whole step leaves the selection of padding rows as the caller had it, and does not read it."""
    c = Cache(new, have, 64, 4, 128, 64, seed=97, pad=70, wide=wide)
    q = torch.randn(c.T, 32, 128, generator=c.g).bfloat16().cuda()
    qi = torch.randn(c.T, 4, 64, generator=c.g).bfloat16().cuda()
    d = c.gpu()
    d_ = msa.chunk_dims(c.S, c.T, c.max_pages, c.n_pages, 32, 4, 128, 64, 64, 16)
    ws = torch.empty(msa.paged_chunk_fp8_workspace_size(d_), dtype=torch.uint8, device="cuda")
    idx = torch.full((c.T, 4, 16), -9, dtype=torch.int32, device="cuda")
    msa.paged_chunk_fp8(q, qi, d["new_k"], d["new_v"], d["new_i"], *c.pools(d), d["table"], d["cu"], d["len"], 16,
                        idx_out=idx, workspace=ws)
    assert msa.device_status(ws) == (0, 0)
    live = (c.positions() >= 0).cuda()
    assert bool((idx[~live] == -9).all()) and bool((idx[live] >= -1).all())


def test_a_timeout_takes_the_place_of_another_error(msa):
    """An ignored entry, recorded first, does not hide that a wait gave up: outputs are invalid then.
    (The entry's code is written here while the self-test's wait is running.)"""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    word = ws.view(torch.int32)
    bad_index = torch.tensor([2, 141], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    waits, other = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):  # again where the host was held up for longer than the wait
        msa.selftest_bounded_wait(ws, stream=waits)
        time.sleep(0.3)  # of the wait's two seconds
        with torch.cuda.stream(other):
            word[:2].copy_(bad_index)
        other.synchronize()
        running = not waits.query()
        status = msa.device_status(ws, stream=waits)
        if running:
            break
    assert running and status == (1, 99)
