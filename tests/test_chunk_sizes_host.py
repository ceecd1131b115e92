"""Sizes that the C ABI's fields cannot hold are refused by the binding, not cut
to their low bits."""
from __future__ import annotations

import pytest


@pytest.fixture(scope="module")
def capi():
    from block_sparse_gqa_idx_b200 import build

    build.build()
    from block_sparse_gqa_idx_b200 import _capi

    return _capi


SIZES = dict(S=3, T=16, max_pages=8, n_pages=32, H_q=8, H_kv=2, d_h=128, d_idx=64, B_k=128, k=4)


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("by", [2**32, -(2**32), 2**64])
def test_chunk_sizes_that_do_not_fit(capi, name, by):
    if name == "n_pages" and abs(by) < 2**63:
        assert capi.chunk_dims(**dict(SIZES, n_pages=SIZES[name] + by)).n_pages == SIZES[name] + by
        return
    with pytest.raises(ValueError, match=name):
        capi.chunk_dims(**dict(SIZES, **{name: SIZES[name] + by}))


def test_the_largest_sizes_pass_through(capi):
    d = capi.chunk_dims(**dict(SIZES, T=2**31 - 1, max_pages=-(2**31), n_pages=2**63 - 1))
    assert (d.T, d.max_pages, d.n_pages) == (2**31 - 1, -(2**31), 2**63 - 1)


@pytest.mark.parametrize("at", range(5))
def test_norm_rope_sizes_that_do_not_fit(capi, at):
    sizes = [16, 8, 2, 128, 64, 0, 1e-6]
    assert capi._norm_rope_dims(*sizes)[0].T == 16
    sizes[at] += 2**32
    with pytest.raises(ValueError):
        capi._norm_rope_dims(*sizes)


def test_host_tensors_are_refused(capi):
    """As by every entry point: there is no other implementation to fall back to."""
    import torch

    T, S, P, B, H, d, di = 4, 2, 6, 64, 2, 64, 64
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    pages = [u8(P, B, H, d), torch.zeros(P, B, H), u8(P, B, H, d), torch.zeros(P, B, H)]
    pools = [*pages, u8(P, B, di), torch.zeros(P, B)]
    seqs = [i32(S, 3), i32(S + 1), i32(S)]
    q, k, qi, ki = bf(T, 2 * H, d), bf(T, H, d), bf(T, H, di), bf(T, di)
    w = bf(d)
    for call in (lambda: capi.qk_norm_rope(q, k, w, w, i32(T)),
                 lambda: capi.qk_norm_rope_bwd(q, k, w, w, i32(T), q, k),
                 lambda: capi.chunk_positions(seqs[1], seqs[2], T),
                 lambda: capi.paged_append_fp8(k, k, ki, *pools, *seqs),
                 lambda: capi.paged_gather_fp8(*pools, *seqs, T),
                 lambda: capi.paged_index_scores_fp8(qi, *pools[4:], *seqs),
                 lambda: capi.block_topk(torch.zeros(T, H, 3), i32(T), B, 2),
                 lambda: capi.paged_sparse_attn_fp8(q, i32(T, H, 2), *pages, *seqs),
                 lambda: capi.paged_chunk_fp8(q, qi, k, k, ki, *pools, *seqs, 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
