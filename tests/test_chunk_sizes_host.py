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
