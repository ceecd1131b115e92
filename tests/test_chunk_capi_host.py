"""CPU-side checks of the C ABI of the chunk operators: sizes and pointers are
refused on the host before anything is launched."""
from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module")
def capi():
    from block_sparse_gqa_idx_b200 import build

    build.build()
    from block_sparse_gqa_idx_b200 import _capi

    return _capi


FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 2)


def freqs(n, value=0.5):
    return (ctypes.c_double * n)(*[value] * n)


@pytest.mark.parametrize("field,value,status", [
    ("T", -1, 1), ("H_q", 0, 1), ("H_k", 0, 1), ("rot", -16, 1), ("rot", 144, 1), ("interleaved", 2, 1),
    ("eps", -1.0, 1), ("eps", float("inf"), 1), ("eps", float("nan"), 1), ("d", 96, 2), ("rot", 24, 2),
])
def test_norm_rope_rejects_on_host(capi, field, value, status):
    d = capi.msa_norm_rope_dims(16, 8, 2, 128, 64, 0, 1e-6)
    setattr(d, field, value)
    f = freqs(64)
    assert capi.LIB.msa_qk_norm_rope(ctypes.byref(d), f, *[FAKE] * 7, None) == status
    assert capi.LIB.msa_qk_norm_rope_bwd_workspace(ctypes.byref(d)) == 0
    assert capi.LIB.msa_qk_norm_rope_bwd(ctypes.byref(d), f, *[FAKE] * 12, 1 << 40, None) == status


def test_norm_rope_rejects_pointers_and_frequencies(capi):
    d = capi.msa_norm_rope_dims(16, 8, 2, 128, 64, 0, 1e-6)
    call = capi.LIB.msa_qk_norm_rope
    assert call(ctypes.byref(d), None, *[FAKE] * 7, None) == 1
    for bad in (float("nan"), float("inf"), 1e300):
        assert call(ctypes.byref(d), freqs(32, bad), *[FAKE] * 7, None) == 1
    for at in (0, 1, 4, 5, 6):  # q, k, pos, q_out, k_out
        for p in (None, ODD):
            args = [FAKE] * 7
            args[at] = p
            assert call(ctypes.byref(d), freqs(32), *args, None) == 1
    for at in (2, 3):  # the weights may be absent, but not misaligned
        args = [FAKE] * 7
        args[at] = ODD
        assert call(ctypes.byref(d), freqs(32), *args, None) == 1
    ws = capi.LIB.msa_qk_norm_rope_bwd_workspace(ctypes.byref(d))
    assert ws > 256
    assert capi.LIB.msa_qk_norm_rope_bwd(ctypes.byref(d), freqs(32), *[FAKE] * 12, ws - 1, None) == 3
    d.T = 0  # nothing to do: no pointer is needed
    assert call(ctypes.byref(d), freqs(32), *[None] * 7, None) == 0


def chunk(capi, **kw):
    v = dict(S=3, T=16, max_pages=8, n_pages=32, H_q=8, H_kv=2, d_h=128, d_idx=64, B_k=128, k=4)
    v.update(kw)
    return capi.chunk_dims(**v)


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), 1), (dict(T=-1), 1), (dict(max_pages=0), 1), (dict(n_pages=0), 1), (dict(H_kv=0), 1),
    (dict(B_k=32), 2), (dict(H_kv=9), 2), (dict(d_h=96), 2), (dict(d_idx=32), 2), (dict(attn_scale=-1.0), 1),
    (dict(idx_scale=float("nan")), 1), (dict(max_pages=1 << 25), 2), (dict(n_pages=1 << 31), 2),
    (dict(T=(1 << 31) - 1), 2),
])
def test_cache_calls_reject_sizes_on_host(capi, kw, status):
    d = chunk(capi, **kw)
    assert capi.LIB.msa_paged_append_fp8(ctypes.byref(d), *[FAKE] * 13, 1 << 20, None) == status
    assert capi.LIB.msa_paged_gather_fp8(ctypes.byref(d), *[FAKE] * 13, 1 << 20, None) == status


def test_cache_calls_reject_pointers_on_host(capi):
    d = chunk(capi)
    for fn in (capi.LIB.msa_paged_append_fp8, capi.LIB.msa_paged_gather_fp8):
        for at in range(12):
            for p in (None, ODD):
                args = [FAKE] * 13
                args[at] = p
                assert fn(ctypes.byref(d), *args, 256, None) == 1
        assert fn(ctypes.byref(d), *[FAKE] * 12, ODD, 256, None) == 1
        assert fn(ctypes.byref(d), *[FAKE] * 13, 255, None) == 3
        none = chunk(capi, T=0)
        assert fn(ctypes.byref(none), *[None] * 13, 0, None) == 0
    for at in range(3):
        args = [FAKE] * 3
        args[at] = None
        assert capi.LIB.msa_chunk_positions(ctypes.byref(d), *args, None) == 1


@pytest.mark.parametrize("kw,status", [(dict(S=0), 1), (dict(d_idx=32), 2), (dict(B_k=96), 2), (dict(H_kv=16), 2)])
def test_index_calls_reject_on_host(capi, kw, status):
    d = chunk(capi, **kw)
    assert capi.LIB.msa_paged_index_scores_fp8(ctypes.byref(d), *[FAKE] * 8, 256, None) == status
    d = chunk(capi)
    for at in range(7):
        for p in (None, ODD):
            args = [FAKE] * 8
            args[at] = p
            assert capi.LIB.msa_paged_index_scores_fp8(ctypes.byref(d), *args, 256, None) == 1
    assert capi.LIB.msa_paged_index_scores_fp8(ctypes.byref(d), *[FAKE] * 8, 16, None) == 3


@pytest.mark.parametrize("kw,status", [(dict(k=0), 1), (dict(k=33), 2), (dict(B_k=1), 2), (dict(T=-1), 1)])
def test_topk_rejects_on_host(capi, kw, status):
    d = chunk(capi, **kw)
    assert capi.LIB.msa_block_topk(ctypes.byref(d), FAKE, FAKE, FAKE, None) == status
    d = chunk(capi)
    for args in ((None, FAKE, FAKE), (FAKE, ODD, FAKE), (FAKE, FAKE, None)):
        assert capi.LIB.msa_block_topk(ctypes.byref(d), *args, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), 1), (dict(H_q=0), 1), (dict(H_q=7), 1), (dict(k=0), 1), (dict(k=33), 2), (dict(H_q=34), 2),
    (dict(d_h=32), 2), (dict(B_k=256), 2), (dict(attn_scale=float("inf")), 1), (dict(H_kv=16, H_q=16), 2),
])
def test_attention_rejects_sizes_on_host(capi, kw, status):
    d = chunk(capi, **kw)
    assert capi.LIB.msa_paged_sparse_attn_fp8_workspace(ctypes.byref(d)) == 0
    assert capi.LIB.msa_paged_sparse_attn_fp8(ctypes.byref(d), *[FAKE] * 12, 1 << 40, None) == status


def test_attention_rejects_pointers_on_host(capi):
    d = chunk(capi)
    n = capi.LIB.msa_paged_sparse_attn_fp8_workspace(ctypes.byref(d))
    assert n >= 256
    for at in range(12):
        for p in (None, ODD):
            if at == 10 and p is None:
                continue  # lse may be absent
            args = [FAKE] * 12
            args[at] = p
            assert capi.LIB.msa_paged_sparse_attn_fp8(ctypes.byref(d), *args, n, None) == 1
    assert capi.LIB.msa_paged_sparse_attn_fp8(ctypes.byref(d), *[FAKE] * 12, n - 1, None) == 3
    d = chunk(capi, T=0)
    assert capi.LIB.msa_paged_sparse_attn_fp8(ctypes.byref(d), *[None] * 12, 0, None) == 0


def test_step_rejects_on_host(capi):
    call, size = capi.LIB.msa_paged_chunk_fp8, capi.LIB.msa_paged_chunk_fp8_workspace
    for kw, status in ((dict(S=0), 1), (dict(d_idx=32), 2), (dict(d_h=96), 2), (dict(k=40), 2), (dict(H_q=3), 1)):
        d = chunk(capi, **kw)
        assert size(ctypes.byref(d)) == 0
        assert call(ctypes.byref(d), *[FAKE] * 18, 1 << 40, None) == status
    d = chunk(capi)
    n = size(ctypes.byref(d))
    assert n >= 256 + 4 * 16 + 4 * 16 * 2 * 8
    for at in range(18):
        for p in (None, ODD):
            if at == 15 and p is None:
                continue  # lse may be absent
            args = [FAKE] * 18
            args[at] = p
            assert call(ctypes.byref(d), *args, n, None) == 1
    assert call(ctypes.byref(d), *[FAKE] * 18, n - 1, None) == 3
