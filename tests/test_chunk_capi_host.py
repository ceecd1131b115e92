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
