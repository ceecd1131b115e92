"""paged_decode_fp8 on pages whose unwritten part holds any bytes (memory that
was never cleared): NaN codes and scales behind a sequence change nothing."""
from __future__ import annotations

import pytest
import torch

from tests.chunk_util import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B_k,d_h", [(128, 128), (64, 64), (64, 128), (128, 64)])
def test_stale_bytes_behind_a_sequence(B_k, d_h):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_gqa_idx_b200 as msa

    c = Cache([1, 1, 1], [500, 1300, 127], B_k, 4, d_h, 64, seed=71)
    q = torch.randn(3, 32, d_h, generator=c.g).bfloat16().cuda()
    qi = torch.randn(3, 4, 64, generator=c.g).bfloat16().cuda()
    outs = []
    for clean in (False, True):
        d = c.gpu()
        table = d["table"].clamp(0, c.n_pages - 1)
        if clean:
            for s in range(3):
                page, slot = c.where(s, torch.arange(c.have[s], (c.have[s] + B_k) // B_k * B_k))
                for n in "kvi":
                    d[n + "p"][page.cuda(), slot.cuda()] = 0
                    d[n + "s"][page.cuda(), slot.cuda()] = 1.0
        o, _ = msa.paged_decode_fp8(q, qi, d["new_k"], d["new_v"], d["new_i"], *c.pools(d), table, d["len"], B_k, 5)
        outs.append(o)
    assert bool(torch.isfinite(outs[0]).all()) and torch.equal(*outs)
