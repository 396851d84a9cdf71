"""sd_cache_sparse_decode over values of any finite magnitude, in 64 bits.

Tolerance: 1.25 * 2^-14 A (tests/test_cache_sparse_gpu.py; a weight's two half-precision parts are good to 2^-22 of the
block's largest product of weight and scale, which here lies within 2^12 of all others), and 2^-148 for the last places that
fp32 has below its normal range."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("power", [-118, -112, -100, -60, 0, 60, 100])
@pytest.mark.parametrize("k", [5, 300])
def test_magnitudes(fmt, power, k):
    w = ch.Batch([1, 1], [699, 310], 8, 2, fmt, seed=80)
    w.q *= 0.25                       # weights within some powers of two
    w.src[1] = (w.src[1].float() * 2.0 ** power).bfloat16()
    w.encode()
    d = w.gpu()
    g = torch.Generator().manual_seed(81)
    idx = torch.stack([torch.stack([torch.randperm(w.total[b], generator=g)[:k].sort().values for _ in range(8)]) for b in range(2)])
    idx = idx.to(torch.int32)
    out = torch.full((2, 8, 128), 7.0, dtype=torch.float32, device=DEV)
    shape = w.shape(k)
    sdb.sd_cache_sparse_decode(shape, d.cache, d.q, d.page_table, d.lens, idx.to(DEV), out,
                               sdb.workspace_for(shape, sdb.SD_OP_CACHE_SPARSE, DEV), d.status)
    assert int(d.status.item()) == 0
    out = out.double().cpu()
    for b in range(2):
        K, V = (w.rows(i, b, 0, w.total[b]) for i in (0, 1))
        for h in range(8):
            s = idx[b, h].long()
            wt = torch.softmax(K[s, h // 4] @ w.q[b, h].double() / 128 ** 0.5, 0)
            r, A = wt @ V[s, h // 4], wt @ V[s, h // 4].abs()
            assert ((out[b, h] - r).abs() <= 1.25 * 2.0 ** -14 * A + 2.0 ** -148).all(), (b, h)
