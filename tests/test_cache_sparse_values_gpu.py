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


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("B,Hq,Hkv,N,k", [(4, 64, 8, 32768, 16384), (12, 48, 16, 20000, 10000), (1, 8, 2, 131072, 65536)])
def test_long_selections_keep_fp32_accuracy(fmt, B, Hq, Hkv, N, k):
    """Many steps in one warp's share (148 x 12 warps, 16 rows a step), N(0, 1) rows, relative root mean square error.

    The result is the end of a random walk, so a partial sum after j of n steps is about sqrt(j / n) of it, and n additions
    rounded to nearest (2^-25 of the sum each, root mean square at most) leave sqrt(n / 2) 2^-25.  Each weight is off by its
    score (2^-23 absolute: eight partial sums of magnitude under 2), its exponential (2^-22) and its second half-precision
    part (2^-22), independently of the others and so in the same proportion in the result: under 2^-21 together."""
    G = Hq // Hkv
    pages = (N + 15) // 16
    g = torch.Generator(DEV).manual_seed(82)
    shape = sdb.make_shape(B, Hq, Hkv, pages, k, B * pages)
    cache = sdb.empty_cache(shape, ch.FMTS[fmt], DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.randperm(B * pages, generator=g, device=DEV).to(torch.int32).view(B, pages)
    lens = torch.full((B,), N, dtype=torch.int32, device=DEV)
    rows = torch.arange(B + 1, dtype=torch.int32, device=DEV) * N
    K, V = (torch.randn((B * N, Hkv, 128), generator=g, device=DEV).bfloat16() for _ in range(2))
    sdb.sd_cache_write(shape, cache, table, lens, rows, K, V, None, status)
    sdb.sd_cache_read(shape, cache, table, lens, torch.zeros_like(lens), rows, K, V, status)      # as stored
    q = torch.randn((B, Hq, 128), generator=g, device=DEV).bfloat16()
    idx = torch.stack([torch.rand((Hq, N), generator=g, device=DEV).topk(k, 1).indices.sort(1).values for _ in range(B)]).int()
    out = torch.zeros((B, Hq, 128), device=DEV)
    sdb.sd_cache_sparse_decode(shape, cache, q, table, lens, idx, out, sdb.workspace_for(shape, sdb.SD_OP_CACHE_SPARSE, DEV), status)
    assert int(status.item()) == 0
    err = ref = 0.0
    for b in range(B):
        for h in range(0, Hq, max(1, Hq // 8)):
            s = b * N + idx[b, h].long()
            r = torch.softmax(K[s, h // G].double() @ q[b, h].double() / 128 ** 0.5, 0) @ V[s, h // G].double()
            err += float((out[b, h].double() - r).square().sum())
            ref += float(r.square().sum())
    steps = max(1.0, B * Hq * k / (148 * 12) / 16)
    assert (err / ref) ** 0.5 <= 2.0 ** -25 * (steps / 2) ** 0.5 + 2.0 ** -21
