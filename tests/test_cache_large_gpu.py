"""Caches whose elements pass 32 bits of offset: a small batch whose pages lie at the end of more than 2^31 elements
gives the same as in a small cache, bit for bit (the same tiles, in the same order)."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_pages_past_32_bits(fmt):
    Hkv = 8
    w = ch.Batch([3, 1, 40], [300, 90, 17], 16, Hkv, fmt, seed=3)
    d = w.gpu()
    small = d.chunk()
    pages = (1 << 31) // (16 * Hkv * 128) + w.num_pages + 5
    shift = pages - w.num_pages
    el = d.K.dtype
    K, V = (torch.zeros((pages, 16, Hkv, 128), dtype=torch.uint8 if el != torch.bfloat16 else el, device=DEV) for _ in range(2))
    K[shift:] = d.K if el == torch.bfloat16 else d.K.view(torch.uint8)
    V[shift:] = d.V if el == torch.bfloat16 else d.V.view(torch.uint8)
    sc = None
    if d.scales is not None:
        sc = torch.zeros((pages, Hkv, 16, 2, 4), dtype=torch.uint8, device=DEV)
        sc[shift:] = d.scales
    cache = sdb.make_cache(ch.FMTS[fmt], K, V, sc)
    table = torch.where(d.page_table < w.num_pages, d.page_table + shift, d.page_table)
    shape = sdb.make_shape(w.B, w.Hq, Hkv, w.max_pages, 1, pages)
    out = torch.full_like(small, 7.0)
    sdb.sd_chunk_attention(shape, cache, d.q, table, d.lens, d.row_start, out, sdb.workspace_for(shape, sdb.SD_OP_CHUNK, DEV),
                           d.status)
    assert torch.equal(out, small)
    # the chunks' rows read back, and written again
    first = d.lens - torch.tensor(w.n, dtype=torch.int32, device=DEV)
    k, v = (torch.zeros((w.T, Hkv, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sdb.sd_cache_read(shape, cache, table, d.lens, first, d.row_start, k, v, d.status)
    for i, got in enumerate((k, v)):
        for b in range(w.B):
            assert torch.equal(got[w.start[b]:w.start[b + 1]].double().cpu(), w.rows(i, b, w.total[b] - w.n[b], w.total[b]))
    before = [x[shift:].clone() for x in (K, V)]
    boxes = torch.zeros((pages, Hkv, 2, 128), dtype=torch.bfloat16, device=DEV)
    sdb.sd_cache_write(shape, cache, table, d.lens, d.row_start, k, v, boxes, d.status)   # stored values are fixed points
    ko = torch.zeros_like(k)
    sdb.sd_cache_read(shape, cache, table, d.lens, first, d.row_start, ko, None, d.status)
    assert torch.equal(ko, k)
    assert not K[:shift].any() and not boxes[:shift].any()
    if fmt == "bf16":
        assert torch.equal(before[0], K[shift:])
    else:
        idx = torch.arange(0, 90, 3, dtype=torch.int32, device=DEV).expand(w.B, w.Hq, 30).clone()
        idx[2, :, 18:] = -1
        outs = []
        for c, t, n in ((d.cache, d.page_table, w.num_pages), (cache, table, pages)):
            s = sdb.make_shape(w.B, w.Hq, Hkv, w.max_pages, 30, n)
            o = torch.zeros((w.B, w.Hq, 128), dtype=torch.float32, device=DEV)
            sdb.sd_cache_sparse_decode(s, c, d.q[:w.B], t, d.lens, idx, o, sdb.workspace_for(s, sdb.SD_OP_CACHE_SPARSE, DEV), d.status)
            outs.append(o)
        assert (outs[0] - outs[1]).abs().max() <= 1e-5      # (rows were written again: the same values, maybe other scales)
    assert int(d.status.item()) == 0
