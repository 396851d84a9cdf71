"""sd_chunk_attention where each CTA (or warp) goes through many consecutive key/value tiles of an item: rings of copies that
wrap, sums and products over many tiles against a reference that lags or is taken anew.  References in 64 bits on the
GPU, from the values that sd_cache_read gives (which has exact tests of its own).

How long the stretches are: items of 2 floor(128 / G) tokens have a unit per 128 positions (and three more), the units of a
batch are cut evenly over 148 CTAs.  200 tokens: 4 requests x 8 heads x 4 items x 96 units, 83 to a CTA (the two tiles of
an item side by side); 20 tokens: one item of one tile per head, 20 to a CTA (its units alternate between two sides).  Over
8-bit caches one or two tokens are streamed by 1776 warps, 22 pages each.

Tolerance: tests/cache_helpers.py.  Scores here reach 2^9, in base-2 units 2^9.5; q.K and the exponent's fused product are
rounded at that magnitude, 2^-24 of it each, a few times: under 2^-12 in the exponent, which leaves more than half of the
quarter of 2^-8 that is in the bound for it.  Half-precision weights: tests/test_chunk_extremes_gpu.py."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
Hq, Hkv, G = 32, 8, 4
CTX = [12000, 11900, 12111, 11777]


def _keys(what, N, g):
    """K rows [N][Hkv][128] and q rows' common part."""
    k = torch.randn((N, Hkv, 128), generator=g, device=DEV)
    u = torch.where(torch.arange(128, device=DEV) % 2 == 0, 1.0, -1.0)
    p = torch.arange(N, device=DEV)
    if what == "random":
        return k, 0 * u
    if what == "growing":        # by some 70 over the context, in every tile
        return k + (p / N * 3.0)[:, None, None] * u, 2.0 * u
    if what == "falling":        # the first tiles hold the maximum, later ones lose it slowly
        return k - (p / N * 3.0)[:, None, None] * u, 2.0 * u
    # jumps by hundreds up and down, at positions inside every CTA's stretch
    step = torch.tensor([0.0, 1.0, -1.0, 6.0, 6.0, 14.0, 2.0, 14.5], device=DEV)[(p // 700) % 8]
    return 0.25 * k + step[:, None, None] * u, 1.0 * u


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("n", [1, 2, 20, 200])
@pytest.mark.parametrize("what", ["random", "growing", "falling", "jumping"])
def test_many_tiles(fmt, n, what):
    g = torch.Generator(DEV).manual_seed(60 + n)
    total = [c + n for c in CTX]
    pages = [(t + 15) // 16 for t in total]
    table = torch.zeros((4, max(pages)), dtype=torch.int32)
    perm, at = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(n)).to(torch.int32), 0
    for b, k in enumerate(pages):
        table[b, :k] = perm[at:at + k]
        at += k
    table = table.to(DEV)
    shape = sdb.make_shape(4, Hq, Hkv, max(pages), 1, sum(pages))
    cache = sdb.empty_cache(shape, ch.FMTS[fmt], DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.tensor(total, dtype=torch.int32, device=DEV)
    all_rows = torch.tensor([0] + total, dtype=torch.int32, device=DEV).cumsum(0, dtype=torch.int32)
    parts = [_keys(what, t, g) for t in total]
    K = torch.cat([k for k, _ in parts]).bfloat16()
    V = torch.randn(K.shape, generator=g, device=DEV).bfloat16()
    sdb.sd_cache_write(shape, cache, table, lens, all_rows, K, V, None, status)
    sdb.sd_cache_read(shape, cache, table, lens, torch.zeros_like(lens), all_rows, K, V, status)   # as stored
    q = (torch.randn((4 * n, Hq, 128), generator=g, device=DEV) + parts[0][1]).bfloat16()
    out = torch.full((4 * n, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    start = torch.arange(0, 4 * n + 1, n, dtype=torch.int32, device=DEV)
    ws = sdb.workspace_for(shape, sdb.SD_OP_CHUNK, DEV)
    sdb.sd_chunk_attention(shape, cache, q, table, lens, start, out, ws, status)
    assert int(status.item()) == 0
    at = 0
    for b, t in enumerate(total):
        k, v = (x[at:at + t].double().permute(1, 0, 2) for x in (K, V))               # [Hkv][N][128]
        half = None
        if fmt != "bf16" and n * G <= 8:
            pos = torch.arange(t, device=DEV)
            byte = cache.tensors[2][table[b].long()[pos // 16], :, pos % 16, 1].double()
            S = torch.exp2(byte - 127.0).repeat_interleave(32, 2).permute(1, 0, 2)      # [Hkv][N][128]
            half = (S, (v / S).abs())
        at += t
        for j in sorted({0, 1, 31, 32, 63, 64, 65, 127, 128, n // 2, n - 2, n - 1} & set(range(n))):
            seen = t - n + j + 1
            s = torch.einsum("hgd,hnd->hgn", q[b * n + j].double().view(Hkv, G, 128), k[:, :seen]) / 128 ** 0.5
            w = torch.softmax(s, 2)
            r, A = torch.einsum("hgn,hnd->hgd", w, v[:, :seen]), torch.einsum("hgn,hnd->hgd", w, v[:, :seen].abs())
            bound = 2.0 ** -8 * r.abs() + 1.25 * 2.0 ** -8 * A + 2.0 ** -134
            if half is not None:
                top = torch.stack([(w[:, i, :, None] * half[0][:, :seen]).amax(1) for i in range(G)], 1)
                bound = bound + 2.0 ** -30 * top * half[1][:, :seen].sum(1)[:, None]
            bad = ~((out[b * n + j].double().view(Hkv, G, 128) - r).abs() <= bound)
            assert not bad.any(), (b, j, float(((out[b * n + j].double().view(Hkv, G, 128) - r).abs() / bound).max()))
