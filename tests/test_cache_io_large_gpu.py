"""sd_cache_write with boxes and sd_cache_read of batches so large that runs are not taken in parts (the box comes out of the
same pass over the rows) and every group of lanes takes several units: bit-exact against the formats' definition, worked
out on the GPU in 64 bits (checked against the references of the small tests first)."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _quantise(x, fmt):
    """(elements, scale bytes [..., 4], stored values as bf16) of finite bf16 rows on the GPU."""
    f = x.double().unflatten(-1, (4, 32))
    a = f.abs().amax(-1)
    lo, hi, most, bias = (-124, 119, 448.0, 127) if fmt == "mxfp8" else (-133, 121, 127.0, 133)
    e = torch.full(a.shape, hi, dtype=torch.int64, device=x.device)
    for k in range(hi, lo - 1, -1):
        y = a * 2.0 ** -k
        e = torch.where((y if fmt == "mxfp8" else y.round()) <= most, k, e)
    scale = torch.ldexp(torch.ones_like(a), e)[..., None]
    y = (f / scale).clamp(-most, most)
    el = y.float().to(torch.float8_e4m3fn) if fmt == "mxfp8" else y.round().to(torch.int8)
    return el.flatten(-2), (e + bias).to(torch.uint8), (el.double() * scale).flatten(-2).bfloat16()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_quantiser(fmt):
    x = torch.cat([torch.randn((50, 128)) * 2.0 ** k for k in (-125, -20, 0, 3, 100)]).bfloat16()
    el, by, val = _quantise(x.to(DEV), fmt)
    el0, by0 = ch.quantise(x, fmt)
    assert torch.equal(el.view(torch.uint8).cpu(), el0) and torch.equal(by.cpu(), by0)
    assert torch.equal(val.double().cpu(), ch.values(el0, by0, fmt))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_large_batches(fmt):
    Hkv, n, ctx = 16, [5000, 4999, 5017, 4983], [5, 16, 0, 37]
    total = [a + c for a, c in zip(n, ctx)]
    g = torch.Generator(DEV).manual_seed(70)
    pages = [(t + 15) // 16 for t in total]
    table = torch.zeros((4, max(pages)), dtype=torch.int32)
    perm, at = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(71)).to(torch.int32), 0
    for b, k in enumerate(pages):
        table[b, :k] = perm[at:at + k]
        at += k
    table = table.to(DEV)
    shape = sdb.make_shape(4, Hkv, Hkv, max(pages), 1, sum(pages))
    cache = sdb.empty_cache(shape, ch.FMTS[fmt], DEV)
    boxes = torch.full((sum(pages), Hkv, 2, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    starts = [torch.tensor([0] + x, dtype=torch.int32, device=DEV).cumsum(0, dtype=torch.int32) for x in (ctx, n, total)]
    new = [[(torch.randn((sum(x), Hkv, 128), generator=g, device=DEV) * 2).bfloat16() for x in (ctx, n)] for _ in range(2)]
    for i, (lens, at) in enumerate(((ctx, starts[0]), (total, starts[1]))):
        sdb.sd_cache_write(shape, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), at, new[0][i], new[1][i],
                           boxes, status)
    lens = torch.tensor(total, dtype=torch.int32, device=DEV)
    got = [torch.full((sum(total), Hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    sdb.sd_cache_read(shape, cache, table, lens, torch.zeros_like(lens), starts[2], got[0], got[1], status)
    assert int(status.item()) == 0
    row = 0
    for b in range(4):
        pos = torch.arange(total[b], device=DEV)
        pg, sl = table[b].long()[pos // 16], pos % 16
        for i in range(2):
            lo, hi = [sum(x[:b]) for x in (ctx, n)], [sum(x[:b + 1]) for x in (ctx, n)]
            want = torch.cat([new[i][s][lo[s]:hi[s]] for s in range(2)])
            if fmt != "bf16":
                el, by, want = _quantise(want, fmt)
                assert torch.equal(cache.tensors[i][pg, sl].view(torch.uint8), el.view(torch.uint8))
                assert torch.equal(cache.tensors[2][pg, :, sl, i], by)
            else:
                assert torch.equal(cache.tensors[i][pg, sl], want)
            assert torch.equal(got[i][row:row + total[b]], want)
            if i == 0:
                pad = torch.full((pages[b] * 16 - total[b], Hkv, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
                rows = torch.cat([want, pad]).view(pages[b], 16, Hkv, 128).float()
                box = boxes[table[b, :pages[b]].long()].float()
                assert torch.equal(box[:, :, 0], rows.nan_to_num(nan=float("inf")).amin(1))
                assert torch.equal(box[:, :, 1], rows.nan_to_num(nan=-float("inf")).amax(1))
        row += total[b]
