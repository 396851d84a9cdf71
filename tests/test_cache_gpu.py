"""sd_cache_write and sd_cache_read: bit-exact against the formats' definition, at block borders, ties, zeros,
subnormals, infinities and NaN, over ragged batches; the Quest boxes that a write keeps; bad inputs.  Quantised
bytes have to be equal: every step but the rounding is exact, so there is no tolerance."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _special_rows(g):
    """Rows [m][1][128] at the formats' borders."""
    x = torch.randn((40, 128), generator=g)
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 2.0 ** -133                          # bf16's smallest
    x[3] = 127 * 2.0 ** -133
    x[4, ::3] = 3.3895313892515355e38           # its largest
    x[5] = torch.linspace(-1, 1, 128) * 448.0
    x[6] = torch.linspace(-1, 1, 128) * 449.0   # amax just above 448 after rounding to bf16
    x[6, 0] = 450.0
    x[7] = torch.linspace(-1, 1, 128) * 127.0
    x[8] = torch.linspace(-1, 1, 128) * 127.5   # 127.5 would round to 128
    x[9, 5], x[9, 40] = float("inf"), -float("inf")
    x[10, 127] = float("nan")
    x[11] = torch.arange(128) * 0.5             # ties
    x[12] = (torch.arange(128) - 64) * 2.0 ** -9
    x[13] = 2.0 ** -126
    x[14, :32], x[14, 32:64], x[14, 64:96], x[14, 96:] = 1e-38, 1.0, 1e30, 0.0
    x[15:25] *= 2.0 ** torch.arange(-130, 120, 25)[:10, None].float()
    x[25:] *= torch.exp(3 * torch.randn((15, 128), generator=g))
    return x.bfloat16()[:, None]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_write_and_read_of_border_values(fmt):
    g = torch.Generator().manual_seed(3)
    rows = _special_rows(g)
    m = rows.shape[0]
    w = ch.Batch([m], [0], 1, 1, fmt)
    d = w.gpu()
    d.K.view(torch.uint8).zero_()
    d.V.view(torch.uint8).zero_()
    k, v = rows.to(DEV), rows.flip(0).contiguous().to(DEV)
    sdb.sd_cache_write(d.shape, d.cache, d.page_table, d.lens, d.row_start, k, v, None, d.status)
    ko, vo = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
    first = torch.zeros(1, dtype=torch.int32, device=DEV)
    sdb.sd_cache_read(d.shape, d.cache, d.page_table, d.lens, first, d.row_start, ko, vo, d.status)
    assert int(d.status.item()) == 0
    pos = torch.arange(m)
    pg = w.page_table[0].long()[pos // 16]
    for i, (src, cache, back) in enumerate(((k, d.K, ko), (v, d.V, vo))):
        if fmt == "bf16":
            assert torch.equal(back.view(torch.int16), src.view(torch.int16))
            continue
        el, by = ch.quantise(src, fmt)
        assert torch.equal(cache.cpu().view(torch.uint8)[pg, pos % 16], el)
        assert torch.equal(d.scales.cpu()[pg, :, pos % 16, i], by)
        assert torch.equal(torch.nan_to_num(back.double().cpu(), nan=1e300), torch.nan_to_num(ch.values(el, by, fmt), nan=1e300))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_every_element_code_reads_back(fmt):
    """All codes under all scale bytes the format can store."""
    codes = [u for u in range(256) if not (fmt == "mxfp8" and (u & 127) == 127) and not (fmt == "mxint8" and u == 128)]
    by_all = list(range(3, 247)) if fmt == "mxfp8" else list(range(0, 255))
    rows = len(by_all) * 2
    w = ch.Batch([rows], [0], 1, 1, fmt, spare=0)
    el = torch.tensor((codes * 2)[:256], dtype=torch.uint8).view(1, 2, 128).expand(len(by_all), 2, 128).reshape(rows, 128)
    by = torch.tensor(by_all, dtype=torch.uint8).repeat_interleave(2)[:, None].expand(rows, 4)
    pos = torch.arange(rows)
    pg = w.page_table[0].long()[pos // 16]
    K = torch.zeros((w.num_pages, 16, 1, 128), dtype=torch.uint8)
    sc = torch.zeros((w.num_pages, 1, 16, 2, 4), dtype=torch.uint8)
    K[pg, pos % 16, 0] = el
    sc[pg, 0, pos % 16, 0] = by
    sc[pg, 0, pos % 16, 1] = by
    K, sc = K.to(DEV), sc.to(DEV)
    d = w.gpu()
    cache = sdb.make_cache(ch.FMTS[fmt], K, K, sc)
    out = torch.zeros((rows, 1, 128), dtype=torch.bfloat16, device=DEV)
    first = torch.zeros(1, dtype=torch.int32, device=DEV)
    sdb.sd_cache_read(d.shape, cache, d.page_table, d.lens, first, d.row_start, out, None, d.status)
    assert int(d.status.item()) == 0
    assert torch.equal(out[:, 0].double().cpu(), ch.values(el.contiguous(), by.contiguous(), fmt))


CASES = [
    # n, ctx, Hkv, pad, lead
    ([1], [0], 1, 0, 0),
    ([1, 1, 1], [15, 16, 17], 2, 0, 0),
    ([0, 5, 0, 33, 1], [7, 0, 0, 30, 63], 3, 4, 2),
    ([200, 17], [9, 640], 8, 0, 0),
    ([3] * 40, list(range(40)), 5, 1, 0),
    ([700], [5], 16, 0, 3),
]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("boxes", [False, True])
def test_ragged_write(fmt, case, boxes):
    n, ctx, Hkv, pad, lead = case
    w = ch.Batch(n, ctx, Hkv, Hkv, fmt, seed=len(n), pad=pad, lead=lead)
    new = [torch.randn((w.T, Hkv, 128), generator=torch.Generator().manual_seed(9 + i)).bfloat16() for i in range(2)]
    d = w.gpu()
    box0 = torch.full((w.num_pages, Hkv, 2, 128), 3.0, dtype=torch.bfloat16)
    if boxes:       # the pages that new rows join hold the boxes of their earlier rows
        for b in range(w.B):
            old = w.total[b] - w.n[b]
            if old % 16 and w.n[b]:
                k = w.rows(0, b, old // 16 * 16, old)
                pg = int(w.page_table[b, old // 16])
                box0[pg, :, 0], box0[pg, :, 1] = k.amin(0).bfloat16(), k.amax(0).bfloat16()
    box = box0.to(DEV) if boxes else None
    sdb.sd_cache_write(d.shape, d.cache, d.page_table, d.lens, d.row_start, new[0].to(DEV), new[1].to(DEV), box, d.status)
    assert int(d.status.item()) == 0
    for b in range(w.B):
        for j in range(w.n[b]):
            p = w.total[b] - w.n[b] + j
            pg, sl = int(w.page_table[b, p // 16]), p % 16
            for i in range(2):
                w.src[i][pg, sl] = new[i][w.start[b] + j]
    w.encode()
    for got, want in zip((d.K, d.V), w.kv):       # rows that were not written are as they were
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
    if fmt != "bf16":
        assert torch.equal(d.scales.cpu(), w.scales)
    if boxes:
        want = box0.clone()
        for b in range(w.B):
            lo = (w.total[b] - w.n[b]) // 16 if w.n[b] else 1 << 30
            for pi in range(lo, (w.total[b] + 15) // 16):
                k = w.rows(0, b, pi * 16, min(w.total[b], pi * 16 + 16))
                pg = int(w.page_table[b, pi])
                want[pg, :, 0], want[pg, :, 1] = k.amin(0).bfloat16(), k.amax(0).bfloat16()
        assert torch.equal(box.cpu(), want)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("case", CASES)
def test_ragged_read(fmt, case):
    n, ctx, Hkv, pad, lead = case
    w = ch.Batch(n, ctx, Hkv, Hkv, fmt, seed=50 + len(n), pad=pad, lead=lead)
    d = w.gpu()
    first_l = [c // 2 for c in ctx]
    first = torch.tensor(first_l, dtype=torch.int32, device=DEV)
    for want_k, want_v in ((True, True), (True, False), (False, True)):
        ko = torch.full((w.T, Hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV) if want_k else None
        vo = torch.full((w.T, Hkv, 128), 7.0, dtype=torch.bfloat16, device=DEV) if want_v else None
        sdb.sd_cache_read(d.shape, d.cache, d.page_table, d.lens, first, d.row_start, ko, vo, d.status)
        assert int(d.status.item()) == 0
        for i, out in enumerate((ko, vo)):
            if out is None:
                continue
            want = torch.full((w.T, Hkv, 128), 7.0, dtype=torch.float64)
            for b in range(w.B):
                want[w.start[b]:w.start[b + 1]] = w.rows(i, b, first_l[b], first_l[b] + w.n[b])
            assert torch.equal(out.double().cpu(), want)


@pytest.mark.parametrize("what,code", [("row_start falls", sdb.SD_ERR_INVALID_ARG), ("row_start past the end", sdb.SD_ERR_INVALID_ARG),
                                       ("row_start negative", sdb.SD_ERR_INVALID_ARG),
                                       ("more rows than lens", sdb.SD_ERR_INVALID_ARG), ("bad length", sdb.SD_ERR_INVALID_ARG),
                                       ("bad page", sdb.SD_ERR_INDEX_OOB), ("negative page", sdb.SD_ERR_INDEX_OOB)])
@pytest.mark.parametrize("op", ["write", "read"])
def test_bad_device_inputs(what, code, op):
    w = ch.Batch([4, 20], [3, 0], 2, 2, "mxfp8")
    d = w.gpu()
    if what == "row_start falls":
        d.row_start[1] = 30
    elif what == "row_start past the end":
        d.row_start[2] = w.T + 1
    elif what == "row_start negative":
        d.row_start[0] = -1
    elif what == "more rows than lens":
        d.lens[1] = 19
    elif what == "bad length":
        d.lens[0] = w.max_pages * 16 + 1
    elif what == "bad page":
        d.page_table[1, 0] = w.num_pages
    else:
        d.page_table[1, 0] = -1
    before = [x.clone() for x in (d.K.view(torch.uint8), d.V.view(torch.uint8), d.scales)]
    k, v = torch.ones((w.T, 2, 128), dtype=torch.bfloat16, device=DEV), torch.ones((w.T, 2, 128), dtype=torch.bfloat16, device=DEV)
    if op == "write":
        sdb.sd_cache_write(d.shape, d.cache, d.page_table, d.lens, d.row_start, k, v, None, d.status)
    else:
        first = torch.zeros(2, dtype=torch.int32, device=DEV)
        sdb.sd_cache_read(d.shape, d.cache, d.page_table, d.lens, first, d.row_start, k, v, d.status)
    assert int(d.status.item()) == code
    if what.startswith("row_start") and op == "write":     # nothing is done
        for x, y in zip(before, (d.K.view(torch.uint8), d.V.view(torch.uint8), d.scales)):
            assert torch.equal(x, y)


def test_read_out_of_range_is_refused():
    w = ch.Batch([4], [8], 2, 2, "bf16")
    d = w.gpu()
    for first_v in (-1, 9):
        d.status.zero_()
        out = torch.full((w.T, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        first = torch.tensor([first_v], dtype=torch.int32, device=DEV)
        sdb.sd_cache_read(d.shape, d.cache, d.page_table, d.lens, first, d.row_start, out, None, d.status)
        assert int(d.status.item()) == sdb.SD_ERR_INVALID_ARG
        assert (out == 7.0).all()


def test_many_requests():
    """4096 requests, the most the library takes, one row each."""
    B = 4096
    w = ch.Batch([1] * B, [b % 5 for b in range(B)], 1, 1, "mxint8", spare=0)
    d = w.gpu()
    k = torch.randn((B, 1, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    sdb.sd_cache_write(d.shape, d.cache, d.page_table, d.lens, d.row_start, k.to(DEV), k.to(DEV), None, d.status)
    ko = torch.zeros((B, 1, 128), dtype=torch.bfloat16, device=DEV)
    first = torch.tensor([b % 5 for b in range(B)], dtype=torch.int32, device=DEV)
    sdb.sd_cache_read(d.shape, d.cache, d.page_table, d.lens, first, d.row_start, ko, None, d.status)
    assert int(d.status.item()) == 0
    el, by = ch.quantise(k, "mxint8")
    assert torch.equal(ko.double().cpu(), ch.values(el, by, "mxint8"))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_no_rows_at_all(fmt):
    """Requests without new rows, empty contexts: nothing is touched."""
    w = ch.Batch([0, 0, 0], [0, 40, 16], 2, 2, fmt, pad=5)
    d = w.gpu()
    before = [x.clone() for x in (d.K.view(torch.uint8), d.V.view(torch.uint8))]
    k = torch.ones((w.T, 2, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(k, 7.0)
    first = torch.tensor([0, 40, 3], dtype=torch.int32, device=DEV)
    sdb.sd_cache_write(d.shape, d.cache, d.page_table, d.lens, d.row_start, k, k, None, d.status)
    sdb.sd_cache_read(d.shape, d.cache, d.page_table, d.lens, first, d.row_start, out, None, d.status)
    att = d.chunk()
    assert int(d.status.item()) == 0
    assert (out == 7.0).all() and (att == 7.0).all()
    for x, y in zip(before, (d.K.view(torch.uint8), d.V.view(torch.uint8))):
        assert torch.equal(x, y)


def test_write_and_read_captured():
    """One graph of write and read, replayed with other rows and other lengths in the same buffers."""
    w = ch.Batch([2, 30], [60, 40], 2, 2, "mxint8", seed=4)
    d = w.gpu()
    k, v, ko, vo = (torch.zeros((w.T, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(4))
    first = torch.zeros(2, dtype=torch.int32, device=DEV)

    def step():
        sdb.sd_cache_write(d.shape, d.cache, d.page_table, d.lens, d.row_start, k, v, None, d.status)
        sdb.sd_cache_read(d.shape, d.cache, d.page_table, d.lens, first, d.row_start, ko, vo, d.status)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, lens in ((1, [62, 70]), (2, [50, 33])):
        src = [torch.randn((w.T, 2, 128), generator=torch.Generator().manual_seed(seed + 9 * i)).bfloat16() for i in range(2)]
        k.copy_(src[0])
        v.copy_(src[1])
        d.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        first.copy_(torch.tensor([n - m for n, m in zip(lens, w.n)], dtype=torch.int32))
        g.replay()
        assert int(d.status.item()) == 0
        for s, o in zip(src, (ko, vo)):
            assert torch.equal(o.double().cpu(), ch.values(*ch.quantise(s, "mxint8"), "mxint8"))
