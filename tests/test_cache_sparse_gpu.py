"""sd_cache_sparse_decode against 64-bit attention over the selected rows of the values the cache holds, its
checks of idx, and a decode loop over an 8-bit cache through the Quest indexer.

Tolerance (fp32 output o, reference r in 64 bits, A = sum_i w_i |V_i|).  A score adds 128 exact products in fp32
with at most 16 roundings on any product's way, so it is off by at most 16 * 2^-24 sum |q k|; for N(0, 1) rows
sum |q k| < 2^8 and the softmax scale is 2^-3.5: 2^-15.5 in the exponent.  A weight carried as two bf16 parts is off
by 2^-17, the exponential by 2^-22, and the running sums of up to 2^12 rows by less than 2^-17.  A weight's error
counts in the numerator and in the sum: |o - r| <= 2 (2^-15.5 + 2^-17 + 2^-22 + 2^-17) A < 2^-14 A * 1.1;
the bound is 1.25 * 2^-14 A."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _select(w, k, seed=0):
    """idx [B][Hq][k_max]: random ascending positions, min(k_b, N_b) of them, then -1."""
    g = torch.Generator().manual_seed(seed)
    k_max = max(1, max(min(a, b) for a, b in zip(k, w.total)))
    idx = torch.full((w.B, w.Hq, k_max), -1, dtype=torch.int32)
    for b in range(w.B):
        m = min(k[b], w.total[b])
        for h in range(w.Hq):
            idx[b, h, :m] = torch.randperm(w.total[b], generator=g)[:m].sort().values.to(torch.int32)
    return idx


def _run(d, idx, ws=None, out=None, **kw):
    w = d.w
    shape = w.shape(idx.shape[2])
    ws = sdb.workspace_for(shape, sdb.SD_OP_CACHE_SPARSE, DEV) if ws is None else ws
    out = torch.full((w.B, w.Hq, 128), 7.0, dtype=torch.float32, device=DEV) if out is None else out
    sdb.sd_cache_sparse_decode(shape, d.cache, d.q, d.page_table, d.lens, idx, out, ws, d.status, **kw)
    return out


def _check(out, w, idx):
    out = out.double().cpu()
    assert torch.isfinite(out).all()
    for b in range(w.B):
        K, V = w.rows(0, b, 0, w.total[b]), w.rows(1, b, 0, w.total[b])
        for h in range(w.Hq):
            s = idx[b, h]
            neg = (s < 0).nonzero()
            s = s[:int(neg[0])] if len(neg) else s
            s = s.long()
            if not len(s):
                assert (out[b, h] == 0).all()
                continue
            wt = torch.softmax(K[s, h // w.G] @ w.q[b, h].double() / 128 ** 0.5, 0)
            r, A = wt @ V[s, h // w.G], wt @ V[s, h // w.G].abs()
            err = ((out[b, h] - r).abs() / (1.25 * 2.0 ** -14 * A + 1e-30)).max()
            assert err <= 1, (b, h, float(err))


CASES = [
    # lens, k, Hq, Hkv
    ([1], [1], 1, 1),
    ([100, 0, 17], [5, 3, 17], 8, 2),
    ([300, 33, 1000], [64, 33, 7], 6, 2),
    ([2048], [1], 32, 2),
    ([511, 513], [511, 256], 4, 4),
    ([5000, 40], [2500, 40], 16, 16),
    ([700] * 9, [15, 16, 17, 31, 32, 33, 47, 48, 700], 5, 1),
    ([64] * 33, [3 * i + 1 for i in range(33)], 14, 2),
]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(case, fmt):
    lens, k, Hq, Hkv = CASES[case]
    w = ch.Batch([1] * len(lens), [n - 1 for n in lens], Hq, Hkv, fmt, seed=case)
    d = w.gpu()
    idx = _select(w, k, seed=case)
    out = _run(d, idx.to(DEV))
    assert int(d.status.item()) == 0
    _check(out, w, idx)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_rows_of_every_length(fmt):
    """Ragged rows in one call: heads with no entry, one entry, whole contexts, and any negative padding."""
    w = ch.Batch([1, 1], [399, 99], 8, 2, fmt, seed=21)
    idx = torch.full((2, 8, 400), -3, dtype=torch.int32)
    for h, m in enumerate((0, 1, 15, 16, 17, 399, 400, 200)):
        idx[0, h, :m] = torch.arange(m, dtype=torch.int32) + (400 - m) // 2
        idx[1, h, :min(m, 100)] = torch.arange(min(m, 100), dtype=torch.int32)
    d = w.gpu()
    out = _run(d, idx.to(DEV))
    assert int(d.status.item()) == 0
    _check(out, w, idx)


def test_large_scores_and_shared_rows():
    w = ch.Batch([1], [3000], 16, 2, "mxfp8", seed=8, scale=4.0)
    idx = _select(w, [600], seed=8)
    idx[0, 1:8] = idx[0, 0]          # a whole group on the same rows
    d = w.gpu()
    out = _run(d, idx.to(DEV))
    assert int(d.status.item()) == 0
    out = out.double().cpu()
    K, V = w.rows(0, 0, 0, 3001), w.rows(1, 0, 0, 3001)
    for h in range(16):              # scores four times as large: the score term of the bound times four
        s = idx[0, h].long()
        wt = torch.softmax(K[s, h // 8] @ w.q[0, h].double() / 128 ** 0.5, 0)
        r, A = wt @ V[s, h // 8], wt @ V[s, h // 8].abs()
        assert ((out[0, h] - r).abs() <= 1.25 * 2.0 ** -12 * A).all()


def test_same_result_every_time_and_dirty_workspace():
    w = ch.Batch([1] * 3, [4000, 10, 900], 16, 4, "mxint8", seed=2)
    d = w.gpu()
    idx = _select(w, [1500, 11, 300]).to(DEV)
    ws = sdb.workspace_for(w.shape(idx.shape[2]), sdb.SD_OP_CACHE_SPARSE, DEV)
    a = _run(d, idx, ws)
    for fill in (0, 255):
        ws.fill_(fill)
        assert torch.equal(a, _run(d, idx, ws))


@pytest.mark.parametrize("what,code", [
    ("past the length", sdb.SD_ERR_INDEX_OOB), ("page", sdb.SD_ERR_INDEX_OOB), ("twice", sdb.SD_ERR_ORDER),
    ("falls", sdb.SD_ERR_ORDER), ("falls across 32", sdb.SD_ERR_ORDER), ("after padding", sdb.SD_ERR_ORDER),
    ("after a long padding", sdb.SD_ERR_ORDER), ("length", sdb.SD_ERR_INVALID_ARG)])
def test_bad_rows(what, code):
    w = ch.Batch([1, 1], [499, 299], 4, 2, "mxfp8", seed=3)
    d = w.gpu()
    idx = _select(w, [200, 100])
    if what == "past the length":
        idx[1, 2, 99] = 300
    elif what == "page":
        d.page_table[0, int(idx[0, 1, 50]) // 16] = -1
    elif what == "twice":
        idx[0, 3, 11] = idx[0, 3, 10]
    elif what == "falls":
        idx[1, 0, 40], idx[1, 0, 41] = int(idx[1, 0, 41]), int(idx[1, 0, 40])
    elif what == "falls across 32":
        idx[1, 0, 31], idx[1, 0, 32] = int(idx[1, 0, 32]), int(idx[1, 0, 31])
    elif what == "after padding":
        idx[0, 2, 60] = -1
    elif what == "after a long padding":
        idx[1, 3, 199] = 299
    else:
        d.lens[1] = w.max_pages * 16 + 1
    _run(d, idx.to(DEV))
    assert int(d.status.item()) == code


def test_captured_and_replayed():
    w = ch.Batch([1, 1], [1999, 600], 8, 2, "mxfp8", seed=5)
    d = w.gpu()
    idx = _select(w, [300, 200], seed=1).to(DEV)
    ws = sdb.workspace_for(w.shape(idx.shape[2]), sdb.SD_OP_CACHE_SPARSE, DEV)
    out = _run(d, idx, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(d, idx, ws, out)
    for seed in (2, 3):
        new = _select(w, [300, 150 + seed], seed=seed)
        idx.copy_(new)
        out.fill_(7.0)
        g.replay()
        assert int(d.status.item()) == 0
        _check(out, w, new)


def test_two_streams_at_once():
    bs = [ch.Batch([1] * 2, [2500, 700], 8, 2, f, seed=i) for i, f in enumerate(("mxfp8", "mxint8"))]
    ds = [b.gpu() for b in bs]
    idx = [_select(b, [500, 100], seed=i) for i, b in enumerate(bs)]
    dev = [i.to(DEV) for i in idx]
    ws = [sdb.workspace_for(b.shape(i.shape[2]), sdb.SD_OP_CACHE_SPARSE, DEV) for b, i in zip(bs, idx)]
    outs = [torch.zeros((2, 8, 128), dtype=torch.float32, device=DEV) for _ in bs]
    st = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            _run(ds[i], dev[i], ws[i], outs[i], stream=st[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert int(ds[i].status.item()) == 0
        _check(outs[i], bs[i], idx[i])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_serving_over_an_8_bit_cache(fmt):
    """As a server uses it: prompts written in chunks with their Quest boxes and attended to, then decode steps:
    write a row, index by boxes, sparse decode; at the end the cache is read back in bf16 and the library's bf16
    sparse decode on it agrees."""
    B, Hq, Hkv, prompt, steps = 2, 8, 2, [270, 95], 20
    w = ch.Batch(prompt, [steps] * B, Hq, Hkv, fmt, seed=31)       # positions 0 .. prompt + steps - 1 have pages
    d = w.gpu()
    total = [p + steps for p in prompt]
    src = [[torch.stack([w.src[i][int(w.page_table[b, p // 16]), p % 16] for p in range(total[b])]) for b in range(B)] for i in (0, 1)]
    shape1 = w.shape()
    cache = sdb.empty_cache(shape1, ch.FMTS[fmt], DEV)
    boxes = sdb.quest_boxes_for(shape1, DEV).zero_()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    wsc = sdb.workspace_for(shape1, sdb.SD_OP_CHUNK, DEV)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    done = [0, 0]
    for share in (0.4, 0.3, 0.3):                                  # the prompts in chunks
        m = [min(int(share * p) + 1, p - x) for p, x in zip(prompt, done)]
        rs = [0, m[0], m[0] + m[1]]
        k, v = (torch.cat([src[i][b][done[b]:done[b] + m[b]] for b in range(B)]).to(DEV) for i in (0, 1))
        done = [x + y for x, y in zip(done, m)]
        sdb.sd_cache_write(shape1, cache, d.page_table, i32(done), i32(rs), k, v, boxes, status)
        q = torch.randn((rs[-1], Hq, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
        out = torch.zeros((rs[-1], Hq, 128), dtype=torch.bfloat16, device=DEV)
        sdb.sd_chunk_attention(shape1, cache, q.to(DEV), d.page_table, i32(done), i32(rs), out, wsc, status)
        part = ch.Batch.__new__(ch.Batch)
        part.__dict__.update(w.__dict__, n=m, total=list(done), start=rs, T=rs[-1], q=q)
        ch.check_attention(out, part)
    assert done == prompt
    k_tok = [64, 48]
    shape = w.shape(128)
    wsq = sdb.workspace_for(shape, sdb.SD_OP_QUEST, DEV)
    wss = sdb.workspace_for(shape, sdb.SD_OP_CACHE_SPARSE, DEV)
    idx = torch.zeros((B, Hq, 128), dtype=torch.int32, device=DEV)
    out = torch.zeros((B, Hq, 128), dtype=torch.float32, device=DEV)
    for s in range(steps):
        lens = i32([p + s + 1 for p in prompt])
        k, v = (torch.stack([src[i][b][prompt[b] + s] for b in range(B)]).to(DEV) for i in (0, 1))
        sdb.sd_cache_write(shape, cache, d.page_table, lens, i32([0, 1, 2]), k, v, boxes, status)
        q = torch.randn((B, Hq, 128), generator=torch.Generator().manual_seed(100 + s)).bfloat16().to(DEV)
        sdb.sd_quest_index(shape, q, boxes, d.page_table, lens, i32(k_tok), idx, wsq, status)
        sdb.sd_cache_sparse_decode(shape, cache, q, d.page_table, lens, idx, out, wss, status)
    assert int(status.item()) == 0
    # the boxes are those of the cache as stored
    kb = torch.zeros((sum((t + 15) // 16 * 16 for t in total), Hkv, 128), dtype=torch.bfloat16, device=DEV)
    vb = torch.zeros_like(kb)
    starts = [0, (total[0] + 15) // 16 * 16]
    table = torch.zeros((B, w.max_pages), dtype=torch.int32)
    for b in range(B):              # each request read back to whole pages of its own
        rs = [starts[b]] * (b + 1) + [starts[b] + total[b]] * (B - b)
        sdb.sd_cache_read(shape, cache, d.page_table, i32(total), i32([0] * B), i32(rs), kb, vb, status)
        table[b, :(total[b] + 15) // 16] = starts[b] // 16 + torch.arange((total[b] + 15) // 16)
    assert int(status.item()) == 0
    pages = kb.shape[0] // 16
    shb = sdb.make_shape(B, Hq, Hkv, w.max_pages, 128, pages)
    kb, vb, table = kb.view(pages, 16, Hkv, 128), vb.view(pages, 16, Hkv, 128), table.to(DEV)
    bx = sdb.quest_boxes_for(shb, DEV).zero_()
    sdb.sd_quest_summarize(shb, kb, table, i32(total), bx, status)
    for b in range(B):
        n = (total[b] + 15) // 16
        assert torch.equal(bx[table[b, :n].long()], boxes[d.page_table[b, :n].long()])
    ref = torch.zeros_like(out)
    sdb.sd_sparse_decode(shb, q, kb, vb, table, i32(total), idx, ref, sdb.workspace_for(shb, sdb.SD_OP_SPARSE, DEV), status)
    assert int(status.item()) == 0
    assert (out - ref).abs().max() <= 2e-4


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("which", [0, 1])
def test_rows_that_read_as_nan(fmt, which):
    """Block 2 of every selected row of one request reads as NaN, and of one row of another: K makes the whole output
    NaN, V that block's; the third request is as ever."""
    w = ch.Batch([1] * 3, [40, 50, 60], 4, 2, fmt, seed=22)
    d = w.gpu()
    idx = _select(w, [7, 20, 61], seed=22)
    for b, rows in ((0, range(41)), (1, [int(idx[1, 0, 3])])):
        for p in rows:
            page, slot = int(w.page_table[b, p // 16]), p % 16
            d.scales[page, :, slot, which, 2] = 255
            (d.K, d.V)[which].view(torch.uint8)[page, slot, :, 64:96] = 0
    out = _run(d, idx.to(DEV)).cpu()
    assert int(d.status.item()) == 0
    dims = slice(0, 128) if which == 0 else slice(64, 96)
    assert out[0][:, dims].isnan().all() and out[1, 0, dims].isnan().all()
    if which == 1:
        assert out[:2, :, :64].isfinite().all() and out[:2, :, 96:].isfinite().all()
    assert out[2].isfinite().all()


@pytest.mark.parametrize("Hq,Hkv,k", [(1, 1, 9000), (3, 1, 4000), (8, 2, 1500)])
def test_few_rows_of_many_parts(Hq, Hkv, k):
    """Few heads with many entries: every warp of the wave has a part of the same row."""
    w = ch.Batch([1], [17999], Hq, Hkv, "mxfp8", seed=23)
    idx = _select(w, [k], seed=23)
    d = w.gpu()
    out = _run(d, idx.to(DEV))
    assert int(d.status.item()) == 0
    _check(out, w, idx)
    assert torch.equal(out, _run(d, idx.to(DEV)))
