"""sd_chunk_attention against 64-bit attention over the values the cache holds: chunks from one token on,
tile borders, groups of every size, all formats; what must not matter (memory behind the lengths, rows of no
request); bad inputs; repeated, captured and concurrent calls.  Tolerances: tests/cache_helpers.py."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

CASES = [
    # n, ctx, Hq, Hkv, pad, lead
    ([1], [0], 1, 1, 0, 0),
    ([1], [300], 4, 1, 0, 0),
    ([2, 1, 3], [0, 127, 128], 8, 2, 0, 0),
    ([0, 40, 0, 129, 1], [9, 0, 0, 70, 255], 6, 2, 5, 2),       # G = 3: 42 tokens to a tile
    ([33, 64, 31], [95, 64, 97], 8, 2, 0, 0),                   # tiles that end at a border
    ([17, 300], [500, 3], 32, 2, 1, 0),                         # G = 16
    ([130, 7], [10, 1000], 4, 4, 0, 0),                         # G = 1: 128 tokens to a tile
    ([50, 50], [77, 200], 14, 2, 0, 1),                         # G = 7
    ([5] * 20, [13 * i for i in range(20)], 10, 2, 0, 0),
    ([600], [5], 5, 1, 0, 0),
    ([1] * 70, [3 * i for i in range(70)], 16, 16, 0, 0),
    ([1], [5000], 8, 8, 0, 0),
]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(case, fmt):
    n, ctx, Hq, Hkv, pad, lead = CASES[case]
    w = ch.Batch(n, ctx, Hq, Hkv, fmt, seed=case, pad=pad, lead=lead)
    d = w.gpu()
    out = d.chunk()
    assert int(d.status.item()) == 0
    ch.check_attention(out, w)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_peaked_and_growing_scores(fmt):
    """Scores that grow along the context by far more than a factor (the running maximum moves in every tile),
    and one position that takes nearly everything."""
    w = ch.Batch([9, 40], [900, 300], 8, 2, fmt, seed=4)
    for b in range(2):
        for p in range(w.total[b]):
            pg, sl = int(w.page_table[b, p // 16]), p % 16
            w.src[0][pg, sl] = (w.q[w.start[b], ::4].float() * (p / w.total[b]) * 1.2).bfloat16()
    w.encode()
    d = w.gpu()
    ch.check_attention(d.chunk(), w)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_memory_behind_the_lengths_does_not_matter(fmt):
    """Pages that no request holds, and the rows of the last pages behind lens, filled with NaN or infinities."""
    w = ch.Batch([20, 1, 3], [37, 10, 200], 8, 2, fmt, seed=5)
    d = w.gpu()
    held = torch.zeros((w.num_pages, 16), dtype=torch.bool)
    for b in range(w.B):
        pos = torch.arange(w.total[b])
        held[w.page_table[b].long()[pos // 16], pos % 16] = True
    free = ~held.to(DEV)
    ref = w.attention()
    for fill in (float("nan"), float("inf"), -float("inf")):
        if fmt == "bf16":
            d.K[free], d.V[free] = fill, fill
        else:
            d.scales.transpose(1, 2)[free] = 255
        ch.check_attention(d.chunk(), w, ref)
    assert int(d.status.item()) == 0


def test_same_result_every_time():
    w = ch.Batch([3, 70, 1], [2000, 900, 4000], 16, 4, "bf16", seed=6)
    d = w.gpu()
    ws = sdb.workspace_for(d.shape, sdb.SD_OP_CHUNK, DEV)
    a = d.chunk(ws=ws)
    for fill in (0, 255):
        ws.fill_(fill)                 # the workspace needs no initialisation
        assert torch.equal(a, d.chunk(ws=ws))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_one_token_agrees_with_dense_decode(fmt):
    """Single tokens: the dense decode over the same values (fp32), rounded to bf16, within the bound."""
    w = ch.Batch([1] * 6, [0, 15, 16, 500, 2049, 3000], 16, 4, fmt, seed=7)
    d = w.gpu()
    out = d.chunk()
    k, v = (torch.zeros((w.num_pages, 16, w.Hkv, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for b in range(w.B):               # the cache in bf16, page by page in place
        for i, t in enumerate((k, v)):
            pos = torch.arange(w.total[b])
            t[w.page_table[b].long()[pos // 16].to(DEV), (pos % 16).to(DEV)] = w.rows(i, b, 0, w.total[b]).bfloat16().to(DEV)
    dense = torch.zeros((w.B, w.Hq, 128), dtype=torch.float32, device=DEV)
    ws = sdb.workspace_for(d.shape, sdb.SD_OP_DENSE, DEV)
    sdb.sd_dense_decode(d.shape, d.q, k, v, d.page_table, d.lens, dense, ws, d.status)
    assert int(d.status.item()) == 0
    ref = w.attention()
    for b in range(w.B):
        r, A = ref[b]
        assert ((dense[b].double().cpu() - r).abs() <= 2e-4).all()
        assert ((out[b].double().cpu() - dense[b].double().cpu()).abs() <= 2.0 ** -8 * r.abs() + 1.25 * 2.0 ** -8 * A + 2e-4).all()


@pytest.mark.parametrize("what,code", [("row_start falls", sdb.SD_ERR_INVALID_ARG), ("row_start past the end", sdb.SD_ERR_INVALID_ARG),
                                       ("row_start negative", sdb.SD_ERR_INVALID_ARG),
                                       ("more rows than lens", sdb.SD_ERR_INVALID_ARG), ("bad length", sdb.SD_ERR_INVALID_ARG),
                                       ("negative length", sdb.SD_ERR_INVALID_ARG),
                                       ("bad page", sdb.SD_ERR_INDEX_OOB), ("negative page", sdb.SD_ERR_INDEX_OOB)])
@pytest.mark.parametrize("fmt", ["bf16", "mxint8"])
def test_bad_device_inputs(what, code, fmt):
    w = ch.Batch([4, 20], [3, 200], 4, 2, fmt)
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
    elif what == "negative length":
        d.lens[0] = -5
    elif what == "bad page":
        d.page_table[1, 2] = w.num_pages
    else:
        d.page_table[1, 0] = -1
    out = d.chunk()
    assert int(d.status.item()) == code
    if what.startswith("row_start"):
        assert (out == 7.0).all()
    if what == "more rows than lens":
        assert (out[4:] == 7.0).all()


def test_captured_and_replayed():
    """One graph of write + attention, replayed over new inputs in the same buffers."""
    w = ch.Batch([5, 1, 30], [50, 333, 100], 8, 2, "mxfp8", seed=11)
    d = w.gpu()
    new = [torch.zeros((w.T, w.Hkv, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = torch.zeros((w.T, w.Hq, 128), dtype=torch.bfloat16, device=DEV)
    ws = sdb.workspace_for(d.shape, sdb.SD_OP_CHUNK, DEV)

    def step():
        sdb.sd_cache_write(d.shape, d.cache, d.page_table, d.lens, d.row_start, new[0], new[1], None, d.status)
        sdb.sd_chunk_attention(d.shape, d.cache, d.q, d.page_table, d.lens, d.row_start, out, ws, d.status)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        src = [torch.randn((w.T, w.Hkv, 128), generator=torch.Generator().manual_seed(seed * 10 + i)).bfloat16() for i in range(2)]
        for a, s in zip(new, src):
            a.copy_(s)
        g.replay()
        torch.cuda.synchronize()
        for b in range(w.B):
            for j in range(w.n[b]):
                p = w.total[b] - w.n[b] + j
                for i in range(2):
                    w.src[i][int(w.page_table[b, p // 16]), p % 16] = src[i][w.start[b] + j]
        w.encode()
        assert int(d.status.item()) == 0
        ch.check_attention(out, w)


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    ws_, ds, outs = [], [], []
    for seed in (1, 2):
        w = ch.Batch([40, 3], [700, 2500], 8, 2, "bf16", seed=seed)
        ws_.append(w)
        ds.append(w.gpu())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = [sdb.workspace_for(d.shape, sdb.SD_OP_CHUNK, DEV) for d in ds]
    outs = [torch.full((w.T, w.Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV) for w in ws_]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s, o, k in zip(ds, streams, outs, work):
            d.chunk(out=o, ws=k, stream=s)
    torch.cuda.synchronize()
    for w, d, o in zip(ws_, ds, outs):
        assert int(d.status.item()) == 0
        ch.check_attention(o, w)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_prompt_in_chunks_equals_the_prompt(fmt):
    """A prompt written and attended to at once, and in chunks: every position within the bound either way."""
    n = 300
    w = ch.Batch([n], [0], 8, 2, fmt, seed=13)
    d = w.gpu()
    ref = w.attention()
    ch.check_attention(d.chunk(), w, ref)
    k, v = (torch.stack([w.src[i][int(w.page_table[0, p // 16]), p % 16] for p in range(n)]).to(DEV) for i in (0, 1))
    out = torch.zeros((n, w.Hq, 128), dtype=torch.bfloat16, device=DEV)
    cache = sdb.empty_cache(d.shape, ch.FMTS[fmt], DEV)
    ws = sdb.workspace_for(d.shape, sdb.SD_OP_CHUNK, DEV)
    at = 0
    for m in (1, 16, 100, 33, 128, 22):
        rs = torch.tensor([0, m], dtype=torch.int32, device=DEV)
        lens = torch.tensor([at + m], dtype=torch.int32, device=DEV)
        sdb.sd_cache_write(d.shape, cache, d.page_table, lens, rs, k[at:at + m], v[at:at + m], None, d.status)
        sdb.sd_chunk_attention(d.shape, cache, d.q[at:at + m], d.page_table, lens, rs, out[at:at + m], ws, d.status)
        at += m
    assert at == n and int(d.status.item()) == 0
    ch.check_attention(out, w, ref)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_scores_far_above_the_first_tile(fmt):
    """Scores that jump by hundreds of powers of two between tiles, up and down, and stay equal: the reference of a row
    is taken anew where they rise, and small weights vanish where they fall.  (q and K are exact powers of two here, so
    scores are exact and the bound of the weights' rounding alone holds.)"""
    w = ch.Batch([2, 150], [600, 500], 8, 2, fmt, seed=14)
    w.q = torch.ones_like(w.q)
    for b in range(2):
        for p in range(w.total[b]):
            step = [0.0, 4.0, -2.0, 16.0, 16.0, 64.0, 1.0][(p // 100) % 7]
            w.src[0][int(w.page_table[b, p // 16]), p % 16] = step
    w.encode()
    d = w.gpu()
    ch.check_attention(d.chunk(), w)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt", ["bf16", "mxint8"])
def test_many_requests_and_idle_ones(fmt):
    """More requests than the threads that plan the shares, most of them without rows."""
    B = 1500
    n = [1 if b % 7 == 3 else 0 for b in range(B)]
    w = ch.Batch(n, [b % 40 for b in range(B)], 4, 2, fmt, seed=15)
    d = w.gpu()
    ch.check_attention(d.chunk(), w)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_workspace_shared_in_one_stream(fmt):
    """Calls of different batches one after the other through one workspace, and two graphs that hold it."""
    ws_ = [ch.Batch([3, 70], [900, 100], 8, 2, fmt, seed=16), ch.Batch([1] * 9, [100 * i for i in range(9)], 16, 4, fmt, seed=17)]
    ds = [w.gpu() for w in ws_]
    work = sdb.workspace_for(ds[0].shape, sdb.SD_OP_CHUNK, DEV)
    refs = [w.attention() for w in ws_]
    outs = [torch.full((w.T, w.Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV) for w in ws_]
    graphs = []
    for d, o in zip(ds, outs):
        d.chunk(out=o, ws=work)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.chunk(out=o, ws=work)
        graphs.append(g)
    for _ in range(2):
        for g, o in zip(graphs, outs):
            o.fill_(7.0)
            g.replay()
        for o, w, r in zip(outs, ws_, refs):
            ch.check_attention(o, w, r)
    assert all(int(d.status.item()) == 0 for d in ds)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("n", [1, 40])
def test_large_values_under_small_weights(fmt, n):
    """Positions whose V is 2^40 times the others' (and some 2^-90 times) but whose scores leave them nothing, at the
    beginning, in between and at the end; and whole contexts of tiny and of huge values.  What a row weighs with 2^-60
    must not cost the others their precision: its share of A is part of the bound."""
    w = ch.Batch([n] * 4, [400, 70, 200, 333], 8, 2, fmt, seed=18)
    w.q = torch.ones_like(w.q)
    for b in range(4):
        for p in range(w.total[b]):
            pg, sl = int(w.page_table[b, p // 16]), p % 16
            if b < 2:
                w.src[0][pg, sl] = -8.0 if p % 37 in (0, 20, 36) else 0.0       # score -90 against 0
                w.src[1][pg, sl] *= 2.0 ** (40 if p % 37 in (0, 36) else -90 if p % 37 == 20 else 0)
            else:
                w.src[1][pg, sl] *= 2.0 ** (-110 if b == 2 else 100)
    w.encode()
    d = w.gpu()
    ch.check_attention(d.chunk(), w)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 2), (8, 1), (4, 4), (14, 2)])
def test_tokens_prompts_and_drafts_in_one_call(fmt, Hq, Hkv):
    """Single tokens, drafts of a few, a prompt and idle requests together: requests of few and of many rows take
    different kernels of the call."""
    n = [1, 1, 200, 2, 0, 1, 3, 1, 8, 9, 1, 0]
    w = ch.Batch(n, [700, 0, 60, 33, 5, 2000, 150, 15, 90, 300, 127, 40], Hq, Hkv, fmt, seed=19, pad=3, lead=1)
    d = w.gpu()
    out = d.chunk()
    assert int(d.status.item()) == 0
    ch.check_attention(out, w)
    assert (out[:1] == 7.0).all() and (out[w.T - 3:] == 7.0).all()   # rows of no request


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (7, 1)])
def test_one_prompt_among_idle_requests(fmt, Hq, Hkv):
    """No more rows than requests, but one request has nearly all of them."""
    n = [0] * 60
    n[7], n[30], n[59] = 1, 50, 2
    w = ch.Batch(n, [(37 * b) % 300 for b in range(60)], Hq, Hkv, fmt, seed=20)
    d = w.gpu()
    ch.check_attention(d.chunk(), w)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_captured_call_over_changing_batches(fmt):
    """One captured call replayed while the batch changes: which request has how many rows, and every length."""
    batches = [ch.Batch(n, ctx, 8, 2, fmt, seed=24, spare=200)
               for n, ctx in (([1, 1, 30, 2], [400, 20, 100, 33]), ([30, 1, 2, 1], [0, 500, 7, 64]), ([0, 0, 0, 34], [5, 16, 3, 300]),
                              ([9, 8, 9, 8], [100, 128, 1, 90]))]
    pages = max(w.max_pages for w in batches)
    num = max(w.num_pages for w in batches)
    shape = sdb.make_shape(4, 8, 2, pages, 1, num)
    cache = sdb.empty_cache(shape, ch.FMTS[fmt], DEV)
    q = torch.zeros((34, 8, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.zeros((34, 8, 128), dtype=torch.bfloat16, device=DEV)
    table = torch.zeros((4, pages), dtype=torch.int32, device=DEV)
    lens = torch.zeros(4, dtype=torch.int32, device=DEV)
    start = torch.zeros(5, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = sdb.workspace_for(shape, sdb.SD_OP_CHUNK, DEV)

    def load(w):
        for t, x in zip(cache.tensors, (*w.kv, w.scales)):
            if t is not None:
                t[:w.num_pages].copy_(x)
        table[:, :w.max_pages].copy_(w.page_table)
        q.copy_(w.q)
        lens.copy_(w.lens)
        start.copy_(w.row_start)

    def call():
        sdb.sd_chunk_attention(shape, cache, q, table, lens, start, out, ws, status)

    load(batches[0])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for w in batches + batches[:1]:
        load(w)
        out.fill_(7.0)
        g.replay()
        ch.check_attention(out, w)
        assert int(status.item()) == 0
