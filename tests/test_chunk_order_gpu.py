"""sd_chunk_attention behind work of the same stream: everything it reads (q, rows, lengths, pages, cache) written by the
operations just before it, and its output and workspace taken over by the ones just behind it.  The same batches with
the device idle between all steps give the same bits."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_inputs_written_just_before(fmt):
    B, T, Hq, Hkv = 4, 150, 8, 2
    rows = [([1, 1, 140, 3], [900, 20, 100, 33]), ([140, 1, 2, 7], [0, 500, 7, 64]), ([0, 2, 146, 1], [5, 16, 3, 3000]),
            ([9, 8, 1, 132], [100, 128, 1, 1900])]
    pages = max(sum((a + c + 15) // 16 for a, c in zip(*r)) for r in rows)
    shape = sdb.make_shape(B, Hq, Hkv, pages, 1, pages)
    g = torch.Generator(DEV).manual_seed(40)
    new = [torch.randn((4, T, Hkv, 128), generator=g, device=DEV).bfloat16() for _ in range(2)]
    qs = torch.randn((4, T, Hq, 128), generator=g, device=DEV).bfloat16()
    starts = torch.zeros((4, B + 1), dtype=torch.int32)
    lens = torch.zeros((4, B), dtype=torch.int32)
    tables = torch.zeros((4, B, pages), dtype=torch.int32)
    for i, (n, ctx) in enumerate(rows):
        starts[i, 1:] = torch.tensor(n).cumsum(0)
        at, perm = 0, torch.randperm(pages, generator=torch.Generator().manual_seed(i))
        for b in range(B):
            lens[i, b] = n[b] + ctx[b]
            k = (n[b] + ctx[b] + 15) // 16
            tables[i, b, :k] = perm[at:at + k]
            at += k
    starts, lens, tables = starts.to(DEV), lens.to(DEV), tables.to(DEV)

    def steps(wait):
        cache = sdb.empty_cache(shape, ch.FMTS[fmt], DEV)
        if fmt == "bf16":       # some context: finite rows everywhere
            for t in cache.tensors[:2]:
                t.copy_(torch.randn(t.shape, generator=torch.Generator(DEV).manual_seed(41), device=DEV))
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = sdb.workspace_for(shape, sdb.SD_OP_CHUNK, DEV)
        rs, ln, pt = torch.zeros_like(starts[0]), torch.zeros_like(lens[0]), torch.zeros_like(tables[0])
        q, out, got = torch.zeros_like(qs[0]), torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device=DEV), []
        torch.cuda.synchronize()
        for rep in range(6):
            for i in range(4):
                for dst, src in ((rs, starts[i]), (ln, lens[i]), (pt, tables[i]), (q, qs[i])):
                    dst.copy_(src)
                out.fill_(7.0)
                wait()
                sdb.sd_cache_write(shape, cache, pt, ln, rs, new[0][i], new[1][i], None, status)
                wait()
                sdb.sd_chunk_attention(shape, cache, q, pt, ln, rs, out, ws, status)
                wait()
                got.append(out.clone())
                ws.fill_(255)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return got

    for a, b in zip(steps(lambda: None), steps(torch.cuda.synchronize)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_batches_of_both_kinds_on_two_streams(fmt):
    """Calls that launch both attention kernels, at once on two streams with a workspace each, eager and replayed."""
    ws_ = [ch.Batch([1, 70, 1, 2], [900, 300, 2000, 17], 8, 2, fmt, seed=42), ch.Batch([40, 1, 3], [700, 2500, 60], 8, 2, fmt, seed=43)]
    ds = [w.gpu() for w in ws_]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = [sdb.workspace_for(d.shape, sdb.SD_OP_CHUNK, DEV) for d in ds]
    outs = [torch.full((w.T, w.Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV) for w in ws_]
    refs = [w.attention() for w in ws_]
    graphs = []
    for d, s, o, k in zip(ds, streams, outs, work):
        d.chunk(out=o, ws=k)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            d.chunk(out=o, ws=k)
        graphs.append(g)
    for replay in (False, True):
        for o, k in zip(outs, work):
            o.fill_(7.0)
            k.fill_(255)
        torch.cuda.synchronize()
        for _ in range(10):
            for d, g, s, o, k in zip(ds, graphs, streams, outs, work):
                with torch.cuda.stream(s):
                    if replay:
                        g.replay()
                    else:
                        d.chunk(out=o, ws=k)
        torch.cuda.synchronize()
        for w, d, o, r in zip(ws_, ds, outs, refs):
            assert int(d.status.item()) == 0
            ch.check_attention(o, w, r)
