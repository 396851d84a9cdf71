"""Which kernel of sd_chunk_attention takes a request over an 8-bit cache depends on its own rows, not on how many requests
of the batch are idle: the same bits with and without them."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("n", [17, 50, 200])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (8, 1), (10, 2)])
def test_a_chunk_among_idle_slots_is_taken_as_alone(fmt, n, Hq, Hkv):
    """256 slots, one chunk: alone it is taken by 128-row tiles, which the key/value rows of a group's tokens share; in
    pieces of eight rows each piece would read the cache again (and round differently)."""
    B, at = 256, 77
    w = ch.Batch([n if b == at else 0 for b in range(B)], [3000 if b == at else 5 for b in range(B)], Hq, Hkv, fmt, seed=50)
    d = w.gpu()
    among = d.chunk()
    alone = torch.full_like(among, 7.0)
    shape = sdb.make_shape(1, Hq, Hkv, w.max_pages, 1, w.num_pages)
    sdb.sd_chunk_attention(shape, d.cache, d.q, d.page_table[at:at + 1].contiguous(), d.lens[at:at + 1].contiguous(),
                           torch.tensor([0, n], dtype=torch.int32, device=DEV), alone,
                           sdb.workspace_for(shape, sdb.SD_OP_CHUNK, DEV), d.status)
    assert int(d.status.item()) == 0
    assert torch.equal(among, alone)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2), (7, 1), (32, 2)])
@pytest.mark.parametrize("rows", [1, 2, 3, 7, 8, 9, 31, 32, 33])
def test_batches_around_the_limits_of_the_choice(fmt, Hq, Hkv, rows):
    """All rows in one request, one row each, and in between; as many requests as rows, fewer and more."""
    for n in ([rows], [1] * rows, [0] * 40 + [rows] + [0] * 2, [rows // 2, 0, rows - rows // 2]):
        w = ch.Batch(n, [(53 * b + 20) % 300 for b in range(len(n))], Hq, Hkv, fmt, seed=51)
        d = w.gpu()
        ch.check_attention(d.chunk(), w)
        assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_bad_rows_in_a_call_of_both_kinds(fmt):
    """row_start that is not valid: nothing is done by either kernel, whatever the call before left in the workspace."""
    w = ch.Batch([40, 1, 1], [300, 20, 700], 8, 2, fmt, seed=52)
    d = w.gpu()
    ws = sdb.workspace_for(d.shape, sdb.SD_OP_CHUNK, DEV)
    ch.check_attention(d.chunk(ws=ws), w)
    good = d.row_start.clone()
    for bad in ([0, 40, 39, 42], [0, 40, 41, 43], [-1, 40, 41, 42]):
        d.status.zero_()
        d.row_start.copy_(torch.tensor(bad, dtype=torch.int32))
        assert (d.chunk(ws=ws) == 7.0).all()
        assert int(d.status.item()) == sdb.SD_ERR_INVALID_ARG
    d.status.zero_()
    d.row_start.copy_(good)
    ch.check_attention(d.chunk(ws=ws), w)
    assert int(d.status.item()) == 0
