"""The Quest boxes that sd_cache_write keeps are those of the rows that the cache holds: after drafts that were rejected and
written over, over boxes of any content, in batches small and large.  Values have to be equal: a box is a minimum and
a maximum of stored values."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _stored(k, fmt):
    """bf16 values as a cache of the format holds them."""
    return k if fmt == "bf16" else ch.values(*ch.quantise(k, fmt), fmt).bfloat16()


class Cache:
    """A paged cache of `caps` positions per request with boxes, written through the library, and its rows in order."""

    def __init__(self, fmt, caps, Hkv, seed):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.Hkv = fmt, Hkv
        pages = [(c + 15) // 16 for c in caps]
        self.table = torch.zeros((len(caps), max(pages)), dtype=torch.int32)
        at, perm = 0, torch.randperm(sum(pages), generator=g).to(torch.int32)
        for b, p in enumerate(pages):
            self.table[b, :p] = perm[at:at + p]
            at += p
        self.shape = sdb.make_shape(len(caps), Hkv, Hkv, max(pages), 1, sum(pages))
        self.cache = sdb.empty_cache(self.shape, ch.FMTS[fmt], DEV)
        self.boxes = torch.full((sum(pages), Hkv, 2, 128), 1e30, dtype=torch.bfloat16, device=DEV)   # nothing valid
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.rows = [torch.zeros((0, Hkv, 128), dtype=torch.bfloat16) for _ in caps]
        self.g = g

    def write(self, lens, n, scale=1.0):
        """The last n[b] of lens[b] positions get new rows."""
        new = (torch.randn((max(1, sum(n)), self.Hkv, 128), generator=self.g) * scale).bfloat16()
        start = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32)
        for b in range(len(n)):
            self.rows[b] = torch.cat([self.rows[b][:lens[b] - n[b]], new[start[b]:start[b + 1]]])
            assert len(self.rows[b]) == lens[b]
        new = new.to(DEV)
        sdb.sd_cache_write(self.shape, self.cache, self.table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                           start.to(DEV), new, new, self.boxes, self.status)
        assert int(self.status.item()) == 0

    def check(self):
        got = self.boxes.cpu()
        for b, r in enumerate(self.rows):
            r = _stored(r, self.fmt)
            for p in range((len(r) + 15) // 16):
                page = r[16 * p:16 * p + 16]
                pg = int(self.table[b, p])
                assert torch.equal(got[pg, :, 0], page.amin(0)), (b, p)
                assert torch.equal(got[pg, :, 1], page.amax(0)), (b, p)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("Hkv", [1, 3, 16])
def test_rejected_drafts_leave_nothing_in_the_boxes(fmt, Hkv):
    c = Cache(fmt, [200, 90, 64, 33], Hkv, seed=1)
    c.write([101, 7, 31, 16], [101, 7, 31, 16])
    c.check()
    c.write([106, 12, 36, 21], [5, 5, 5, 5], scale=50.0)      # drafts of five
    c.check()
    c.write([103, 8, 32, 17], [2, 1, 1, 1])                   # two, one, one and one of them kept in length, written anew
    c.check()
    c.write([119, 24, 48, 33], [16, 16, 16, 16], scale=20.0)
    c.write([104, 9, 33, 18], [1, 1, 1, 1])
    c.check()
    for step in range(20):                                    # single rows, over the page's end
        c.write([105 + step, 10 + step, 34 + step, 19 + min(step, 14)], [1, 1, 1, 1 if step < 15 else 0])
        if step in (0, 5, 6, 19):
            c.check()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
def test_nan_rows_leave_the_bounds_of_the_others(fmt):
    c = Cache(fmt, [40], 2, seed=2)
    c.write([5], [5])
    nan = torch.full((1, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    sdb.sd_cache_write(c.shape, c.cache, c.table.to(DEV), torch.tensor([6], dtype=torch.int32, device=DEV),
                       torch.tensor([0, 1], dtype=torch.int32, device=DEV), nan, nan, c.boxes, c.status)
    c.rows[0] = torch.cat([c.rows[0], c.rows[0][:1]])         # (counts as one of the others)
    c.check()
    c.write([8], [2])
    c.check()
