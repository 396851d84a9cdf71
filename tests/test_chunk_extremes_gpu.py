"""sd_chunk_attention over finite but extreme K and V: scores that jump further than a 32-bit exponential reaches, values
whose magnitudes lie far apart, and the smallest ones.  References in 64 bits.

Tolerance: that of tests/cache_helpers.py, with q and K powers of two so that scores are exact; the absolute term is what
bf16 itself leaves open, half of its smallest step, 2^-134, so that results of any magnitude are told from zeros.

Requests of few rows over an 8-bit cache take products of weight and block scale as half precision, scaled so that the
row's largest one in a block of 32 dimensions is at least 2^5.  Half precision's steps never get smaller than 2^-24, so
each product may be off by 2^-25 there, that is by 2^-30 of the largest; it multiplies the position's element.  With
S_i the scale of position i's block that is 2^-30 max_i(w_i S_i) sum_i |V_i / S_i|, over the positions that count (w_i above
2^-126, the least that the exponential gives)."""
from __future__ import annotations

import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _half_steps(w):
    """{row: the last term above, [Hq][128]} for the rows of such requests."""
    got = {}
    for b in range(w.B):
        if w.fmt == "bf16" or w.n[b] * w.G > 8:
            continue
        K, V = (w.rows(i, b, 0, w.total[b]).repeat_interleave(w.G, 1) for i in (0, 1))
        pos = torch.arange(w.total[b])
        byte = w.scales[w.page_table[b].long()[pos // 16], :, pos % 16, 1].double()      # [N][Hkv][4]
        S = torch.exp2(byte - 127.0).repeat_interleave(32, 2).repeat_interleave(w.G, 1)   # [N][Hq][128]
        for j in range(w.n[b]):
            t, seen = w.start[b] + j, w.total[b] - w.n[b] + j + 1
            p = torch.softmax(torch.einsum("hd,nhd->hn", w.q[t].double(), K[:seen]) / 128 ** 0.5, 1)
            p = torch.where(p > 2.0 ** -126, p, 0.0).T[:, :, None]                        # [N][Hq][1]
            got[t] = 2.0 ** -30 * (p * S[:seen]).amax(0) * torch.where(p > 0, (V / S)[:seen].abs(), 0.0).sum(0)
    return got


def _check(out, w, ref=None):
    out, ref = out.double().cpu(), w.attention() if ref is None else ref
    half = _half_steps(w)
    for t, (r, A) in ref.items():
        bad = ~((out[t] - r).abs() <= 2.0 ** -8 * r.abs() + 1.25 * 2.0 ** -8 * A + half.get(t, 0.0) + 2.0 ** -134)
        assert not bad.any(), (t, bad.nonzero()[0].tolist(), float(out[t][bad][0]), float(r[bad][0]))


def _place(w, b, p):
    return int(w.page_table[b, p // 16]), p % 16


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("n", [1, 2, 40])
@pytest.mark.parametrize("power", [0, 36, 42, 50, 100])
def test_far_jumps_of_the_maximum_under_large_values(fmt, n, power):
    """Scores rise by more than 2^7 in base-2 units in one step (what came before then counts nothing) while V is large."""
    w = ch.Batch([n] * 4, [70, 150, 200, 333], 8, 2, fmt, seed=30)
    w.q = torch.ones_like(w.q)
    for b in range(4):
        for p in range(w.total[b]):
            pg, sl = _place(w, b, p)
            w.src[0][pg, sl] = [-32.0, -16.0, 0.0, 32.0][min(3, p // (10, 40, 64, 90)[b])]   # 16 in K: 261
            w.src[1][pg, sl] *= 2.0 ** power
    w.encode()
    d = w.gpu()
    _check(d.chunk(), w)
    assert int(d.status.item()) == 0


def _huge_beside_small(fmt, n):
    """V of 2^100 at positions that count nothing (scores -362 and less, and a chunk's last token, which only its own
    row sees) among values near 2^-30."""
    w = ch.Batch([n] * 3, [70, 500, 1], 8, 2, fmt, seed=31)
    w.q = torch.ones_like(w.q)
    for b in range(3):
        for p in range(w.total[b]):
            pg, sl = _place(w, b, p)
            far = p % 23 == 7
            w.src[0][pg, sl] = -32.0 if far else 0.0
            w.src[1][pg, sl] *= 2.0 ** (100 if far or p == w.total[b] - 1 else -30)
    w.encode()
    d = w.gpu()
    _check(d.chunk(), w)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("n", [1, 2])
def test_huge_values_with_weight_zero_in_single_tokens_and_drafts(fmt, n):
    _huge_beside_small(fmt, n)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
@pytest.mark.parametrize("n,power", [(1, -90), (1, -110), (1, -118), (2, -112), (40, -100)])
def test_tiny_values(fmt, n, power):
    w = ch.Batch([n] * 3, [70, 700, 1], 8, 2, fmt, seed=32)
    for b in range(3):
        for p in range(w.total[b]):
            w.src[1][_place(w, b, p)] *= 2.0 ** power
    w.encode()
    d = w.gpu()
    _check(d.chunk(), w)
    assert int(d.status.item()) == 0


@pytest.mark.parametrize("fmt,n", [("bf16", 1), ("bf16", 2), ("bf16", 40), ("mxfp8", 40), ("mxint8", 40)])
def test_huge_values_with_weight_zero_in_tiles(fmt, n):
    _huge_beside_small(fmt, n)


@pytest.mark.parametrize("fmt,n", [("bf16", 1), ("bf16", 2), ("bf16", 40), ("mxfp8", 40), ("mxint8", 40)])
def test_huge_values_with_weight_zero_in_tiles(fmt, n):
    _huge_beside_small(fmt, n)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxint8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 1)])
def test_a_query_that_is_not_finite_gives_nan(fmt, bad, Hq, Hkv):
    """Its own row and head, wherever its positions fall in a tile; the others are not touched."""
    w = ch.Batch([1, 1, 2, 40, 3], [0, 3, 1, 2, 700], Hq, Hkv, fmt, seed=33)
    hurt = [(t, (3 * t + 1) % Hq) for t in range(w.T)]
    for t, h in hurt:
        w.q[t, h, (5 * t) % 128] = bad
    d = w.gpu()
    out = d.chunk()
    assert int(d.status.item()) == 0
    clean = torch.ones((w.T, Hq), dtype=torch.bool)
    for t, h in hurt:
        assert out[t, h].isnan().all(), (t, h)
        clean[t, h] = False
        w.q[t, h] = 0.0
    out = out.double().cpu()
    for t, (r, A) in w.attention().items():
        ok = (out[t] - r).abs() <= 2.0 ** -8 * r.abs() + 1.25 * 2.0 ** -8 * A + 2.0 ** -134
        assert ok[clean[t]].all(), t
