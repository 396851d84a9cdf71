"""sd_chunk_attention over finite but extreme K and V: scores that jump further than a 32-bit exponential reaches, values
whose magnitudes lie far apart, and the smallest ones.  References in 64 bits.

Tolerance: that of tests/cache_helpers.py, with q and K powers of two so that scores are exact; the absolute term is what
bf16 itself leaves open, half of its smallest step, 2^-134, so that results of any magnitude are told from zeros."""
from __future__ import annotations

import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _check(out, w, ref=None):
    out, ref = out.double().cpu(), w.attention() if ref is None else ref
    for t, (r, A) in ref.items():
        bad = ~((out[t] - r).abs() <= 2.0 ** -8 * r.abs() + 1.25 * 2.0 ** -8 * A + 2.0 ** -134)
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
