"""Plain 64-bit references of the cache formats and of attention over a cache, and small ragged batches.

Formats: blocks of 32 values share 2^e.  MXFP8: e the least integer in [-124, 119] with amax <= 448 * 2^e,
elements on the e4m3 grid; MXINT8: e the least integer in [-133, 121] for which amax * 2^-e rounds to at most 127;
elements saturate where no exponent is left.  Everything is
found by search and table here (no bit tricks), in numpy float64, where each step is exact.

Tolerance of chunk attention (bf16 output o, reference r in 64 bits, A = sum_i w_i |V_i| per element):
  * each probability is rounded to bf16 (half a step: 2^-9 relative to a value's binade, at most 2^-8 of it), so
    the sum moves by at most 2^-8 A; the unrounded sum below is in fp32 (2^-24 a term: under 2^-12 over the
    lengths tested);
  * scores: products of bf16 values are exact in fp32; 128 of them are added in fp32, and the exponent is off by
    at most 2^-16 (|s| < 2^6): relative 2^-15 in a weight;
  * the result is rounded once to bf16: 2^-8 |r| at most (half a step of 2^-7 relative to the binade's low end).
So |o - r| <= 2^-8 |r| + (2^-8 + 2^-11) A, taken as 2^-8 |r| + 1.25 * 2^-8 A.
"""
from __future__ import annotations

import numpy as np
import torch

from sparse_attention_decode_sd_b200 import binding as sdb

FMTS = {"bf16": sdb.SD_CACHE_BF16, "mxfp8": sdb.SD_CACHE_MXFP8, "mxint8": sdb.SD_CACHE_MXINT8}


def e4m3_table() -> np.ndarray:
    """Value of each of the 256 codes (NaN at 0x7f and 0xff)."""
    v = np.empty(256)
    for u in range(256):
        s, e, m = (-1.0 if u & 128 else 1.0), (u >> 3) & 15, u & 7
        v[u] = np.nan if (u & 127) == 127 else s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return v


_POS = e4m3_table()[:127]


def _to_e4m3(y: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values, ties to the even code."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x: torch.Tensor, fmt: str):
    """(element bytes uint8 [..., 128], scale bytes uint8 [..., 4]) of bf16 rows."""
    f = x.double().cpu().numpy().reshape(*x.shape[:-1], 4, 32)
    a = np.abs(f).max(-1)
    fine = np.isfinite(a)
    aa = np.where(fine, a, 0.0)
    lo, hi = (-124, 119) if fmt == "mxfp8" else (-133, 121)
    e = np.full(a.shape, hi)
    for k in range(hi, lo - 1, -1):      # the least exponent that still fits
        with np.errstate(over="ignore"):
            y = np.ldexp(aa, -k)
        fits = y <= 448.0 if fmt == "mxfp8" else np.rint(y) <= 127
        e = np.where(fits, k, e)
    y = np.ldexp(np.where(fine[..., None], f, 0.0), -e[..., None])
    el = _to_e4m3(np.clip(y, -448, 448)) if fmt == "mxfp8" else np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    by = np.where(fine, e + (127 if fmt == "mxfp8" else 133), 255).astype(np.uint8)
    el = np.where(fine[..., None], el, 0).astype(np.uint8)
    return torch.from_numpy(el.reshape(x.shape)), torch.from_numpy(by)


def values(el: torch.Tensor, by: torch.Tensor, fmt: str) -> torch.Tensor:
    """float64 values of element bytes [..., 128] and scale bytes [..., 4]."""
    u = el.cpu().numpy()
    v = (e4m3_table()[u] if fmt == "mxfp8" else u.view(np.int8).astype(np.float64)).reshape(*u.shape[:-1], 4, 32)
    b = by.cpu().numpy().astype(np.int64)
    s = np.ldexp(v, (b - (127 if fmt == "mxfp8" else 133))[..., None])
    s = np.where((b == 255)[..., None], np.nan, s)
    return torch.from_numpy(s.reshape(u.shape))


class Batch:
    """A ragged batch over a paged cache, on the CPU; to_gpu() gives the device tensors of the calls."""

    def __init__(self, n, ctx, Hq, Hkv, fmt, seed=0, pad=0, lead=0, spare=3, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.total = list(n), [a + c for a, c in zip(n, ctx)]
        self.B, self.Hq, self.Hkv, self.G, self.fmt = len(n), Hq, Hkv, Hq // Hkv, fmt
        pages = [(t + 15) // 16 for t in self.total]
        self.max_pages, self.num_pages = max(1, max(pages)) + 1, sum(pages) + spare
        perm = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        self.page_table = torch.full((self.B, self.max_pages), 0x7ffffff0, dtype=torch.int32)   # never read
        off = 0
        for b, k in enumerate(pages):
            self.page_table[b, :k] = perm[off:off + k]
            off += k
        start = [lead]
        for x in self.n:
            start.append(start[-1] + x)
        self.start, self.T = start, max(1, start[-1] + pad)
        self.row_start = torch.tensor(start, dtype=torch.int32)
        self.lens = torch.tensor(self.total, dtype=torch.int32)
        size = (self.num_pages, 16, Hkv, 128)
        self.src = [(torch.randn(size, generator=g) * scale).bfloat16() for _ in range(2)]   # K, V as given
        self.q = torch.randn((self.T, Hq, 128), generator=g).bfloat16()
        self.encode()

    def encode(self):
        """The cache's tensors (and their 64-bit values) from src."""
        self.scales = None
        if self.fmt == "bf16":
            self.kv, self.val = [s.clone() for s in self.src], [s.double() for s in self.src]
            return
        self.kv, self.val = [], []
        self.scales = torch.zeros((self.num_pages, self.Hkv, 16, 2, 4), dtype=torch.uint8)
        for i, s in enumerate(self.src):
            el, by = quantise(s, self.fmt)
            self.kv.append(el.view(torch.float8_e4m3fn if self.fmt == "mxfp8" else torch.int8))
            self.scales[:, :, :, i] = by.transpose(1, 2)
            self.val.append(values(el, by, self.fmt))

    def shape(self, k_max=1):
        return sdb.make_shape(self.B, self.Hq, self.Hkv, self.max_pages, k_max, self.num_pages)

    def rows(self, i, b, lo, hi):
        """64-bit values of K (i = 0) or V (1) at positions lo..hi of request b."""
        pos = torch.arange(lo, hi)
        return self.val[i][self.page_table[b].long()[pos // 16], pos % 16]

    def attention(self):
        """{row: (reference [Hq][128], A = sum w |V| [Hq][128])} in 64 bits."""
        got = {}
        for b in range(self.B):
            K, V = self.rows(0, b, 0, self.total[b]), self.rows(1, b, 0, self.total[b])
            K, V = K.repeat_interleave(self.G, 1), V.repeat_interleave(self.G, 1)
            for j in range(self.n[b]):
                t, seen = self.start[b] + j, self.total[b] - self.n[b] + j + 1
                s = torch.einsum("hd,nhd->hn", self.q[t].double(), K[:seen]) / 128 ** 0.5
                w = torch.softmax(s, 1)
                got[t] = (torch.einsum("hn,nhd->hd", w, V[:seen]), torch.einsum("hn,nhd->hd", w, V[:seen].abs()))
        return got

    def gpu(self, dev="cuda:0"):
        return Gpu(self, dev)


class Gpu:
    def __init__(self, w: Batch, dev):
        self.w, self.dev = w, dev
        self.shape = w.shape()
        for name in ("page_table", "lens", "row_start", "q"):
            setattr(self, name, getattr(w, name).to(dev))
        self.K, self.V = (x.to(dev) for x in w.kv)
        self.scales = None if w.scales is None else w.scales.to(dev)
        self.cache = sdb.make_cache(FMTS[w.fmt], self.K, self.V, self.scales)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def chunk(self, out=None, ws=None, **kw):
        out = torch.full((self.w.T, self.w.Hq, 128), 7.0, dtype=torch.bfloat16, device=self.dev) if out is None else out
        ws = sdb.workspace_for(self.shape, sdb.SD_OP_CHUNK, self.dev) if ws is None else ws
        sdb.sd_chunk_attention(self.shape, self.cache, self.q, self.page_table, self.lens, self.row_start, out, ws,
                               self.status, **kw)
        return out


def check_attention(out: torch.Tensor, w: Batch, ref=None):
    """Every row within the derived bound, rows of no request as they were (7.0)."""
    out = out.double().cpu()
    ref = w.attention() if ref is None else ref
    for t in range(w.T):
        if t not in ref:
            assert (out[t] == 7.0).all(), t
            continue
        r, A = ref[t]
        bound = 2.0 ** -8 * r.abs() + 1.25 * 2.0 ** -8 * A + 1e-30
        bad = (out[t] - r).abs() > bound
        assert not bad.any(), (t, float(((out[t] - r).abs() / bound).max()))
