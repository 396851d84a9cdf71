"""What the Python binding of the cache and chunk calls refuses before it hands addresses to the library: tensors that the
call would read or write past their end, of other types, strided, or on another device.  CPU only."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb

B, Hq, Hkv, PAGES, T = 3, 8, 2, 10, 12
BF = torch.bfloat16


def _cache(fmt=sdb.SD_CACHE_MXFP8, pages=PAGES, heads=Hkv):
    return sdb.empty_cache(sdb.make_shape(B, heads, heads, 4, 1, pages), fmt, "cpu")


def _rows(n=T, h=Hkv, dtype=BF):
    return torch.zeros((n, h, 128), dtype=dtype)


def _ints(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def _call(op, cache=None, a=None, b=None, rs=None, lens=None, first=None):
    shape = sdb.make_shape(B, Hq, Hkv, 4, 1, PAGES)
    h = Hq if op == "chunk" else Hkv
    cache = cache or _cache()
    a, b = _rows(h=h) if a is None else a, _rows(h=h) if b is None else b
    rs, lens, first = (_ints(n) if t is None else t for t, n in ((rs, B + 1), (lens, B), (first, B)))
    pt, st = _ints(B * 4), _ints(1)
    if op == "write":
        return sdb.sd_cache_write(shape, cache, pt, lens, rs, a, b, None, st, stream=0)
    if op == "read":
        return sdb.sd_cache_read(shape, cache, pt, lens, first, rs, a, b, st, stream=0)
    return sdb.sd_chunk_attention(shape, cache, a, pt, lens, rs, b, torch.zeros(16, dtype=torch.uint8), st, stream=0)


@pytest.mark.parametrize("op", ["write", "read", "chunk"])
def test_row_arrays(op):
    h = Hq if op == "chunk" else Hkv
    for bad in (_rows(T - 1, h), _rows(T, h)[:, :, :64], _rows(T, h, torch.float16), _rows(T, h, torch.float32),
                torch.zeros((h, T, 128), dtype=BF).transpose(0, 1), _rows(T, 2 * h)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous bf16 rows"):
            _call(op, b=bad)
    for bad in (_rows(T, h - 1), _rows(T, h, torch.float16), torch.zeros((h, T, 128), dtype=BF).transpose(0, 1)):
        with pytest.raises(ValueError, match="contiguous bf16 rows"):
            _call(op, a=bad)


@pytest.mark.parametrize("op", ["write", "read", "chunk"])
def test_host_tensors(op):
    with pytest.raises(ValueError, match="current CUDA device"):
        _call(op)


@pytest.mark.parametrize("op", ["write", "read", "chunk"])
def test_counts(op):
    for kw in (dict(rs=_ints(B)), dict(rs=_ints(B + 1, torch.int64)), dict(rs=_ints(2 * B + 2)[::2])) + (
            (dict(first=_ints(B - 1)), dict(first=_ints(B, torch.int64))) if op == "read" else ()):
        with pytest.raises(ValueError, match="contiguous int32"):
            _call(op, **kw)


@pytest.mark.parametrize("op", ["write", "read", "chunk", "sparse"])
def test_caches_of_other_sizes(op):
    for c in (_cache(pages=PAGES - 1), _cache(heads=Hkv + 1), _cache(heads=1)):
        with pytest.raises(ValueError, match="pages"):
            if op == "sparse":
                sdb.sd_cache_sparse_decode(sdb.make_shape(B, Hq, Hkv, 4, 1, PAGES), c, 0, 0, 0, 0, 0, None, 0, stream=0)
            else:
                _call(op, cache=c)


def _bytes(*size, dtype=torch.uint8):
    return torch.zeros(size, dtype=dtype)


@pytest.mark.parametrize("fmt,dtype", [(sdb.SD_CACHE_BF16, BF), (sdb.SD_CACHE_MXFP8, torch.float8_e4m3fn),
                                       (sdb.SD_CACHE_MXINT8, torch.int8)])
def test_make_cache(fmt, dtype):
    K = _bytes(4, 16, 2, 128, dtype=dtype)
    sc = None if fmt == sdb.SD_CACHE_BF16 else _bytes(4, 2, 16, 2, 4)
    assert sdb.make_cache(fmt, K, K.clone(), sc).heads == 2
    other = torch.float16 if fmt == sdb.SD_CACHE_BF16 else BF
    for k, v in ((K.to(other), K), (K, K.to(other)), (K[:3], K), (K[:, :8].contiguous(), K[:, :8].contiguous()),
                 (K[..., :64].contiguous(), K[..., :64].contiguous()), (K.view(4, 16, 256), K.view(4, 16, 256))):
        with pytest.raises(ValueError, match="make_cache"):
            sdb.make_cache(fmt, k, v, sc)
    with pytest.raises(ValueError, match="format"):
        sdb.make_cache(7, K, K, sc)
    if sc is not None:
        u = K.view(torch.uint8)
        assert sdb.make_cache(fmt, u, u, sc).pages == 4
        for bad in (None, sc[:3], sc.view(torch.int8), _bytes(4, 16, 2, 2, 4), sc.transpose(1, 2)):
            with pytest.raises(ValueError, match="make_cache"):
                sdb.make_cache(fmt, K, K, bad)
