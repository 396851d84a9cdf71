"""Host validation of the cache and chunk entry points, and the references of the GPU tests.  CPU only: no call
here reaches a kernel."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from sparse_attention_decode_sd_b200 import binding as sdb
from sparse_attention_decode_sd_b200 import build as sdbuild
from tests import cache_helpers as ch


@pytest.fixture(scope="module")
def lib():
    sdbuild.build()
    return sdb.load()


FAKE, ODD = 1 << 20, (1 << 20) + 2      # never dereferenced: validation fails first
WS = ctypes.c_size_t(1 << 40)


def _shape(**kw):
    base = dict(B=4, Hq=64, Hkv=8, max_pages=8192, k_max=2621, num_pages=32768)
    base.update(kw)
    return sdb.make_shape(**base)


def _cache(fmt=sdb.SD_CACHE_MXFP8, K=FAKE, V=FAKE, scales=FAKE, reserved=0):
    return sdb.SdCache(fmt, reserved, K, V, scales)


def _write(lib, s=None, c=None, pt=FAKE, lens=FAKE, rs=FAKE, rows=8, k=FAKE, v=FAKE, boxes=None, st=FAKE):
    return lib.sd_cache_write(ctypes.byref(s or _shape()), ctypes.byref(c) if c is not None else None, pt, lens, rs, rows, k, v,
                              boxes, st, None)


def _read(lib, s=None, c=None, pt=FAKE, lens=FAKE, first=FAKE, rs=FAKE, rows=8, k=FAKE, v=FAKE, st=FAKE):
    return lib.sd_cache_read(ctypes.byref(s or _shape()), ctypes.byref(c) if c is not None else None, pt, lens, first, rs, rows,
                             k, v, st, None)


def _chunk(lib, s=None, c=None, q=FAKE, pt=FAKE, lens=FAKE, rs=FAKE, rows=8, out=FAKE, ws=FAKE, n=WS, st=FAKE):
    return lib.sd_chunk_attention(ctypes.byref(s or _shape()), ctypes.byref(c) if c is not None else None, q, pt, lens, rs, rows,
                                  out, ws, n, st, None)


def _sparse(lib, s=None, c=None, q=FAKE, pt=FAKE, lens=FAKE, idx=FAKE, out=FAKE, ws=FAKE, n=WS, st=FAKE):
    return lib.sd_cache_sparse_decode(ctypes.byref(s or _shape()), ctypes.byref(c) if c is not None else None, q, pt, lens, idx,
                                      out, ws, n, st, None)


CALLS = [_write, _read, _chunk, _sparse]


@pytest.mark.parametrize("call", CALLS)
def test_cache_handle_is_checked(lib, call):
    bad = [None, _cache(fmt=3), _cache(fmt=-1), _cache(K=None), _cache(V=None), _cache(scales=None), _cache(K=ODD),
           _cache(V=FAKE + 8), _cache(scales=FAKE + 4), _cache(reserved=1)]
    for c in bad:
        assert call(lib, c=c) == sdb.SD_ERR_INVALID_ARG


@pytest.mark.parametrize("call", CALLS)
def test_shapes_are_checked(lib, call):
    assert call(lib, c=_cache(), s=_shape(Hq=60)) == sdb.SD_ERR_INVALID_ARG
    assert call(lib, c=_cache(), s=_shape(head_dim=64)) == sdb.SD_ERR_UNSUPPORTED
    assert call(lib, c=_cache(), s=_shape(Hq=136, Hkv=4)) == sdb.SD_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,names", [(_write, ("pt", "lens", "rs", "k", "v", "st")), (_read, ("pt", "lens", "first", "rs", "st")),
                                        (_chunk, ("q", "pt", "lens", "rs", "out", "ws", "st")),
                                        (_sparse, ("q", "pt", "lens", "idx", "out", "ws", "st"))])
def test_null_and_misaligned_pointers(lib, call, names):
    for name in names:
        assert call(lib, c=_cache(), **{name: None}) == sdb.SD_ERR_INVALID_ARG, name
        assert call(lib, c=_cache(), **{name: ODD}) == sdb.SD_ERR_INVALID_ARG, name


def test_read_needs_one_output_and_write_aligned_boxes(lib):
    assert _read(lib, c=_cache(), k=None, v=None) == sdb.SD_ERR_INVALID_ARG
    assert _read(lib, c=_cache(), k=None, v=ODD) == sdb.SD_ERR_INVALID_ARG
    assert _write(lib, c=_cache(), boxes=ODD) == sdb.SD_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_write, _read, _chunk])
def test_row_counts(lib, call):
    assert call(lib, c=_cache(), rows=0) == sdb.SD_ERR_INVALID_ARG
    assert call(lib, c=_cache(), rows=-1) == sdb.SD_ERR_INVALID_ARG
    assert call(lib, c=_cache(), rows=1 << 25) == sdb.SD_ERR_UNSUPPORTED      # times 64 heads: 2^31
    assert call(lib, c=_cache(), s=_shape(Hq=1, Hkv=1), rows=0x7fffffff) == sdb.SD_ERR_UNSUPPORTED


def test_sparse_refuses_bf16_and_too_many_entries(lib):
    assert _sparse(lib, c=_cache(fmt=sdb.SD_CACHE_BF16)) == sdb.SD_ERR_UNSUPPORTED
    big = _shape(B=64, Hq=128, Hkv=8, k_max=1 << 18, max_pages=1 << 14)
    assert _sparse(lib, c=_cache(), s=big) == sdb.SD_ERR_UNSUPPORTED
    n = ctypes.c_size_t(0)
    assert lib.sd_workspace_size(ctypes.byref(big), sdb.SD_OP_CACHE_SPARSE, ctypes.byref(n)) == sdb.SD_ERR_UNSUPPORTED


def test_workspaces(lib):
    for call, op in ((_chunk, sdb.SD_OP_CHUNK), (_sparse, sdb.SD_OP_CACHE_SPARSE)):
        need = sdb.sd_workspace_size(_shape(), op)
        assert need % 256 == 0 and need > 0
        assert call(lib, c=_cache(), n=ctypes.c_size_t(need - 1)) == sdb.SD_ERR_WORKSPACE
        assert call(lib, c=_cache(), ws=FAKE + 16) == sdb.SD_ERR_INVALID_ARG


# ---- the references used on the GPU, against torch's own conversions and closed forms ----------------------

def test_e4m3_table_is_torchs():
    u = torch.arange(256).to(torch.uint8)
    want = u.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ch.e4m3_table(), want, equal_nan=True)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_quantiser_keeps_half_a_step(fmt):
    x = (torch.randn((64, 128), generator=torch.Generator().manual_seed(1)) * 3).bfloat16()
    el, by = ch.quantise(x, fmt)
    v = ch.values(el, by, fmt)
    blk = x.double().view(64, 4, 32)
    amax = blk.abs().amax(-1, keepdim=True)
    if fmt == "mxint8":      # step <= amax / 63.5: half of it
        bound = amax / 127 + 0 * blk
    else:                    # half of a 2^-3 step of the value's binade, or of the smallest step
        bound = torch.maximum(blk.abs() * 2.0 ** -4, amax * 2.0 ** -9 * 2.0 ** -8)
    assert ((v.view(64, 4, 32) - blk).abs() <= bound).all()
    if fmt == "mxfp8":
        e = by.double() - 127
        y = (blk * torch.exp2(-e)[..., None]).float()
        assert torch.equal(y.to(torch.float8_e4m3fn).view(torch.uint8).view(64, 128), el)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxint8"])
def test_every_stored_value_is_exact_in_bf16(fmt):
    x = torch.cat([torch.randn((32, 128)) * 2.0 ** k for k in (-130, -120, -3, 0, 60, 124)]).bfloat16()
    v = ch.values(*ch.quantise(x, fmt), fmt)
    assert torch.equal(v.bfloat16().double(), v)


def test_reference_attention_is_sdpa():
    w = ch.Batch([5, 0, 3], [4, 2, 30], 4, 2, "bf16", pad=2, lead=1)
    ref = w.attention()
    assert sorted(ref) == [1, 2, 3, 4, 5, 6, 7, 8]
    for b in range(3):
        if not w.n[b]:
            continue
        k, v = (w.rows(i, b, 0, w.total[b]).repeat_interleave(2, 1).transpose(0, 1) for i in (0, 1))
        q = w.q[w.start[b]:w.start[b + 1]].double().transpose(0, 1)
        mask = torch.ones(w.n[b], w.total[b], dtype=torch.bool).tril(w.total[b] - w.n[b])
        o = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=mask)
        got = torch.stack([ref[t][0] for t in range(w.start[b], w.start[b + 1])], 1)
        assert (got - o).abs().max() < 1e-12


def test_make_cache_refuses_strided_tensors():
    K = torch.zeros((2, 16, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="contiguous"):
        sdb.make_cache(sdb.SD_CACHE_BF16, K.transpose(1, 2), K)
    assert sdb.make_cache(sdb.SD_CACHE_BF16, K, K.clone()).tensors[0] is K
