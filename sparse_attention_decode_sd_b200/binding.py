"""ctypes binding of libsparsedecode (include/sparsedecode.h): argument marshalling only.

Every function takes torch tensors that already live on the current CUDA device, passes their
device pointers to the C entry point of the same name on the current stream (or `stream`), and
returns the host status.  No computation happens here and there is no fallback: if the shared
library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsparsedecode.so")
_lib = None

SD_OK = 0
SD_ERR_INVALID_ARG = 1
SD_ERR_UNSUPPORTED = 2
SD_ERR_CUDA = 3
SD_ERR_INDEX_OOB = 4
SD_ERR_TIMEOUT = 5
SD_ERR_WORKSPACE = 6
SD_ERR_ORDER = 7

SD_OP_TOPK = 1
SD_OP_SPARSE = 2
SD_OP_DENSE = 3
SD_OP_QUEST = 4
SD_OP_CHUNK = 5
SD_OP_CACHE_SPARSE = 6

SD_CACHE_BF16 = 0
SD_CACHE_MXFP8 = 1
SD_CACHE_MXINT8 = 2

SD_SAMPLED_FLAG = 1 << 30   # idx entry of a row drawn by sd_stochastic_index (position in the low 30 bits)

EXPORTED = ("sd_workspace_size", "sd_topk_index", "sd_topk_scores", "sd_topk_select", "sd_topk_index_static",
            "sd_sparse_decode", "sd_stochastic_index", "sd_sparse_decode_sampled", "sd_dense_decode", "sd_append_kv",
            "sd_quest_summarize", "sd_quest_append_kv", "sd_quest_index", "sd_cache_write", "sd_cache_read", "sd_chunk_attention",
            "sd_cache_sparse_decode", "sd_selftest_wait_timeout", "sd_status_string",
            "sd_last_cuda_error", "sd_version")


class SdShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages_per_req", ctypes.c_int32),
                ("k_max", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


class SdCache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("reserved", ctypes.c_int32), ("K", ctypes.c_void_p),
                ("V", ctypes.c_void_p), ("scales", ctypes.c_void_p)]
    pages = heads = None   # of the tensors behind it, where make_cache() made it


class SdError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = f"{what}: {status_string(status)} (status {status})"
        if status == SD_ERR_CUDA:
            code, name = last_cuda_error()
            msg += f": {name} ({code})"
        super().__init__(msg)
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load():
    """Loads libsparsedecode.so (built by sparse_attention_decode_sd_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libsparsedecode.so not found at {_LIB_PATH}; run "
                           "`python -m sparse_attention_decode_sd_b200.build` first")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    SH = ctypes.POINTER(SdShape)
    lib.sd_workspace_size.argtypes = [SH, I32, ctypes.POINTER(SZ)]
    lib.sd_topk_index.argtypes = [SH, P, P, P, P, P, P, P, SZ, P, P]
    lib.sd_topk_scores.argtypes = [SH, P, P, P, P, P, P, SZ, P, P]
    lib.sd_topk_select.argtypes = [SH, P, P, P, P, SZ, P, P]
    lib.sd_topk_index_static.argtypes = [SH, P, P, P, P, P, P, P, P]
    lib.sd_topk_index_static.restype = I32
    lib.sd_sparse_decode.argtypes = [SH, P, P, P, P, P, P, P, P, SZ, P, P]
    lib.sd_sparse_decode_sampled.argtypes = [SH, P, P, P, P, P, P, P, P, SZ, P, P]
    lib.sd_stochastic_index.argtypes = [SH, P, P, P, P, P, P, ctypes.c_uint64, ctypes.c_uint32, P, P, SZ, P, P]
    lib.sd_dense_decode.argtypes = [SH, P, P, P, P, P, P, P, SZ, P, P]
    lib.sd_append_kv.argtypes = [SH, P, P, P, P, P, P, P, I32, P, P]
    lib.sd_quest_append_kv.argtypes = [SH, P, P, P, P, P, P, P, I32, P, P, P]
    lib.sd_quest_summarize.argtypes = [SH, P, P, P, P, I32, P, P]
    lib.sd_quest_index.argtypes = [SH, P, P, P, P, P, P, P, SZ, P, P]
    CH = ctypes.POINTER(SdCache)
    lib.sd_cache_write.argtypes = [SH, CH, P, P, P, I32, P, P, P, P, P]
    lib.sd_cache_read.argtypes = [SH, CH, P, P, P, P, I32, P, P, P, P]
    lib.sd_chunk_attention.argtypes = [SH, CH, P, P, P, P, I32, P, P, SZ, P, P]
    lib.sd_cache_sparse_decode.argtypes = [SH, CH, P, P, P, P, P, P, SZ, P, P]
    lib.sd_selftest_wait_timeout.argtypes = [ctypes.c_uint32, P, P]
    lib.sd_selftest_wait_timeout.restype = I32
    for f in (lib.sd_workspace_size, lib.sd_topk_index, lib.sd_topk_scores, lib.sd_topk_select, lib.sd_sparse_decode,
              lib.sd_sparse_decode_sampled, lib.sd_stochastic_index, lib.sd_dense_decode, lib.sd_append_kv,
              lib.sd_quest_summarize, lib.sd_quest_append_kv, lib.sd_quest_index, lib.sd_cache_write, lib.sd_cache_read,
              lib.sd_chunk_attention, lib.sd_cache_sparse_decode):
        f.restype = I32
    lib.sd_status_string.argtypes = [I32]
    lib.sd_status_string.restype = ctypes.c_char_p
    lib.sd_last_cuda_error.argtypes = [ctypes.POINTER(ctypes.c_char_p)]
    lib.sd_last_cuda_error.restype = I32
    lib.sd_version.argtypes = []
    lib.sd_version.restype = I32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().sd_status_string(int(status)).decode()


def last_cuda_error() -> tuple[int, str]:
    """(cudaError_t value, its name) behind the last SD_ERR_CUDA on this thread."""
    name = ctypes.c_char_p()
    code = load().sd_last_cuda_error(ctypes.byref(name))
    return int(code), (name.value or b"").decode()


def version() -> int:
    return int(load().sd_version())


def make_shape(B, Hq, Hkv, max_pages, k_max, num_pages, head_dim=128, page_size=16) -> SdShape:
    return SdShape(int(B), int(Hq), int(Hkv), int(head_dim), int(page_size), int(max_pages), int(k_max), int(num_pages))


def shape_of(w) -> SdShape:
    """SdShape of a workloads.Workload."""
    return make_shape(w.B, w.Hq, w.Hkv, w.max_pages, w.k_max, w.num_pages, w.d, w.P)


def _ptr(t):
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream(stream):
    if stream is None:   # the current stream's handle, without making a Stream object for each call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, what: str, check: bool) -> int:
    if check and status != SD_OK:
        raise SdError(status, what)
    return status


def sd_workspace_size(shape: SdShape, op: int) -> int:
    n = ctypes.c_size_t(0)
    st = load().sd_workspace_size(ctypes.byref(shape), int(op), ctypes.byref(n))
    _check(st, "sd_workspace_size", True)
    return int(n.value)


def _ws_bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def sd_topk_index(shape, q, K, page_table, lens, k, idx, workspace, dev_status, stream=None, check=True) -> int:
    st = load().sd_topk_index(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(page_table), _ptr(lens), _ptr(k), _ptr(idx),
                              _ptr(workspace), _ws_bytes(workspace), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_topk_index", check)


def sd_topk_scores(shape, q, K, page_table, lens, k, workspace, dev_status, stream=None, check=True) -> int:
    st = load().sd_topk_scores(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(page_table), _ptr(lens), _ptr(k),
                               _ptr(workspace), _ws_bytes(workspace), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_topk_scores", check)


def sd_topk_select(shape, lens, k, idx, workspace, dev_status, stream=None, check=True) -> int:
    st = load().sd_topk_select(ctypes.byref(shape), _ptr(lens), _ptr(k), _ptr(idx), _ptr(workspace),
                               _ws_bytes(workspace), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_topk_select", check)


def sd_topk_index_static(shape, q, K, page_table, lens, k, idx, dev_status, stream=None, check=True) -> int:
    """sd_topk_index with the library's own static 48 MiB scratch (no workspace argument)."""
    st = load().sd_topk_index_static(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(page_table), _ptr(lens), _ptr(k),
                                     _ptr(idx), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_topk_index_static", check)


def sd_sparse_decode(shape, q, K, V, page_table, lens, idx, out, workspace, dev_status, stream=None,
                     check=True) -> int:
    st = load().sd_sparse_decode(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V), _ptr(page_table), _ptr(lens),
                                 _ptr(idx), _ptr(out), _ptr(workspace), _ws_bytes(workspace), _ptr(dev_status),
                                 _stream(stream))
    return _check(st, "sd_sparse_decode", check)


def sd_stochastic_index(shape, q, K, page_table, lens, k_det, k_samp, seed, step, idx, workspace, dev_status,
                        stream=None, check=True) -> int:
    st = load().sd_stochastic_index(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(page_table), _ptr(lens), _ptr(k_det),
                                    _ptr(k_samp), ctypes.c_uint64(int(seed) & 0xFFFFFFFFFFFFFFFF),
                                    ctypes.c_uint32(int(step) & 0xFFFFFFFF), _ptr(idx), _ptr(workspace),
                                    _ws_bytes(workspace), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_stochastic_index", check)


def sd_sparse_decode_sampled(shape, q, K, V, page_table, lens, idx, out, workspace, dev_status, stream=None,
                             check=True) -> int:
    st = load().sd_sparse_decode_sampled(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V), _ptr(page_table),
                                         _ptr(lens), _ptr(idx), _ptr(out), _ptr(workspace), _ws_bytes(workspace),
                                         _ptr(dev_status), _stream(stream))
    return _check(st, "sd_sparse_decode_sampled", check)


def sd_dense_decode(shape, q, K, V, page_table, lens, out, workspace, dev_status, stream=None, check=True) -> int:
    st = load().sd_dense_decode(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V), _ptr(page_table), _ptr(lens),
                                _ptr(out), _ptr(workspace), _ws_bytes(workspace), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_dense_decode", check)


def sd_quest_summarize(shape, K, page_table, lens, boxes, dev_status, last_page_only=False, stream=None,
                       check=True) -> int:
    st = load().sd_quest_summarize(ctypes.byref(shape), _ptr(K), _ptr(page_table), _ptr(lens), _ptr(boxes),
                                   int(bool(last_page_only)), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_quest_summarize", check)


def sd_quest_index(shape, q, boxes, page_table, lens, k, idx, workspace, dev_status, stream=None, check=True) -> int:
    st = load().sd_quest_index(ctypes.byref(shape), _ptr(q), _ptr(boxes), _ptr(page_table), _ptr(lens), _ptr(k),
                               _ptr(idx), _ptr(workspace), ctypes.c_size_t(workspace.numel()), _ptr(dev_status),
                               _stream(stream))
    return _check(st, "sd_quest_index", check)


def sd_selftest_wait_timeout(wait_ms: int, dev_status, stream=None, check=True) -> int:
    st = load().sd_selftest_wait_timeout(int(wait_ms), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_selftest_wait_timeout", check)


def quest_boxes_for(shape: SdShape, device=None) -> torch.Tensor:
    """A caller-side buffer for the Quest page boxes: bf16 [num_pages][Hkv][2][head_dim]."""
    return torch.empty((shape.num_pages, shape.num_kv_heads, 2, shape.head_dim), dtype=torch.bfloat16,
                       device=device or "cuda")


def sd_append_kv(shape, K, V, page_table, lens, k_new, v_new, k_sel, ratio, dev_status, stream=None,
                 check=True) -> int:
    st = load().sd_append_kv(ctypes.byref(shape), _ptr(K), _ptr(V), _ptr(page_table), _ptr(lens), _ptr(k_new),
                             _ptr(v_new), _ptr(k_sel), int(ratio), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_append_kv", check)


def sd_quest_append_kv(shape, K, V, page_table, lens, k_new, v_new, k_sel, ratio, boxes, dev_status, stream=None,
                       check=True) -> int:
    """sd_append_kv that also brings the Quest box of each written page up to date."""
    st = load().sd_quest_append_kv(ctypes.byref(shape), _ptr(K), _ptr(V), _ptr(page_table), _ptr(lens), _ptr(k_new),
                                   _ptr(v_new), _ptr(k_sel), int(ratio), _ptr(boxes), _ptr(dev_status),
                                   _stream(stream))
    return _check(st, "sd_quest_append_kv", check)


_CACHE_DTYPE = {SD_CACHE_BF16: torch.bfloat16, SD_CACHE_MXFP8: torch.float8_e4m3fn, SD_CACHE_MXINT8: torch.int8}


def make_cache(fmt: int, K, V, scales=None) -> SdCache:
    """Handle of a paged cache: K, V [num_pages][P][Hkv][d] of the format's element type (8-bit formats: or uint8) and, for
    the 8-bit formats, scales uint8 [num_pages][Hkv][P][2][4].  It keeps the tensors alive."""
    fmt = int(fmt)
    if fmt not in _CACHE_DTYPE:
        raise ValueError(f"make_cache: unknown format {fmt}")
    if any(t is not None and not t.is_contiguous() for t in (K, V, scales)):
        raise ValueError("make_cache: the tensors must be contiguous")
    types = (_CACHE_DTYPE[fmt],) if fmt == SD_CACHE_BF16 else (_CACHE_DTYPE[fmt], torch.uint8)
    if K.dtype not in types or V.dtype not in types:
        raise ValueError(f"make_cache: K and V must be {types[0]}, not {K.dtype} and {V.dtype}")
    if K.dim() != 4 or K.shape[1] != 16 or K.shape[3] != 128 or V.shape != K.shape:
        raise ValueError(f"make_cache: K and V must be [num_pages][16][Hkv][128], not {list(K.shape)} and {list(V.shape)}")
    if fmt != SD_CACHE_BF16:
        want = (K.shape[0], K.shape[2], 16, 2, 4)
        if scales is None or scales.dtype != torch.uint8 or tuple(scales.shape) != want:
            raise ValueError(f"make_cache: scales must be uint8 {list(want)}")
    if any(t is not None and t.device != K.device for t in (V, scales)):
        raise ValueError("make_cache: the tensors must be on one device")
    addr = [None if t is None else t.data_ptr() for t in (K, V, scales)]
    c = SdCache(fmt, 0, *addr)
    c.tensors = (K, V, scales)
    c.pages, c.heads = int(K.shape[0]), int(K.shape[2])
    return c


def empty_cache(shape: SdShape, fmt: int, device=None) -> SdCache:
    """A zeroed cache of the shape's pages in the given format (its tensors: `.tensors`)."""
    dev = device or "cuda"
    size = (shape.num_pages, shape.page_size, shape.num_kv_heads, shape.head_dim)
    K, V = (torch.zeros(size, dtype=_CACHE_DTYPE[fmt], device=dev) for _ in range(2))
    sc = None if fmt == SD_CACHE_BF16 else torch.zeros((shape.num_pages, shape.num_kv_heads, shape.page_size, 2, 4),
                                                       dtype=torch.uint8, device=dev)
    return make_cache(fmt, K, V, sc)


_BF16, _I32 = torch.bfloat16, torch.int32


def _cache_ok(what, shape, cache):
    pages = cache.pages
    if pages is not None and (pages < shape.num_pages or cache.heads != shape.num_kv_heads):
        raise ValueError(f"{what}: a cache of {pages} pages and {cache.heads} KV heads for a shape of "
                         f"{shape.num_pages} and {shape.num_kv_heads}")


def _batch_ok(what, rows, heads, a, b, row_start, B):
    """The arrays of a ragged batch, whose sizes sd_shape does not give: a, b bf16 [rows][heads][d] (or longer) on the current
    device, row_start int32 [B + 1], all contiguous.  Addresses (int) are taken as they are.  One expression where all is
    well: a call of a few rows takes hardly longer than this."""
    n = rows * heads * 128
    try:
        if (a.dtype is _BF16 and b.dtype is _BF16 and a.is_contiguous() and b.is_contiguous() and a.numel() >= n
                and b.numel() >= n and row_start.dtype is _I32 and row_start.is_contiguous() and row_start.numel() > B
                and a.get_device() == torch._C._cuda_getDevice() == b.get_device()):
            return
    except (AttributeError, RuntimeError):   # an address; no device at all
        pass
    arrays = [t for t in (a, b) if not isinstance(t, int)]
    for t in arrays:
        if t.dtype is not _BF16 or not t.is_contiguous() or t.numel() < n:
            raise ValueError(f"{what}: expected contiguous bf16 rows [{rows}][{heads}][128], got {t.dtype} {list(t.shape)}"
                             f"{'' if t.is_contiguous() else ', not contiguous'}")
    _counts_ok(what, row_start, B + 1)
    for t in arrays:
        if not t.is_cuda or t.get_device() != torch._C._cuda_getDevice():
            raise ValueError(f"{what}: the tensors must be on the current CUDA device, not on {t.device}")


def _counts_ok(what, t, n):
    if not isinstance(t, int) and (t.dtype is not _I32 or not t.is_contiguous() or t.numel() < n):
        raise ValueError(f"{what}: expected contiguous int32 [{n}], got {t.dtype} {list(t.shape)}")


def sd_cache_write(shape, cache, page_table, lens, row_start, k_new, v_new, boxes, dev_status, stream=None,
                   check=True) -> int:
    rows = k_new.shape[0]
    _cache_ok("sd_cache_write", shape, cache)
    _batch_ok("sd_cache_write", rows, shape.num_kv_heads, k_new, v_new, row_start, shape.batch)
    st = load().sd_cache_write(ctypes.byref(shape), ctypes.byref(cache), _ptr(page_table), _ptr(lens), _ptr(row_start),
                               rows, k_new.data_ptr(), _ptr(v_new), _ptr(boxes), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_cache_write", check)


def sd_cache_read(shape, cache, page_table, lens, first, row_start, k_out, v_out, dev_status, stream=None,
                  check=True) -> int:
    a, b = (v_out if k_out is None else k_out), (k_out if v_out is None else v_out)
    rows = a.shape[0]
    _cache_ok("sd_cache_read", shape, cache)
    _counts_ok("sd_cache_read", first, shape.batch)
    _batch_ok("sd_cache_read", rows, shape.num_kv_heads, a, b, row_start, shape.batch)
    st = load().sd_cache_read(ctypes.byref(shape), ctypes.byref(cache), _ptr(page_table), _ptr(lens), _ptr(first),
                              _ptr(row_start), rows, _ptr(k_out), _ptr(v_out), _ptr(dev_status), _stream(stream))
    return _check(st, "sd_cache_read", check)


def sd_chunk_attention(shape, cache, q, page_table, lens, row_start, out, workspace, dev_status, stream=None,
                       check=True) -> int:
    rows = q.shape[0]
    _cache_ok("sd_chunk_attention", shape, cache)
    _batch_ok("sd_chunk_attention", rows, shape.num_q_heads, q, out, row_start, shape.batch)
    st = load().sd_chunk_attention(ctypes.byref(shape), ctypes.byref(cache), q.data_ptr(), _ptr(page_table), _ptr(lens),
                                   _ptr(row_start), rows, _ptr(out), _ptr(workspace), _ws_bytes(workspace),
                                   _ptr(dev_status), _stream(stream))
    return _check(st, "sd_chunk_attention", check)


def sd_cache_sparse_decode(shape, cache, q, page_table, lens, idx, out, workspace, dev_status, stream=None,
                           check=True) -> int:
    _cache_ok("sd_cache_sparse_decode", shape, cache)
    st = load().sd_cache_sparse_decode(ctypes.byref(shape), ctypes.byref(cache), _ptr(q), _ptr(page_table), _ptr(lens),
                                       _ptr(idx), _ptr(out), _ptr(workspace), _ws_bytes(workspace), _ptr(dev_status),
                                       _stream(stream))
    return _check(st, "sd_cache_sparse_decode", check)


def workspace_for(shape: SdShape, op: int, device=None) -> torch.Tensor:
    """A caller-side workspace buffer of the size the library asks for (uint8, 256-byte aligned)."""
    n = sd_workspace_size(shape, op)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def read_status(dev_status: torch.Tensor) -> int:
    """Synchronises dev_status's stream and returns the device-side status word."""
    return int(dev_status.item())
