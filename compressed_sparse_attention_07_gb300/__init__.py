"""GB300 (sm_103a) CSA2 compressed sparse attention.

Thin ctypes binding over the C ABI in ``include/csa2.h`` (libcsa2.so, built
in-tree from ``csrc/``).  PyTorch only provides device memory and streams:
every step of the path runs in the library's CUDA kernels, and the binding
raises if the library cannot be built or loaded -- there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import math
import threading

import torch

from . import build as _build

__all__ = [
    "Cfg", "PagedCache", "GroupState", "load", "compress", "index_workspace_bytes", "index_topk", "attend",
    "gather_dequant", "layer", "status_string", "CsaError", "CACHE_FP4", "CACHE_BF16", "MODE_FULL",
    "MODE_REINDEX", "MODE_REUSE", "PAGE", "library_path", "capture", "swa_encode", "CACHE_FP4_S32",
    "FMT_IDX_68B", "FMT_SWA_FP8", "FMT_IDX_QFP4", "SWA_FP8_ROW", "KVCfg", "KVCache", "kv_append", "kv_attend",
    "kv_cross_attend", "kv_workspace_bytes", "rope_table", "ROPE_INTERLEAVED", "ROPE_HALF",
    "kv_append_axes", "kv_reorder", "beam_select", "beam_workspace_bytes", "Fp4Weights", "fp4_linear",
]

CACHE_FP4, CACHE_BF16, CACHE_FP4_S32 = 0, 1, 2
FMT_IDX_68B, FMT_SWA_FP8, FMT_IDX_QFP4 = 1, 2, 4
SWA_FP8_ROW = 528  # bytes of one MXFP8 window row
MODE_FULL, MODE_REINDEX, MODE_REUSE = 0, 1, 2
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
PAGE = 64


class CsaError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__("%s failed: %s (%d)" % (fn, status_string(code) if _lib else code, code))
        self.code = code


class Cfg(C.Structure):
    """csa2_cfg: defaults are the model's sizes (64 x 512 latent, 64 RoPE
    dims, indexer 32 x 128, top-512, window 128, HSI 2048 x 8); `formats`
    takes FMT_IDX_68B (indexer entries with one scale per 32 channels),
    FMT_SWA_FP8 (MXFP8 window rows) and FMT_IDX_QFP4 (FP4 indexer queries)."""
    _fields_ = [("dim", C.c_int32), ("rope_dims", C.c_int32), ("n_heads", C.c_int32), ("idx_heads", C.c_int32),
                ("idx_dim", C.c_int32), ("topk", C.c_int32), ("window", C.c_int32), ("ratio", C.c_int32),
                ("hsi_blocks", C.c_int32), ("hsi_block", C.c_int32), ("cache_dtype", C.c_int32),
                ("formats", C.c_int32), ("rope_theta", C.c_double)]

    def __init__(self, ratio=2, cache_dtype=CACHE_FP4, topk=512, window=128, hsi_blocks=0, rope_theta=1e4,
                 formats=0):
        super().__init__(512, 64, 64, 32, 128, topk, window, ratio, hsi_blocks, 8, cache_dtype, formats, rope_theta)

    @property
    def idx_dtype(self) -> int:
        """Format of the indexer cache under this configuration."""
        return CACHE_FP4_S32 if (self.cache_dtype == CACHE_FP4 and self.formats & FMT_IDX_68B) else self.cache_dtype


class _CacheDesc(C.Structure):
    _fields_ = [("data", C.c_void_p), ("scales", C.c_void_p), ("block_table", C.c_void_p), ("max_pages", C.c_int32),
                ("num_pages", C.c_int32), ("channels", C.c_int32), ("reserved", C.c_int32)]


class _GroupState(C.Structure):
    _fields_ = [("main_cache", _CacheDesc), ("idx_cache", _CacheDesc), ("n_entries", C.c_void_p),
                ("max_entries", C.c_int32), ("reserved", C.c_int32), ("topk", C.c_void_p), ("pool", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t), ("status", C.c_void_p)]


class _LayerIO(C.Structure):
    _fields_ = [("B", C.c_int32), ("Tq", C.c_int32), ("q_pos", C.c_void_p), ("T", C.c_int32), ("x", C.c_void_p),
                ("pos0", C.c_void_p), ("merge_w", C.c_void_p), ("w_idx", C.c_void_p), ("q_idx", C.c_void_p),
                ("head_w", C.c_void_p), ("q", C.c_void_p), ("swa", C.c_void_p), ("S", C.c_int32),
                ("swa_len", C.c_void_p), ("swa_pos0", C.c_void_p), ("scale", C.c_float), ("out", C.c_void_p),
                ("lse", C.c_void_p)]


class KVCfg(C.Structure):
    """csa2_kv_cfg: an ordinary grouped-query layer -- `n_heads` query heads over `kv_heads` key / value heads of
    `head_dim` (64 or 128) channels, an FP4 or BF16 cache, a sliding `window` (0: none) and RoPE over the first
    `rope_dims` channels (ROPE_INTERLEAVED pairs, or ROPE_HALF)."""
    _fields_ = [("n_heads", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32), ("cache_dtype", C.c_int32),
                ("window", C.c_int32), ("rope_dims", C.c_int32), ("rope_style", C.c_int32), ("reserved", C.c_int32)]

    def __init__(self, n_heads=64, kv_heads=8, head_dim=128, cache_dtype=CACHE_FP4, window=0, rope_dims=64,
                 rope_style=ROPE_INTERLEAVED):
        super().__init__(n_heads, kv_heads, head_dim, cache_dtype, window, rope_dims, rope_style, 0)


class _Fp4Desc(C.Structure):
    _fields_ = [("data", C.c_void_p), ("n", C.c_int32), ("k", C.c_int32), ("alpha", C.c_float), ("reserved", C.c_int32)]


class _KVCacheDesc(C.Structure):
    _fields_ = [("k_data", C.c_void_p), ("k_scales", C.c_void_p), ("v_data", C.c_void_p), ("v_scales", C.c_void_p),
                ("block_table", C.c_void_p), ("max_pages", C.c_int32), ("num_pages", C.c_int32)]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load():
    """Build (if stale) and load libcsa2.so; raises when that is impossible."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build()
        L = C.CDLL(path)
        vp, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
        L.csa2_page_bytes.restype = sz
        L.csa2_page_bytes.argtypes = [i32, i32, i32]
        L.csa2_status_string.restype = C.c_char_p
        L.csa2_status_string.argtypes = [i32]
        L.csa2_compress.restype = i32
        L.csa2_compress.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.csa2_index_workspace_bytes.restype = sz
        L.csa2_index_workspace_bytes.argtypes = [vp, i32, i32, i32, i32]
        L.csa2_index_topk.restype = i32
        L.csa2_index_topk.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp, vp]
        L.csa2_index_score.restype = i32
        L.csa2_index_score.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, i32, vp, i32, vp, sz, vp, vp]
        L.csa2_index_select.restype = i32
        L.csa2_index_select.argtypes = [vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp, vp]
        L.csa2_attend.restype = i32
        L.csa2_attend.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, C.c_float, vp, vp, vp, vp]
        L.csa2_gather_dequant.restype = i32
        L.csa2_gather_dequant.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
        L.csa2_layer.restype = i32
        L.csa2_layer.argtypes = [vp, i32, vp, vp, vp]
        L.csa2_swa_encode.restype = i32
        L.csa2_swa_encode.argtypes = [i32, i32, vp, vp, vp, i32, vp, vp]
        i64, kvc = C.c_int64, C.POINTER(KVCfg)
        kvd = C.POINTER(_KVCacheDesc)
        L.csa2_kv_page_bytes.restype = sz
        L.csa2_kv_page_bytes.argtypes = [kvc, i32]
        L.csa2_kv_workspace_bytes.restype = sz
        L.csa2_kv_workspace_bytes.argtypes = [kvc, i32, i32, i32, i32]
        L.csa2_kv_append.restype = i32
        L.csa2_kv_append.argtypes = [kvc, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, kvd, vp, i64, vp, vp,
                                     vp, vp]
        L.csa2_kv_append_axes.restype = i32
        L.csa2_kv_append_axes.argtypes = [kvc, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, i32, C.c_char_p, vp, i64,
                                          kvd, vp, i64, vp, vp, vp, vp]
        L.csa2_kv_reorder.restype = i32
        L.csa2_kv_reorder.argtypes = [kvc, i32, vp, i32, i32, vp, vp, vp, vp]
        L.csa2_beam_workspace_bytes.restype = sz
        L.csa2_beam_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.csa2_beam_select.restype = i32
        L.csa2_beam_select.argtypes = [i32, i32, i32, i32, vp, i32, i64, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp]
        L.csa2_fp4_weight_bytes.restype = sz
        L.csa2_fp4_weight_bytes.argtypes = [i32, i32]
        L.csa2_fp4_encode.restype = i32
        L.csa2_fp4_encode.argtypes = [i32, i32, vp, i64, C.c_float, vp, vp, vp]
        L.csa2_fp4_pack.restype = i32
        L.csa2_fp4_pack.argtypes = [i32, i32, vp, vp, vp, vp, vp]
        L.csa2_fp4_linear.restype = i32
        L.csa2_fp4_linear.argtypes = [C.POINTER(_Fp4Desc), i32, vp, i64, vp, vp, i32, i64, vp, vp]
        for f in (L.csa2_kv_attend, L.csa2_kv_cross_attend):
            f.restype = i32
            f.argtypes = [kvc, i32, i32, vp, i64, vp, kvd, vp, i32, i32, C.c_float, vp, i64, vp, vp, sz, vp, vp]
        _lib = L
        return L


def status_string(code: int) -> str:
    return load().csa2_status_string(int(code)).decode()


def _check(fn, rc):
    if rc != 0:
        raise CsaError(fn, rc)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _bf16(t, name):
    if t is None:
        return None
    if t.dtype == torch.bfloat16:
        return _ptr(t, None, name)
    return _ptr(t, torch.int16, name) if t.dtype == torch.int16 else _ptr(t, torch.uint16, name)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


class PagedCache:
    """Device pages for one cache (main KV: 512 channels; indexer K: 128) of
    `batch` sequences with `capacity` entries each.  Pages are handed out in
    `page_order` (a permutation of range(num_pages); identity by default)."""

    def __init__(self, batch: int, capacity: int, channels: int, cache_dtype: int, device="cuda",
                 page_order=None, spare_pages: int = 0):
        lib = load()
        self.batch, self.channels, self.cache_dtype = batch, channels, cache_dtype
        self.max_pages = max(1, math.ceil(capacity / PAGE))
        self.capacity = self.max_pages * PAGE
        self.num_pages = batch * self.max_pages + spare_pages
        db = lib.csa2_page_bytes(channels, cache_dtype, 0)
        sb = lib.csa2_page_bytes(channels, cache_dtype, 1)
        if db == 0:
            raise ValueError("unsupported cache (channels=%d dtype=%d)" % (channels, cache_dtype))
        self.data = torch.zeros((self.num_pages, db), dtype=torch.uint8, device=device)
        self.scales = torch.zeros((self.num_pages, sb), dtype=torch.uint8, device=device) if sb else None
        order = torch.arange(batch * self.max_pages) if page_order is None else torch.as_tensor(page_order)
        self.block_table = order[: batch * self.max_pages].reshape(batch, self.max_pages).to(
            device=device, dtype=torch.int32).contiguous()

    def desc(self) -> _CacheDesc:
        return _CacheDesc(self.data.data_ptr(), self.scales.data_ptr() if self.scales is not None else None,
                          self.block_table.data_ptr(), self.max_pages, self.num_pages, self.channels, 0)


def compress(cfg: Cfg, x, pos0, merge_w, w_idx, main: PagedCache, idx: PagedCache, n_entries, status=None,
             stream=None):
    """a1: x [B][T][512] bf16, pos0 [B] int64, merge_w [r][512] fp32, w_idx [512][128] bf16."""
    B, T, _ = x.shape
    md, idd = main.desc(), idx.desc()
    _check("csa2_compress", load().csa2_compress(
        C.byref(cfg), B, T, _bf16(x, "x"), _ptr(pos0, torch.int64, "pos0"), _ptr(merge_w, torch.float32, "merge_w"),
        _bf16(w_idx, "w_idx"), C.byref(md), C.byref(idd), _ptr(n_entries, torch.int32, "n_entries"),
        _ptr(status, torch.int32, "status"), _stream(stream)))


def index_workspace_bytes(cfg: Cfg, B: int, Tq: int, max_entries: int, reindex: bool = False) -> int:
    return int(load().csa2_index_workspace_bytes(C.byref(cfg), B, Tq, max_entries, int(reindex)))


def index_topk(cfg: Cfg, q_idx, q_pos, idx: PagedCache, n_entries, max_entries: int, topk_out, workspace,
               head_w=None, pool=None, pool_out=None, status=None, stream=None):
    """a3-a6: q_idx [B][Tq][32][128] bf16, q_pos [B][Tq] int64 -> topk_out [B][Tq][k] int32
    (and pool_out [B][Tq][hsi_blocks] for an HSI Full layer; `pool` selects Reindex)."""
    B, Tq = q_idx.shape[:2]
    d = idx.desc()
    _check("csa2_index_topk", load().csa2_index_topk(
        C.byref(cfg), B, Tq, _bf16(q_idx, "q_idx"), _ptr(head_w, torch.float32, "head_w"),
        _ptr(q_pos, torch.int64, "q_pos"), C.byref(d), _ptr(n_entries, torch.int32, "n_entries"), int(max_entries),
        _ptr(pool, torch.int32, "pool"), _ptr(topk_out, torch.int32, "topk_out"),
        _ptr(pool_out, torch.int32, "pool_out"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(status, torch.int32, "status"), _stream(stream)))


def index_score(cfg: Cfg, q_idx, q_pos, idx: PagedCache, n_entries, max_entries: int, workspace, head_w=None,
                pool=None, hsi=False, status=None, stream=None):
    """a3/a5/a6 scores of every query into `workspace` (which holds them all), for index_select."""
    B, Tq = q_idx.shape[:2]
    d = idx.desc()
    _check("csa2_index_score", load().csa2_index_score(
        C.byref(cfg), B, Tq, _bf16(q_idx, "q_idx"), _ptr(head_w, torch.float32, "head_w"),
        _ptr(q_pos, torch.int64, "q_pos"), C.byref(d), _ptr(n_entries, torch.int32, "n_entries"), int(max_entries),
        _ptr(pool, torch.int32, "pool"), 1 if hsi else 0, _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(status, torch.int32, "status"), _stream(stream)))


def index_select(cfg: Cfg, q_pos, idx: PagedCache, n_entries, max_entries: int, topk_out, workspace, pool=None,
                 pool_out=None, status=None, stream=None):
    """a4/a5 from the scores index_score left in `workspace` -> topk_out (and pool_out)."""
    B, Tq = q_pos.shape[:2]
    d = idx.desc()
    _check("csa2_index_select", load().csa2_index_select(
        C.byref(cfg), B, Tq, _ptr(q_pos, torch.int64, "q_pos"), C.byref(d), _ptr(n_entries, torch.int32, "n_entries"),
        int(max_entries), _ptr(pool, torch.int32, "pool"), _ptr(topk_out, torch.int32, "topk_out"),
        _ptr(pool_out, torch.int32, "pool_out"), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(status, torch.int32, "status"), _stream(stream)))


def _swa(cfg: Cfg, swa):
    """Window rows: bf16 [B][S][512], or uint8 MXFP8 rows [B][S][528] under FMT_SWA_FP8."""
    if swa is None:
        return None
    if cfg.formats & FMT_SWA_FP8:
        if swa.shape[-1] != SWA_FP8_ROW:
            raise ValueError("MXFP8 window rows must be [B][S][%d] uint8" % SWA_FP8_ROW)
        return _ptr(swa, torch.uint8, "swa")
    return _bf16(swa, "swa")


def swa_encode(x, row0, rows, status=None, stream=None):
    """FP8 window rows: x [B][T][512] bf16 -> rows[b][row0[b] + i] of rows [B][S][528] uint8 (MXFP8)."""
    B, T = x.shape[:2]
    _check("csa2_swa_encode", load().csa2_swa_encode(
        B, T, _bf16(x, "x"), _ptr(row0, torch.int64, "row0"), _ptr(rows, torch.uint8, "rows"), rows.shape[1],
        _ptr(status, torch.int32, "status"), _stream(stream)))


def attend(cfg: Cfg, q, main: PagedCache, n_entries, topk, swa, swa_len, swa_pos0, q_pos, out, lse=None,
           scale=None, status=None, stream=None):
    """a7: q [B][Tq][64][512] bf16, topk [B][Tq][k], swa [B][S][512] bf16 (or [B][S][528] uint8 MXFP8 rows
    under FMT_SWA_FP8) -> out [B][Tq][64][512] fp32.  q, the window rows, swa_len, swa_pos0 and q_pos are read before
    the wait for the kernel ahead on the stream: enqueue another call between this one and the one that writes them."""
    B, Tq = q.shape[:2]
    S = swa.shape[1] if swa is not None else 0
    d = main.desc()
    scale = 1.0 / math.sqrt(512) if scale is None else float(scale)
    _check("csa2_attend", load().csa2_attend(
        C.byref(cfg), B, Tq, _bf16(q, "q"), C.byref(d), _ptr(n_entries, torch.int32, "n_entries"),
        _ptr(topk, torch.int32, "topk"), _swa(cfg, swa), S, _ptr(swa_len, torch.int32, "swa_len"),
        _ptr(swa_pos0, torch.int64, "swa_pos0"), _ptr(q_pos, torch.int64, "q_pos"), scale,
        _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"), _ptr(status, torch.int32, "status"),
        _stream(stream)))


def gather_dequant(cache: PagedCache, ids, out, status=None, stream=None):
    """Decode entries ids [B][n] of `cache` into out [B][n][channels] fp32."""
    B, n = ids.shape
    d = cache.desc()
    _check("csa2_gather_dequant", load().csa2_gather_dequant(
        C.byref(d), cache.cache_dtype, B, n, _ptr(ids, torch.int32, "ids"), _ptr(out, torch.float32, "out"),
        _ptr(status, torch.int32, "status"), _stream(stream)))


class GroupState:
    """Shared state of one cross-layer group: caches, entry counts, the latest
    published top-k, the HSI pool and the indexer workspace."""

    def __init__(self, main: PagedCache, idx: PagedCache, n_entries, max_entries: int, topk, pool, workspace,
                 status):
        self.main, self.idx, self.n_entries, self.max_entries = main, idx, n_entries, max_entries
        self.topk, self.pool, self.workspace, self.status = topk, pool, workspace, status
        self._c = _GroupState(main.desc(), idx.desc(), _ptr(n_entries, torch.int32, "n_entries"), int(max_entries), 0,
                              _ptr(topk, torch.int32, "topk"), _ptr(pool, torch.int32, "pool"),
                              _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
                              _ptr(status, torch.int32, "status"))


def layer(cfg: Cfg, mode: int, state: GroupState, q_pos, q, swa, swa_len, swa_pos0, out, lse=None, q_idx=None,
          head_w=None, x=None, pos0=None, merge_w=None, w_idx=None, scale=None, stream=None):
    """a8: one CSA2 layer in mode MODE_FULL / MODE_REINDEX / MODE_REUSE."""
    B, Tq = q.shape[:2]
    io = _LayerIO(B, Tq, _ptr(q_pos, torch.int64, "q_pos"), x.shape[1] if x is not None else 0, _bf16(x, "x"),
                  _ptr(pos0, torch.int64, "pos0"), _ptr(merge_w, torch.float32, "merge_w"), _bf16(w_idx, "w_idx"),
                  _bf16(q_idx, "q_idx"), _ptr(head_w, torch.float32, "head_w"), _bf16(q, "q"), _swa(cfg, swa),
                  swa.shape[1] if swa is not None else 0, _ptr(swa_len, torch.int32, "swa_len"),
                  _ptr(swa_pos0, torch.int64, "swa_pos0"), 1.0 / math.sqrt(512) if scale is None else float(scale),
                  _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"))
    _check("csa2_layer", load().csa2_layer(C.byref(cfg), int(mode), C.byref(state._c), C.byref(io), _stream(stream)))


class KVCache:
    """Paged keys and values of `batch` sequences with `capacity` tokens each (layout in include/csa2.h).  Pages are
    handed out in `page_order` (a permutation of range(num_pages); identity by default)."""

    def __init__(self, cfg: KVCfg, batch: int, capacity: int, device="cuda", page_order=None, spare_pages: int = 0):
        max_pages = max(1, math.ceil(capacity / PAGE))
        n = batch * max_pages + spare_pages
        order = torch.arange(batch * max_pages) if page_order is None else torch.as_tensor(page_order)
        table = order[: batch * max_pages].reshape(batch, max_pages).to(device=device, dtype=torch.int32).contiguous()
        h, d = cfg.kv_heads, cfg.head_dim
        if cfg.cache_dtype == CACHE_FP4:
            data = [torch.zeros((n, h, PAGE, d // 2), dtype=torch.uint8, device=device) for _ in "kv"]
            scales = [torch.zeros((n, h, PAGE, d // 16), dtype=torch.uint8, device=device) for _ in "kv"]
        else:
            data = [torch.zeros((n, h, d // 8, PAGE, 8), dtype=torch.bfloat16, device=device) for _ in "kv"]
            scales = [None, None]
        self._set(cfg, data[0], data[1], table, scales[0], scales[1])

    @classmethod
    def over(cls, cfg: KVCfg, k_data, v_data, block_table, k_scales=None, v_scales=None) -> "KVCache":
        """A cache over pages that the caller holds: data [pages][kv_heads][64][head_dim / 2] uint8 with scales
        [pages][kv_heads][64][head_dim / 16] uint8 (FP4), or [pages][kv_heads][head_dim / 8][64][8] bf16; block_table
        [batch][max_pages] int32.  `block_table` may be rewritten in place between calls."""
        self = cls.__new__(cls)
        self._set(cfg, k_data, v_data, block_table, k_scales, v_scales)
        return self

    def _set(self, cfg, k_data, v_data, block_table, k_scales, v_scales):
        n, h, d = k_data.shape[0], cfg.kv_heads, cfg.head_dim
        fp4 = cfg.cache_dtype == CACHE_FP4
        if load().csa2_kv_page_bytes(C.byref(cfg), 0) == 0:
            raise ValueError("unsupported KV configuration")
        want = (n, h, PAGE, d // 2) if fp4 else (n, h, d // 8, PAGE, 8)
        parts = [("k_data", k_data, want, torch.uint8 if fp4 else torch.bfloat16),
                 ("v_data", v_data, want, torch.uint8 if fp4 else torch.bfloat16)]
        if fp4:
            parts += [(m, t, (n, h, PAGE, d // 16), torch.uint8) for m, t in (("k_scales", k_scales), ("v_scales", v_scales))]
        elif k_scales is not None or v_scales is not None:
            raise ValueError("a BF16 cache has no scales")
        for name, t, shape, dtype in parts:
            if t is None or tuple(t.shape) != shape:
                raise ValueError("%s must be %s" % (name, list(shape)))
            _ptr(t, dtype, name)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [batch][max_pages]")
        _ptr(block_table, torch.int32, "block_table")
        if len({t.device for t in (k_data, v_data, block_table, *(s for s in (k_scales, v_scales) if s is not None))}) > 1:
            raise ValueError("the pages and the block table must be on one device")
        self.k_data, self.v_data, self.k_scales, self.v_scales = k_data, v_data, k_scales, v_scales
        self.block_table, self.device, self.device_index = block_table, k_data.device, k_data.get_device()
        self.batch, self.max_pages, self.num_pages = block_table.shape[0], block_table.shape[1], n
        self.capacity = self.max_pages * PAGE
        self.layout = (h, d, cfg.cache_dtype)
        self.place = (block_table.data_ptr(), self.batch, self.max_pages, self.device_index)
        self._c = _KVCacheDesc(k_data.data_ptr(), k_scales.data_ptr() if fp4 else None, v_data.data_ptr(),
                               v_scales.data_ptr() if fp4 else None, block_table.data_ptr(), self.max_pages, n)


def rope_table(n: int, rope_dims: int, theta: float = 1e4, device="cuda"):
    """(cos, sin) of positions 0 .. n - 1 for kv_append: [n][rope_dims / 2][2] fp32, angles position *
    theta^(-2i / rope_dims) formed in fp64."""
    half = rope_dims // 2
    freq = float(theta) ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(n, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()


def _kv_rows(t, heads, dim, name, device):
    """Address and row distance of [T][heads][dim] bf16 rows; a row is contiguous, the rows may stand apart."""
    shape, stride = t.shape, t.stride()
    if t.dtype is torch.bfloat16 and t.get_device() == device and len(shape) == 3 and shape[1] == heads and \
            shape[2] == dim and stride[2] == 1 and (stride[1] == dim or heads == 1):
        return t.data_ptr(), (stride[0] if shape[0] > 1 else heads * dim)
    if t.dtype != torch.bfloat16:
        raise TypeError("%s must be torch.bfloat16, got %s" % (name, t.dtype))
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError("%s must be [T][%d][%d], got %s" % (name, heads, dim, list(shape)))
    if t.get_device() != device:
        raise ValueError("%s must be on the cache's device" % name)
    raise ValueError("%s: the channels of a row must be contiguous" % name)


def _kv_ptr(t, dtype, shape, name, device):
    """Address of a contiguous tensor of a given shape on the cache's device."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.get_device() != device:
        raise ValueError("%s must be on the cache's device" % name)
    raise ValueError("%s must be contiguous" % name)


# the address of a device's current stream, without a Stream object around it
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(index, fn, stream, *args):
    """Call fn on `stream`, or on the current stream of a device, with that device current."""
    if index == torch.cuda.current_device():
        return fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    with torch.cuda.device(index):
        return fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)


def _kv_same(cfg, cache):
    if cache.layout != (cfg.kv_heads, cfg.head_dim, cfg.cache_dtype):
        raise ValueError("the cache was made for another configuration")


def kv_append(cfg: KVCfg, k, v, cu, pos0, cache: KVCache, rope=None, q=None, q_out=None, k_out=None, v_out=None,
              status=None, stream=None):
    """New tokens of a ragged batch into the cache: k, v [T][kv_heads][head_dim] bf16 (row i of sequence b at
    cu[b] + i, position pos0[b] + i), keys and queries q [T][n_heads][head_dim] rotated by `rope` [rows][rope_dims / 2]
    [2] fp32.  q_out (which may be q) takes the rotated queries, k_out / v_out the values as stored.  (attend, not
    kv_attend, reads its queries ahead of time: see there before handing it these outputs.)"""
    _kv_append(cfg, k, v, cu, pos0, cache, rope, q, q_out, k_out, v_out, status, stream)


def kv_append_axes(cfg: KVCfg, k, v, cu, pos0, cache: KVCache, axes, axis_of, rope, q=None, q_out=None, k_out=None,
                   v_out=None, status=None, stream=None):
    """kv_append with rotary positions of several axes (images, video): axes [T][n_axes] int32 holds each row's positions
    in `rope`, axis_of the axis of each of the rope_dims / 2 pairs (a sequence of small integers, or bytes).  pos0 gives
    the slots in the cache, as before."""
    _kv_append(cfg, k, v, cu, pos0, cache, rope, q, q_out, k_out, v_out, status, stream, axes,
               axis_of if isinstance(axis_of, bytes) else bytes(list(axis_of)))


def _kv_append(cfg, k, v, cu, pos0, cache, rope, q, q_out, k_out, v_out, status, stream, axes=None, axis_of=None):
    _kv_same(cfg, cache)
    dev, h, d = cache.device_index, cfg.kv_heads, cfg.head_dim
    T, B = k.shape[0], cache.batch
    kp, ks = _kv_rows(k, h, d, "k", dev)
    vp, vs = _kv_rows(v, h, d, "v", dev)
    if v.shape[0] != T:
        raise ValueError("k and v must have the same rows")
    rows = 0 if rope is None else rope.shape[0]
    qp = qs = op = os_ = None
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out are given together")
    if q is not None:
        qp, qs = _kv_rows(q, cfg.n_heads, d, "q", dev)
        op, os_ = _kv_rows(q_out, cfg.n_heads, d, "q_out", dev)
        if q.shape[0] != T or q_out.shape[0] != T:
            raise ValueError("q, q_out and k must have the same rows")
    lib, name, where = _lib or load(), "csa2_kv_append", ()
    if axis_of is not None:
        if len(axis_of) != cfg.rope_dims // 2:
            raise ValueError("axis_of must name the axis of each of %d pairs" % (cfg.rope_dims // 2))
        if axes.dim() != 2:
            raise ValueError("axes must be [T][n_axes]")
        n = axes.shape[1]
        name, where = "csa2_kv_append_axes", (_kv_ptr(axes, torch.int32, (T, n), "axes", dev), n, axis_of)
    _check(name, _on(
        cache.device_index, getattr(lib, name), stream, C.byref(cfg), B, T, qp, qs or 0, kp, ks, vp, vs,
        _kv_ptr(cu, torch.int32, (B + 1,), "cu", dev), _kv_ptr(pos0, torch.int64, (B,), "pos0", dev), *where,
        _kv_ptr(rope, torch.float32, (rows, cfg.rope_dims // 2, 2), "rope", dev), rows,
        C.byref(cache._c), op, os_ or 0, _kv_ptr(k_out, torch.bfloat16, (T, h, d), "k_out", dev),
        _kv_ptr(v_out, torch.bfloat16, (T, h, d), "v_out", dev), _kv_ptr(status, torch.int32, (1,), "status", dev)))


def kv_workspace_bytes(cfg: KVCfg, B: int, T: int, max_q: int, max_kv: int) -> int:
    """Workspace with which kv_attend and kv_cross_attend divide keys of these sizes, and decode them ahead, as they
    would best."""
    return int(load().csa2_kv_workspace_bytes(C.byref(cfg), B, T, max_q, max_kv))


def _kv_attend(name, cfg, q, cu, cache, kv_len, max_q, max_kv, out, lse, scale, workspace, status, stream):
    _kv_same(cfg, cache)
    dev, h, d = cache.device_index, cfg.n_heads, cfg.head_dim
    T, B = q.shape[0], cache.batch
    qp, qs = _kv_rows(q, h, d, "q", dev)
    op, os_ = _kv_rows(out, h, d, "out", dev)
    if out.shape[0] != T:
        raise ValueError("q and out must have the same rows")
    wp, wn = None, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on the cache's device")
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    lib = _lib or load()
    _check("csa2_" + name, _on(
        cache.device_index, lib.csa2_kv_attend if name == "kv_attend" else lib.csa2_kv_cross_attend, stream, C.byref(cfg),
        B, T, qp, qs, _kv_ptr(cu, torch.int32, (B + 1,), "cu", dev), C.byref(cache._c),
        _kv_ptr(kv_len, torch.int32, (B,), "kv_len", dev), int(max_q), int(max_kv), scale, op, os_,
        _kv_ptr(lse, torch.float32, (T, h), "lse", dev), wp if wn else None, wn,
        _kv_ptr(status, torch.int32, (1,), "status", dev)))


def kv_attend(cfg: KVCfg, q, cu, cache: KVCache, kv_len, max_q: int, max_kv: int, out, lse=None, scale=None,
              workspace=None, status=None, stream=None):
    """Causal attention (over cfg.window keys if set) of each sequence's last rows, q [T][n_heads][head_dim] bf16 in a
    ragged batch (row i of sequence b at cu[b] + i), over kv_len [B] int32 cached tokens -> out like q, lse
    [T][n_heads] fp32.  `workspace` (kv_workspace_bytes) lets the keys be divided among more CTAs."""
    _kv_attend("kv_attend", cfg, q, cu, cache, kv_len, max_q, max_kv, out, lse, scale, workspace, status, stream)


def kv_cross_attend(cfg: KVCfg, q, cu, cache: KVCache, kv_len, max_q: int, max_kv: int, out, lse=None, scale=None,
                    workspace=None, status=None, stream=None):
    """kv_attend without a causal mask: every row of sequence b sees all kv_len[b] states of the cache (an encoder's)."""
    _kv_attend("kv_cross_attend", cfg, q, cu, cache, kv_len, max_q, max_kv, out, lse, scale, workspace, status, stream)


def kv_reorder(cfg: KVCfg, caches, beams: int, parents, kv_len, status=None, stream=None):
    """The beams' states in the order of a selection: sequence i of the caches goes on from what sequence parents[i] (of
    its group of `beams`, or -1: from nothing) had.  `caches`: the layers' caches, over one block table, which is permuted
    in place; last pages, written in part, are copied where a beam has several children (rules in include/csa2.h)."""
    if not caches:
        raise ValueError("at least one layer's cache is needed")
    first = caches[0]
    layout, place, n = (cfg.kv_heads, cfg.head_dim, cfg.cache_dtype), first.place, first.batch
    for c in caches:
        if c.layout != layout:
            raise ValueError("the cache was made for another configuration")
        if c.place != place:
            raise ValueError("the layers' caches must share one block table")
    if beams < 1 or n % beams:
        raise ValueError("the caches must hold whole groups of beams")
    dev = first.device_index
    _check("csa2_kv_reorder", _on(
        dev, (_lib or load()).csa2_kv_reorder, stream, C.byref(cfg), len(caches),
        (_KVCacheDesc * len(caches))(*[c._c for c in caches]), n // beams, beams,
        _kv_ptr(parents, torch.int32, (n,), "parents", dev), _kv_ptr(kv_len, torch.int32, (n,), "kv_len", dev),
        _kv_ptr(status, torch.int32, (1,), "status", dev)))


def _plain(t, dtype, shape, name, index):
    """Address of a contiguous tensor of a given shape on a given CUDA device."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s must be on the call's device" % name)
    raise ValueError("%s must be contiguous" % name)


def _rows_of(t, width, name, index):
    """Address and row distance of [T][width] rows on a given CUDA device; a row is contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != width:
        raise ValueError("%s must be [T][%d], got %s" % (name, width, list(shape)))
    if t.get_device() != index or index < 0:
        raise ValueError("%s must be on the call's device" % name)
    if stride[1] != 1 and width > 1:
        raise ValueError("%s: a row must be contiguous" % name)
    return t.data_ptr(), (stride[0] if shape[0] > 1 else -(-width // 8) * 8)


_FLOATS = {torch.bfloat16: 0, torch.float32: 1}


def beam_workspace_bytes(groups: int, beams: int, vocab: int, take: int) -> int:
    """Workspace of beam_select for these sizes."""
    return int(load().csa2_beam_workspace_bytes(groups, beams, vocab, take))


def beam_select(logits, cum, scores, parents, tokens, workspace, done=None, end_token: int = 0, lse=None, status=None,
                stream=None):
    """Best continuations of each group of beams: logits [groups * beams][vocab] (bf16 or fp32; rows may stand apart),
    cum [groups][beams] fp32 -> the best scores [groups][take] fp32 (cum + log-softmax) in order, their parents (sequence
    numbers) and tokens [groups][take] int32.  scores may be cum where take == beams.  done [groups][beams] uint8: a beam that has ended proposes end_token alone
    at its score.  lse [groups * beams] fp32 receives the log-sum-exps."""
    groups, beams = cum.shape
    take, dev, vocab = scores.shape[1], logits.get_device(), logits.shape[1]
    if logits.dtype not in _FLOATS:
        raise TypeError("logits must be bf16 or fp32, got %s" % logits.dtype)
    n = groups * beams
    if logits.shape[0] != n:
        raise ValueError("logits must have %d rows" % n)
    p, stride = _rows_of(logits, vocab, "logits", dev)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the call's device")
    _check("csa2_beam_select", _on(
        dev, (_lib or load()).csa2_beam_select, stream, groups, beams, vocab, take, p, _FLOATS[logits.dtype], stride,
        _plain(cum, torch.float32, (groups, beams), "cum", dev), _plain(done, torch.uint8, (groups, beams), "done", dev),
        int(end_token), _plain(scores, torch.float32, (groups, take), "scores", dev),
        _plain(parents, torch.int32, (groups, take), "parents", dev),
        _plain(tokens, torch.int32, (groups, take), "tokens", dev), _plain(lse, torch.float32, (n,), "lse", dev),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _plain(status, torch.int32, (1,), "status", dev)))


class Fp4Weights:
    """Weights [n][k] in the caches' codec (E2M1, one E4M3 scale per 16 channels), laid out for fp4_linear; a weight is
    alpha * code * scale.  pack and encode take the memory for them on the stream that they are given, or the current one:
    it is that stream's, as any tensor made there."""

    def __init__(self, data, n: int, k: int, alpha: float):
        if data.dtype != torch.uint8:
            raise TypeError("data must be torch.uint8, got %s" % data.dtype)
        if not data.is_contiguous() or data.numel() < self._size(n, k):
            raise ValueError("data must be contiguous and hold weights [%d][%d]" % (n, k))
        self.data, self.n, self.k, self.alpha = data, n, k, float(alpha)
        self.device, self.device_index = data.device, data.get_device()
        self._c = _Fp4Desc(data.data_ptr(), n, k, self.alpha, 0)
        self._ref = C.byref(self._c)

    @staticmethod
    def _size(n, k):
        size = load().csa2_fp4_weight_bytes(n, k)
        if size == 0:
            raise ValueError("unsupported weights [%d][%d]: k must be a multiple of 16" % (n, k))
        return size

    @classmethod
    def _room(cls, n, k, device):
        return torch.empty(cls._size(n, k), dtype=torch.uint8, device=device)

    @classmethod
    def pack(cls, codes, scales, alpha: float = 1.0, status=None, stream=None) -> "Fp4Weights":
        """From codes [n][k / 2] (channel 2i in the low nibble of byte i) and E4M3 scales [n][k / 16], both uint8."""
        n, k, dev = codes.shape[0], 2 * codes.shape[1], codes.get_device()
        if not codes.is_cuda:
            raise ValueError("codes must be a CUDA tensor")
        cp = _plain(codes, torch.uint8, (n, k // 2), "codes", dev)
        sp = _plain(scales, torch.uint8, (n, k // 16), "scales", dev)
        st = _plain(status, torch.int32, (1,), "status", dev)
        with torch.cuda.stream(stream):  # the memory's stream too, which knows what else uses it
            data = cls._room(n, k, codes.device)
            _check("csa2_fp4_pack", _on(dev, load().csa2_fp4_pack, stream, n, k, cp, sp, data.data_ptr(), st))
        return cls(data, n, k, alpha)

    @classmethod
    def encode(cls, w, gain=None, status=None, stream=None) -> "Fp4Weights":
        """From bf16 rows w [n][k], encoded times `gain`; alpha becomes 1 / gain.  Without a gain: the power of two that
        brings the largest weight nearest below the codec's largest value, 448 x 6 (read on the host)."""
        n, k = w.shape
        dev = w.get_device()
        if w.dtype != torch.bfloat16:
            raise TypeError("w must be torch.bfloat16, got %s" % w.dtype)
        p, stride = _rows_of(w, k, "w", dev)
        st = _plain(status, torch.int32, (1,), "status", dev)
        with torch.cuda.stream(stream):
            if gain is None:
                most = float(w.abs().amax()) if w.numel() else 0.0
                gain = 2.0 ** min(126, math.floor(math.log2(448 * 6 / most))) if 0 < most < math.inf else 1.0
            if not 2.0 ** -126 <= abs(gain) <= 2.0 ** 126:
                raise ValueError("gain must be one that fp32 has with its reciprocal, got %r" % gain)
            data = cls._room(n, k, w.device)
            _check("csa2_fp4_encode", _on(dev, load().csa2_fp4_encode, stream, n, k, p, stride, float(gain),
                                          data.data_ptr(), st))
        return cls(data, n, k, 1.0 / gain)


def fp4_linear(x, weights: Fp4Weights, out, bias=None, status=None, stream=None):
    """out [T][n] (bf16 or fp32) = x [T][k] bf16 times the weights' transpose (+ bias [n] bf16).  Rows of x and out may
    stand apart."""
    n, dev = weights.n, weights.device_index
    if x.dtype is not torch.bfloat16:
        raise TypeError("x must be torch.bfloat16, got %s" % x.dtype)
    if out.dtype not in _FLOATS:
        raise TypeError("out must be bf16 or fp32, got %s" % out.dtype)
    xp, xs = _rows_of(x, weights.k, "x", dev)
    op, os_ = _rows_of(out, n, "out", dev)
    T = x.shape[0]
    if out.shape[0] != T:
        raise ValueError("x and out must have the same rows")
    _check("csa2_fp4_linear", _on(
        dev, (_lib or load()).csa2_fp4_linear, stream, weights._ref, T, xp, xs,
        _plain(bias, torch.bfloat16, (n,), "bias", dev), op, _FLOATS[out.dtype], os_,
        _plain(status, torch.int32, (1,), "status", dev)))


class Captured:
    """A sequence of library calls (and the caller's copies) recorded once as
    a CUDA graph and replayed with one launch: the same kernels on the same
    buffers, without the host-side cost of issuing them call by call.  Every
    buffer the calls touch must stay alive and in place; a call's host-side
    arguments (sizes, configs, pointers) are those of the capture."""

    def __init__(self, fn, warmup: int = 1):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(warmup):
                fn()
        torch.cuda.current_stream().wait_stream(s)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            fn()

    def __call__(self):
        self.graph.replay()


def capture(fn, warmup: int = 1) -> Captured:
    """Record ``fn`` (library calls on the current stream) for replay."""
    return Captured(fn, warmup)

