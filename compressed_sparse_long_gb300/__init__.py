"""v4a: one layer of DeepSeek-V4-style hybrid compressed attention on GB300 (sm_103a).

Python binding of ``libv4a.so`` (the C ABI declared in ``include/v4a.h``). The functions
below carry the C names and only marshal arguments: torch tensors become device
pointers, the current torch stream becomes the CUDA stream. Every step of the layer runs
in the library's CUDA kernels; there is no other implementation to fall back to, and
importing this package fails if the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "V4AError", "LayerCfg", "Cache", "library", "layer_cfg", "cache",
    "v4a_compress_insert", "v4a_compress_insert_qnorm", "v4a_index_topk", "v4a_index_topk_workspace_size",
    "v4a_index_scores", "v4a_index_scores_row_stride", "v4a_index_topk_noalloc",
    "v4a_index_topk_noalloc_capacity",
    "v4a_attn_decode", "v4a_attn_prefill", "v4a_attn_workspace_size", "v4a_slot_mapping",
    "v4a_attn_decode_q8", "v4a_attn_q8_workspace_size", "v4a_attn_plan",
    "RopeCfg", "LatentCfg", "rope_cfg", "latent_cfg", "v4a_rope", "v4a_latent_insert",
    "v4a_latent_gather", "v4a_latent_attn", "v4a_latent_attn_workspace_size",
    "v4a_latent_attn_expanded", "v4a_latent_attn_expanded_workspace_size",
    "v4a_latent_attn_window", "v4a_latent_attn_window_workspace_size",
    "PageTableDesc", "Pool", "v4a_pages_workspace_size", "v4a_pages_free", "v4a_pages_grow",
    "v4a_pages_fork", "v4a_pages_copy", "v4a_pages_compact",
    "v4a_get_error", "v4a_version",
    "BF16", "ROPE_INTERLEAVED", "ROPE_HALF", "ROPE_SCALE_NONE", "ROPE_SCALE_LINEAR",
    "ROPE_SCALE_BY_PARTS", "ROPE_SCALE_YARN", "MAX_SEQ", "LATENT_PLAIN", "LATENT_FP4", "MAX_POOLS",
    "DEV_NO_PAGE", "latent_row_bytes",
    "C4A", "C128A", "FP32", "BF16_FP8", "IDX_DEFAULT", "IDX_FP4", "DEV_MISSING_PAGE", "DEV_BAD_PAGE", "DEV_BAD_INDEX", "DEV_BAD_POS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libv4a.so")

C4A, C128A = 0, 1
FP32, BF16_FP8, BF16 = 0, 1, 2
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_BY_PARTS, ROPE_SCALE_YARN = 0, 1, 2, 3
MAX_SEQ, MAX_POOLS = 1024, 64
LATENT_PLAIN, LATENT_FP4 = 0, 1
IDX_DEFAULT, IDX_FP4 = 0, 1
OK, ERR_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE, ERR_TOO_LARGE = 0, -1, -2, -3, -4, -5
DEV_MISSING_PAGE, DEV_BAD_PAGE, DEV_BAD_INDEX, DEV_BAD_POS = 1, 2, 4, 8
DEV_NO_PAGE = 32
_NAMES = {ERR_ARG: "V4A_ERR_ARG", ERR_UNSUPPORTED: "V4A_ERR_UNSUPPORTED",
          ERR_CUDA: "V4A_ERR_CUDA", ERR_DEVICE: "V4A_ERR_DEVICE",
          ERR_TOO_LARGE: "V4A_ERR_TOO_LARGE"}


class V4AError(RuntimeError):
    def __init__(self, fn: str, code: int, flags: int = 0):
        super().__init__("%s returned %s (%d)%s" % (fn, _NAMES.get(code, "?"), code,
                                                    " flags=0x%x" % flags if flags else ""))
        self.code, self.flags = code, flags


class LayerCfg(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("idx_heads", ctypes.c_int32),
                ("idx_dim", ctypes.c_int32), ("window", ctypes.c_int32),
                ("stride", ctypes.c_int32), ("win_off", ctypes.c_int32),
                ("swa", ctypes.c_int32), ("rope_base", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("softmax_scale", ctypes.c_float),
                ("idx_format", ctypes.c_int32)]


class Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int32),
                ("rows_per_block", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("row_width", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class RopeCfg(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("base", ctypes.c_float), ("factor", ctypes.c_float),
                ("orig_max_pos", ctypes.c_float), ("low", ctypes.c_float),
                ("high", ctypes.c_float), ("amplitude", ctypes.c_float)]


class LatentCfg(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("latent_dim", ctypes.c_int32), ("nope_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32), ("cache_format", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("softmax_scale", ctypes.c_float),
                ("rope", RopeCfg)]

    @property
    def reserved(self):
        """cache_format, by the name that the field had before it had a meaning."""
        return self.cache_format

    @reserved.setter
    def reserved(self, value):
        self.cache_format = value


class PageTableDesc(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("n_seq", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("n_pages", ctypes.c_int64)]


class Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("row_bytes", ctypes.c_int64), ("rows_per_block", ctypes.c_int32),
                ("late", ctypes.c_int16), ("reserved", ctypes.c_int16)]


_P = ctypes.c_void_p
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_CFG, _CACHE = ctypes.POINTER(LayerCfg), ctypes.POINTER(Cache)
_ROPE, _LATENT = ctypes.POINTER(RopeCfg), ctypes.POINTER(LatentCfg)
_TABLE, _POOLS = ctypes.POINTER(PageTableDesc), ctypes.POINTER(Pool)

_SIGS = {
    "v4a_version": (_I32, []),
    "v4a_compress_insert": (ctypes.c_int, [_CFG, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                           _CACHE, _CACHE, _CACHE, _CACHE, _P, _P]),
    "v4a_compress_insert_qnorm": (ctypes.c_int, [_CFG, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                                 _P, _P, _CACHE, _CACHE, _CACHE, _CACHE, _I32,
                                                 _P, _P, _P, _P, _P]),
    "v4a_index_topk_workspace_size": (_SZ, [_CFG, _I32, _I64]),
    "v4a_index_topk": (ctypes.c_int, [_CFG, _I32, _P, _P, _I64, _P, _P, _CACHE, _I32, _P, _P,
                                      _SZ, _P, _P]),
    "v4a_attn_workspace_size": (_SZ, [_CFG, _I32, _I64, _I32, _I32]),
    "v4a_attn_plan": (ctypes.c_int, [_CFG, _I32, _I64, _I32, _I32, ctypes.POINTER(_I32),
                                     ctypes.POINTER(_I32)]),
    "v4a_attn_decode": (ctypes.c_int, [_CFG, _I32, _P, _P, _I64, _P, _P, _I32, _CACHE, _CACHE,
                                       _P, _P, _SZ, _P, _P]),
    "v4a_attn_prefill": (ctypes.c_int, [_CFG, _I32, _P, _P, _I64, _P, _P, _I32, _CACHE, _CACHE,
                                        _P, _P, _SZ, _P, _P]),
    "v4a_slot_mapping": (ctypes.c_int, [_CACHE, _I32, _P, _P, _P, _P, _P]),
    "v4a_attn_q8_workspace_size": (_SZ, [_CFG, _I32, _I64, _I32]),
    "v4a_attn_decode_q8": (ctypes.c_int, [_CFG, _I32, _P, _P, _I64, _P, _P, _I32, _CACHE, _CACHE,
                                          _P, _P, _P, _SZ, _P, _P]),
    "v4a_index_scores_row_stride": (_I64, [_CFG, _I64]),
    "v4a_index_scores": (ctypes.c_int, [_CFG, _I32, _P, _P, _I64, _P, _P, _CACHE, _P, _SZ, _P,
                                        _P]),
    "v4a_index_topk_noalloc_capacity": (_SZ, []),
    "v4a_index_topk_noalloc": (ctypes.c_int, [_CFG, _I32, _P, _P, _I64, _P, _P, _CACHE, _I32,
                                              _P, _P, _P]),
    "v4a_rope": (ctypes.c_int, [_ROPE, _I32, _I32, _I32, _P, _P, _I64, _I64, _P, _I64, _I64, _I32,
                                _P, _P]),
    "v4a_latent_insert": (ctypes.c_int, [_LATENT, _I32, _I32, _P, _P, _P, _I64, _P, _I64, _P,
                                         _CACHE, _P, _P]),
    "v4a_latent_gather": (ctypes.c_int, [_LATENT, _I32, _I32, _P, _P, _CACHE, _P, _P, _P]),
    "v4a_latent_attn_workspace_size": (_SZ, [_LATENT, _I32, _I32, _I64]),
    "v4a_latent_attn": (ctypes.c_int, [_LATENT, _I32, _I32, _P, _P, _I64, _P, _CACHE, _P, _P, _SZ,
                                       _P, _P]),
    "v4a_latent_attn_window_workspace_size": (_SZ, [_LATENT, _I32, _I32, _I64, _I64, _I64]),
    "v4a_latent_attn_window": (ctypes.c_int, [_LATENT, _I32, _I32, _P, _P, _I64, _I64, _I64, _P,
                                              _CACHE, _P, _P, _SZ, _P, _P]),
    "v4a_pages_workspace_size": (_SZ, [_TABLE]),
    "v4a_pages_free": (ctypes.c_int, [_TABLE, _P, _P, _P, _P]),
    "v4a_pages_grow": (ctypes.c_int, [_TABLE, _P, _P, _P, _SZ, _P, _P]),
    "v4a_pages_fork": (ctypes.c_int, [_TABLE, _POOLS, _I32, _I32, _P, _P, _P, _P, _SZ, _P, _P]),
    "v4a_pages_copy": (ctypes.c_int, [_TABLE, _POOLS, _I32, _I32, _P, _P, _P, _P]),
    "v4a_pages_compact": (ctypes.c_int, [_TABLE, _POOLS, _I32, _P, _P, _P, _SZ, _P, _P]),
    "v4a_latent_attn_expanded": (ctypes.c_int, [_LATENT, _I32, _I32, _P, _I32, _P, _P, _P, _I64,
                                                _I64, _P, _I64, _P, _I64, _I64, _I32, _P, _P,
                                                _SZ, _P, _P]),
    "v4a_latent_attn_expanded_workspace_size": (_SZ, [_LATENT, _I32, _I32, _I32]),
    "v4a_get_error": (ctypes.c_int, [_P, _P, ctypes.POINTER(_I32)]),
}

_lib = None


def library() -> ctypes.CDLL:
    """Load libv4a.so (built in-tree by ``compressed_sparse_long_gb300.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libv4a.so is not built (%s); run "
                              "`python -m compressed_sparse_long_gb300.build`. There is no "
                              "fallback implementation." % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if t.numel() and not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(fn: str, rc: int):
    if rc != OK:
        raise V4AError(fn, rc)


def layer_cfg(kind: int, dtype: int, head_dim: int, rope_dim: int, n_heads: int,
              idx_heads: int, idx_dim: int, window: int, stride: int, win_off: int = 0,
              swa: int = 128, rope_base: float = 10000.0, rms_eps: float = 1e-6,
              softmax_scale: float | None = None, idx_format: int = 0) -> LayerCfg:
    return LayerCfg(kind, dtype, head_dim, rope_dim, n_heads, idx_heads, idx_dim, window,
                    stride, win_off, swa, rope_base, rms_eps,
                    softmax_scale if softmax_scale else head_dim ** -0.5, idx_format)


def cache(data: torch.Tensor, scale: torch.Tensor | None, block_table: torch.Tensor,
          rows_per_block: int, elems_per_byte: int = 1) -> Cache:
    """Describe a paged pool. The tensors must stay alive while the library uses them.
    elems_per_byte = 2 for a pool of packed fp4 rows (uint8 data, two elements a byte)."""
    assert data.dim() == 2 and block_table.dim() == 2 and block_table.dtype == torch.int32
    return Cache(data.data_ptr(), None if scale is None else scale.data_ptr(),
                 block_table.data_ptr(), block_table.shape[1], rows_per_block,
                 data.shape[0] // rows_per_block, data.shape[1] * elems_per_byte, 0)


def v4a_version() -> int:
    return library().v4a_version()


def v4a_compress_insert(cfg, n_seq, n_tokens, cu_tokens, start_pos, kv, score, bias, gamma,
                        ikv, iscore, ibias, attn, idx, swa, state, dev_err=None, stream=None):
    _check("v4a_compress_insert", library().v4a_compress_insert(
        ctypes.byref(cfg), n_seq, n_tokens, _ptr(cu_tokens), _ptr(start_pos), _ptr(kv),
        _ptr(score), _ptr(bias), _ptr(gamma), _ptr(ikv), _ptr(iscore), _ptr(ibias),
        ctypes.byref(attn), None if idx is None else ctypes.byref(idx), ctypes.byref(swa),
        ctypes.byref(state), _ptr(dev_err), _stream(stream)))


def _cref(c):
    return None if c is None else ctypes.byref(c)


def v4a_compress_insert_qnorm(cfg, n_seq, n_tokens, cu_tokens, start_pos, kv, score, bias,
                              gamma, ikv, iscore, ibias, attn, idx, swa, state, n_q, q, q_gamma,
                              q_out, dev_err=None, stream=None):
    _check("v4a_compress_insert_qnorm", library().v4a_compress_insert_qnorm(
        ctypes.byref(cfg), n_seq, n_tokens, _ptr(cu_tokens), _ptr(start_pos), _ptr(kv),
        _ptr(score), _ptr(bias), _ptr(gamma), _ptr(ikv), _ptr(iscore), _ptr(ibias),
        _cref(attn), _cref(idx), _cref(swa), _cref(state), n_q, _ptr(q), _ptr(q_gamma),
        _ptr(q_out), _ptr(dev_err), _stream(stream)))


def v4a_index_topk_workspace_size(cfg, n_q, max_pos) -> int:
    return library().v4a_index_topk_workspace_size(ctypes.byref(cfg), n_q, max_pos)


def v4a_index_topk(cfg, n_q, q_seq, q_pos, max_pos, q_idx, w, idx, k, topk_out, workspace,
                   dev_err=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("v4a_index_topk", library().v4a_index_topk(
        ctypes.byref(cfg), n_q, _ptr(q_seq), _ptr(q_pos), max_pos, _ptr(q_idx), _ptr(w),
        ctypes.byref(idx), k, _ptr(topk_out), _ptr(workspace), ws_bytes, _ptr(dev_err),
        _stream(stream)))


def v4a_index_scores_row_stride(cfg, max_pos) -> int:
    return library().v4a_index_scores_row_stride(ctypes.byref(cfg), max_pos)


def v4a_index_scores(cfg, n_q, q_seq, q_pos, max_pos, q_idx, w, idx, scores, dev_err=None,
                     stream=None):
    """Indexer score rows alone: scores [n_q, v4a_index_scores_row_stride(cfg, max_pos)] fp32."""
    nb = 0 if scores is None else scores.numel() * scores.element_size()
    _check("v4a_index_scores", library().v4a_index_scores(
        ctypes.byref(cfg), n_q, _ptr(q_seq), _ptr(q_pos), max_pos, _ptr(q_idx), _ptr(w),
        ctypes.byref(idx), _ptr(scores), nb, _ptr(dev_err), _stream(stream)))


def v4a_index_topk_noalloc_capacity() -> int:
    return library().v4a_index_topk_noalloc_capacity()


def v4a_index_topk_noalloc(cfg, n_q, q_seq, q_pos, max_pos, q_idx, w, idx, k, topk_out,
                           dev_err=None, stream=None):
    """v4a_index_topk for callers that cannot provide or allocate a workspace: the scores
    go to the library's fixed device scratch (see include/v4a.h for its limit and rules)."""
    _check("v4a_index_topk_noalloc", library().v4a_index_topk_noalloc(
        ctypes.byref(cfg), n_q, _ptr(q_seq), _ptr(q_pos), max_pos, _ptr(q_idx), _ptr(w),
        ctypes.byref(idx), k, _ptr(topk_out), _ptr(dev_err), _stream(stream)))


def v4a_attn_workspace_size(cfg, n_q, max_pos, k, prefill) -> int:
    return library().v4a_attn_workspace_size(ctypes.byref(cfg), n_q, max_pos, k, int(prefill))


def _attn(name, cfg, n_q, q_seq, q_pos, max_pos, q, topk, k, attn, swa, out, workspace,
          dev_err, stream):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(name, getattr(library(), name)(
        ctypes.byref(cfg), n_q, _ptr(q_seq), _ptr(q_pos), max_pos, _ptr(q), _ptr(topk), k,
        ctypes.byref(attn), ctypes.byref(swa), _ptr(out), _ptr(workspace), ws_bytes,
        _ptr(dev_err), _stream(stream)))


def v4a_attn_decode(cfg, n_q, q_seq, q_pos, max_pos, q, topk, k, attn, swa, out, workspace,
                    dev_err=None, stream=None):
    _attn("v4a_attn_decode", cfg, n_q, q_seq, q_pos, max_pos, q, topk, k, attn, swa, out,
          workspace, dev_err, stream)


def v4a_attn_q8_workspace_size(cfg, n_q, max_pos, k) -> int:
    return library().v4a_attn_q8_workspace_size(ctypes.byref(cfg), n_q, max_pos, k)


def v4a_attn_plan(cfg, n_q, max_pos, k, prefill=False):
    """(key ranges per query, kernels per call) of an attention call of this shape."""
    ns, nk = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("v4a_attn_plan", library().v4a_attn_plan(ctypes.byref(cfg), n_q, max_pos, k,
                                                     int(prefill), ctypes.byref(ns),
                                                     ctypes.byref(nk)))
    return ns.value, nk.value


def v4a_attn_decode_q8(cfg, n_q, q_seq, q_pos, max_pos, q, topk, k, attn, swa, out_codes,
                       out_scale, workspace, dev_err=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("v4a_attn_decode_q8", library().v4a_attn_decode_q8(
        ctypes.byref(cfg), n_q, _ptr(q_seq), _ptr(q_pos), max_pos, _ptr(q), _ptr(topk), k,
        ctypes.byref(attn), ctypes.byref(swa), _ptr(out_codes), _ptr(out_scale), _ptr(workspace),
        ws_bytes, _ptr(dev_err), _stream(stream)))


def v4a_attn_prefill(cfg, n_q, q_seq, q_pos, max_pos, q, topk, k, attn, swa, out, workspace,
                     dev_err=None, stream=None):
    _attn("v4a_attn_prefill", cfg, n_q, q_seq, q_pos, max_pos, q, topk, k, attn, swa, out,
          workspace, dev_err, stream)


def v4a_slot_mapping(c, n, seq, row, slots, dev_err=None, stream=None):
    _check("v4a_slot_mapping", library().v4a_slot_mapping(
        ctypes.byref(c), n, _ptr(seq), _ptr(row), _ptr(slots), _ptr(dev_err), _stream(stream)))


def rope_cfg(dim: int, layout: int = ROPE_INTERLEAVED, base: float = 10000.0,
             scaling: int = ROPE_SCALE_NONE, factor: float = 1.0, orig_max_pos: float = 0.0,
             low: float = 0.0, high: float = 0.0, amplitude: float = 1.0) -> RopeCfg:
    """A rotation of `dim` values a row (see v4a_rope_cfg in include/v4a.h)."""
    return RopeCfg(dim, layout, scaling, 0, base, factor, orig_max_pos, low, high, amplitude)


def latent_cfg(dtype: int, n_heads: int, latent_dim: int, rope: RopeCfg, nope_dim: int = 128,
               v_dim: int = 128, rms_eps: float = 1e-6, softmax_scale: float | None = None,
               cache_format: int = LATENT_PLAIN) -> LatentCfg:
    """A latent-attention layer; the softmax scale defaults to the expanded key's width ^ -1/2.
    cache_format: LATENT_PLAIN, or LATENT_FP4 for a cache in 4 bits (see include/v4a.h)."""
    return LatentCfg(dtype, n_heads, latent_dim, nope_dim, v_dim, cache_format, rms_eps,
                     softmax_scale if softmax_scale else (nope_dim + rope.dim) ** -0.5, rope)


def latent_row_bytes(cfg: LatentCfg) -> int:
    """Bytes of a row of the layer's pool (an FP4 row's scale besides)."""
    if cfg.cache_format == LATENT_FP4:
        return -(-(cfg.latent_dim // 2 + 2 * cfg.rope.dim + cfg.latent_dim // 16) // 16) * 16
    return (cfg.latent_dim + cfg.rope.dim) * (2 if cfg.dtype == BF16 else 4)


def v4a_rope(rope, dtype, n_tokens, n_heads, pos, x, x_token_stride, x_head_stride, y,
             y_token_stride, y_head_stride, inverse=False, dev_err=None, stream=None):
    _check("v4a_rope", library().v4a_rope(
        ctypes.byref(rope), dtype, n_tokens, n_heads, _ptr(pos), _ptr(x), x_token_stride,
        x_head_stride, _ptr(y), y_token_stride, y_head_stride, int(inverse), _ptr(dev_err),
        _stream(stream)))


def v4a_latent_insert(cfg, n_seq, n_tokens, cu_tokens, start_pos, c, c_stride, k_pe, k_stride,
                      gamma, cache, dev_err=None, stream=None):
    _check("v4a_latent_insert", library().v4a_latent_insert(
        ctypes.byref(cfg), n_seq, n_tokens, _ptr(cu_tokens), _ptr(start_pos), _ptr(c), c_stride,
        _ptr(k_pe), k_stride, _ptr(gamma), ctypes.byref(cache), _ptr(dev_err), _stream(stream)))


def v4a_latent_gather(cfg, n_seq, n_rows, cu_rows, start_pos, cache, out, dev_err=None,
                      stream=None):
    _check("v4a_latent_gather", library().v4a_latent_gather(
        ctypes.byref(cfg), n_seq, n_rows, _ptr(cu_rows), _ptr(start_pos), ctypes.byref(cache),
        _ptr(out), _ptr(dev_err), _stream(stream)))


def v4a_latent_attn_workspace_size(cfg, n_seq, n_tokens, max_pos) -> int:
    return library().v4a_latent_attn_workspace_size(ctypes.byref(cfg), n_seq, n_tokens, max_pos)


def v4a_latent_attn(cfg, n_seq, n_tokens, cu_tokens, start_pos, max_pos, q, cache, out, workspace,
                    dev_err=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("v4a_latent_attn", library().v4a_latent_attn(
        ctypes.byref(cfg), n_seq, n_tokens, _ptr(cu_tokens), _ptr(start_pos), max_pos, _ptr(q),
        ctypes.byref(cache), _ptr(out), _ptr(workspace), ws_bytes, _ptr(dev_err),
        _stream(stream)))


def v4a_latent_attn_window_workspace_size(cfg, n_seq, n_tokens, max_pos, window, sinks) -> int:
    return library().v4a_latent_attn_window_workspace_size(ctypes.byref(cfg), n_seq, n_tokens,
                                                           max_pos, window, sinks)


def v4a_latent_attn_window(cfg, n_seq, n_tokens, cu_tokens, start_pos, max_pos, window, sinks, q,
                           cache, out, workspace, dev_err=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("v4a_latent_attn_window", library().v4a_latent_attn_window(
        ctypes.byref(cfg), n_seq, n_tokens, _ptr(cu_tokens), _ptr(start_pos), max_pos, window,
        sinks, _ptr(q), ctypes.byref(cache), _ptr(out), _ptr(workspace), ws_bytes, _ptr(dev_err),
        _stream(stream)))


def v4a_latent_attn_expanded(cfg, n_seq, n_q, cu_q, n_k, cu_k, q, k, k_token_stride,
                             k_head_stride, k_pe, k_pe_stride, v, v_token_stride, v_head_stride,
                             causal, out, workspace, dev_err=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("v4a_latent_attn_expanded", library().v4a_latent_attn_expanded(
        ctypes.byref(cfg), n_seq, n_q, _ptr(cu_q), n_k, _ptr(cu_k), _ptr(q), _ptr(k),
        k_token_stride, k_head_stride, _ptr(k_pe), k_pe_stride, _ptr(v), v_token_stride,
        v_head_stride, int(causal), _ptr(out), _ptr(workspace), ws_bytes, _ptr(dev_err),
        _stream(stream)))


def v4a_latent_attn_expanded_workspace_size(cfg, n_seq, n_q, n_k) -> int:
    return library().v4a_latent_attn_expanded_workspace_size(ctypes.byref(cfg), n_seq, n_q, n_k)


def _pools(pools):
    return (Pool * len(pools))(*pools) if pools else None


def _bytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def v4a_pages_workspace_size(table) -> int:
    return library().v4a_pages_workspace_size(ctypes.byref(table))


def v4a_pages_free(table, first, last, dev_err=None, stream=None):
    _check("v4a_pages_free", library().v4a_pages_free(
        ctypes.byref(table), _ptr(first), _ptr(last), _ptr(dev_err), _stream(stream)))


def v4a_pages_grow(table, first, last, workspace, dev_err=None, stream=None):
    _check("v4a_pages_grow", library().v4a_pages_grow(
        ctypes.byref(table), _ptr(first), _ptr(last), _ptr(workspace), _bytes(workspace),
        _ptr(dev_err), _stream(stream)))


def v4a_pages_fork(table, pools, n, src, dst, length, workspace, dev_err=None, stream=None):
    """pools: a sequence of Pool."""
    _check("v4a_pages_fork", library().v4a_pages_fork(
        ctypes.byref(table), _pools(pools), len(pools), n, _ptr(src), _ptr(dst), _ptr(length),
        _ptr(workspace), _bytes(workspace), _ptr(dev_err), _stream(stream)))


def v4a_pages_copy(table, pools, n, src, dst, dev_err=None, stream=None):
    _check("v4a_pages_copy", library().v4a_pages_copy(
        ctypes.byref(table), _pools(pools), len(pools), n, _ptr(src), _ptr(dst), _ptr(dev_err),
        _stream(stream)))


def v4a_pages_compact(table, pools, n_used, moved, workspace, dev_err=None, stream=None):
    _check("v4a_pages_compact", library().v4a_pages_compact(
        ctypes.byref(table), _pools(pools), len(pools), _ptr(n_used), _ptr(moved),
        _ptr(workspace), _bytes(workspace), _ptr(dev_err), _stream(stream)))


def v4a_get_error(dev_err, stream=None) -> int:
    """Synchronise the stream, return and clear the device error bits."""
    flags = _I32(0)
    rc = library().v4a_get_error(_ptr(dev_err), _stream(stream), ctypes.byref(flags))
    if rc not in (OK, ERR_DEVICE):
        raise V4AError("v4a_get_error", rc)
    return flags.value
