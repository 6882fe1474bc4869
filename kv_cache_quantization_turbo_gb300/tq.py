"""ctypes binding of libtq.so (include/tq.h): argument marshalling only.

Every function keeps the C name.  Device buffers are passed as torch tensors
(their data_ptr()) or raw integer addresses; streams as torch.cuda.Stream or
raw handles.  The compute runs in the library's CUDA kernels; importing this
module without the built library raises, there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtq.so")

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_WORKSPACE, TQ_ERR_CUDA, TQ_ERR_OOM = range(6)

FORMATS = {
    "turbo2": 0, "turbo3": 1, "turbo4": 2,
    "turbo2_mse": 3, "turbo3_mse": 4, "turbo4_mse": 5,
    "q8_0": 6, "minmax": 7,
}

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with kv_cache_quantization_turbo_gb300.build.build()")
_lib = ctypes.CDLL(LIB_PATH)


class tq_cache_view(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("n_layers", ctypes.c_int32),
        ("bits", ctypes.c_int32), ("payload", ctypes.c_void_p), ("header", ctypes.c_void_p),
    ]


class tq_rope_params(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("scaling", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
        ("original_ctx", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
        ("attn_factor", ctypes.c_double),
    ]


class tq_rope_table(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("attn_factor", ctypes.c_float), ("turns", ctypes.c_uint64 * 128),
    ]


class tq_batch(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
        ("max_ctx", ctypes.c_int32), ("max_blocks", ctypes.c_int32), ("cu_tokens", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
    ]


class tq_score_mods(ctypes.Structure):
    _fields_ = [
        ("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("slopes", ctypes.c_void_p),
        ("first_keys", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p),
    ]


_P = ctypes.c_void_p
_I = ctypes.c_int
_U32 = ctypes.c_uint32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_VP = ctypes.POINTER(tq_cache_view)

_SIGS = {
    "tq_status_string": (ctypes.c_char_p, [_I]),
    "tq_format_name": (ctypes.c_char_p, [_I]),
    "tq_payload_bytes": (_SZ, [_I, _I, _I]),
    "tq_header_bytes": (_SZ, [_I, _I, _I]),
    "tq_vector_bytes": (_SZ, [_I, _I, _I]),
    "tq_codebook_build": (_I, [_I, _I, _P, _P]),
    "tq_signs_generate": (_I, [_U32, _I, _P]),
    "tq_qjl_matrix_generate": (_I, [_U32, _I, _P]),
    "tq_context_create": (_I, [_I, _U32, _U32, _P, _P, ctypes.POINTER(_P)]),
    "tq_context_destroy": (_I, [_P]),
    "tq_context_get_tables": (_I, [_P, _P, _P, _P, _P]),
    "tq_get_status": (_I, [_P, ctypes.POINTER(_U32)]),
    "tq_encode_kv": (_I, [_P, _VP, _P, _VP, _P, _I, _I, _I, _I64, _I64, _P, _I64, _P]),
    "tq_decode_workspace_bytes": (_SZ, [_P, _I, _I, _I, _I]),
    "tq_decode_attention": (_I, [_P, _P, _I, _I, _I, _I, _VP, _VP, _I, _P, _I, _P, _I, _F, _F, _P, _SZ,
                                 _P, _P]),
    "tq_dequantize": (_I, [_P, _VP, _I, _P, _I64, _I, _I, _P, _P]),
    "tq_decode_attention_static": (_I, [_P, _P, _I, _I, _I, _I, _VP, _VP, _I, _P, _I, _P, _I, _F, _F, _P, _P]),
    "tq_encode_kv_layers": (_I, [_P, _VP, _P, _VP, _P, _I, _P, _P, _I, _I64, _I64, _P, _I64, _P]),
    "tq_decode_attention_layers": (_I, [_P, _P, _I, _I, _I, _I, _VP, _P, _VP, _P, _P, _I, _P, _I, _F, _F, _P, _SZ,
                                        _P, _P]),
    "tq_prefill_workspace_bytes": (_SZ, [_P, _I, _I]),
    "tq_prefill_attention": (_I, [_P, _P, _I, _I, _I, _VP, _VP, _I, _I, _P, _I, _I, _F, _P, _SZ, _P, _P]),
    "tq_rope_build": (_I, [ctypes.POINTER(tq_rope_params), ctypes.POINTER(tq_rope_table)]),
    "tq_rope": (_I, [_P, ctypes.POINTER(tq_rope_table), _P, _I, _I, _I, _I64, _P, _I, _P, _I64, _P]),
    "tq_append_kv": (_I, [_P, ctypes.POINTER(tq_batch), _P, _I64, _P, _I64, _I, ctypes.POINTER(tq_rope_table), _P,
                          _VP, _VP, _I, _P]),
    "tq_read_kv": (_I, [_P, ctypes.POINTER(tq_batch), _VP, _P, _VP, _P, _I, _I, _P]),
    "tq_chunk_workspace_bytes": (_SZ, [_P, ctypes.POINTER(tq_batch), _I, _I]),
    "tq_chunk_attention": (_I, [_P, ctypes.POINTER(tq_batch), _P, _I, _I64, _I, _VP, _VP, _I, _F,
                                ctypes.POINTER(tq_score_mods), _P, _SZ, _P, _I, _P]),
    "tq_context_tables_hash": (_I, [_P, ctypes.POINTER(ctypes.c_uint64)]),
    "tq_cache_save": (_I, [_P, _VP, _I, ctypes.c_char_p]),
    "tq_cache_file_info": (_I, [ctypes.c_char_p, _VP, ctypes.POINTER(ctypes.c_uint64)]),
    "tq_cache_load": (_I, [_P, _VP, _I, ctypes.c_char_p]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class TQError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {tq_status_string(status)} ({status})")
        self.status = status


def _check(status: int, what: str) -> int:
    if status != TQ_OK:
        raise TQError(status, what)
    return status


def _ptr(x) -> int | None:
    """Device/host address of a tensor, an ndarray, an int, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError(type(x))


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _fmt(f) -> int:
    return FORMATS[f] if isinstance(f, str) else int(f)


# ---- pure host functions ----

def tq_status_string(status: int) -> str:
    return _lib.tq_status_string(status).decode()


def tq_format_name(fmt) -> str:
    return _lib.tq_format_name(_fmt(fmt)).decode()


def tq_payload_bytes(fmt, head_dim: int, bits: int = 0) -> int:
    return _lib.tq_payload_bytes(_fmt(fmt), head_dim, bits)


def tq_header_bytes(fmt, head_dim: int, bits: int = 0) -> int:
    return _lib.tq_header_bytes(_fmt(fmt), head_dim, bits)


def tq_vector_bytes(fmt, head_dim: int, bits: int = 0) -> int:
    return _lib.tq_vector_bytes(_fmt(fmt), head_dim, bits)


def tq_codebook_build(bits: int, head_dim: int):
    """Returns (centroids, boundaries) as numpy float32 arrays."""
    import numpy as np

    c = np.zeros(1 << bits, np.float32)
    b = np.zeros(max((1 << bits) - 1, 1), np.float32)
    _check(_lib.tq_codebook_build(bits, head_dim, c.ctypes.data, b.ctypes.data), "tq_codebook_build")
    return c, b[: (1 << bits) - 1]


def tq_signs_generate(seed: int, head_dim: int):
    import numpy as np

    s = np.zeros(head_dim, np.int8)
    _check(_lib.tq_signs_generate(seed, head_dim, s.ctypes.data), "tq_signs_generate")
    return s


def tq_qjl_matrix_generate(seed: int, head_dim: int):
    import numpy as np

    S = np.zeros((head_dim, head_dim), np.float32)
    _check(_lib.tq_qjl_matrix_generate(seed, head_dim, S.ctypes.data), "tq_qjl_matrix_generate")
    return S


# ---- context ----

def tq_context_create(head_dim: int, wht_seed: int = 1, qjl_seed: int = 2, signs=None, qjl=None) -> int:
    """Returns the context handle (an integer).  signs/qjl: host numpy arrays or None."""
    import numpy as np

    out = _P()
    s = None if signs is None else np.ascontiguousarray(signs, dtype=np.int8)
    S = None if qjl is None else np.ascontiguousarray(qjl, dtype=np.float32)
    _check(_lib.tq_context_create(head_dim, wht_seed, qjl_seed, _ptr(s), _ptr(S), ctypes.byref(out)),
           "tq_context_create")
    return out.value


def tq_context_destroy(ctx: int) -> None:
    _check(_lib.tq_context_destroy(ctx), "tq_context_destroy")


def tq_context_get_tables(ctx: int, head_dim: int):
    """Returns (signs int8 [d], S float32 [d, d], centroids [3, 8], boundaries [3, 7])."""
    import numpy as np

    s = np.zeros(head_dim, np.int8)
    S = np.zeros((head_dim, head_dim), np.float32)
    c = np.zeros((3, 8), np.float32)
    b = np.zeros((3, 7), np.float32)
    _check(_lib.tq_context_get_tables(ctx, s.ctypes.data, S.ctypes.data, c.ctypes.data, b.ctypes.data),
           "tq_context_get_tables")
    return s, S, c, b


def tq_get_status(ctx: int) -> tuple[int, int]:
    """Returns (status, flags); synchronises the device."""
    f = _U32(0)
    st = _lib.tq_get_status(ctx, ctypes.byref(f))
    return st, f.value


# ---- views ----

@dataclass
class CacheView:
    """A cache view plus the torch tensors that own its memory."""
    fmt: str
    head_dim: int
    n_kv_heads: int
    page_size: int
    num_pages: int
    n_layers: int
    payload: object
    header: object
    bits: int = 0

    def c_view(self) -> tq_cache_view:
        return tq_cache_view(_fmt(self.fmt), self.head_dim, self.n_kv_heads, self.page_size, self.num_pages,
                             self.n_layers, self.bits, _ptr(self.payload), _ptr(self.header))

    @property
    def compressed_bytes_per_vector(self) -> int:
        return tq_vector_bytes(self.fmt, self.head_dim, self.bits)


def alloc_view(fmt, head_dim: int, n_kv_heads: int, page_size: int, num_pages: int, n_layers: int = 1,
               bits: int = 0, device="cuda") -> CacheView:
    """Allocates a zeroed view's payload and header with torch (the caller owns them)."""
    import torch

    n = n_layers * num_pages * n_kv_heads * page_size
    pb, hb = tq_payload_bytes(fmt, head_dim, bits), tq_header_bytes(fmt, head_dim, bits)
    if pb == 0:
        raise ValueError(f"unsupported view: {fmt} d={head_dim} bits={bits}")
    payload = torch.zeros(n * pb, dtype=torch.uint8, device=device)
    header = torch.zeros(n * hb, dtype=torch.uint8, device=device)
    return CacheView(fmt if isinstance(fmt, str) else tq_format_name(fmt), head_dim, n_kv_heads, page_size,
                     num_pages, n_layers, payload, header, bits)


def _view_arg(v):
    if v is None:
        return None
    cv = v.c_view() if isinstance(v, CacheView) else v
    return ctypes.byref(cv), cv


# ---- device entry points ----

def tq_encode_kv(ctx: int, k_view, k, v_view, v, layer_begin: int, n_layers: int, n_tokens: int,
                 in_layer_stride: int, in_token_stride: int, slots=None, slot_begin: int = 0,
                 stream=None) -> int:
    ka, va = _view_arg(k_view), _view_arg(v_view)
    return _lib.tq_encode_kv(ctx, ka[0] if ka else None, _ptr(k), va[0] if va else None, _ptr(v), layer_begin,
                             n_layers, n_tokens, in_layer_stride, in_token_stride, _ptr(slots), slot_begin,
                             _stream(stream))


def tq_decode_workspace_bytes(ctx: int, n_layers: int, batch: int, n_q_heads: int, max_ctx: int) -> int:
    return _lib.tq_decode_workspace_bytes(ctx, n_layers, batch, n_q_heads, max_ctx)


def tq_decode_attention(ctx: int, q, q_is_fp16: int, n_layers: int, batch: int, n_q_heads: int, k_view, v_view,
                        layer_begin: int, seq_lens, max_ctx: int, block_table, max_blocks_per_seq: int,
                        softmax_scale: float, skip_threshold: float, workspace, workspace_bytes: int, out,
                        stream=None) -> int:
    ka, va = _view_arg(k_view), _view_arg(v_view)
    return _lib.tq_decode_attention(ctx, _ptr(q), q_is_fp16, n_layers, batch, n_q_heads, ka[0], va[0], layer_begin,
                                    _ptr(seq_lens), max_ctx, _ptr(block_table), max_blocks_per_seq,
                                    softmax_scale, skip_threshold, _ptr(workspace), workspace_bytes, _ptr(out),
                                    _stream(stream))


def tq_decode_attention_static(ctx: int, q, q_is_fp16: int, n_layers: int, batch: int, n_q_heads: int, k_view,
                               v_view, layer_begin: int, seq_lens, max_ctx: int, block_table,
                               max_blocks_per_seq: int, softmax_scale: float, skip_threshold: float, out,
                               stream=None) -> int:
    ka, va = _view_arg(k_view), _view_arg(v_view)
    return _lib.tq_decode_attention_static(ctx, _ptr(q), q_is_fp16, n_layers, batch, n_q_heads, ka[0], va[0],
                                           layer_begin, _ptr(seq_lens), max_ctx, _ptr(block_table),
                                           max_blocks_per_seq, softmax_scale, skip_threshold, _ptr(out),
                                           _stream(stream))


def tq_dequantize(ctx: int, view, layer: int, slots, slot_begin: int, n: int, include_qjl: int, out,
                  stream=None) -> int:
    va = _view_arg(view)
    return _lib.tq_dequantize(ctx, va[0], layer, _ptr(slots), slot_begin, n, include_qjl, _ptr(out),
                              _stream(stream))


# ---- persistence ----

def _host_view(v) -> tuple:
    """(c view, host_memory flag) for a CacheView over torch tensors or numpy arrays."""
    cv = v.c_view() if isinstance(v, CacheView) else v
    host = 1
    if isinstance(v, CacheView) and hasattr(v.payload, "is_cuda") and v.payload.is_cuda:
        host = 0
    return cv, host


def tq_context_tables_hash(ctx: int) -> int:
    h = ctypes.c_uint64(0)
    _check(_lib.tq_context_tables_hash(ctx, ctypes.byref(h)), "tq_context_tables_hash")
    return h.value


def tq_cache_save(ctx, view, path: str) -> int:
    """Saves a view (device tensors or host arrays); ctx may be None.  Returns the status."""
    cv, host = _host_view(view)
    return _lib.tq_cache_save(ctx, ctypes.byref(cv), host, os.fsencode(path))


def tq_cache_file_info(path: str):
    """Returns (status, geometry dict, tables_hash)."""
    cv = tq_cache_view()
    h = ctypes.c_uint64(0)
    st = _lib.tq_cache_file_info(os.fsencode(path), ctypes.byref(cv), ctypes.byref(h))
    geo = {k: getattr(cv, k) for k in ("format", "head_dim", "n_kv_heads", "page_size", "num_pages", "n_layers",
                                       "bits")}
    return st, geo, h.value


def tq_cache_load(ctx, view, path: str) -> int:
    """Loads a file into a view of the same geometry (device tensors or host arrays); ctx may be None."""
    cv, host = _host_view(view)
    return _lib.tq_cache_load(ctx, ctypes.byref(cv), host, os.fsencode(path))


# ---- per-layer views ----

def _view_array(views):
    """(ctypes array of tq_cache_view, keep-alive) for a list of CacheView, or (None, None)."""
    if views is None:
        return None, None
    arr = (tq_cache_view * len(views))(*[v.c_view() if isinstance(v, CacheView) else v for v in views])
    return arr, arr


def _layer_array(layers):
    if layers is None:
        return None
    return (ctypes.c_int32 * len(layers))(*[int(x) for x in layers])


def tq_encode_kv_layers(ctx: int, k_views, k_view_layers, v_views, v_view_layers, n_layers: int, k, v,
                        n_tokens: int, in_layer_stride: int, in_token_stride: int, slots=None, slot_begin: int = 0,
                        stream=None) -> int:
    """k_views / v_views: lists of n_layers CacheView (or None); *_view_layers: lists of ints."""
    ka, kkeep = _view_array(k_views)
    va, vkeep = _view_array(v_views)
    kl, vl = _layer_array(k_view_layers), _layer_array(v_view_layers)
    return _lib.tq_encode_kv_layers(ctx, ka, kl, va, vl, n_layers, _ptr(k), _ptr(v), n_tokens, in_layer_stride,
                                    in_token_stride, _ptr(slots), slot_begin, _stream(stream))


def tq_decode_attention_layers(ctx: int, q, q_is_fp16: int, n_layers: int, batch: int, n_q_heads: int, k_views,
                               k_view_layers, v_views, v_view_layers, seq_lens, max_ctx: int, block_table,
                               max_blocks_per_seq: int, softmax_scale: float, skip_threshold: float, workspace,
                               workspace_bytes: int, out, stream=None) -> int:
    ka, kkeep = _view_array(k_views)
    va, vkeep = _view_array(v_views)
    return _lib.tq_decode_attention_layers(ctx, _ptr(q), q_is_fp16, n_layers, batch, n_q_heads, ka,
                                           _layer_array(k_view_layers), va, _layer_array(v_view_layers),
                                           _ptr(seq_lens), max_ctx, _ptr(block_table), max_blocks_per_seq,
                                           softmax_scale, skip_threshold, _ptr(workspace), workspace_bytes, _ptr(out),
                                           _stream(stream))


# ---- chunked-prefill attention ----

def tq_prefill_workspace_bytes(ctx: int, n_tokens: int, n_q_heads: int) -> int:
    return _lib.tq_prefill_workspace_bytes(ctx, n_tokens, n_q_heads)


def tq_prefill_attention(ctx: int, q, q_is_fp16: int, n_tokens: int, n_q_heads: int, k_view, v_view, layer: int,
                         seq: int, block_table, max_blocks: int, start: int, softmax_scale: float, workspace,
                         workspace_bytes: int, out, stream=None) -> int:
    ka, va = _view_arg(k_view), _view_arg(v_view)
    return _lib.tq_prefill_attention(ctx, _ptr(q), q_is_fp16, n_tokens, n_q_heads, ka[0], va[0], layer, seq,
                                     _ptr(block_table), max_blocks, start, softmax_scale, _ptr(workspace),
                                     workspace_bytes, _ptr(out), _stream(stream))


# ---- one serving step: rotate, append, attend a ragged batch ----

DTYPES = {"float32": 0, "float16": 1, "bfloat16": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "wavelength": 3, "yarn": 4}


_DTYPE_OF: dict = {}  # torch dtype -> element type, filled as types come up


def _dtype(t) -> int:
    """The library's element type of a tensor; -1 (refused by every call) for any other."""
    d = t.dtype
    code = _DTYPE_OF.get(d)
    if code is None:
        code = _DTYPE_OF[d] = DTYPES.get(_short(t), -1)
    return code


def _rows(t, shape, heads: int | None = None) -> int:
    """Token stride of a [tokens, heads, d] tensor on a GPU whose heads are consecutive d-vectors; shape: t.shape."""
    if not t.is_cuda:
        raise ValueError(f"a tensor on the GPU is wanted, not on {t.device}")
    if len(shape) != 3 or (heads is not None and shape[1] != heads):
        raise ValueError(f"a [tokens, {'heads' if heads is None else heads}, d] tensor is wanted: {tuple(shape)}")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 or (h > 1 and s1 != d)) and n * h * d:
        raise ValueError(f"heads have to be consecutive vectors: {tuple(shape)}, strides {t.stride()}")
    return s0 if n > 1 else h * d


@dataclass(frozen=True, eq=False)
class Batch:
    """A ragged batch (tq_batch) and the device tensors that own its arrays (int32): cu_tokens [n_seqs + 1],
    seq_lens [n_seqs], block_table [n_seqs, max_blocks] or None.  The tensors' contents may change between calls, the
    fields not."""
    cu_tokens: object
    seq_lens: object
    block_table: object
    n_tokens: int
    max_tokens: int
    max_ctx: int

    def __post_init__(self):
        n = self.seq_lens.numel()
        if self.cu_tokens.numel() != n + 1:
            raise ValueError(f"cu_tokens has {self.cu_tokens.numel()} entries for {n} sequences")
        bt = self.block_table
        if bt is not None and (bt.dim() != 2 or bt.shape[0] != n or (n and not bt.shape[1])):
            raise ValueError(f"block_table {tuple(bt.shape)} for {n} sequences")
        for t in (self.cu_tokens, self.seq_lens, bt):
            if t is not None and (_short(t) != "int32" or not t.is_contiguous() or not t.is_cuda):
                raise ValueError("the batch's arrays are contiguous int32 tensors on the GPU")
        object.__setattr__(self, "_c", tq_batch(n, self.n_tokens, self.max_tokens, self.max_ctx,
                                                0 if bt is None else bt.shape[1], _ptr(self.cu_tokens),
                                                _ptr(self.seq_lens), _ptr(bt)))

    def c_batch(self) -> tq_batch:
        return self._c


@dataclass(frozen=True, eq=False)
class ScoreMods:
    """Changes to the scores (tq_score_mods) and the device tensors they read: slopes float32 [n_q_heads],
    first_keys int32 [n_tokens], prefix_lens int32 [n_seqs], each None for none; contents may change between calls."""
    softcap: float = 0.0
    window: int = 0
    slopes: object = None
    first_keys: object = None
    prefix_lens: object = None

    def __post_init__(self):
        for t, want in ((self.slopes, "float32"), (self.first_keys, "int32"), (self.prefix_lens, "int32")):
            if t is not None and (_short(t) != want or not t.is_contiguous() or not t.is_cuda):
                raise ValueError(f"a contiguous {want} tensor on the GPU is wanted: {t.dtype}, strides {t.stride()}, "
                                 f"{t.device}")
        object.__setattr__(self, "_c", tq_score_mods(self.softcap, self.window, _ptr(self.slopes),
                                                     _ptr(self.first_keys), _ptr(self.prefix_lens)))

    def c_mods(self) -> tq_score_mods:
        return self._c


_NAME_OF: dict = {}  # torch dtype -> its name


def _short(t) -> str:
    d = t.dtype
    name = _NAME_OF.get(d)
    if name is None:
        name = _NAME_OF[d] = str(d).rsplit(".", 1)[-1]
    return name


def _positions(positions, n: int):
    if positions is None:
        return None
    if _short(positions) != "int32" or positions.numel() != n or not positions.is_contiguous() or \
            not positions.is_cuda:
        raise ValueError(f"positions: {n} contiguous int32 values on the GPU are wanted")
    return positions.data_ptr()


def tq_rope_build(head_dim: int, rotary_dim: int | None = None, layout="half", scaling="none", base: float = 10000.0,
                  factor: float = 1.0, original_ctx: float = 0.0, low: float = 0.0, high: float = 0.0,
                  attn_factor: float = 0.0) -> tq_rope_table:
    """The rotation's table (a host structure that later calls take by value)."""
    p = tq_rope_params(head_dim, head_dim if rotary_dim is None else rotary_dim,
                       ROPE_LAYOUTS[layout] if isinstance(layout, str) else layout,
                       ROPE_SCALINGS[scaling] if isinstance(scaling, str) else scaling, base, factor, original_ctx,
                       low, high, attn_factor)
    t = tq_rope_table()
    _check(_lib.tq_rope_build(ctypes.byref(p), ctypes.byref(t)), "tq_rope_build")
    return t


def tq_rope(ctx: int, table: tq_rope_table, x, positions, out, inverse: bool = False, stream=None) -> int:
    """x, out: [tokens, heads, d] tensors of one type (out may be x); positions: int32 [tokens]."""
    shape = x.shape
    if len(shape) != 3 or out.shape != shape or out.dtype != x.dtype or shape[-1] != table.head_dim:
        raise ValueError(f"x {tuple(shape)} {x.dtype}, out {tuple(out.shape)} {out.dtype}")
    return _lib.tq_rope(ctx, ctypes.byref(table), x.data_ptr(), _dtype(x), shape[0], shape[1], _rows(x, shape),
                        _positions(positions, shape[0]), int(inverse), out.data_ptr(), _rows(out, shape),
                        _stream(stream))


def tq_append_kv(ctx: int, batch: Batch, k, v, k_view, v_view, layer: int, rope: tq_rope_table | None = None,
                 positions=None, stream=None) -> int:
    """k, v: [n_tokens, H, d] tensors of one type (slices of a fused projection are fine)."""
    shape = k.shape
    if k.dtype != v.dtype or shape != v.shape or shape[0] != batch.n_tokens or shape[-1] != k_view.head_dim:
        raise ValueError(f"k {tuple(shape)} {k.dtype}, v {tuple(v.shape)} {v.dtype}, {batch.n_tokens} tokens")
    ka, va = _view_arg(k_view), _view_arg(v_view)
    return _lib.tq_append_kv(ctx, ctypes.byref(batch.c_batch()), k.data_ptr(), _rows(k, shape, k_view.n_kv_heads),
                             v.data_ptr(), _rows(v, shape, v_view.n_kv_heads), _dtype(k),
                             None if rope is None else ctypes.byref(rope), _positions(positions, batch.n_tokens),
                             ka[0], va[0], layer, _stream(stream))


def tq_read_kv(ctx: int, batch: Batch, k_view, k_out, v_view, v_out, layer: int, stream=None) -> int:
    """k_out, v_out: contiguous [n_tokens, H, d] tensors of one type; a pair may be None."""
    outs = [(view, t) for view, t in ((k_view, k_out), (v_view, v_out)) if t is not None]
    for view, t in outs:
        if view is None:
            raise ValueError("an output without the view it is read from")
        if t.shape != (batch.n_tokens, view.n_kv_heads, view.head_dim) or not t.is_contiguous() or not t.is_cuda or \
                t.dtype != outs[0][1].dtype:
            raise ValueError(f"output {tuple(t.shape)} {t.dtype} for {batch.n_tokens} tokens")
    ka, va = _view_arg(k_view), _view_arg(v_view)
    return _lib.tq_read_kv(ctx, ctypes.byref(batch.c_batch()), ka[0] if ka else None, _ptr(k_out),
                           va[0] if va else None, _ptr(v_out), _dtype(outs[0][1]) if outs else 0, layer,
                           _stream(stream))


def tq_chunk_workspace_bytes(ctx: int, batch: Batch, n_q_heads: int, n_kv_heads: int) -> int:
    return _lib.tq_chunk_workspace_bytes(ctx, ctypes.byref(batch.c_batch()), n_q_heads, n_kv_heads)


def tq_chunk_attention(ctx: int, batch: Batch, q, k_view, v_view, layer: int, softmax_scale: float, workspace,
                       workspace_bytes: int, out, mods: ScoreMods | None = None, stream=None) -> int:
    """q: [n_tokens, n_q_heads, d]; out: contiguous, the same shape, its type may differ."""
    shape = q.shape
    if shape[0] != batch.n_tokens or out.shape != shape or not out.is_contiguous() or not out.is_cuda or \
            shape[-1] != k_view.head_dim:
        raise ValueError(f"q {tuple(shape)}, out {tuple(out.shape)} for {batch.n_tokens} tokens")
    if mods is not None:
        for t, n in ((mods.slopes, shape[1]), (mods.first_keys, batch.n_tokens),
                     (mods.prefix_lens, batch.seq_lens.numel())):
            if t is not None and t.numel() != n:
                raise ValueError(f"{n} values are wanted: {tuple(t.shape)}")
    ka, va = _view_arg(k_view), _view_arg(v_view)
    return _lib.tq_chunk_attention(ctx, ctypes.byref(batch.c_batch()), q.data_ptr(), _dtype(q), _rows(q, shape),
                                   shape[1], ka[0], va[0], layer, softmax_scale,
                                   None if mods is None else ctypes.byref(mods.c_mods()), _ptr(workspace),
                                   workspace_bytes, _ptr(out), _dtype(out), _stream(stream))
