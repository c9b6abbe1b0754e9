"""Thin ctypes binding of libpa (include/pa.h): the same entry points, with
torch tensors in and out.  It only checks dtypes/devices and marshals
pointers; every step of the computation runs in the library's kernels.  If
libpa.so has not been built, every call raises (there is no fallback).
"""

from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_WORKSPACE = 0, 1, 2, 3, 4
PA_DEV_BAD_SLOT, PA_DEV_BAD_POSITION, PA_DEV_BAD_BLOCK = 1, 2, 4
PA_DEV_BAD_LENGTH, PA_DEV_TIMEOUT, PA_DEV_WORKSPACE = 8, 16, 32

# every symbol include/pa.h declares
EXPORTS = (
    "pa_cache_bytes", "pa_alloc_cache", "pa_free_cache", "pa_prepare_prefill",
    "pa_prepare_decode", "pa_rope_table_bytes", "pa_rope_table_init", "pa_rope_kv_write",
    "pa_prefill_varlen", "pa_decode_workspace_bytes", "pa_decode", "pa_strerror",
    "pa_check_device", "pa_decode_noalloc", "pa_decode_step", "pa_prefill_step",
    "pa_step_graph_create",
    "pa_step_graph_launch", "pa_step_graph_destroy", "pa_step_graph_create_io",
    "pa_bm_create", "pa_bm_destroy", "pa_bm_num_free", "pa_bm_blocks_needed", "pa_bm_allocate",
    "pa_bm_next_chunk", "pa_bm_mark_computed", "pa_bm_can_append", "pa_bm_append",
    "pa_bm_num_tokens", "pa_bm_block_table", "pa_bm_free", "pa_selftest_wait_timeout",
    "pa_cache_i8_bytes", "pa_alloc_cache_i8", "pa_free_cache_i8", "pa_rope_kv_write_i8",
    "pa_decode_i8",
    "pa_cache_i4_bytes", "pa_alloc_cache_i4", "pa_free_cache_i4", "pa_rope_kv_write_i4",
    "pa_kv_read_i4", "pa_decode_i4_workspace_bytes", "pa_decode_i4",
    "pa_prefill_i4_workspace_bytes", "pa_prefill_varlen_i4",
    "pa_rope_kv_write_layout", "pa_rope_table_init_scaled", "pa_prepare_shared",
    "pa_decode_shared_workspace_bytes", "pa_decode_shared",
    "pa_decode_weights_workspace_bytes", "pa_decode_weights",
    "pa_kv_evict_workspace_bytes", "pa_kv_evict", "pa_bm_evict_begin", "pa_bm_evict_end",
)


class PaCache(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("layers", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("owns", ctypes.c_int32), ("layer_stride", ctypes.c_int64),
                ("kv_stride", ctypes.c_int64)]


class PaCacheI8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("layers", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("owns", ctypes.c_int32)]


class PaCacheI4(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("layers", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("owns", ctypes.c_int32)]


class PaRopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("original_positions", ctypes.c_int32),
                ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("attention", ctypes.c_double)]


class PAError(RuntimeError):
    def __init__(self, name, code):
        super().__init__(f"{name} failed: {strerror(code)} (code {code})")
        self.code = code


_lib = None

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "pa_cache_bytes": (_sz, [_i32] * 5),
    "pa_alloc_cache": (_i32, [ctypes.POINTER(PaCache)] + [_i32] * 5 + [_vp]),
    "pa_free_cache": (_i32, [ctypes.POINTER(PaCache)]),
    "pa_prepare_prefill": (_i32, [_i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "pa_prepare_decode": (_i32, [_i32, _vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "pa_rope_table_bytes": (_sz, [_i32, _i32]),
    "pa_rope_table_init": (_i32, [_vp, _i32, _i32, ctypes.c_double, _vp]),
    "pa_rope_kv_write": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32,
                                ctypes.POINTER(PaCache), _i32, _vp, _vp]),
    "pa_prefill_varlen": (_i32, [_vp, _i32, ctypes.POINTER(PaCache), _i32, _vp, _vp, _vp, _i32,
                                 _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _vp, _vp]),
    "pa_decode_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "pa_decode": (_i32, [_vp, ctypes.POINTER(PaCache), _i32, _vp, _i32, _vp, _i32, _i32, _i32,
                         _i32, ctypes.c_float, _vp, _sz, _vp, _vp, _vp]),
    "pa_decode_noalloc": (_i32, [_vp, ctypes.POINTER(PaCache), _i32, _vp, _i32, _vp, _i32, _i32,
                                 _i32, _i32, ctypes.c_float, _vp, _vp, _vp]),
    "pa_decode_step": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, ctypes.POINTER(PaCache), _i32,
                              _vp, _i32, _vp, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _sz,
                              _vp, _vp, _vp]),
    "pa_prefill_step": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, ctypes.POINTER(PaCache), _i32,
                               _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                               ctypes.c_float, _vp, _vp, _vp]),
    "pa_step_graph_create": (_i32, [ctypes.POINTER(_vp), _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                    ctypes.POINTER(PaCache), _i32, _vp, _i32, _vp, _i32, _i32,
                                    _i32, _i32, ctypes.c_float, _vp, _sz, _vp, _vp]),
    "pa_step_graph_create_io": (_i32, [ctypes.POINTER(_vp), _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                       ctypes.POINTER(PaCache), _i32, _vp, _i32, _vp, _i32, _i32,
                                       _i32, _i32, ctypes.c_float, _vp, _sz, _vp, _vp, _vp, _vp,
                                       _sz, _vp]),
    "pa_step_graph_launch": (_i32, [_vp, _vp]),
    "pa_step_graph_destroy": (_i32, [_vp]),
    "pa_bm_create": (_vp, [_i32, _i32]),
    "pa_bm_destroy": (None, [_vp]),
    "pa_bm_num_free": (_i32, [_vp]),
    "pa_bm_blocks_needed": (_i32, [_vp, _i32]),
    "pa_bm_allocate": (_i32, [_vp, _i64, _vp, _i32, ctypes.POINTER(_i32)]),
    "pa_bm_next_chunk": (_i32, [_vp, _i64, _i32, ctypes.POINTER(_i32), ctypes.POINTER(_i32)]),
    "pa_bm_mark_computed": (_i32, [_vp, _i64, _i32]),
    "pa_bm_can_append": (_i32, [_vp, _i64]),
    "pa_bm_append": (_i32, [_vp, _i64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]),
    "pa_bm_num_tokens": (_i32, [_vp, _i64]),
    "pa_bm_block_table": (_i32, [_vp, _i64, _vp, _i32, ctypes.POINTER(_i32)]),
    "pa_bm_free": (_i32, [_vp, _i64]),
    "pa_bm_evict_begin": (_i32, [_vp, _i64, _i32]),
    "pa_bm_evict_end": (_i32, [_vp, _i64]),
    "pa_selftest_wait_timeout": (_i32, [_vp, _vp]),
    "pa_cache_i8_bytes": (_sz, [_i32] * 5),
    "pa_alloc_cache_i8": (_i32, [ctypes.POINTER(PaCacheI8)] + [_i32] * 5 + [_vp]),
    "pa_free_cache_i8": (_i32, [ctypes.POINTER(PaCacheI8)]),
    "pa_rope_kv_write_i8": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32,
                                   ctypes.POINTER(PaCacheI8), _i32, _vp, _vp]),
    "pa_decode_i8": (_i32, [_vp, ctypes.POINTER(PaCacheI8), _i32, _vp, _i32, _vp, _i32, _i32,
                            _i32, _i32, ctypes.c_float, _vp, _sz, _vp, _vp, _vp]),
    "pa_cache_i4_bytes": (_sz, [_i32] * 5),
    "pa_alloc_cache_i4": (_i32, [ctypes.POINTER(PaCacheI4)] + [_i32] * 5 + [_vp]),
    "pa_free_cache_i4": (_i32, [ctypes.POINTER(PaCacheI4)]),
    "pa_rope_kv_write_i4": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                                   _i32, ctypes.POINTER(PaCacheI4), _i32, _vp, _vp]),
    "pa_kv_read_i4": (_i32, [ctypes.POINTER(PaCacheI4), _i32, _vp, _i32, _vp, _vp, _vp, _i32,
                             _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "pa_decode_i4_workspace_bytes": (_sz, [_i32] * 4),
    "pa_decode_i4": (_i32, [_vp, ctypes.POINTER(PaCacheI4), _i32, _vp, _i32, _vp, _i32, _i32,
                            _i32, _i32, ctypes.c_float, _vp, _sz, _vp, _vp, _vp]),
    "pa_prefill_i4_workspace_bytes": (_sz, [_i32] * 5),
    "pa_prefill_varlen_i4": (_i32, [_vp, _i32, ctypes.POINTER(PaCacheI4), _i32, _vp, _vp, _vp,
                                    _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _sz,
                                    _vp, _vp, _vp]),
    "pa_rope_kv_write_layout": (_i32, [_vp] * 6 + [_i32] * 6 + [_vp, _i32, ctypes.POINTER(PaCache),
                                                                _i32, _vp, _vp]),
    "pa_rope_table_init_scaled": (_i32, [_vp, _i32, _i32, ctypes.c_double,
                                         ctypes.POINTER(PaRopeScaling), _vp]),
    "pa_prepare_shared": (_i32, [_i32, _vp, _i32, _vp, _i32, _vp, _vp, ctypes.POINTER(_i32)]),
    "pa_decode_shared_workspace_bytes": (_sz, [_i32] * 4),
    "pa_decode_shared": (_i32, [_vp, ctypes.POINTER(PaCache), _i32, _vp, _i32, _vp, _i32, _vp, _vp,
                                _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _sz, _vp, _vp, _vp]),
    "pa_decode_weights_workspace_bytes": (_sz, [_i32] * 4 + [_i64]),
    "pa_decode_weights": (_i32, [_vp, ctypes.POINTER(PaCache), _i32, _vp, _i32, _vp, _i32, _i32,
                                 _i32, _i32, ctypes.c_float, _vp, _vp, _i64, _vp, _sz, _vp, _vp,
                                 _vp]),
    "pa_kv_evict_workspace_bytes": (_sz, [_i32] * 3),
    "pa_kv_evict": (_i32, [ctypes.POINTER(PaCache), _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp,
                           _vp, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _sz, _vp, _vp]),
    "pa_strerror": (ctypes.c_char_p, [_i32]),
    "pa_check_device": (_i32, []),
}


def lib() -> ctypes.CDLL:
    """Load libpa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m paged_kv_gqa_rope_gb300.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(l, name)
            fn.restype, fn.argtypes = res, args
        _lib = l
    return _lib


def strerror(code: int) -> str:
    return lib().pa_strerror(int(code)).decode()


def _check(name, rc):
    if rc != PA_OK:
        raise PAError(name, rc)


def _p(t):
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(ctypes.c_void_p)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, dtype, name, shape=None):
    """A contiguous CUDA tensor of `dtype`; with `shape`, of exactly that shape
    (None entries free).  The library sees only pointers, so the sizes its
    kernels index by are checked here."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous CUDA {dtype} tensor")
    if shape is not None:
        _check_shape(t, shape, name)
    return t


def _check_shape(t, shape, name):
    if t.dim() != len(shape) or any(want is not None and got != want
                                    for got, want in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"{tuple('*' if w is None else w for w in shape)}")


def _table_width(block_tables):
    """max_blocks_per_seq; the kernels bound lengths by it * 16 in int32."""
    w = block_tables.shape[1]
    if w * 16 > 2**31 - 1:
        raise ValueError(f"block_tables rows of {w} entries: max_blocks_per_seq * 16 "
                         "must stay within int32")
    return w


def _bound(n):
    """A bound on lengths as an int32 (a larger one would reach the library cut to
    its low 32 bits)."""
    return min(int(n), 2**31 - 1)


def _int32(**numbers):
    """Refuses numbers that the library would see cut to their low 32 bits."""
    for name, x in numbers.items():
        if not -2**31 <= x < 2**31:
            raise ValueError(f"{name} {x} does not fit int32")


def _opt(t, dtype, name, shape):
    return None if t is None else _dev(t, dtype, name, shape)


def _out(out, like, stream=None):
    if out is None:
        return _new_out(like, stream)
    return _dev(out, like.dtype, "out", tuple(like.shape))


def _new_out(like, stream):
    """A tensor like `like` from the memory of the stream that will write it: of
    another stream's, the work before may still be using it."""
    if stream is None:
        return torch.empty_like(like)
    with torch.cuda.stream(stream):
        return torch.empty_like(like)


def check_device() -> int:
    return lib().pa_check_device()


# ------------------------------------------------------------------ host metadata

def prepare_prefill(num_cached, num_new, block_tables, block_size=16):
    nc = np.ascontiguousarray(num_cached, np.int32)
    nn = np.ascontiguousarray(num_new, np.int32)
    bt = np.ascontiguousarray(block_tables, np.int32)
    B = len(nn)
    T = int(nn.sum())
    pos = np.empty(max(T, 1), np.int32)
    slots = np.empty(max(T, 1), np.int32)
    cuq = np.empty(B + 1, np.int32)
    cuk = np.empty(B + 1, np.int32)
    mq, mk = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("pa_prepare_prefill", lib().pa_prepare_prefill(
        B, _p(nc), _p(nn), _p(bt), bt.shape[1] if bt.ndim == 2 else 0, block_size, _p(pos),
        _p(slots), _p(cuq), _p(cuk), ctypes.byref(mq), ctypes.byref(mk)))
    return dict(positions=pos[:T], slot_mapping=slots[:T], cu_seqlens_q=cuq, cu_seqlens_k=cuk,
                max_seqlen_q=mq.value, max_seqlen_k=mk.value)


def prepare_decode(num_cached, block_tables, block_size=16):
    nc = np.ascontiguousarray(num_cached, np.int32)
    bt = np.ascontiguousarray(block_tables, np.int32)
    B = len(nc)
    pos, slots, ctx = (np.empty(max(B, 1), np.int32) for _ in range(3))
    _check("pa_prepare_decode", lib().pa_prepare_decode(
        B, _p(nc), _p(bt), bt.shape[1], block_size, _p(pos), _p(slots), _p(ctx)))
    return dict(positions=pos[:B], slot_mapping=slots[:B], context_lens=ctx[:B])


# ------------------------------------------------------------------ cache and table

class Cache:
    """The block pool [2, layers, num_blocks, block_size, n_kv_heads, head_dim]
    fp16.  By default the memory is a torch tensor (``self.tensor``) that the
    library wraps; `tensor` takes a caller's own, a contiguous CUDA fp16 tensor
    of that shape; ``library_owned=True`` lets pa_alloc_cache allocate it."""

    def __init__(self, layers, num_blocks, n_kv_heads, head_dim, block_size=16, device="cuda",
                 library_owned=False, tensor=None):
        self.desc = PaCache()
        self.tensor = None
        shape = (2, layers, num_blocks, block_size, n_kv_heads, head_dim)
        if library_owned:
            if tensor is not None:
                raise ValueError("a library-owned pool takes no tensor")
            base = None
        else:
            self.tensor = (torch.empty(shape, dtype=torch.float16, device=device)
                           if tensor is None else _dev(tensor, torch.float16, "tensor", shape))
            base = _p(self.tensor)
        _check("pa_alloc_cache", lib().pa_alloc_cache(
            ctypes.byref(self.desc), layers, num_blocks, block_size, n_kv_heads, head_dim, base))

    def free(self):
        if self.desc.base:
            _check("pa_free_cache", lib().pa_free_cache(ctypes.byref(self.desc)))
        self.tensor = None

    def __del__(self):
        try:
            if self.desc.owns and self.desc.base:
                lib().pa_free_cache(ctypes.byref(self.desc))
        except Exception:
            pass


def cache_bytes(layers, num_blocks, block_size, n_kv_heads, head_dim) -> int:
    return lib().pa_cache_bytes(layers, num_blocks, block_size, n_kv_heads, head_dim)


def rope_table(max_positions, head_dim, theta=10000.0, device="cuda", stream=None):
    nbytes = lib().pa_rope_table_bytes(max_positions, head_dim)
    if nbytes == 0:
        raise ValueError("bad RoPE table shape")
    t = torch.empty((max_positions, head_dim // 2, 2), dtype=torch.float32, device=device)
    _check("pa_rope_table_init", lib().pa_rope_table_init(
        _p(t), max_positions, head_dim, float(theta), _stream(stream)))
    return t


def new_status(device="cuda"):
    return torch.zeros(1, dtype=torch.int32, device=device)


# ------------------------------------------------------------------ the hot path

def _rope_args(q, k, v, positions, slot_mapping, table, status):
    _dev(q, torch.float16, "q", (None, None, None))
    T, H, d = q.shape
    _dev(k, torch.float16, "k", (T, None, d))
    _dev(v, torch.float16, "v", tuple(k.shape))
    _dev(positions, torch.int32, "positions", (T,))
    _dev(slot_mapping, torch.int32, "slot_mapping", (T,))
    _dev(table, torch.float32, "table", (None, d // 2, 2))
    _opt(status, torch.int32, "status", (1,))
    return T, H, k.shape[1], d


def rope_kv_write(q, k, v, positions, slot_mapping, table, cache: Cache, layer=0, status=None,
                  stream=None):
    T, H, Hk, d = _rope_args(q, k, v, positions, slot_mapping, table, status)
    _check("pa_rope_kv_write", lib().pa_rope_kv_write(
        _p(q), _p(k), _p(v), _p(positions), _p(slot_mapping), T, H, Hk, d, _p(table),
        table.shape[0], ctypes.byref(cache.desc), layer, _p(status), _stream(stream)))


def prefill_varlen(q, cache: Cache, cu_seqlens_q, cu_seqlens_k, block_tables, max_seqlen_q,
                   n_kv_heads, layer=0, scale=0.0, out=None, status=None, stream=None):
    _dev(q, torch.float16, "q", (None, None, None))
    T, H, d = q.shape
    _dev(cu_seqlens_q, torch.int32, "cu_seqlens_q", (None,))
    B = cu_seqlens_q.shape[0] - 1
    _dev(cu_seqlens_k, torch.int32, "cu_seqlens_k", (B + 1,))
    _dev(block_tables, torch.int32, "block_tables", (B, None))
    _table_width(block_tables)
    _opt(status, torch.int32, "status", (1,))
    out = _out(out, q, stream)
    _check("pa_prefill_varlen", lib().pa_prefill_varlen(
        _p(q), T, ctypes.byref(cache.desc), layer, _p(cu_seqlens_q), _p(cu_seqlens_k),
        _p(block_tables), block_tables.shape[1], B, _bound(max_seqlen_q), H,
        n_kv_heads, d, float(scale), _p(out), _p(status), _stream(stream)))
    return out


def prefill_step(q, k, v, positions, slot_mapping, rope_table, cache: Cache, cu_seqlens_q,
                 cu_seqlens_k, block_tables, max_seqlen_q, n_kv_heads, layer=0, scale=0.0,
                 out=None, status=None, stream=None):
    """pa_prefill_step: RoPE + append of the new tokens, then the varlen prefill."""
    T, H, Hk, d = _rope_args(q, k, v, positions, slot_mapping, rope_table, status)
    _dev(cu_seqlens_q, torch.int32, "cu_seqlens_q", (None,))
    B = cu_seqlens_q.shape[0] - 1
    _dev(cu_seqlens_k, torch.int32, "cu_seqlens_k", (B + 1,))
    _dev(block_tables, torch.int32, "block_tables", (B, None))
    _table_width(block_tables)
    if Hk != n_kv_heads:
        raise ValueError(f"k has {Hk} KV heads, n_kv_heads is {n_kv_heads}")
    out = _out(out, q, stream)
    _check("pa_prefill_step", lib().pa_prefill_step(
        _p(q), _p(k), _p(v), _p(positions), _p(slot_mapping), _p(rope_table),
        rope_table.shape[0], ctypes.byref(cache.desc), layer, _p(cu_seqlens_q), _p(cu_seqlens_k),
        _p(block_tables), block_tables.shape[1], B, T, _bound(max_seqlen_q), H, n_kv_heads, d,
        float(scale), _p(out), _p(status), _stream(stream)))
    return out


def decode_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim) -> int:
    return lib().pa_decode_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim)


def decode_workspace(num_seqs, n_heads, n_kv_heads, head_dim, device="cuda", nbytes=None):
    """A zeroed workspace for pa_decode (its counters must start at zero);
    `nbytes` overrides the size (a smaller one narrows the grid)."""
    n = decode_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim) if nbytes is None else nbytes
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _decode_args(q, block_tables, context_lens, workspace, status):
    _dev(q, torch.float16, "q", (None, None, None))
    B = q.shape[0]
    _dev(block_tables, torch.int32, "block_tables", (B, None))
    _table_width(block_tables)
    _dev(context_lens, torch.int32, "context_lens", (B,))
    _dev(workspace, torch.uint8, "workspace", (None,))
    _opt(status, torch.int32, "status", (1,))
    return q.shape


def decode(q, cache: Cache, block_tables, context_lens, workspace, n_kv_heads, layer=0, scale=0.0,
           out=None, status=None, stream=None):
    B, H, d = _decode_args(q, block_tables, context_lens, workspace, status)
    out = _out(out, q, stream)
    _check("pa_decode", lib().pa_decode(
        _p(q), ctypes.byref(cache.desc), layer, _p(block_tables), block_tables.shape[1],
        _p(context_lens), B, H, n_kv_heads, d, float(scale), _p(workspace), workspace.numel(),
        _p(out), _p(status), _stream(stream)))
    return out


def _step_args(q, k, v, positions, slot_mapping, rope_table, cache, block_tables, context_lens,
               workspace, n_kv_heads, layer, scale, out, status):
    _rope_args(q, k, v, positions, slot_mapping, rope_table, status)
    B, H, d = _decode_args(q, block_tables, context_lens, workspace, status)
    _dev(out, torch.float16, "out", (B, H, d))
    return [_p(q), _p(k), _p(v), _p(positions), _p(slot_mapping), _p(rope_table),
            rope_table.shape[0], ctypes.byref(cache.desc), layer, _p(block_tables),
            block_tables.shape[1], _p(context_lens), B, H, n_kv_heads, d, float(scale),
            _p(workspace), workspace.numel(), _p(out), _p(status)]


def decode_step(q, k, v, positions, slot_mapping, rope_table, cache: Cache, block_tables,
                context_lens, workspace, n_kv_heads, layer=0, scale=0.0, out=None, status=None,
                stream=None):
    """pa_decode_step: RoPE + append of the new tokens, then decode."""
    out = _out(out, q, stream)
    args = _step_args(q, k, v, positions, slot_mapping, rope_table, cache, block_tables,
                      context_lens, workspace, n_kv_heads, layer, scale, out, status)
    _check("pa_decode_step", lib().pa_decode_step(*args, _stream(stream)))
    return out


class StepGraph:
    """pa_step_graph_*: a decode step captured once, replayed by launch().
    The tensors passed in are the step's buffers for every replay; refill
    them in place between replays.  References are kept so they outlive
    the graph.

    With `host_in` (a pinned uint8 host tensor) and `dev_in` (the device
    uint8 tensor of the same size that the input tensors are views of), a
    replay first copies host_in to dev_in; with `host_out` (a pinned host
    tensor shaped like q), it ends by copying the output there
    (pa_step_graph_create_io): one launch per step, I/O included."""

    def __init__(self, q, k, v, positions, slot_mapping, rope_table, cache: Cache, block_tables,
                 context_lens, workspace, n_kv_heads, layer=0, scale=0.0, out=None,
                 status=None, host_in=None, dev_in=None, host_out=None):
        self.out = _out(out, q)
        self._keep = (q, k, v, positions, slot_mapping, rope_table, cache, block_tables,
                      context_lens, workspace, status, host_in, dev_in, host_out)
        args = _step_args(q, k, v, positions, slot_mapping, rope_table, cache, block_tables,
                          context_lens, workspace, n_kv_heads, layer, scale, self.out, status)
        h = ctypes.c_void_p()
        if host_in is None and dev_in is None and host_out is None:
            _check("pa_step_graph_create", lib().pa_step_graph_create(ctypes.byref(h), *args))
        else:
            nin = 0
            if host_in is not None or dev_in is not None:
                if not (isinstance(host_in, torch.Tensor) and not host_in.is_cuda
                        and host_in.is_pinned() and host_in.dtype == torch.uint8
                        and host_in.is_contiguous()):
                    raise TypeError("host_in must be a contiguous pinned host uint8 tensor")
                _dev(dev_in, torch.uint8, "dev_in", (host_in.numel(),))
                nin = host_in.numel()
            if host_out is not None:
                if not (isinstance(host_out, torch.Tensor) and not host_out.is_cuda
                        and host_out.is_pinned() and host_out.dtype == torch.float16
                        and host_out.is_contiguous()):
                    raise TypeError("host_out must be a contiguous pinned host fp16 tensor")
                _check_shape(host_out, tuple(q.shape), "host_out")
            _check("pa_step_graph_create_io", lib().pa_step_graph_create_io(
                ctypes.byref(h), *args, _p(host_in), _p(dev_in), nin, _p(host_out)))
        self._h = h

    def launch(self, stream=None):
        _check("pa_step_graph_launch", lib().pa_step_graph_launch(self._h, _stream(stream)))
        return self.out

    def close(self):
        if self._h:
            _check("pa_step_graph_destroy", lib().pa_step_graph_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BlockManager:
    """pa_bm_*: the host block manager (block ownership, prefix-cache reuse,
    chunked-prefill progress); its tables feed prepare_prefill/decode."""

    def __init__(self, num_blocks, block_size=16):
        self._h = lib().pa_bm_create(num_blocks, block_size)
        if not self._h:
            raise ValueError("bad block manager sizes")
        self.block_size = block_size

    def num_free(self):
        return lib().pa_bm_num_free(self._h)

    def blocks_needed(self, num_tokens):
        return lib().pa_bm_blocks_needed(self._h, num_tokens)

    def allocate(self, seq_id, tokens):
        """Admit a prompt; returns the number of tokens already cached."""
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        n = ctypes.c_int()
        _check("pa_bm_allocate", lib().pa_bm_allocate(self._h, seq_id, _p(t), t.size,
                                                       ctypes.byref(n)))
        return n.value

    def next_chunk(self, seq_id, max_tokens):
        c, n = ctypes.c_int(), ctypes.c_int()
        _check("pa_bm_next_chunk", lib().pa_bm_next_chunk(self._h, seq_id, max_tokens,
                                                           ctypes.byref(c), ctypes.byref(n)))
        return c.value, n.value

    def mark_computed(self, seq_id, num_tokens):
        _check("pa_bm_mark_computed", lib().pa_bm_mark_computed(self._h, seq_id, num_tokens))

    def can_append(self, seq_id):
        r = lib().pa_bm_can_append(self._h, seq_id)
        if r < 0:
            raise PAError("pa_bm_can_append", -r)
        return bool(r)

    def append(self, seq_id, token):
        """Append a decoded token; returns its cache slot."""
        slot = ctypes.c_int32()
        _check("pa_bm_append", lib().pa_bm_append(self._h, seq_id, int(token), ctypes.byref(slot)))
        return slot.value

    def num_tokens(self, seq_id):
        return lib().pa_bm_num_tokens(self._h, seq_id)

    def block_table(self, seq_id):
        n = ctypes.c_int()
        lib().pa_bm_block_table(self._h, seq_id, None, 0, ctypes.byref(n))
        out = np.zeros(max(n.value, 1), np.int32)
        _check("pa_bm_block_table", lib().pa_bm_block_table(self._h, seq_id, _p(out), out.size,
                                                             ctypes.byref(n)))
        return out[:n.value]

    def evict_begin(self, seq_id, num_keep):
        """Switch to the table of the kept rows (kv_evict's out_block_tables)."""
        _check("pa_bm_evict_begin", lib().pa_bm_evict_begin(self._h, seq_id,
                                                            _bound(max(num_keep, 0))))

    def evict_end(self, seq_id):
        """The evictions are enqueued: the blocks left behind may be reused."""
        _check("pa_bm_evict_end", lib().pa_bm_evict_end(self._h, seq_id))

    def free(self, seq_id):
        _check("pa_bm_free", lib().pa_bm_free(self._h, seq_id))

    def close(self):
        if self._h:
            lib().pa_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def selftest_wait_timeout(status, stream=None):
    """pa_selftest_wait_timeout: a bounded wait that runs out (about 1 s)."""
    _dev(status, torch.int32, "status", (1,))
    _check("pa_selftest_wait_timeout", lib().pa_selftest_wait_timeout(_p(status), _stream(stream)))


class CacheI8:
    """The int8 pool: ``codes`` int8 [2, layers, num_blocks, block_size,
    n_kv_heads, head_dim] and ``scales`` float32 [2, layers, num_blocks,
    n_kv_heads, block_size], views of one torch allocation the library
    wraps."""

    def __init__(self, layers, num_blocks, n_kv_heads, head_dim, block_size=16, device="cuda"):
        self.desc = PaCacheI8()
        n = lib().pa_cache_i8_bytes(layers, num_blocks, block_size, n_kv_heads, head_dim)
        if n == 0:
            raise ValueError("bad int8 cache shape")
        self.buffer = torch.empty(n, dtype=torch.uint8, device=device)
        _check("pa_alloc_cache_i8", lib().pa_alloc_cache_i8(
            ctypes.byref(self.desc), layers, num_blocks, block_size, n_kv_heads, head_dim,
            _p(self.buffer)))
        nc = 2 * layers * num_blocks * block_size * n_kv_heads * head_dim
        off = self.desc.scales - self.desc.codes
        self.codes = self.buffer[:nc].view(torch.int8).view(
            2, layers, num_blocks, block_size, n_kv_heads, head_dim)
        self.scales = self.buffer[off:].view(torch.float32).view(
            2, layers, num_blocks, n_kv_heads, block_size)


def rope_kv_write_i8(q, k, v, positions, slot_mapping, table, cache: CacheI8, layer=0,
                     status=None, stream=None):
    T, H, Hk, d = _rope_args(q, k, v, positions, slot_mapping, table, status)
    _check("pa_rope_kv_write_i8", lib().pa_rope_kv_write_i8(
        _p(q), _p(k), _p(v), _p(positions), _p(slot_mapping), T, H, Hk, d, _p(table),
        table.shape[0], ctypes.byref(cache.desc), layer, _p(status), _stream(stream)))


def decode_i8(q, cache: CacheI8, block_tables, context_lens, workspace, n_kv_heads, layer=0,
              scale=0.0, out=None, status=None, stream=None):
    B, H, d = _decode_args(q, block_tables, context_lens, workspace, status)
    out = _out(out, q, stream)
    _check("pa_decode_i8", lib().pa_decode_i8(
        _p(q), ctypes.byref(cache.desc), layer, _p(block_tables), block_tables.shape[1],
        _p(context_lens), B, H, n_kv_heads, d, float(scale), _p(workspace), workspace.numel(),
        _p(out), _p(status), _stream(stream)))
    return out


class CacheI4:
    """The 4-bit pool: ``tiles`` uint8 [layers, num_blocks, n_kv_heads, 2 (K, V),
    10 * head_dim] (the tile's layout is in include/pa.h), a view of ``buffer``,
    the torch allocation the library wraps.  `buffer` takes a caller's own: a
    contiguous CUDA uint8 tensor of at least cache_i4_bytes(...) elements,
    256-byte aligned."""

    def __init__(self, layers, num_blocks, n_kv_heads, head_dim, block_size=16, device="cuda",
                 buffer=None):
        self.desc = PaCacheI4()
        n = cache_i4_bytes(layers, num_blocks, block_size, n_kv_heads, head_dim)
        if n == 0:
            raise ValueError("bad 4-bit cache shape")
        if buffer is None:
            buffer = torch.empty(n, dtype=torch.uint8, device=device)
        elif _dev(buffer, torch.uint8, "buffer", (None,)).numel() < n:
            raise ValueError(f"buffer holds {buffer.numel()} bytes, the pool needs {n}")
        if not buffer.is_cuda:
            raise ValueError(f"the 4-bit pool cannot be on {buffer.device}")
        self.buffer = buffer
        _check("pa_alloc_cache_i4", lib().pa_alloc_cache_i4(
            ctypes.byref(self.desc), layers, num_blocks, block_size, n_kv_heads, head_dim,
            _p(buffer)))
        self.tiles = buffer[:n].view(layers, num_blocks, n_kv_heads, 2, 10 * head_dim)


def cache_i4_bytes(layers, num_blocks, block_size, n_kv_heads, head_dim) -> int:
    return lib().pa_cache_i4_bytes(layers, num_blocks, block_size, n_kv_heads, head_dim)


# The 4-bit entry points check their tensors with `_on` and pass addresses as
# plain integers: on a small batch the Python of a call takes longer than its
# kernel.

def _on(dev, t, dtype, name, *shape):
    """The address of a contiguous CUDA tensor of `dtype` and exactly `shape` on
    device number `dev`."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtype, name, shape)
    raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's device is cuda:{dev}")


def _refuse_rank(*tensors):
    """The error of a call whose tensors' sizes could not be read: (tensor,
    dimensions, name) of each."""
    for t, n, name in tensors:
        if not (isinstance(t, torch.Tensor) and t.is_cuda):
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dim() != n:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {n} dimensions")
    raise TypeError("arguments are not CUDA tensors")


# The handle of a device's current stream, without a Stream object around it
# where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call_on(dev, name, stream, *args):
    """lib().<name>(*args, stream) with device `dev` current, on `stream` or that
    device's current stream."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index == dev:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"{name}: tensors on cuda:{dev}, stream on {stream.device}")
    fn = getattr(_lib or lib(), name)
    if dev == torch.cuda.current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != PA_OK:
        raise PAError(name, rc)


def _cache_i4(dev, cache):
    if not isinstance(cache, CacheI4):
        raise TypeError(f"cache must be a CacheI4, not {type(cache).__name__}")
    if cache.buffer.get_device() != dev:
        raise ValueError(f"the cache is on {cache.buffer.device}, the call's device is cuda:{dev}")
    return ctypes.byref(cache.desc)


def _layer_i4(layer):
    """The library checks it against the pool; past int32 it would see another one."""
    if not -2**31 <= layer < 2**31:
        raise ValueError(f"layer {layer} is not one of the pool's")
    return layer


def _status_i4(dev, status):
    return None if status is None else _on(dev, status, torch.int32, "status", 1)


def rope_kv_write_i4(q, k, v, positions, slot_mapping, table, cache: CacheI4, layer=0,
                     q_out=None, status=None, stream=None):
    """pa_rope_kv_write_i4: rotates Q (in place, or into `q_out`) and appends the
    quantised rotated K and V (both left as they are).  Returns the rotated Q."""
    try:
        (T, H, d), (_, Hk, _), (rows, _, _) = q.shape, k.shape, table.shape
        dev = q.get_device()
        if dev < 0:  # a host tensor
            raise ValueError
    except (AttributeError, ValueError):
        _refuse_rank((q, 3, "q"), (k, 3, "k"), (table, 3, "table"))
    if q_out is None:
        q_out = q
    _call_on(dev, "pa_rope_kv_write_i4", stream, _on(dev, q, torch.float16, "q", T, H, d),
             _on(dev, q_out, torch.float16, "q_out", T, H, d),
             _on(dev, k, torch.float16, "k", T, Hk, d), _on(dev, v, torch.float16, "v", T, Hk, d),
             _on(dev, positions, torch.int32, "positions", T),
             _on(dev, slot_mapping, torch.int32, "slot_mapping", T), T, H, Hk, d,
             _on(dev, table, torch.float32, "table", rows, d // 2, 2), rows,
             _cache_i4(dev, cache), _layer_i4(layer), _status_i4(dev, status))
    return q_out


def kv_read_i4(cache: CacheI4, block_tables, lengths, row_starts, k_out=None, v_out=None,
               first_tokens=None, layer=0, status=None, stream=None):
    """pa_kv_read_i4: tokens first_tokens[s] .. + lengths[s] - 1 of every sequence
    (from its first token by default) as fp16 into rows row_starts[s] .. of k_out
    and v_out [rows, n_kv_heads, head_dim] (None: not read).  Returns (k_out, v_out)."""
    if not isinstance(cache, CacheI4):
        raise TypeError(f"cache must be a CacheI4, not {type(cache).__name__}")
    dev = cache.buffer.get_device()
    Hk, d = cache.desc.n_kv_heads, cache.desc.head_dim
    out, rows = (k_out, "k_out") if k_out is not None else (v_out, "v_out"), 0
    try:
        B, width = block_tables.shape
        if out[0] is not None:
            rows, _, _ = out[0].shape
    except (AttributeError, ValueError):
        _refuse_rank((block_tables, 2, "block_tables"), (out[0], 3, out[1]))
    if rows > 2**31 - 1:
        raise ValueError(f"{rows} output rows: they must stay within int32")
    _call_on(dev, "pa_kv_read_i4", stream, ctypes.byref(cache.desc), _layer_i4(layer),
             _on(dev, block_tables, torch.int32, "block_tables", B, width),
             _table_width(block_tables), _on(dev, lengths, torch.int32, "lengths", B),
             None if first_tokens is None else
             _on(dev, first_tokens, torch.int32, "first_tokens", B),
             _on(dev, row_starts, torch.int32, "row_starts", B), B, rows, Hk, d,
             None if k_out is None else _on(dev, k_out, torch.float16, "k_out", rows, Hk, d),
             None if v_out is None else _on(dev, v_out, torch.float16, "v_out", rows, Hk, d),
             _status_i4(dev, status))
    return k_out, v_out


def decode_i4_workspace(num_seqs, n_heads, n_kv_heads, head_dim, device="cuda"):
    """A zeroed workspace for pa_decode_i4 (its counters must start at zero)."""
    return torch.zeros(lib().pa_decode_i4_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim),
                       dtype=torch.uint8, device=device)


def decode_i4(q, cache: CacheI4, block_tables, context_lens, workspace, n_kv_heads, layer=0,
              scale=0.0, out=None, status=None, stream=None):
    try:
        (B, H, d), (_, width), (nbytes,) = q.shape, block_tables.shape, workspace.shape
        dev = q.get_device()
        if dev < 0:  # a host tensor
            raise ValueError
    except (AttributeError, ValueError):
        _refuse_rank((q, 3, "q"), (block_tables, 2, "block_tables"), (workspace, 1, "workspace"))
    if out is None:
        out = _new_out(q, stream)
    _call_on(dev, "pa_decode_i4", stream, _on(dev, q, torch.float16, "q", B, H, d),
             _cache_i4(dev, cache), _layer_i4(layer),
             _on(dev, block_tables, torch.int32, "block_tables", B, width),
             _table_width(block_tables), _on(dev, context_lens, torch.int32, "context_lens", B), B,
             H, n_kv_heads, d, scale, _on(dev, workspace, torch.uint8, "workspace", nbytes), nbytes,
             _on(dev, out, torch.float16, "out", B, H, d), _status_i4(dev, status))
    return out


def prefill_i4_workspace(scratch_blocks, num_seqs, max_blocks_per_seq, n_kv_heads, head_dim,
                         device="cuda"):
    """A workspace for pa_prefill_varlen_i4 batches in which the contexts of the
    sequences with new tokens take at most `scratch_blocks` blocks of 16 tokens
    together."""
    n = lib().pa_prefill_i4_workspace_bytes(scratch_blocks, num_seqs, max_blocks_per_seq,
                                            n_kv_heads, head_dim)
    if n == 0:
        raise ValueError("bad 4-bit prefill workspace shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def prefill_varlen_i4(q, cache: CacheI4, cu_seqlens_q, cu_seqlens_k, block_tables, max_seqlen_q,
                      n_kv_heads, workspace, layer=0, scale=0.0, out=None, status=None,
                      stream=None):
    """pa_prefill_varlen_i4: varlen causal prefill over the 4-bit pool."""
    try:
        (T, H, d), (B, width), (nbytes,) = q.shape, block_tables.shape, workspace.shape
        dev = q.get_device()
        if dev < 0:  # a host tensor
            raise ValueError
    except (AttributeError, ValueError):
        _refuse_rank((q, 3, "q"), (block_tables, 2, "block_tables"), (workspace, 1, "workspace"))
    if out is None:
        out = _new_out(q, stream)
    _call_on(dev, "pa_prefill_varlen_i4", stream, _on(dev, q, torch.float16, "q", T, H, d), T,
             _cache_i4(dev, cache), _layer_i4(layer),
             _on(dev, cu_seqlens_q, torch.int32, "cu_seqlens_q", B + 1),
             _on(dev, cu_seqlens_k, torch.int32, "cu_seqlens_k", B + 1),
             _on(dev, block_tables, torch.int32, "block_tables", B, width),
             _table_width(block_tables), B, _bound(max_seqlen_q), H, n_kv_heads, d, scale,
             _on(dev, workspace, torch.uint8, "workspace", nbytes), nbytes,
             _on(dev, out, torch.float16, "out", T, H, d), _status_i4(dev, status))
    return out


# ------------------------------------------------------------------ long contexts

def _cache_f16(dev, cache):
    """The descriptor of an fp16 pool on device number `dev` (a library-owned pool
    names no device: it is taken to be on the call's)."""
    if not isinstance(cache, Cache):
        raise TypeError(f"cache must be a Cache, not {type(cache).__name__}")
    if cache.tensor is not None and cache.tensor.get_device() != dev:
        raise ValueError(f"the cache is on {cache.tensor.device}, the call's device is cuda:{dev}")
    return ctypes.byref(cache.desc)


ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def rope_kv_write_layout(q, k, v, positions, slot_mapping, table, cache: Cache, layout, layer=0,
                         q_out=None, status=None, stream=None):
    """pa_rope_kv_write_layout: turns the first 2 * table.shape[1] values of every Q
    row (in place, or into `q_out`) and of K, `layout` "interleaved" or "half", and
    appends K and V (both left as they are).  Returns the rotated Q."""
    try:
        (T, H, d), (_, Hk, _), (rows, pairs, _) = q.shape, k.shape, table.shape
        dev = q.get_device()
        if dev < 0:  # a host tensor
            raise ValueError
    except (AttributeError, ValueError):
        _refuse_rank((q, 3, "q"), (k, 3, "k"), (table, 3, "table"))
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout {layout!r} is none of {', '.join(ROPE_LAYOUTS)}")
    if q_out is None:
        q_out = q
    _call_on(dev, "pa_rope_kv_write_layout", stream, _on(dev, q, torch.float16, "q", T, H, d),
             _on(dev, q_out, torch.float16, "q_out", T, H, d),
             _on(dev, k, torch.float16, "k", T, Hk, d), _on(dev, v, torch.float16, "v", T, Hk, d),
             _on(dev, positions, torch.int32, "positions", T),
             _on(dev, slot_mapping, torch.int32, "slot_mapping", T), T, H, Hk, d,
             ROPE_LAYOUTS[layout], 2 * pairs,
             _on(dev, table, torch.float32, "table", rows, pairs, 2), rows,
             _cache_f16(dev, cache), _layer_i4(layer), _status_i4(dev, status))
    return q_out


def rope_table_scaled(max_positions, rotary_dim, theta=10000.0, scaling=None, factor=1.0,
                      original_positions=0, low=1.0, high=None, attention=0.0, device="cuda",
                      stream=None):
    """pa_rope_table_init_scaled: a table [max_positions, rotary_dim / 2, 2] for
    rope_kv_write_layout.  `scaling`: None, "linear", "ntk", "yarn" or "bands" (`low` and
    `high` turns over `original_positions`; high is 32 for "yarn" and 4 for "bands"
    unless given)."""
    if scaling is not None and scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r} is none of {', '.join(ROPE_SCALINGS)}")
    _int32(max_positions=max_positions, rotary_dim=rotary_dim,
           original_positions=original_positions)
    if lib().pa_rope_table_bytes(max_positions, rotary_dim) == 0:
        raise ValueError("bad RoPE table shape")
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if torch.device(device).type != "cuda":
        raise ValueError(f"a RoPE table cannot be on {device}")
    with torch.cuda.stream(stream):  # (None: as it is)
        t = torch.empty((max_positions, rotary_dim // 2, 2), dtype=torch.float32, device=device)
    sc = PaRopeScaling(ROPE_SCALINGS.get(scaling, 0), original_positions, factor, low, high,
                       attention)
    _call_on(t.get_device(), "pa_rope_table_init_scaled", stream, t.data_ptr(), max_positions,
             rotary_dim, float(theta), ctypes.byref(sc))
    return t


def prepare_shared(block_tables, context_lens, block_size=16):
    """pa_prepare_shared: the groups of neighbouring sequences whose block tables begin
    alike, as group_starts [groups + 1] and shared_blocks [groups] (numpy)."""
    _int32(block_size=block_size)
    bt = np.ascontiguousarray(block_tables, np.int32)
    ctx = np.ascontiguousarray(context_lens, np.int32)
    if bt.ndim != 2 or ctx.shape != bt.shape[:1]:
        raise ValueError(f"block_tables {bt.shape} and context_lens {ctx.shape} do not match")
    B = len(ctx)
    starts, blocks, n = np.zeros(B + 1, np.int32), np.zeros(max(B, 1), np.int32), _i32()
    _check("pa_prepare_shared", lib().pa_prepare_shared(
        B, _p(bt), bt.shape[1], _p(ctx), block_size, _p(starts), _p(blocks), ctypes.byref(n)))
    return dict(group_starts=starts[:n.value + 1].copy(), shared_blocks=blocks[:n.value].copy())


def decode_shared_workspace(num_seqs, n_heads, n_kv_heads, head_dim, device="cuda"):
    """A workspace for pa_decode_shared."""
    _int32(num_seqs=num_seqs, n_heads=n_heads, n_kv_heads=n_kv_heads, head_dim=head_dim)
    n = lib().pa_decode_shared_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim)
    if n == 0:
        raise ValueError("bad shared decode workspace shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def decode_shared(q, cache: Cache, block_tables, context_lens, group_starts, shared_blocks,
                  workspace, n_kv_heads, layer=0, scale=0.0, out=None, status=None, stream=None):
    """pa_decode_shared: decode of sequences group_starts[r] .. group_starts[r + 1] - 1
    that share their first shared_blocks[r] blocks, read once for the group.
    `context_lens`, `group_starts` and `shared_blocks` are read before the wait for the
    work ahead in the stream: torch operations, copies and this library's calls may write
    them directly before, a kernel that lets its dependents launch early
    (griddepcontrol.launch_dependents, programmatic launches of compiled kernels) may
    not."""
    try:
        (B, H, d), (_, width), (nbytes,) = q.shape, block_tables.shape, workspace.shape
        (groups,) = shared_blocks.shape
        dev = q.get_device()
        if dev < 0:  # a host tensor
            raise ValueError
    except (AttributeError, ValueError):
        _refuse_rank((q, 3, "q"), (block_tables, 2, "block_tables"), (workspace, 1, "workspace"),
                     (shared_blocks, 1, "shared_blocks"))
    if out is None:
        out = _new_out(q, stream)
    _call_on(dev, "pa_decode_shared", stream, _on(dev, q, torch.float16, "q", B, H, d),
             _cache_f16(dev, cache), _layer_i4(layer),
             _on(dev, block_tables, torch.int32, "block_tables", B, width),
             _table_width(block_tables), _on(dev, context_lens, torch.int32, "context_lens", B), B,
             _on(dev, group_starts, torch.int32, "group_starts", groups + 1),
             _on(dev, shared_blocks, torch.int32, "shared_blocks", groups), groups,
             H, n_kv_heads, d, scale, _on(dev, workspace, torch.uint8, "workspace", nbytes), nbytes,
             _on(dev, out, torch.float16, "out", B, H, d), _status_i4(dev, status))
    return out


def decode_weights_workspace(num_seqs, n_heads, n_kv_heads, head_dim, score_blocks,
                             device="cuda"):
    """A workspace for pa_decode_weights batches whose contexts take at most
    `score_blocks` blocks of 16 tokens together."""
    _int32(num_seqs=num_seqs, n_heads=n_heads, n_kv_heads=n_kv_heads, head_dim=head_dim)
    n = lib().pa_decode_weights_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim,
                                                score_blocks)
    if n == 0:
        raise ValueError("bad weights workspace shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def decode_weights(q, cache: Cache, block_tables, context_lens, weights, workspace, n_kv_heads,
                   weights_out=None, layer=0, scale=0.0, out=None, status=None, stream=None):
    """pa_decode_weights: decode, and weights_out[s, kv head, t] = weights + the attention
    weight of token t in the KV head's Q heads.  `weights` fp32 [B, n_kv_heads, stride]
    is updated in place unless `weights_out` is given; None stands for zeros (weights_out
    is then needed).  `context_lens` are read before the wait for the work ahead in the
    stream, as decode_shared's.  The weights stand by batch row: a sequence that changes
    its row takes them along.  Returns (out, weights_out)."""
    if weights_out is None:
        weights_out = weights
    try:
        (B, H, d), (_, width), (nbytes,) = q.shape, block_tables.shape, workspace.shape
        _, _, stride = weights_out.shape
        dev = q.get_device()
        if dev < 0:  # a host tensor
            raise ValueError
    except (AttributeError, ValueError):
        _refuse_rank((q, 3, "q"), (block_tables, 2, "block_tables"), (workspace, 1, "workspace"),
                     (weights_out, 3, "weights_out"))
    if out is None:
        out = _new_out(q, stream)
    _call_on(dev, "pa_decode_weights", stream, _on(dev, q, torch.float16, "q", B, H, d),
             _cache_f16(dev, cache), _layer_i4(layer),
             _on(dev, block_tables, torch.int32, "block_tables", B, width),
             _table_width(block_tables), _on(dev, context_lens, torch.int32, "context_lens", B), B,
             H, n_kv_heads, d, scale,
             None if weights is None else
             _on(dev, weights, torch.float32, "weights", B, n_kv_heads, stride),
             _on(dev, weights_out, torch.float32, "weights_out", B, n_kv_heads, stride), stride,
             _on(dev, workspace, torch.uint8, "workspace", nbytes), nbytes,
             _on(dev, out, torch.float16, "out", B, H, d), _status_i4(dev, status))
    return out, weights_out


def kv_evict_workspace(num_seqs, n_kv_heads, budget, device="cuda"):
    """A workspace for pa_kv_evict."""
    _int32(num_seqs=num_seqs, n_kv_heads=n_kv_heads, budget=budget)
    n = lib().pa_kv_evict_workspace_bytes(num_seqs, n_kv_heads, budget)
    if n == 0:
        raise ValueError("bad eviction workspace shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kv_evict(cache: Cache, block_tables, context_lens, weights, budget, workspace, sinks=0,
             recent=0, out_block_tables=None, out_context_lens=None, weights_out=None, layer=0,
             status=None, stream=None):
    """pa_kv_evict: every KV head keeps `budget` of a sequence's tokens, the first `sinks`,
    the last `recent` and those of the largest weights, K and V rows and weights [B,
    n_kv_heads, stride] moved to the first places.  Tables, lengths and weights are
    worked on in place unless their `out` is given.  One call is one layer's: with more
    layers give `out_context_lens`, since every layer starts from the old lengths.
    Returns (weights_out, out_context_lens)."""
    if out_block_tables is None:
        out_block_tables = block_tables
    if out_context_lens is None:
        out_context_lens = context_lens
    if weights_out is None:
        weights_out = weights
    try:
        (B, width), (_, out_width), (nbytes,) = (block_tables.shape, out_block_tables.shape,
                                                 workspace.shape)
        _, Hk, stride = weights.shape
        dev = weights.get_device()
        if dev < 0:  # a host tensor
            raise ValueError
    except (AttributeError, ValueError):
        _refuse_rank((block_tables, 2, "block_tables"), (out_block_tables, 2, "out_block_tables"),
                     (workspace, 1, "workspace"), (weights, 3, "weights"))
    desc = _cache_f16(dev, cache)
    _int32(budget=budget, sinks=sinks, recent=recent)
    _call_on(dev, "pa_kv_evict", stream, desc, _layer_i4(layer),
             _on(dev, block_tables, torch.int32, "block_tables", B, width),
             _table_width(block_tables), _on(dev, context_lens, torch.int32, "context_lens", B), B,
             Hk, cache.desc.head_dim, _on(dev, weights, torch.float32, "weights", B, Hk, stride),
             _on(dev, weights_out, torch.float32, "weights_out", B, Hk, stride), stride, budget,
             sinks, recent,
             _on(dev, out_block_tables, torch.int32, "out_block_tables", B, out_width),
             _table_width(out_block_tables),
             _on(dev, out_context_lens, torch.int32, "out_context_lens", B),
             _on(dev, workspace, torch.uint8, "workspace", nbytes), nbytes,
             _status_i4(dev, status))
    return weights_out, out_context_lens
