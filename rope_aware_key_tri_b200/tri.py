"""Thin Python binding of the C ABI in ``include/tri.h`` (ctypes).

Argument marshalling only: every step of the pass runs in the CUDA library
``lib/libtri_b200.so``. Importing this module loads that library and fails
loudly if it is missing; there is no fallback of any kind.

The module-level functions carry the C names (``tri_create``, ``tri_prune`` ...)
and take raw handles; :class:`TriContext` wraps them for torch tensors.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libtri_b200.so")

TRI_OK, TRI_EINVAL, TRI_ENOMEM, TRI_ECUDA, TRI_ESTATE, TRI_EDEVICE, TRI_EUNSUPPORTED = range(7)
TRI_ROPE_HALF, TRI_ROPE_INTERLEAVED = 0, 1
TRI_OFFSETS_MEAN, TRI_OFFSETS_MAX = 0, 1
TRI_ROPE_PLAIN, TRI_ROPE_LINEAR, TRI_ROPE_NTK, TRI_ROPE_YARN, TRI_ROPE_SMOOTH = range(5)
TRI_ENGINE_AUTO, TRI_ENGINE_CUDA_CORES, TRI_ENGINE_TENSOR = 0, 1, 2
TRI_DEV_NONE, TRI_DEV_LEN_GT_CAP, TRI_DEV_BAD_PAGE, TRI_DEV_TIMEOUT, TRI_DEV_INTERNAL, TRI_DEV_T_NOT_AFTER_POS = range(6)
TRI_DEV_BAD_RANGE = 6


class tri_kv(ctypes.Structure):
    _fields_ = [
        ("K", ctypes.c_void_p),
        ("V", ctypes.c_void_p),
        ("pos", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("lens_out", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("batch", ctypes.c_int32),
        ("cap", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("layer_begin", ctypes.c_int32),
        ("n_layers", ctypes.c_int32),
    ]


class tri_rows(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("layer_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


class TriError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}" + (f" [{detail}]" if detail else ""))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"the CUDA library {LIB_PATH} is missing; build it with "
            "`python -m rope_aware_key_tri_b200.build` (nvcc, sm_100a)")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    L.tri_create.argtypes = [ctypes.POINTER(P), ctypes.c_int]
    L.tri_destroy.argtypes = [P]
    L.tri_calibrate_load.argtypes = [P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, D,
                                     ctypes.c_int, P, P, P, P, ctypes.c_int]
    L.tri_prune.argtypes = [P, ctypes.POINTER(tri_kv), P, I32, P]
    L.tri_prune_noalloc.argtypes = [P, ctypes.POINTER(tri_kv), P, I32, P]
    L.tri_score.argtypes = [P, ctypes.POINTER(tri_kv), P, P, P, P]
    L.tri_calibrate_estimate.argtypes = [P, P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_int, P, P, P, P]
    L.tri_append.argtypes = [P, ctypes.POINTER(tri_kv), P, P, P, P]
    L.tri_append_advance.argtypes = [P, ctypes.POINTER(tri_kv), P, P, P, P]
    L.tri_get_error.argtypes = [P, P, ctypes.POINTER(I32), ctypes.POINTER(I64)]
    L.tri_get_failed_units.argtypes = [P, P, P, I32, ctypes.POINTER(I32)]
    L.tri_decode_attention.argtypes = [P, ctypes.POINTER(tri_kv), P, P, P]
    L.tri_set_test_fault.argtypes = [P, I64, I32]
    R = ctypes.POINTER(tri_rows)
    L.tri_rope_frequencies.argtypes = [ctypes.c_int, D, ctypes.c_int, D, D, D, D, P, ctypes.POINTER(D)]
    L.tri_rope_load.argtypes = [P, ctypes.c_int, ctypes.c_int, P, D]
    L.tri_rope.argtypes = [P, R, R, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, P, ctypes.c_int, P]
    L.tri_append_chunk.argtypes = [P, ctypes.POINTER(tri_kv), R, R, P, P, ctypes.c_int, ctypes.c_int, R, R, P]
    L.tri_chunk_attention.argtypes = [P, ctypes.POINTER(tri_kv), R, P, ctypes.c_int, D, ctypes.c_int, R, P, P]
    L.tri_set_tuning.argtypes = [P, ctypes.c_int, ctypes.c_int]
    L.tri_set_offset_combine.argtypes = [P, ctypes.c_int]
    L.tri_set_score_engine.argtypes = [P, ctypes.c_int]
    L.tri_last_error.argtypes = [P]
    L.tri_last_error.restype = ctypes.c_char_p
    L.tri_status_str.argtypes = [ctypes.c_int]
    L.tri_status_str.restype = ctypes.c_char_p
    for fn in ("tri_create", "tri_destroy", "tri_calibrate_load", "tri_prune", "tri_prune_noalloc", "tri_score",
               "tri_calibrate_estimate", "tri_append", "tri_append_advance", "tri_get_error", "tri_set_tuning",
               "tri_set_offset_combine",
               "tri_get_failed_units", "tri_set_test_fault", "tri_decode_attention", "tri_set_score_engine",
               "tri_rope_frequencies", "tri_rope_load", "tri_rope", "tri_append_chunk", "tri_chunk_attention",
               "tri_version"):
        getattr(L, fn).restype = ctypes.c_int
    return L


_lib = _load()


def library():
    return _lib


def status_str(st: int) -> str:
    return _lib.tri_status_str(int(st)).decode()


# ---- raw C names -----------------------------------------------------------------------

def tri_version() -> int:
    return _lib.tri_version()


def tri_status_str(st: int) -> str:
    return status_str(st)


def tri_create(device: int = 0) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    st = _lib.tri_create(ctypes.byref(h), int(device))
    if st != TRI_OK:
        raise TriError(st, "tri_create")
    return h


def tri_destroy(ctx) -> int:
    return _lib.tri_destroy(ctx)


def tri_calibrate_load(ctx, n_layers, n_kv_heads, group, head_dim, rope_base, layout,
                       q_mean, q_norm_mean, R, offsets) -> int:
    qm = np.ascontiguousarray(q_mean, dtype=np.float32)
    qn = np.ascontiguousarray(q_norm_mean, dtype=np.float32)
    rr = np.ascontiguousarray(R, dtype=np.float32)
    off = np.ascontiguousarray(offsets, dtype=np.int64)
    return _lib.tri_calibrate_load(ctx, int(n_layers), int(n_kv_heads), int(group), int(head_dim),
                                   float(rope_base), int(layout), qm.ctypes.data, qn.ctypes.data,
                                   rr.ctypes.data, off.ctypes.data, int(off.shape[0]))


def tri_prune(ctx, kv: tri_kv, t_ptr: int, budget: int, stream: int) -> int:
    return _lib.tri_prune(ctx, ctypes.byref(kv), t_ptr, int(budget), stream)


def tri_prune_noalloc(ctx, kv: tri_kv, t_ptr: int, budget: int, stream: int) -> int:
    return _lib.tri_prune_noalloc(ctx, ctypes.byref(kv), t_ptr, int(budget), stream)


def tri_score(ctx, kv: tri_kv, t_ptr: int, raw_ptr: int, zmax_ptr: int, stream: int) -> int:
    return _lib.tri_score(ctx, ctypes.byref(kv), t_ptr, raw_ptr, zmax_ptr, stream)


def tri_calibrate_estimate(ctx, q_ptr: int, n_layers: int, T: int, n_q_heads: int, head_dim: int, layout: int,
                           q_mean_ptr: int, q_norm_mean_ptr: int, R_ptr: int, stream: int) -> int:
    return _lib.tri_calibrate_estimate(ctx, q_ptr, int(n_layers), int(T), int(n_q_heads), int(head_dim),
                                       int(layout), q_mean_ptr, q_norm_mean_ptr, R_ptr, stream)


def tri_decode_attention(ctx, kv: tri_kv, q_ptr: int, out_ptr: int, stream: int) -> int:
    return _lib.tri_decode_attention(ctx, ctypes.byref(kv), q_ptr, out_ptr, stream)


def tri_append(ctx, kv: tri_kv, k_new_ptr: int, v_new_ptr: int, pos_new_ptr: int, stream: int) -> int:
    return _lib.tri_append(ctx, ctypes.byref(kv), k_new_ptr, v_new_ptr, pos_new_ptr, stream)


def tri_append_advance(ctx, kv: tri_kv, k_new_ptr: int, v_new_ptr: int, pos_ptr: int, stream: int) -> int:
    return _lib.tri_append_advance(ctx, ctypes.byref(kv), k_new_ptr, v_new_ptr, pos_ptr, stream)


_SCALINGS = {"plain": TRI_ROPE_PLAIN, "linear": TRI_ROPE_LINEAR, "ntk": TRI_ROPE_NTK, "yarn": TRI_ROPE_YARN,
             "smooth": TRI_ROPE_SMOOTH}


def rope_frequencies(rotary_dim, base, scaling="plain", factor=1.0, original_length=0.0, low=1.0, high=None):
    """(omega fp64 [rotary_dim/2], magnitude) for :meth:`TriContext.rope_load`: "plain", "linear", "ntk", "yarn" or
    "smooth" (or the TRI_ROPE_* value). low, high: the turns over original_length between which "yarn" and "smooth" go from
    interpolated to unscaled (high=None: 32 for "yarn", 4 for "smooth", their usual values). Host only."""
    kind = int(_SCALINGS.get(scaling, scaling))
    if high is None:
        high = 4.0 if kind == TRI_ROPE_SMOOTH else 32.0
    omega = np.empty(max(0, int(rotary_dim)) // 2, dtype=np.float64)
    mag = ctypes.c_double()
    st = _lib.tri_rope_frequencies(int(rotary_dim), float(base), kind, float(factor), float(original_length), float(low),
                                   float(high), omega.ctypes.data, ctypes.byref(mag))
    if st != TRI_OK:
        raise TriError(st, "tri_rope_frequencies")
    return omega, mag.value


def tri_rope_load(ctx, rotary_dim: int, layout: int, omega, magnitude: float) -> int:
    om = np.ascontiguousarray(omega, dtype=np.float64)
    return _lib.tri_rope_load(ctx, int(rotary_dim), int(layout), om.ctypes.data, float(magnitude))


# (the prompt side's calls are short: structures and numbers are converted by the argtypes alone)
def tri_rope(ctx, x: tri_rows, out: tri_rows, n_layers: int, n_tokens: int, n_heads: int, head_dim: int, pos_ptr: int,
             inverse: int, stream: int) -> int:
    return _lib.tri_rope(ctx, x, out, n_layers, n_tokens, n_heads, head_dim, pos_ptr, inverse, stream)


def tri_append_chunk(ctx, kv: tri_kv, K_new: tri_rows, V_new: tri_rows, cu_ptr: int, pos_ptr: int, n_tokens: int,
                     rotate: int, q: Optional[tri_rows], q_out: Optional[tri_rows], stream: int) -> int:
    return _lib.tri_append_chunk(ctx, kv, K_new, V_new, cu_ptr, pos_ptr, n_tokens, rotate, q, q_out, stream)


def tri_chunk_attention(ctx, kv: tri_kv, q: tri_rows, cu_ptr: int, n_tokens: int, scale: float, causal: int,
                        out: tri_rows, lse_ptr: Optional[int], stream: int) -> int:
    return _lib.tri_chunk_attention(ctx, kv, q, cu_ptr, n_tokens, scale, causal, out, lse_ptr, stream)


def tri_get_error(ctx, stream: int):
    code = ctypes.c_int32()
    unit = ctypes.c_int64()
    st = _lib.tri_get_error(ctx, stream, ctypes.byref(code), ctypes.byref(unit))
    return st, code.value, unit.value


def tri_get_failed_units(ctx, stream: int, capacity: int = 4096):
    """(status, total count, list of unit indices) of units left uncompacted by unit-level failures."""
    buf = (ctypes.c_int32 * max(1, capacity))()
    n = ctypes.c_int32()
    st = _lib.tri_get_failed_units(ctx, stream, buf, int(capacity), ctypes.byref(n))
    return st, n.value, [buf[i] for i in range(min(n.value, capacity))]


def tri_set_test_fault(ctx, unit: int = -1, wait_tries: int = 0) -> int:
    return _lib.tri_set_test_fault(ctx, int(unit), int(wait_tries))


def tri_last_error(ctx) -> str:
    r = _lib.tri_last_error(ctx)
    return r.decode() if r else ""


def tri_set_tuning(ctx, cluster_size: int = 0, buffers_per_warp: int = 0) -> int:
    return _lib.tri_set_tuning(ctx, int(cluster_size), int(buffers_per_warp))


def tri_set_offset_combine(ctx, combine: int) -> int:
    return _lib.tri_set_offset_combine(ctx, int(combine))


def tri_set_score_engine(ctx, engine: int) -> int:
    return _lib.tri_set_score_engine(ctx, int(engine))


# ---- torch-facing wrapper ----------------------------------------------------------------

def _ptr(x: Optional[torch.Tensor]) -> Optional[int]:
    return None if x is None else x.data_ptr()


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _new(shape, dtype, device, stream):
    """A result's memory, of the stream that writes it: what the current stream freed may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check_t(t, lens):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.shape != lens.shape:
        raise ValueError(f"t must be a contiguous CUDA int32 tensor shaped like lens {tuple(lens.shape)}")


def make_kv(K, V, pos, lens, lens_out=None, block_table=None, n_pages=None, layer_begin=0) -> tri_kv:
    """Describe a cache held in torch tensors.

    Dense: K, V bf16 [L][batch][Hkv][cap][d], pos int32 [L][batch][Hkv][cap].
    Paged: K, V bf16 [L][pages][Hkv][page_size][d], pos int32 [L][pages][Hkv][page_size],
           block_table int32 [batch][max_pages].
    """
    for name, x, dt in (("K", K, torch.bfloat16), ("V", V, torch.bfloat16), ("pos", pos, torch.int32),
                        ("lens", lens, torch.int32), ("lens_out", lens_out, torch.int32),
                        ("block_table", block_table, torch.int32)):
        if x is None:
            continue
        if x.dtype != dt or not x.is_cuda or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor of {dt}")
    # the C ABI sees plain pointers: check here that every buffer holds what the call describes
    batch = int(lens.shape[0])
    if K.dim() != 5 or (V is not None and V.shape != K.shape):
        raise ValueError("K (and V) must be 5-D: [L][batch][Hkv][cap][d] dense or [L][pages][Hkv][page][d] paged")
    if pos is not None and tuple(pos.shape) != tuple(K.shape[:4]):
        raise ValueError(f"pos must be {tuple(K.shape[:4])}, got {tuple(pos.shape)}")
    if block_table is None and int(K.shape[1]) != batch:
        raise ValueError(f"dense cache holds {int(K.shape[1])} sequences, lens describes {batch}")
    if block_table is not None and (block_table.dim() != 2 or int(block_table.shape[0]) != batch):
        raise ValueError(f"block_table must be [batch={batch}][max_pages]")
    kv = tri_kv()
    kv.K, kv.V, kv.pos = _ptr(K), _ptr(V), _ptr(pos)
    kv.lens, kv.lens_out, kv.block_table = _ptr(lens), _ptr(lens_out), _ptr(block_table)
    kv.batch = int(lens.shape[0])
    kv.layer_begin = int(layer_begin)
    kv.n_layers = int(K.shape[0])
    if block_table is None:
        kv.cap = int(K.shape[3])
    else:
        kv.page_size = int(K.shape[3])
        kv.max_pages = int(block_table.shape[1])
        kv.n_pages = int(K.shape[1]) if n_pages is None else int(n_pages)
    return kv


def make_rows(x: torch.Tensor, name: str = "x", device: Optional[int] = None) -> tri_rows:
    """Describe bf16 rows held in a torch tensor [tokens][heads][d] or [layers][tokens][heads][d]: any strides that are
    multiples of 8 elements, each row contiguous."""
    shape, stride = x.shape, x.stride()
    n = len(shape)
    if x.dtype is not torch.bfloat16 or not x.is_cuda or n not in (3, 4):
        raise ValueError(f"{name} must be a CUDA tensor of torch.bfloat16 [tokens][heads][d] or [layers][tokens][heads][d]")
    if device is not None and x.get_device() != device:
        raise ValueError(f"{name} is on {x.device}, the context on cuda:{device}")
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # (data, layer, token and head stride: a dimension of one element has no stride of its own)
    return tri_rows(x.data_ptr(), stride[0] if n == 4 and shape[0] > 1 else 0, stride[-3] if shape[-3] > 1 else 0,
                    stride[-2] if shape[-2] > 1 else 0)


class TriContext:
    """One library context on one CUDA device."""

    def __init__(self, device: int = 0):
        self.device = int(device)
        self.handle = tri_create(self.device)
        self.shape = None  # (n_layers, n_kv_heads, group, head_dim) of the loaded statistics

    # the C ABI takes the head counts and head_dim from the statistics: what the tensors hold must agree (_cache, _heads)
    def _heads(self, name, q):
        Hq, d = q.shape[-2], q.shape[-1]
        if self.shape is not None and (Hq, d) != (self.shape[1] * self.shape[2], self.shape[3]):
            raise ValueError(f"{name} has {Hq} heads of {d}, the loaded statistics {self.shape[1] * self.shape[2]} of "
                             f"{self.shape[3]}")
        return Hq

    def close(self):
        if self.handle is not None:
            tri_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def calibrate_load(self, n_layers, n_kv_heads, group, head_dim, rope_base, layout,
                       q_mean, q_norm_mean, R, offsets):
        st = tri_calibrate_load(self.handle, n_layers, n_kv_heads, group, head_dim, rope_base, layout,
                                q_mean, q_norm_mean, R, offsets)
        if st != TRI_OK:
            raise TriError(st, "tri_calibrate_load")
        self.shape = (int(n_layers), int(n_kv_heads), int(group), int(head_dim))

    def set_offset_combine(self, combine):
        """"mean" (the default) or "max" over the future offsets (or the TRI_OFFSETS_* value)."""
        code = {"mean": TRI_OFFSETS_MEAN, "max": TRI_OFFSETS_MAX}.get(combine, combine)
        st = tri_set_offset_combine(self.handle, code)
        if st != TRI_OK:
            raise TriError(st, "tri_set_offset_combine")

    def set_score_engine(self, engine):
        """"auto" (the default), "cuda_cores" or "tensor" (or the TRI_ENGINE_* value)."""
        code = {"auto": TRI_ENGINE_AUTO, "cuda_cores": TRI_ENGINE_CUDA_CORES, "tensor": TRI_ENGINE_TENSOR}.get(
            engine, engine)
        st = tri_set_score_engine(self.handle, code)
        if st != TRI_OK:
            raise TriError(st, "tri_set_score_engine")

    def set_tuning(self, cluster_size=0, buffers_per_warp=0):
        st = tri_set_tuning(self.handle, cluster_size, buffers_per_warp)
        if st != TRI_OK:
            raise TriError(st, "tri_set_tuning")

    def prune(self, K, V, pos, lens, t, budget, lens_out="inplace", block_table=None,
              layer_begin=0, stream=None, check=True):
        if isinstance(lens_out, str):
            lens_out = lens
        kv = make_kv(K, V, pos, lens, lens_out, block_table, layer_begin=layer_begin)
        _check_t(t, lens)
        st = tri_prune(self.handle, kv, t.data_ptr(), budget, _stream_handle(stream))
        if check and st != TRI_OK:
            raise TriError(st, "tri_prune", tri_last_error(self.handle))
        return st

    def prune_noalloc(self, K, V, pos, lens, t, budget, lens_out="inplace", block_table=None,
                      layer_begin=0, stream=None, check=True):
        """tri_prune_noalloc: the same prune with fixed, library-held scratch (no allocation)."""
        if isinstance(lens_out, str):
            lens_out = lens
        kv = make_kv(K, V, pos, lens, lens_out, block_table, layer_begin=layer_begin)
        _check_t(t, lens)
        st = tri_prune_noalloc(self.handle, kv, t.data_ptr(), budget, _stream_handle(stream))
        if check and st != TRI_OK:
            raise TriError(st, "tri_prune_noalloc", tri_last_error(self.handle))
        return st

    def score(self, K, lens, t, raw=None, zmax=None, block_table=None, layer_begin=0,
              stream=None, check=True):
        kv = make_kv(K, None, None, lens, None, block_table, layer_begin=layer_begin)
        _check_t(t, lens)
        st = tri_score(self.handle, kv, t.data_ptr(), _ptr(raw), _ptr(zmax), _stream_handle(stream))
        if check and st != TRI_OK:
            raise TriError(st, "tri_score", tri_last_error(self.handle))
        return st

    def append(self, K, V, pos, lens, block_table, K_new, V_new, pos_new, lens_out="inplace", n_pages=None,
               layer_begin=0, stream=None, check=True, advance=False):
        """Append one token per sequence to a paged cache (see make_kv for the layouts):
        K_new, V_new bf16 [n_layers][batch][n_kv_heads][head_dim], pos_new int32 [batch].
        advance=True: tri_append_advance (pos_new then holds the next positions)."""
        if isinstance(lens_out, str):
            lens_out = lens
        kv = make_kv(K, V, pos, lens, lens_out, block_table, n_pages=n_pages, layer_begin=layer_begin)
        for name, x, dt in (("K_new", K_new, torch.bfloat16), ("V_new", V_new, torch.bfloat16),
                            ("pos_new", pos_new, torch.int32)):
            if x.dtype != dt or not x.is_cuda or not x.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA tensor of {dt}")
        fn = tri_append_advance if advance else tri_append
        st = fn(self.handle, kv, K_new.data_ptr(), V_new.data_ptr(), pos_new.data_ptr(), _stream_handle(stream))
        if check and st != TRI_OK:
            raise TriError(st, fn.__name__, tri_last_error(self.handle))
        return st

    def decode_attention(self, K, V, lens, q, out=None, block_table=None, n_pages=None, layer_begin=0,
                         stream=None, check=True):
        """Attention of the post-RoPE queries q (bf16 [n_layers][batch][Hq][d]) over the cached
        rows [0, lens[s]) of K/V (layouts as in make_kv). Returns out (fp32, like q), or the
        status when check is False."""
        kv = make_kv(K, V, None, lens, None, block_table, n_pages=n_pages, layer_begin=layer_begin)
        if q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous():
            raise ValueError("q must be a contiguous CUDA tensor of torch.bfloat16")
        if q.dim() != 4 or tuple(q.shape[:2]) != (int(K.shape[0]), int(lens.shape[0])) or q.shape[3] != K.shape[4]:
            raise ValueError(f"q must be [n_layers][batch][Hq][d] for this cache, got {tuple(q.shape)}")
        if out is not None and (out.dtype != torch.float32 or tuple(out.shape) != tuple(q.shape)
                                or not out.is_contiguous()):
            raise ValueError("out must be a contiguous float32 tensor shaped like q")
        if out is None:
            out = _new(q.shape, torch.float32, q.device, stream)
        st = tri_decode_attention(self.handle, kv, q.data_ptr(), out.data_ptr(), _stream_handle(stream))
        if not check:
            return st
        if st != TRI_OK:
            raise TriError(st, "tri_decode_attention", tri_last_error(self.handle))
        return out

    def _flat(self, name, x, dtype, shape=None):
        if x.dtype is not dtype or x.get_device() != self.device or not x.is_contiguous() or (
                shape is not None and x.shape != shape):
            raise ValueError(f"{name} must be a contiguous tensor of {dtype} on cuda:{self.device}"
                             + (f" shaped {tuple(shape)}" if shape is not None else "")
                             + f", got {tuple(x.shape)} of {x.dtype} on {x.device}")
        return x.data_ptr()

    def _stream(self, stream):
        return torch._C._cuda_getCurrentRawStream(self.device) if stream is None else stream.cuda_stream

    def _cache(self, K, V, pos, lens, lens_out, block_table, n_pages, layer_begin):
        """The cache of a call (as make_kv, on this context's device), its layers, KV heads, head_dim and sequences."""
        shape, batch = K.shape, lens.shape
        if len(shape) != 5 or len(batch) != 1:
            raise ValueError("K and V must be 5-D: [L][batch][Hkv][cap][d] dense or [L][pages][Hkv][page][d] paged, lens 1-D")
        L, units, H, rows, d = shape
        if self.shape is not None and (H, d) != (self.shape[1], self.shape[3]):
            raise ValueError(f"the cache has {H} KV heads of {d}, the loaded statistics {self.shape[1]} of {self.shape[3]}")
        B = batch[0]
        if block_table is None:
            if units != B:
                raise ValueError(f"dense cache holds {units} sequences, lens describes {B}")
            table, cap, page, max_pages, n_pages = None, rows, 0, 0, 0
        else:
            if block_table.dim() != 2 or block_table.shape[0] != B:
                raise ValueError(f"block_table must be [batch={B}][max_pages]")
            # (the C ABI steps from layer to layer by n_pages)
            if n_pages is not None and (n_pages > units or L > 1 and n_pages != units):
                raise ValueError(f"n_pages is {n_pages}, the pools of {L} layers hold {units}")
            table, cap, page, max_pages = self._flat("block_table", block_table, torch.int32), 0, rows, block_table.shape[1]
            n_pages = units if n_pages is None else n_pages
        kv = tri_kv(self._flat("K", K, torch.bfloat16), self._flat("V", V, torch.bfloat16, shape),
                    None if pos is None else self._flat("pos", pos, torch.int32, shape[:4]),
                    self._flat("lens", lens, torch.int32),
                    None if lens_out is None else self._flat("lens_out", lens_out, torch.int32, batch), table, B, cap, page,
                    max_pages, n_pages, layer_begin, L)
        return kv, L, H, d, B

    def rope_load(self, omega, layout, magnitude=1.0):
        """The rotation of :meth:`rope` and :meth:`append_chunk`: omega fp64 [rotary_dim/2] radians per position (e.g. of
        :func:`rope_frequencies`), TRI_ROPE_HALF or TRI_ROPE_INTERLEAVED, and the magnitude of the rotated dims."""
        st = tri_rope_load(self.handle, 2 * len(omega), layout, omega, magnitude)
        if st != TRI_OK:
            raise TriError(st, "tri_rope_load", tri_last_error(self.handle))

    def rope(self, x, pos, out=None, inverse=False, stream=None, check=True):
        """Rotate the rows x (bf16 [tokens][heads][d] or [layers][tokens][heads][d], see make_rows) at pos (int32 [tokens]);
        inverse=True rotates back. Returns out (x itself is accepted), or the status when check is False."""
        if out is None:
            out = _new(x.shape, x.dtype, x.device, stream)
        if out.shape != x.shape:
            raise ValueError(f"out must be shaped like x {tuple(x.shape)}, got {tuple(out.shape)}")
        rows, rout = make_rows(x, "x", self.device), make_rows(out, "out", self.device)
        T, H, d = x.shape[-3:]
        st = tri_rope(self.handle, rows, rout, x.shape[0] if x.dim() == 4 else 1, T, H, d,
                      self._flat("pos", pos, torch.int32, (T,)), bool(inverse), self._stream(stream))
        if not check:
            return st
        if st != TRI_OK:
            raise TriError(st, "tri_rope", tri_last_error(self.handle))
        return out

    def _tokens(self, name, x, L, T, heads, d):
        """make_rows of a tensor whose shape the call gives."""
        shape, stride = x.shape, x.stride()
        if len(shape) == 3:
            shape, stride = (1, *shape), (0, *stride)
        if tuple(shape) != (L, T, heads, d):
            raise ValueError(f"{name} must be [{L} layers][{T} tokens][{heads}][{d}], got {tuple(x.shape)}")
        if x.dtype is not torch.bfloat16 or x.get_device() != self.device or stride[3] != 1:
            return make_rows(x, name, self.device)  # says what is wrong
        return tri_rows(x.data_ptr(), stride[0] if L > 1 else 0, stride[1] if T > 1 else 0, stride[2] if heads > 1 else 0)

    def append_chunk(self, K, V, pos, lens, K_new, V_new, cu_new, pos_new, block_table=None, lens_out="inplace",
                     rotate=True, q=None, q_out=None, n_pages=None, layer_begin=0, stream=None, check=True):
        """Append runs of new tokens to a cache (see make_kv for the layouts). K_new, V_new: bf16 rows
        [n_layers][tokens][n_kv_heads][d] (or without layers for one; strided views are accepted), sequence s holding the
        tokens [cu_new[s], cu_new[s + 1]); pos_new int32 [tokens]. rotate: K_new is pre-RoPE and rotated on the way; q
        (rows of the query heads) is then rotated into q_out in the same launch (q_out=None: in place)."""
        if isinstance(lens_out, str):
            lens_out = lens
        kv, L, H, d, B = self._cache(K, V, pos, lens, lens_out, block_table, n_pages, layer_begin)
        T = K_new.shape[-3]
        kn, vn = self._tokens("K_new", K_new, L, T, H, d), self._tokens("V_new", V_new, L, T, H, d)
        qr = qo = None
        if q is not None:
            q_out = q if q_out is None else q_out
            Hq = self._heads("q", q)
            qr, qo = self._tokens("q", q, L, T, Hq, d), self._tokens("q_out", q_out, L, T, Hq, d)
        st = tri_append_chunk(self.handle, kv, kn, vn, self._flat("cu_new", cu_new, torch.int32, (B + 1,)),
                              self._flat("pos_new", pos_new, torch.int32, (T,)), T, bool(rotate), qr, qo, self._stream(stream))
        if check and st != TRI_OK:
            raise TriError(st, "tri_append_chunk", tri_last_error(self.handle))
        return st

    def chunk_attention(self, K, V, lens, q, cu_q, out=None, lse=None, scale=None, causal=True, block_table=None,
                        n_pages=None, layer_begin=0, stream=None, check=True):
        """Attention of the post-RoPE queries q (bf16 rows [n_layers][tokens][Hq][d], or without layers for one;
        sequence s holding the tokens [cu_q[s], cu_q[s + 1])) over the cache that already holds those tokens as the
        last of its lens[s] rows. scale: of the logits (None: 1/sqrt(d)); lse: fp32 [n_layers][tokens][Hq] to receive
        the logarithm of the softmax sums. Returns out (bf16, like q), or the status when check is False."""
        kv, L, H, d, B = self._cache(K, V, None, lens, None, block_table, n_pages, layer_begin)
        T = q.shape[-3]
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        Hq = self._heads("q", q)
        qr, ro = self._tokens("q", q, L, T, Hq, d), self._tokens("out", out, L, T, Hq, d)
        if lse is not None and (lse.dtype is not torch.float32 or lse.numel() != L * T * Hq or not lse.is_contiguous()
                                or lse.get_device() != self.device):
            raise ValueError(f"lse must be a contiguous float32 tensor [{L}][{T}][{Hq}] on cuda:{self.device}")
        st = tri_chunk_attention(self.handle, kv, qr, self._flat("cu_q", cu_q, torch.int32, (B + 1,)), T,
                                 d ** -0.5 if scale is None else scale, bool(causal), ro,
                                 None if lse is None else lse.data_ptr(), self._stream(stream))
        if not check:
            return st
        if st != TRI_OK:
            raise TriError(st, "tri_chunk_attention", tri_last_error(self.handle))
        return out

    def calibrate_estimate(self, Q, layout, out=None, stream=None, check=True):
        """Calibration statistics from pre-RoPE queries Q (bf16 [n_layers][T][n_q_heads][head_dim],
        on this context's device). Returns fp32 device tensors (q_mean [L][Hq][d],
        q_norm_mean [L][Hq][d/2], R [L][Hq][d/2]), or the status when check is False."""
        if Q.dtype != torch.bfloat16 or Q.dim() != 4 or not Q.is_contiguous():
            raise TriError(TRI_EINVAL, "tri_calibrate_estimate", "Q must be a contiguous bf16 [L][T][Hq][d] tensor")
        nl, T, Hq, d = Q.shape
        if out is None:
            out = tuple(_new((nl, Hq, n), torch.float32, Q.device, stream) for n in (d, d // 2, d // 2))
        qm, qn, R = out
        st = tri_calibrate_estimate(self.handle, Q.data_ptr(), nl, T, Hq, d, int(layout), qm.data_ptr(),
                                    qn.data_ptr(), R.data_ptr(), _stream_handle(stream))
        if not check:
            return st
        if st != TRI_OK:
            raise TriError(st, "tri_calibrate_estimate", tri_last_error(self.handle))
        return qm, qn, R

    def get_error(self, stream=None):
        return tri_get_error(self.handle, _stream_handle(stream))

    def failed_units(self, stream=None, capacity=4096):
        """(total count, unit indices) of units left uncompacted by unit-level failures."""
        st, n, units = tri_get_failed_units(self.handle, _stream_handle(stream), capacity)
        if st != TRI_OK:
            raise TriError(st, "tri_get_failed_units")
        return n, units

    def set_test_fault(self, unit=-1, wait_tries=0):
        """Test hook: withhold the first key copy of `unit` on later calls (-1: off)."""
        st = tri_set_test_fault(self.handle, unit, wait_tries)
        if st != TRI_OK:
            raise TriError(st, "tri_set_test_fault")
