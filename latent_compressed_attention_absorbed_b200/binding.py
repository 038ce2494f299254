"""ctypes binding of libmla.so: argument marshalling only.

Every step of the decode runs in the CUDA library; this module turns torch
tensors into the C ABI's pointers, sizes and structs (include/mla.h),
allocates outputs / workspace with torch, and raises on any non-zero return
code.  ``load()`` raises if the library has not been built: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla.so")

MLA_DTYPE_BF16, MLA_DTYPE_F32 = 0, 1
PATH_AUTO, PATH_SM100, PATH_GENERIC = 0, 1, 2
STATUS_BAD_POS, STATUS_BAD_SEQLEN, STATUS_TIMEOUT, STATUS_NONFINITE = 1, 2, 4, 8
CACHE_FULL, CACHE_PACKED = 0, 1
NUM_EVENTS = 6
EV_START, EV_ABSORB_DONE, EV_ATTEND_BEGIN, EV_ATTEND_END, EV_COMBINE_DONE, EV_END = range(6)
ERRORS = {-1: "MLA_ERR_ARG", -2: "MLA_ERR_SHAPE", -3: "MLA_ERR_ALIGN", -4: "MLA_ERR_CUDA",
          -5: "MLA_ERR_TIMEOUT", -6: "MLA_ERR_DEVICE", -7: "MLA_ERR_WORKSPACE", -8: "MLA_ERR_UNSUPPORTED"}

# Every symbol the header declares (checked by the CPU test suite).
EXPORTS = ["mla_append_cache", "mla_workspace_bytes", "mla_decode", "mla_decode_ex", "mla_absorb_query",
           "mla_attend_latent", "mla_project_out", "mla_device_status", "mla_last_error", "mla_last_path",
           "mla_version", "mla_decode_no_alloc", "mla_append_from_hidden", "mla_append_from_hidden_workspace_bytes",
           "mla_output_projection", "mla_output_projection_workspace_bytes", "mla_packed_row_bytes", "mla_append_packed",
           "mla_append_rows", "mla_load_packed", "mla_packed_workspace_bytes", "mla_attend_packed", "mla_decode_packed",
           "mla_attend_latent_lse", "mla_accumulate_weights", "mla_evict_workspace_bytes", "mla_evict", "mla_evict_ex"]


class Dims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d_c", ctypes.c_int32), ("d_r", ctypes.c_int32),
                ("d_n", ctypes.c_int32), ("d_v", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("rope_base", ctypes.c_float), ("softmax_scale", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("B", ctypes.c_int32), ("T_max", ctypes.c_int32),
                ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64)]


class Opts(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("num_pairs", ctypes.c_int32), ("overhead_tiles", ctypes.c_int32),
                ("min_tiles", ctypes.c_int32), ("n_events", ctypes.c_int32),
                ("events", ctypes.POINTER(ctypes.c_void_p)), ("wait_limit_ns", ctypes.c_int64),
                ("withhold_tile", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MLAError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


_P = ctypes.c_void_p
_I = ctypes.c_int32
_SIGS = {
    "mla_append_cache": ([ctypes.POINTER(Dims), _P, _P, _P, _I, _I, ctypes.POINTER(Cache), _P], ctypes.c_int),
    "mla_workspace_bytes": ([ctypes.POINTER(Dims), _I, _I], ctypes.c_size_t),
    "mla_decode": ([ctypes.POINTER(Dims), _P, _P, _P, _P, ctypes.POINTER(Cache), _P, _I, _I, _P, _P,
                    ctypes.c_size_t, _P], ctypes.c_int),
    "mla_decode_ex": ([ctypes.POINTER(Dims), _P, _P, _P, _P, ctypes.POINTER(Cache), _P, _I, _I, _P, _P,
                       ctypes.c_size_t, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_decode_no_alloc": ([ctypes.POINTER(Dims), _P, _P, _P, _P, ctypes.POINTER(Cache), _P, _I, _I, _P, _P],
                            ctypes.c_int),
    "mla_absorb_query": ([ctypes.POINTER(Dims), _P, _P, _P, _P, _I, _I, _P, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_attend_latent": ([ctypes.POINTER(Dims), _P, ctypes.POINTER(Cache), _P, _I, _I, _P, _P, ctypes.c_size_t,
                           ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_project_out": ([ctypes.POINTER(Dims), _P, _P, _I, _P, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_append_from_hidden_workspace_bytes": ([ctypes.POINTER(Dims), _I, _I, _I], ctypes.c_size_t),
    "mla_append_from_hidden": ([ctypes.POINTER(Dims), _P, _P, _P, _P, _I, _I, _I, ctypes.POINTER(Cache), _P,
                                ctypes.c_size_t, _P], ctypes.c_int),
    "mla_output_projection_workspace_bytes": ([ctypes.POINTER(Dims), _I, _I], ctypes.c_size_t),
    "mla_output_projection": ([ctypes.POINTER(Dims), _P, _P, _I, _I, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "mla_packed_row_bytes": ([ctypes.POINTER(Dims)], ctypes.c_size_t),
    "mla_append_packed": ([ctypes.POINTER(Dims), _P, _P, _P, _P, _I, _I, ctypes.POINTER(Cache), _P], ctypes.c_int),
    "mla_append_rows": ([ctypes.POINTER(Dims), _P, _P, _P, _P, _I, _I, ctypes.POINTER(Cache), _P], ctypes.c_int),
    "mla_load_packed": ([ctypes.POINTER(Dims), ctypes.POINTER(Cache), _P, _I, _I, _P, _P], ctypes.c_int),
    "mla_packed_workspace_bytes": ([ctypes.POINTER(Dims), _I, _I], ctypes.c_size_t),
    "mla_attend_packed": ([ctypes.POINTER(Dims), _P, ctypes.POINTER(Cache), _P, _I, _I, _P, _P, _P, ctypes.c_size_t,
                           ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_decode_packed": ([ctypes.POINTER(Dims), _P, _P, _P, _P, ctypes.POINTER(Cache), _P, _P, _I, _I, _P, _P, _P, _P,
                           ctypes.c_size_t, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_attend_latent_lse": ([ctypes.POINTER(Dims), _P, ctypes.POINTER(Cache), _P, _I, _I, _P, _P, _P, ctypes.c_size_t,
                               ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_accumulate_weights": ([ctypes.POINTER(Dims), _P, _P, ctypes.POINTER(Cache), _I, _P, _I, _I, ctypes.c_float, _P,
                                _P, ctypes.c_int64, ctypes.POINTER(Opts), _P], ctypes.c_int),
    "mla_evict_workspace_bytes": ([ctypes.POINTER(Dims), _I, _I, _I], ctypes.c_size_t),
    "mla_evict": ([ctypes.POINTER(Dims), ctypes.POINTER(Cache), _I, _P, ctypes.c_int64, _P, _I, _I, _I, _I,
                   ctypes.POINTER(Cache), _P, ctypes.c_int64, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "mla_evict_ex": ([ctypes.POINTER(Dims), ctypes.POINTER(Cache), _I, _P, ctypes.c_int64, _P, _I, _I, _I, _I,
                      ctypes.POINTER(Cache), _P, ctypes.c_int64, _P, _P, _P, ctypes.c_size_t, ctypes.POINTER(Opts), _P],
                     ctypes.c_int),
    "mla_device_status": ([_P, ctypes.POINTER(_I)], ctypes.c_int),
    "mla_last_error": ([], ctypes.c_char_p),
    "mla_last_path": ([], ctypes.c_char_p),
    "mla_version": ([], ctypes.c_int),
}


def _torch_dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MLA_DTYPE_BF16
    if t.dtype == torch.float32:
        return MLA_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def _expect(t: Optional[torch.Tensor], name: str, dtype, shape: tuple, device):
    """``t`` is a contiguous tensor of that type and shape on ``device``; None passes."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    _need(t, name, dtype=dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def _need_weights(t, name, device, B):
    """Running weights: fp32 [B][>= T_max], unit stride along the rows (a view of a larger array is passed on)."""
    if t.dtype != torch.float32 or t.dim() != 2 or t.shape[0] != B or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be fp32 [{B}, rows] with unit stride along the rows")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor for a call on ``stream``: allocated there, as memory that the allocator hands out for the current
    stream may still be in use on it, and may be handed out again there before ``stream`` has got to the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class Library:
    def __init__(self, path: str = LIB_PATH):
        if not os.path.exists(path):
            raise FileNotFoundError(f"{path} is missing: build it with "
                                    "`python -m latent_compressed_attention_absorbed_b200.build`")
        self.path = path
        self.lib = ctypes.CDLL(path)
        for name, (args, res) in _SIGS.items():
            f = getattr(self.lib, name)
            f.argtypes = args
            f.restype = res

    # ------------------------------------------------------------------ helpers
    def _check(self, rc: int):
        if rc != 0:
            raise MLAError(rc, self.lib.mla_last_error().decode())

    def _call(self, fn, device: torch.device, stream, *args):
        """fn(*args, stream) with ``device`` current, on ``stream`` (default: the device's current stream); raises on error."""
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(device.index)
        else:
            raw = stream.cuda_stream
        if torch._C._cuda_getDevice() == device.index:
            rc = fn(*args, raw)
        else:
            with torch.cuda.device(device):
                rc = fn(*args, raw)
        if rc != 0:
            self._check(rc)

    @staticmethod
    def dims(H, d_c, d_r, d_n, d_v, dtype, rope_base=10000.0, softmax_scale=0.0) -> Dims:
        code = dtype if isinstance(dtype, int) else _torch_dtype_code(torch.empty(0, dtype=dtype))
        return Dims(H, d_c, d_r, d_n, d_v, code, rope_base, softmax_scale)

    @staticmethod
    def cache_desc(cache: torch.Tensor) -> Cache:
        """[B][T_max][row] with unit stride along the row; the other two strides
        are passed on (a view of a larger buffer: padded rows, or a subset of a
        larger batch), and the library checks them."""
        if not cache.is_cuda:
            raise ValueError("cache must be a CUDA tensor")
        if cache.dim() != 3:
            raise ValueError(f"cache must have 3 dims, got {tuple(cache.shape)}")
        shape, stride = cache.shape, cache.stride()
        if stride[2] != 1:
            raise ValueError("cache rows must be contiguous (unit stride along the last dimension)")
        return Cache(cache.data_ptr(), shape[0], shape[1], stride[0], stride[1])

    @staticmethod
    def opts(path=PATH_AUTO, num_pairs=0, overhead_tiles=-1, min_tiles=0, events=None, wait_limit_ns=0,
             withhold_tile=0) -> Opts:
        """``events``: MLA_NUM_EVENTS recorded torch.cuda.Event objects (stage timing).
        ``wait_limit_ns`` / ``withhold_tile``: see mla_decode_opts_t (the latter is a test hook)."""
        o = Opts(path, num_pairs, overhead_tiles, min_tiles, 0, None, wait_limit_ns, withhold_tile, 0)
        if events is not None:
            arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
            o.events = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
            o.n_events = len(events)
            o._keep = arr  # keep the array alive as long as the options
        return o

    def last_path(self) -> str:
        return self.lib.mla_last_path().decode()

    def version(self) -> int:
        return self.lib.mla_version()

    # ------------------------------------------------------------------ entry points
    def workspace_bytes(self, dims: Dims, B: int, q_len: int) -> int:
        return int(self.lib.mla_workspace_bytes(ctypes.byref(dims), B, q_len))

    def append_cache(self, dims: Dims, cache: torch.Tensor, c_kv: torch.Tensor, k_rope: torch.Tensor,
                     pos: torch.Tensor, stream=None):
        """Rows pos[b]+i of cache[b] <- [c_kv[b,i] || RoPE(k_rope[b,i], pos[b]+i)]."""
        _need(c_kv, "c_kv", ndim=3)
        _need(k_rope, "k_rope", ndim=3)
        _need(pos, "pos", dtype=torch.int32, ndim=1)
        B, n_tok = c_kv.shape[0], c_kv.shape[1]
        cd = self.cache_desc(cache)
        self._check(self.lib.mla_append_cache(ctypes.byref(dims), _ptr(c_kv), _ptr(k_rope), _ptr(pos), B, n_tok,
                                              ctypes.byref(cd), _stream(stream)))

    def decode(self, dims: Dims, q_nope, q_rope, W_UK, W_UV, cache, seqlens, out=None, workspace=None,
               opts: Optional[Opts] = None, stream=None):
        """One absorbed-MLA decode step; returns out [B, q_len, H, d_v]."""
        for t, n in ((q_nope, "q_nope"), (q_rope, "q_rope"), (W_UK, "W_UK"), (W_UV, "W_UV")):
            _need(t, n)
        _need(seqlens, "seqlens", dtype=torch.int32, ndim=1)
        B, q_len = q_nope.shape[0], q_nope.shape[1]
        if out is None:
            out = torch.empty((B, q_len, dims.H, dims.d_v), dtype=q_nope.dtype, device=q_nope.device)
        if workspace is None:
            workspace = torch.empty(max(self.workspace_bytes(dims, B, q_len), 16), dtype=torch.uint8,
                                    device=q_nope.device)
        cd = self.cache_desc(cache)
        o = opts if opts is not None else self.opts()
        self._check(self.lib.mla_decode_ex(ctypes.byref(dims), _ptr(q_nope), _ptr(q_rope), _ptr(W_UK), _ptr(W_UV),
                                           ctypes.byref(cd), _ptr(seqlens), B, q_len, _ptr(out), _ptr(workspace),
                                           workspace.numel(), ctypes.byref(o), _stream(stream)))
        return out

    def decode_no_alloc(self, dims: Dims, q_nope, q_rope, W_UK, W_UV, cache, seqlens, out=None, stream=None):
        """Same step as decode() using the library's static device scratch (no workspace argument)."""
        for t, n in ((q_nope, "q_nope"), (q_rope, "q_rope"), (W_UK, "W_UK"), (W_UV, "W_UV")):
            _need(t, n)
        _need(seqlens, "seqlens", dtype=torch.int32, ndim=1)
        B, q_len = q_nope.shape[0], q_nope.shape[1]
        if out is None:
            out = torch.empty((B, q_len, dims.H, dims.d_v), dtype=q_nope.dtype, device=q_nope.device)
        cd = self.cache_desc(cache)
        self._check(self.lib.mla_decode_no_alloc(ctypes.byref(dims), _ptr(q_nope), _ptr(q_rope), _ptr(W_UK),
                                                 _ptr(W_UV), ctypes.byref(cd), _ptr(seqlens), B, q_len, _ptr(out),
                                                 _stream(stream)))
        return out

    def absorb_query(self, dims: Dims, q_nope, q_rope, W_UK, seqlens, out=None, opts=None, stream=None):
        B, q_len = q_nope.shape[0], q_nope.shape[1]
        if out is None:
            out = torch.empty((B, q_len, dims.H, dims.d_c + dims.d_r), dtype=q_nope.dtype, device=q_nope.device)
        o = opts if opts is not None else self.opts()
        self._check(self.lib.mla_absorb_query(ctypes.byref(dims), _ptr(q_nope), _ptr(q_rope), _ptr(W_UK),
                                              _ptr(seqlens), B, q_len, _ptr(out), ctypes.byref(o), _stream(stream)))
        return out

    def attend_latent(self, dims: Dims, q_hat, cache, seqlens, out=None, workspace=None, opts=None, stream=None):
        B, q_len = q_hat.shape[0], q_hat.shape[1]
        if out is None:
            out = torch.empty((B, q_len, dims.H, dims.d_c), dtype=q_hat.dtype, device=q_hat.device)
        if workspace is None:
            workspace = torch.empty(max(self.workspace_bytes(dims, B, q_len), 16), dtype=torch.uint8,
                                    device=q_hat.device)
        cd = self.cache_desc(cache)
        o = opts if opts is not None else self.opts()
        self._check(self.lib.mla_attend_latent(ctypes.byref(dims), _ptr(q_hat), ctypes.byref(cd), _ptr(seqlens), B,
                                               q_len, _ptr(out), _ptr(workspace), workspace.numel(), ctypes.byref(o),
                                               _stream(stream)))
        return out

    def project_out(self, dims: Dims, o_lat, W_UV, out=None, opts=None, stream=None):
        rows = o_lat.shape[0] * o_lat.shape[1]
        if out is None:
            out = torch.empty((o_lat.shape[0], o_lat.shape[1], dims.H, dims.d_v), dtype=o_lat.dtype,
                              device=o_lat.device)
        o = opts if opts is not None else self.opts()
        self._check(self.lib.mla_project_out(ctypes.byref(dims), _ptr(o_lat), _ptr(W_UV), rows, _ptr(out),
                                             ctypes.byref(o), _stream(stream)))
        return out

    def append_from_hidden(self, dims: Dims, cache: torch.Tensor, x: torch.Tensor, W_A: torch.Tensor,
                           gamma: torch.Tensor, pos: torch.Tensor, workspace=None, stream=None):
        """Rows pos[b]+i of cache[b] <- [RMSNorm_gamma(W_DKV x[b,i]) || RoPE(W_KR x[b,i], pos[b]+i)];
        W_A = [W_DKV; W_KR] as [d_c + d_r, d_model]."""
        _need(x, "x", ndim=3)
        _need(W_A, "W_A", ndim=2)
        _need(gamma, "gamma", ndim=1)
        _need(pos, "pos", dtype=torch.int32, ndim=1)
        B, n_tok, d_model = x.shape
        if workspace is None:
            n = self.lib.mla_append_from_hidden_workspace_bytes(ctypes.byref(dims), B, n_tok, d_model)
            workspace = torch.empty(max(int(n), 16), dtype=torch.uint8, device=x.device)
        cd = self.cache_desc(cache)
        self._check(self.lib.mla_append_from_hidden(ctypes.byref(dims), _ptr(x), _ptr(W_A), _ptr(gamma), _ptr(pos),
                                                    B, n_tok, d_model, ctypes.byref(cd), _ptr(workspace),
                                                    workspace.numel(), _stream(stream)))

    def output_projection(self, dims: Dims, attn_out: torch.Tensor, W_O: torch.Tensor, y=None, workspace=None,
                          stream=None):
        """y[r] = W_O attn_out[r] with attn_out viewed as [rows, H * d_v]; W_O is [d_model, H * d_v]."""
        _need(attn_out, "attn_out")
        _need(W_O, "W_O", ndim=2)
        width = dims.H * dims.d_v
        rows, d_model = attn_out.numel() // width, W_O.shape[0]
        if y is None:
            y = torch.empty((rows, d_model), dtype=attn_out.dtype, device=attn_out.device)
        if workspace is None:
            n = self.lib.mla_output_projection_workspace_bytes(ctypes.byref(dims), rows, d_model)
            workspace = torch.empty(max(int(n), 16), dtype=torch.uint8, device=attn_out.device)
        self._check(self.lib.mla_output_projection(ctypes.byref(dims), _ptr(attn_out), _ptr(W_O), rows, d_model,
                                                   _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream)))
        return y

    # ------------------------------------------------------------------ 4-bit cache
    @staticmethod
    def _dtype(dims: Dims) -> torch.dtype:
        return torch.float32 if dims.dtype == MLA_DTYPE_F32 else torch.bfloat16

    def packed_row_bytes(self, dims: Dims) -> int:
        """Bytes of a packed row; a packed cache is a uint8 tensor [B][T_max][row bytes]."""
        n = int(self.lib.mla_packed_row_bytes(ctypes.byref(dims)))
        if n == 0:
            raise ValueError("these dims have no packed row (d_c must be a multiple of 16)")
        return n

    def _row(self, dims: Dims, fmt: int) -> int:
        """Elements of a row of that format (the packed layout of mla.h)."""
        d_c, d_r = dims.d_c, dims.d_r
        if fmt == CACHE_FULL:
            return d_c + d_r
        if d_c % 16:
            raise ValueError("these dims have no packed row (d_c must be a multiple of 16)")
        return ((((d_c // 2 + d_c // 16 + 15) & ~15) + d_r * (4 if dims.dtype == MLA_DTYPE_F32 else 2)) + 15) & ~15

    def _any_cache(self, dims: Dims, cache: torch.Tensor, device, name: str = "cache", want: Optional[int] = None):
        """(descriptor, format) of a full-width or (uint8) packed cache; ``want``: the one format the call takes."""
        fmt = CACHE_PACKED if cache.dtype is torch.uint8 else CACHE_FULL
        if fmt == CACHE_FULL and cache.dtype is not self._dtype(dims):
            raise TypeError(f"{name} must be {self._dtype(dims)} or torch.uint8 (packed), got {cache.dtype}")
        if want is not None and fmt != want:
            raise TypeError(f"the call takes a {('full-width', 'packed (torch.uint8)')[want]} cache, got {cache.dtype}")
        if cache.device != device:
            raise ValueError(f"{name} is on {cache.device}, the other tensors on {device}")
        d = self.cache_desc(cache)
        row = self._row(dims, fmt)
        if cache.shape[2] < row:
            raise ValueError(f"{name} rows hold {cache.shape[2]} elements, {row} are needed")
        return d, fmt

    def _append(self, fn, want, dims, cache, c_kv, k_rope, pos, rows, stream):
        dt, dev = self._dtype(dims), c_kv.device
        cd, _ = self._any_cache(dims, cache, dev, want=want)
        _need(c_kv, "c_kv", ndim=3)
        B, n_tok = c_kv.shape[0], c_kv.shape[1]
        _expect(c_kv, "c_kv", dt, (B, n_tok, dims.d_c), dev)
        _expect(k_rope, "k_rope", dt, (B, n_tok, dims.d_r), dev)
        _expect(pos, "pos", torch.int32, (B,), dev)
        _expect(rows, "rows", torch.int32, (B,), dev)
        self._call(fn, dev, stream, dims, c_kv.data_ptr(), k_rope.data_ptr(), pos.data_ptr(),
                   None if rows is None else rows.data_ptr(), B, n_tok, cd)

    def append_packed(self, dims: Dims, cache: torch.Tensor, c_kv: torch.Tensor, k_rope: torch.Tensor,
                      pos: torch.Tensor, rows: Optional[torch.Tensor] = None, stream=None):
        """Rows rows[b]+i (default pos[b]+i) of the packed cache <- [c_kv[b,i] in 4 bits || RoPE(k_rope[b,i], pos[b]+i)]."""
        self._append(self.lib.mla_append_packed, CACHE_PACKED, dims, cache, c_kv, k_rope, pos, rows, stream)

    def append_rows(self, dims: Dims, cache: torch.Tensor, c_kv: torch.Tensor, k_rope: torch.Tensor, pos: torch.Tensor,
                    rows: torch.Tensor, stream=None):
        """append_cache with the row apart from the position (after rows have been evicted)."""
        self._append(self.lib.mla_append_rows, CACHE_FULL, dims, cache, c_kv, k_rope, pos, rows, stream)

    def load_packed(self, dims: Dims, cache: torch.Tensor, rows: torch.Tensor, n_tok: int, out=None, stream=None):
        """Rows rows[b] .. rows[b]+n_tok-1 as full-width rows [B, n_tok, d_c + d_r]."""
        dt, dev = self._dtype(dims), rows.device
        cd, _ = self._any_cache(dims, cache, dev, want=CACHE_PACKED)
        _need(rows, "rows", dtype=torch.int32, ndim=1)
        B = rows.shape[0]
        shape = (B, n_tok, dims.d_c + dims.d_r)
        if out is None:
            out = _empty(shape, dt, dev, stream)
        else:
            _expect(out, "out", dt, shape, dev)
        self._call(self.lib.mla_load_packed, dev, stream, dims, cd, rows.data_ptr(), B, n_tok, out.data_ptr())
        return out

    def packed_workspace_bytes(self, dims: Dims, B: int, q_len: int) -> int:
        return int(self.lib.mla_packed_workspace_bytes(ctypes.byref(dims), B, q_len))

    @staticmethod
    def _scratch(workspace, nbytes, device, stream):
        """The caller's workspace, or a new one of nbytes() bytes."""
        if workspace is None:
            with torch.cuda.device(device):  # (the size depends on the device)
                n = nbytes()
            return _empty(max(n, 16), torch.uint8, device, stream)
        _need(workspace, "workspace", dtype=torch.uint8)
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, the other tensors on {device}")
        return workspace

    def _attend(self, fn, want, size, dims, q_hat, cache, seqlens, out, lse, workspace, opts, stream):
        dt, dev = self._dtype(dims), q_hat.device
        cd, _ = self._any_cache(dims, cache, dev, want=want)
        _need(q_hat, "q_hat", ndim=4)
        B, q_len = q_hat.shape[0], q_hat.shape[1]
        _expect(q_hat, "q_hat", dt, (B, q_len, dims.H, dims.d_c + dims.d_r), dev)
        _expect(seqlens, "seqlens", torch.int32, (B,), dev)
        _expect(lse, "lse", torch.float32, (B, q_len, dims.H), dev)
        shape = (B, q_len, dims.H, dims.d_c)
        if out is None:
            out = _empty(shape, dt, dev, stream)
        else:
            _expect(out, "out", dt, shape, dev)
        ws = self._scratch(workspace, lambda: size(dims, B, q_len), dev, stream)
        self._call(fn, dev, stream, dims, q_hat.data_ptr(), cd, seqlens.data_ptr(), B, q_len, out.data_ptr(),
                   None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), opts)
        return out

    def attend_packed(self, dims: Dims, q_hat, cache, seqlens, out=None, lse=None, workspace=None,
                      opts: Optional[Opts] = None, stream=None):
        """attend_latent over a packed cache; ``lse`` (fp32 [B, q_len, H]) receives the log-sum-exps if given."""
        return self._attend(self.lib.mla_attend_packed, CACHE_PACKED, self.packed_workspace_bytes, dims, q_hat, cache,
                            seqlens, out, lse, workspace, opts, stream)

    def decode_packed(self, dims: Dims, q_nope, q_rope, W_UK, W_UV, cache, seqlens, n_seen=None, out=None, q_hat=None,
                      lse=None, workspace=None, opts: Optional[Opts] = None, stream=None):
        """One decode step over a packed cache; returns out [B, q_len, H, d_v].  ``seqlens`` counts rows, ``n_seen``
        tokens (default: the same); ``q_hat`` and ``lse`` receive the folded queries and log-sum-exps if given."""
        dt, dev = self._dtype(dims), q_nope.device
        cd, _ = self._any_cache(dims, cache, dev, want=CACHE_PACKED)
        _need(q_nope, "q_nope", ndim=4)
        B, q_len = q_nope.shape[0], q_nope.shape[1]
        _expect(q_nope, "q_nope", dt, (B, q_len, dims.H, dims.d_n), dev)
        _expect(q_rope, "q_rope", dt, (B, q_len, dims.H, dims.d_r), dev)
        _expect(W_UK, "W_UK", dt, (dims.H, dims.d_n, dims.d_c), dev)
        _expect(W_UV, "W_UV", dt, (dims.H, dims.d_v, dims.d_c), dev)
        _expect(seqlens, "seqlens", torch.int32, (B,), dev)
        _expect(n_seen, "n_seen", torch.int32, (B,), dev)
        _expect(q_hat, "q_hat", dt, (B, q_len, dims.H, dims.d_c + dims.d_r), dev)
        _expect(lse, "lse", torch.float32, (B, q_len, dims.H), dev)
        shape = (B, q_len, dims.H, dims.d_v)
        if out is None:
            out = _empty(shape, dt, dev, stream)
        else:
            _expect(out, "out", dt, shape, dev)
        ws = self._scratch(workspace, lambda: self.packed_workspace_bytes(dims, B, q_len), dev, stream)
        self._call(self.lib.mla_decode_packed, dev, stream, dims, q_nope.data_ptr(), q_rope.data_ptr(), W_UK.data_ptr(),
                   W_UV.data_ptr(), cd, seqlens.data_ptr(), None if n_seen is None else n_seen.data_ptr(), B, q_len,
                   out.data_ptr(), None if q_hat is None else q_hat.data_ptr(), None if lse is None else lse.data_ptr(),
                   ws.data_ptr(), ws.numel(), opts)
        return out

    # ------------------------------------------------------------------ eviction by accumulated attention weight
    def attend_latent_lse(self, dims: Dims, q_hat, cache, seqlens, lse, out=None, workspace=None,
                          opts: Optional[Opts] = None, stream=None):
        """attend_latent that also writes the log-sum-exps to ``lse`` (fp32 [B, q_len, H])."""
        if lse is None:
            raise ValueError("lse must be given (attend_latent does without it)")
        return self._attend(self.lib.mla_attend_latent_lse, CACHE_FULL, self.workspace_bytes, dims, q_hat, cache,
                            seqlens, out, lse, workspace, opts, stream)

    def accumulate_weights(self, dims: Dims, q_hat, lse, cache, seqlens, weights, prev=None, decay: float = 1.0,
                           opts: Optional[Opts] = None, stream=None):
        """weights[b, t] = decay * prev[b, t] + the attention weight row t received in this step, summed over heads and
        queries (``prev``: None for zero, or ``weights`` itself); the cache is full-width or packed."""
        dev = q_hat.device
        cd, fmt = self._any_cache(dims, cache, dev)
        _need(q_hat, "q_hat", ndim=4)
        B, q_len, rows = q_hat.shape[0], q_hat.shape[1], cache.shape[1]
        _expect(q_hat, "q_hat", self._dtype(dims), (B, q_len, dims.H, dims.d_c + dims.d_r), dev)
        _expect(lse, "lse", torch.float32, (B, q_len, dims.H), dev)
        _expect(seqlens, "seqlens", torch.int32, (B,), dev)
        _need_weights(weights, "weights", dev, B)
        if weights.shape[1] < rows:
            raise ValueError(f"weights cover {weights.shape[1]} rows, the cache holds {rows}")
        if prev is not None and prev is not weights:
            _need_weights(prev, "prev", dev, B)
            if prev.shape != weights.shape or (B > 1 and prev.stride(0) != weights.stride(0)):
                raise ValueError("prev must have the shape and strides of weights")
        stride = weights.stride(0) if B > 1 else max(weights.stride(0), rows)
        self._call(self.lib.mla_accumulate_weights, dev, stream, dims, q_hat.data_ptr(), lse.data_ptr(), cd, fmt,
                   seqlens.data_ptr(), B, q_len, decay, None if prev is None else prev.data_ptr(), weights.data_ptr(),
                   stride, opts)
        return weights

    def evict_workspace_bytes(self, dims: Dims, B: int, budget: int, packed: bool = False) -> int:
        fmt = CACHE_PACKED if packed else CACHE_FULL
        return int(self.lib.mla_evict_workspace_bytes(ctypes.byref(dims), fmt, B, budget))

    def evict(self, dims: Dims, cache, weights, seqlens, budget: int, n_sink: int = 0, n_recent: int = 0, out=None,
              out_weights=None, out_seqlens=None, kept=None, workspace=None, opts: Optional[Opts] = None, stream=None):
        """Cuts sequences of more than ``budget`` rows down to the first n_sink, the last n_recent and the rows between
        with the largest weights, in their order.  In place unless ``out`` / ``out_weights`` / ``out_seqlens`` are
        given; ``kept`` (int32 [B, budget]) receives the kept rows' indexes, -1 past their number."""
        _need(seqlens, "seqlens", dtype=torch.int32, ndim=1)
        dev, B = seqlens.device, seqlens.shape[0]
        cd, fmt = self._any_cache(dims, cache, dev)
        od = cd if out is None else self._any_cache(dims, out, dev, "out", want=fmt)[0]
        rows = cache.shape[1]
        most = min(budget, rows)
        _need_weights(weights, "weights", dev, B)
        sw = weights.stride(0) if B > 1 else max(weights.stride(0), rows)
        if out_weights is None or out_weights is weights:
            out_weights, so = weights, sw
        else:
            _need_weights(out_weights, "out_weights", dev, B)
            so = out_weights.stride(0) if B > 1 else max(out_weights.stride(0), most)
        if weights.shape[1] < rows or out_weights.shape[1] < most:
            raise ValueError(f"weights must cover {rows} rows and out_weights {most}")
        if out_seqlens is None:
            out_seqlens = seqlens
        else:
            _expect(out_seqlens, "out_seqlens", torch.int32, (B,), dev)
        _expect(kept, "kept", torch.int32, (B, budget), dev)
        ws = self._scratch(workspace, lambda: self.evict_workspace_bytes(dims, B, budget, fmt == CACHE_PACKED), dev,
                           stream)
        self._call(self.lib.mla_evict_ex, dev, stream, dims, cd, fmt, weights.data_ptr(), sw, seqlens.data_ptr(), B, budget,
                   n_sink, n_recent, od, out_weights.data_ptr(), so, out_seqlens.data_ptr(),
                   None if kept is None else kept.data_ptr(), ws.data_ptr(), ws.numel(), opts)

    def device_status(self, stream=None) -> int:
        """Synchronises the stream, returns and clears the device status bits."""
        v = ctypes.c_int32(0)
        rc = self.lib.mla_device_status(_stream(stream), ctypes.byref(v))
        if rc not in (0, -6):
            self._check(rc)
        return int(v.value)


_lock = threading.Lock()
_lib: Optional[Library] = None


def load(path: str = LIB_PATH) -> Library:
    """The CUDA library (loaded once).  Raises if it is not built."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = Library(path)
        return _lib
