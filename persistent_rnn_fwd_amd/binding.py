"""ctypes binding of libprnn.so (the C ABI declared in include/prnn.h).

Argument marshalling only: torch tensors supply device memory and the current
stream; every step of the recurrence runs in the library's HIP kernels.  If the
library has not been built, every entry point raises; nothing falls back to
another implementation.
"""
from __future__ import annotations

import atexit
import ctypes
import os
import struct
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libprnn.so")

STATUS_NAMES = {
    0: "PRNN_STATUS_SUCCESS",
    1: "PRNN_STATUS_BAD_PARAM",
    2: "PRNN_STATUS_NOT_SUPPORTED",
    3: "PRNN_STATUS_ALLOC_FAILED",
    4: "PRNN_STATUS_EXECUTION_FAILED",
    5: "PRNN_STATUS_INTERNAL_ERROR",
}
SUCCESS, BAD_PARAM, NOT_SUPPORTED, ALLOC_FAILED, EXECUTION_FAILED, INTERNAL_ERROR = range(6)
DATA_FLOAT, DATA_HALF, DATA_BFLOAT, DATA_E4M3 = 0, 1, 2, 3
EXCHANGE_AUTO, EXCHANGE_DIRECT, EXCHANGE_RELAY = 0, 1, 2
LAYOUT_AUTO, LAYOUT_SPREAD, LAYOUT_TEAM = 0, 1, 2
MATH_AUTO, MATH_EXACT, MATH_SPLIT, MATH_HALF = 0, 1, 2, 3
STACK_AUTO, STACK_BLOCKED, STACK_FUSED, STACK_LAYERS = 0, 1, 2, 3
LAUNCH_COOPERATIVE, LAUNCH_PLAIN = 0, 1
TRACE_WORDS = 8  # per-wave trace record: see Handle.get_trace

# Every function include/prnn.h declares, with its ctypes signature.
_H = ctypes.c_void_p
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
SIGNATURES = {
    "prnn_create": (_I, [ctypes.POINTER(_H)]),
    "prnn_destroy": (_I, [_H]),
    "prnn_forward_dense": (_I, [_H, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "prnn_forward_sparse": (_I, [_H, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P]),
    "prnn_forward_sparse_rows": (_I, [_H, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P]),
    "prnn_sync_floor": (_I, [_H, _I, _I, _I, _P, _P]),
    "prnn_synchronize": (_I, [_H, _P]),
    "prnn_set_grid": (_I, [_H, _I]),
    "prnn_set_team_waves": (_I, [_H, _I]),
    "prnn_set_xcds_per_row": (_I, [_H, _I]),
    "prnn_set_watchdog_us": (_I, [_H, ctypes.c_uint32]),
    "prnn_set_exchange": (_I, [_H, _I]),
    "prnn_set_layout": (_I, [_H, _I]),
    "prnn_set_math": (_I, [_H, _I]),
    "prnn_get_last_plan": (_I, [_H, _P]),
    "prnn_debug_skip_publish": (_I, [_H, _I, _I]),
    "prnn_debug_jitter": (_I, [_H, ctypes.c_uint32, _I]),
    "prnn_set_trace": (_I, [_H, _I]),
    "prnn_get_trace": (_I, [_H, _P, ctypes.c_size_t, ctypes.POINTER(_I), _P]),
    "prnn_status_string": (ctypes.c_char_p, [_I]),
    "prnn_project": (_I, [_H, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P]),
    "prnn_forward_layer_dense": (_I, [_H, _I, _I, _I, _I, _I, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P]),
    "prnn_forward_layer_sparse": (_I, [_H, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P]),
    "prnn_forward_stack_dense": (_I, [_H, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "prnn_forward_stack_sparse": (_I, [_H, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P]),
    "prnn_set_stack_mode": (_I, [_H, _I]),
    "prnn_set_launch": (_I, [_H, _I]),
    "prnn_forward_dense_noalloc": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "prnn_linear_attention": (_I, [_H, _P, _P, _P, _P, _P, _P, _P, _P]),
    "prnn_linear_attention_backward": (_I, [_H, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "prnn_linear_attention_step": (_I, [_H, _P, _P, _P, _P, _P, _P, _P, _P]),
    "prnn_layer_norm": (_I, [_H, _L, _I, _I, _P, _L, _I, _P, _P, ctypes.c_float, _P, _L, _P, _P, _P]),
    "prnn_layer_norm_backward": (_I, [_H, _L, _I, _I, _P, _L, _P, _L, _P, _P, _I, _P, _P, _L, _P, _P, _P]),
    "prnn_gated_delta_rule": (_I, [_H, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "prnn_gated_delta_rule_backward": (_I, [_H, *[_P] * 16]),
    "prnn_gated_delta_rule_step": (_I, [_H, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "prnn_rms_norm": (_I, [_H, _L, _I, _I, _P, _L, _P, _L, _I, _P, ctypes.c_float, _P, _L, _I, _P, _L, _P, _I, _P, _P]),
    "prnn_rms_norm_backward": (_I, [_H, _L, _I, _I, _P, _L, _P, _L, _P, _I, _P, _P, _L, _P, _L, _P, _P]),
}

ATTENTION_MAX_D = 256  # PRNN_ATTENTION_MAX_D
SEQUENCE_TYPES = {torch.float32: DATA_FLOAT, torch.float16: DATA_HALF, torch.bfloat16: DATA_BFLOAT}


# prnnAttention_t, prnnDeltaRule_t, and prnnSequence_t: data, token, batch, head
_ATTENTION = struct.Struct("@7if3Pq")
_DELTA_RULE = struct.Struct("@7if2Pq")
_SEQUENCE = struct.Struct("@P3q")
_DELTA_FORWARD = struct.Struct("@7if2Pq" + 6 * "P3q")
_DELTA_BACKWARD = struct.Struct("@7if2Pq" + 11 * "P3q")
_NO_SEQUENCE = (0, 0, 0, 0)
ABSENT = object()  # in a stream's place: an output that is not made
RMS_GROUP = 128  # columns that share a scale of rms_norm_e4m3's groups


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("layout", ctypes.c_int),
        ("grid", ctypes.c_int),
        ("waves_per_wg", ctypes.c_int),
        ("rows_per_wave", ctypes.c_int),
        ("rmax", ctypes.c_int),
        ("chunks", ctypes.c_int),
        ("lds_bytes", ctypes.c_int),
        ("relay_slice", ctypes.c_int),
        ("first_step", ctypes.c_uint64),
        ("math", ctypes.c_int),
        ("xcds_per_row", ctypes.c_int),
    ]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class PrnnError(RuntimeError):
    def __init__(self, where: str, status: int):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_lib = None


def load_library() -> ctypes.CDLL:
    """Loads libprnn.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m persistent_rnn_fwd_amd.build` "
                "(the HIP library is required; there is no fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(where: str, status: int):
    if status != SUCCESS:
        raise PrnnError(where, status)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


try:  # the stream's pointer alone, without a Stream object
    from torch._C import _cuda_getCurrentRawStream as _current_raw_stream
except ImportError:
    def _current_raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _need(t: torch.Tensor, name: str, dtypes, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_strided(t: torch.Tensor, name: str, device: torch.device, dtypes, shape):
    """_need for a tensor whose rows may lie at any strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")


def _empty(like: torch.Tensor, shape, dtype, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A new output that belongs to the stream the call runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _ptr(t: Optional[torch.Tensor]):
    return t.data_ptr() if t is not None else None


class Handle:
    """A library handle (prnn_create) bound to the current GPU."""

    def __init__(self):
        self._lib = load_library()
        h = _H()
        _check("prnn_create", self._lib.prnn_create(ctypes.byref(h)))
        self._h = h
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        # descriptors of one call (an attention and up to 7 sequences, or a delta
        # rule and up to 11); the library reads them before it returns
        self._desc = ctypes.create_string_buffer(_ATTENTION.size + 11 * _SEQUENCE.size)
        self._desc_at = ctypes.addressof(self._desc)

    # -- lifetime ---------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            st = self._lib.prnn_destroy(self._h)
            self._h = None
            _check("prnn_destroy", st)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            if getattr(self, "_h", None):
                self._lib.prnn_destroy(self._h)
                self._h = None
        except Exception:
            pass

    # -- options ------------------------------------------------------------
    def set_grid(self, workgroups: int):
        _check("prnn_set_grid", self._lib.prnn_set_grid(self._h, int(workgroups)))

    def set_team_waves(self, waves: int):
        """Waves per team-layout workgroup for later calls: 0 (automatic), 8, 12 or 16."""
        _check("prnn_set_team_waves", self._lib.prnn_set_team_waves(self._h, int(waves)))

    def set_exchange(self, mode: int):
        """EXCHANGE_AUTO, EXCHANGE_DIRECT or EXCHANGE_RELAY for later calls."""
        _check("prnn_set_exchange", self._lib.prnn_set_exchange(self._h, int(mode)))

    def set_layout(self, layout: int):
        """LAYOUT_AUTO, LAYOUT_SPREAD or LAYOUT_TEAM for later calls."""
        _check("prnn_set_layout", self._lib.prnn_set_layout(self._h, int(layout)))

    def set_stack_mode(self, mode: int):
        """STACK_AUTO, STACK_BLOCKED, STACK_FUSED or STACK_LAYERS for later stack calls."""
        _check("prnn_set_stack_mode", self._lib.prnn_set_stack_mode(self._h, mode))

    def set_math(self, mode: int):
        """MATH_AUTO, MATH_EXACT, MATH_SPLIT or MATH_HALF (dense fp16) for later calls."""
        _check("prnn_set_math", self._lib.prnn_set_math(self._h, int(mode)))

    def set_xcds_per_row(self, xcds: int):
        """XCDs per batch row of dense fp16 layers for later calls: 0 (automatic), 1, 2 or 4."""
        _check("prnn_set_xcds_per_row", self._lib.prnn_set_xcds_per_row(self._h, int(xcds)))

    def set_launch(self, kind: int):
        """LAUNCH_COOPERATIVE or LAUNCH_PLAIN dispatch of the persistent kernels for later calls."""
        _check("prnn_set_launch", self._lib.prnn_set_launch(self._h, int(kind)))

    def set_watchdog_us(self, us: int):
        _check("prnn_set_watchdog_us", self._lib.prnn_set_watchdog_us(self._h, int(us)))

    def debug_skip_publish(self, wg: int, step: int):
        _check("prnn_debug_skip_publish", self._lib.prnn_debug_skip_publish(self._h, int(wg), int(step)))

    def debug_jitter(self, seed: int, span: int):
        """Test only: random publish delays of up to ``span`` sleep periods (0: off)."""
        _check("prnn_debug_jitter", self._lib.prnn_debug_jitter(self._h, int(seed) & 0xFFFFFFFF, int(span)))

    def last_plan(self) -> dict:
        info = PlanInfo()
        _check("prnn_get_last_plan", self._lib.prnn_get_last_plan(self._h, ctypes.byref(info)))
        return info.as_dict()

    def synchronize(self, stream: Optional[torch.cuda.Stream] = None):
        _check("prnn_synchronize", self._lib.prnn_synchronize(self._h, _stream_ptr(stream)))

    def set_trace(self, enable: bool):
        _check("prnn_set_trace", self._lib.prnn_set_trace(self._h, 1 if enable else 0))

    def get_trace(self, stream: Optional[torch.cuda.Stream] = None):
        """Phase records of the last traced call: uint64 array [grid * waves_per_wg, 8]
        (stage, barrier, compute, reduce, epilogue cycles; loop cycles; loop
        ticks of the 100 MHz clock; steps), one row per wave."""
        import numpy as np
        records = ctypes.c_int(0)
        st = self._lib.prnn_get_trace(self._h, None, 0, ctypes.byref(records), _stream_ptr(stream))
        if records.value <= 0:
            _check("prnn_get_trace", st)
        buf = np.zeros((records.value, TRACE_WORDS), dtype=np.uint64)
        _check("prnn_get_trace", self._lib.prnn_get_trace(self._h, buf.ctypes.data, buf.size, ctypes.byref(records),
                                                          _stream_ptr(stream)))
        return buf

    # -- the recurrence -----------------------------------------------------
    def forward_dense(self, W: torch.Tensor, X: torch.Tensor, h0: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """H[t] = relu(X[t] + H[t-1] W^T); W [N, N] fp32/fp16, X [T, B, N] fp32."""
        T, B, N = X.shape
        _need(W, "W", (torch.float32, torch.float16), (N, N))
        _need(X, "X", (torch.float32,), (T, B, N))
        if h0 is not None:
            _need(h0, "h0", (torch.float32,), (B, N))
        if out is None:
            out = torch.empty((T, B, N), dtype=torch.float32, device=X.device)
        _need(out, "out", (torch.float32,), (T, B, N))
        wt = DATA_FLOAT if W.dtype == torch.float32 else DATA_HALF
        st = self._lib.prnn_forward_dense(self._h, N, B, T, wt, W.data_ptr(), X.data_ptr(),
                                          h0.data_ptr() if h0 is not None else None, out.data_ptr(),
                                          _stream_ptr(stream))
        _check("prnn_forward_dense", st)
        return out

    def forward_sparse(self, col: torch.Tensor, val: torch.Tensor, X: torch.Tensor,
                       h0: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
        """Row-balanced sparse W: col int16 [N, K], val fp16/fp32 [N, K]."""
        T, B, N = X.shape
        K = col.shape[1] if col.dim() == 2 else -1
        _need(col, "col", (torch.int16,), (N, K))
        _need(val, "val", (torch.float32, torch.float16), (N, K))
        _need(X, "X", (torch.float32,), (T, B, N))
        if h0 is not None:
            _need(h0, "h0", (torch.float32,), (B, N))
        if out is None:
            out = torch.empty((T, B, N), dtype=torch.float32, device=X.device)
        _need(out, "out", (torch.float32,), (T, B, N))
        vt = DATA_FLOAT if val.dtype == torch.float32 else DATA_HALF
        st = self._lib.prnn_forward_sparse(self._h, N, B, T, K, col.data_ptr(), vt, val.data_ptr(),
                                           X.data_ptr(), h0.data_ptr() if h0 is not None else None,
                                           out.data_ptr(), _stream_ptr(stream))
        _check("prnn_forward_sparse", st)
        return out

    def forward_sparse_rows(self, col: torch.Tensor, val: torch.Tensor, row_len: torch.Tensor, X: torch.Tensor,
                            h0: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
        """Sparse W with rows of unequal length: col int16 [N, K], val fp16 [N, K],
        row_len int32 [N] (row i is its first row_len[i] pairs)."""
        T, B, N = X.shape
        K = col.shape[1] if col.dim() == 2 else -1
        _need(col, "col", (torch.int16,), (N, K))
        _need(val, "val", (torch.float32, torch.float16), (N, K))
        _need(row_len, "row_len", (torch.int32,), (N,))
        _need(X, "X", (torch.float32,), (T, B, N))
        if h0 is not None:
            _need(h0, "h0", (torch.float32,), (B, N))
        if out is None:
            out = torch.empty((T, B, N), dtype=torch.float32, device=X.device)
        _need(out, "out", (torch.float32,), (T, B, N))
        vt = DATA_FLOAT if val.dtype == torch.float32 else DATA_HALF
        st = self._lib.prnn_forward_sparse_rows(self._h, N, B, T, K, col.data_ptr(), vt, val.data_ptr(),
                                                row_len.data_ptr(), X.data_ptr(),
                                                h0.data_ptr() if h0 is not None else None, out.data_ptr(),
                                                _stream_ptr(stream))
        _check("prnn_forward_sparse_rows", st)
        return out

    # -- the input projection and whole layers ------------------------------
    def project(self, U: torch.Tensor, x: torch.Tensor, bias: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """X[..., n] = bias[n] + sum_i U[n, i] x[..., i]; U fp16 [N, I], x fp32/fp16 [..., I]."""
        N, I = U.shape
        lead = tuple(x.shape[:-1])
        M = 1
        for d in lead:
            M *= int(d)
        _need(U, "U", (torch.float16,), (N, I))
        _need(x, "x", (torch.float32, torch.float16), lead + (I,))
        if bias is not None:
            _need(bias, "bias", (torch.float32,), (N,))
        if out is None:
            out = torch.empty(lead + (N,), dtype=torch.float32, device=x.device)
        _need(out, "out", (torch.float32,), lead + (N,))
        xt = DATA_FLOAT if x.dtype == torch.float32 else DATA_HALF
        st = self._lib.prnn_project(self._h, M, N, I, xt, x.data_ptr(), DATA_HALF, U.data_ptr(),
                                    bias.data_ptr() if bias is not None else None, out.data_ptr(),
                                    _stream_ptr(stream))
        _check("prnn_project", st)
        return out

    def _layer_buffers(self, x, U, bias, h0, N, workspace, out):
        T, B, I = x.shape
        _need(U, "U", (torch.float16,), (N, I))
        _need(x, "x", (torch.float32, torch.float16), (T, B, I))
        if bias is not None:
            _need(bias, "bias", (torch.float32,), (N,))
        if h0 is not None:
            _need(h0, "h0", (torch.float32,), (B, N))
        if workspace is None:
            workspace = torch.empty((T, B, N), dtype=torch.float32, device=x.device)
        _need(workspace, "workspace", (torch.float32,), (T, B, N))
        if out is None:
            out = torch.empty((T, B, N), dtype=torch.float32, device=x.device)
        _need(out, "out", (torch.float32,), (T, B, N))
        return T, B, I, workspace, out

    def forward_layer_dense(self, U: torch.Tensor, bias: Optional[torch.Tensor], W: torch.Tensor, x: torch.Tensor,
                            h0: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One dense layer: X = x U^T + bias into `workspace` [T, B, N], then the recurrence."""
        N = W.shape[0]
        _need(W, "W", (torch.float32, torch.float16), (N, N))
        T, B, I, workspace, out = self._layer_buffers(x, U, bias, h0, N, workspace, out)
        xt = DATA_FLOAT if x.dtype == torch.float32 else DATA_HALF
        wt = DATA_FLOAT if W.dtype == torch.float32 else DATA_HALF
        st = self._lib.prnn_forward_layer_dense(
            self._h, N, I, B, T, xt, x.data_ptr(), DATA_HALF, U.data_ptr(),
            bias.data_ptr() if bias is not None else None, wt, W.data_ptr(),
            h0.data_ptr() if h0 is not None else None, workspace.data_ptr(), out.data_ptr(), _stream_ptr(stream))
        _check("prnn_forward_layer_dense", st)
        return out

    def forward_layer_sparse(self, U: torch.Tensor, bias: Optional[torch.Tensor], col: torch.Tensor,
                             val: torch.Tensor, x: torch.Tensor, h0: Optional[torch.Tensor] = None,
                             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
        """One row-balanced sparse layer: the projection, then the sparse recurrence."""
        N = col.shape[0]
        K = col.shape[1] if col.dim() == 2 else -1
        _need(col, "col", (torch.int16,), (N, K))
        _need(val, "val", (torch.float32, torch.float16), (N, K))
        T, B, I, workspace, out = self._layer_buffers(x, U, bias, h0, N, workspace, out)
        xt = DATA_FLOAT if x.dtype == torch.float32 else DATA_HALF
        vt = DATA_FLOAT if val.dtype == torch.float32 else DATA_HALF
        st = self._lib.prnn_forward_layer_sparse(
            self._h, N, I, B, T, K, xt, x.data_ptr(), DATA_HALF, U.data_ptr(),
            bias.data_ptr() if bias is not None else None, col.data_ptr(), vt, val.data_ptr(),
            h0.data_ptr() if h0 is not None else None, workspace.data_ptr(), out.data_ptr(), _stream_ptr(stream))
        _check("prnn_forward_layer_sparse", st)
        return out

    def forward_stack_dense(self, layers, x: torch.Tensor, h0s=None, outs=None,
                            workspace: Optional[torch.Tensor] = None, stream=None):
        """A stack of dense fp16 layers as one wavefront.  layers: list of dicts
        with U (fp16 [N, I] for the first, [N, N] after), bias (fp32 [N] or
        None) and W (fp16 [N, N]); x [T, B, I]; h0s: None or one [B, N] (or
        None) per layer.  Returns the list of every layer's H [T, B, N]."""
        L = len(layers)
        T, B, I = x.shape
        N = layers[0]["W"].shape[0]
        _need(x, "x", (torch.float32, torch.float16), (T, B, I))
        for l, ly in enumerate(layers):
            _need(ly["U"], f"layers[{l}].U", (torch.float16,), (N, I if l == 0 else N))
            _need(ly["W"], f"layers[{l}].W", (torch.float16,), (N, N))
            if ly.get("bias") is not None:
                _need(ly["bias"], f"layers[{l}].bias", (torch.float32,), (N,))
            if h0s is not None and h0s[l] is not None:
                _need(h0s[l], f"h0s[{l}]", (torch.float32,), (B, N))
        if workspace is None:
            workspace = torch.empty((T, B, N), dtype=torch.float32, device=x.device)
        _need(workspace, "workspace", (torch.float32,), (T, B, N))
        if outs is None:
            outs = [torch.empty((T, B, N), dtype=torch.float32, device=x.device) for _ in range(L)]
        for l, o in enumerate(outs):
            _need(o, f"outs[{l}]", (torch.float32,), (T, B, N))
        ptrs = lambda ts: (ctypes.c_void_p * L)(*[(t.data_ptr() if t is not None else None) for t in ts])
        Up, Wp, Hp = ptrs([ly["U"] for ly in layers]), ptrs([ly["W"] for ly in layers]), ptrs(outs)
        bp = ptrs([ly.get("bias") for ly in layers])
        hp = ptrs(h0s) if h0s is not None else None
        xt = DATA_FLOAT if x.dtype == torch.float32 else DATA_HALF
        st = self._lib.prnn_forward_stack_dense(self._h, L, N, I, B, T, xt, x.data_ptr(), Up, bp, Wp, hp,
                                                workspace.data_ptr(), Hp, _stream_ptr(stream))
        _check("prnn_forward_stack_dense", st)
        return outs

    def forward_stack_sparse(self, layers, x: torch.Tensor, h0s=None, outs=None,
                             workspace: Optional[torch.Tensor] = None, stream=None):
        """A stack of row-balanced sparse layers, one after another.  layers: list
        of dicts with U (fp16 [N, I] for the first, [N, N] after), bias (fp32
        [N] or None), col (int16 [N, K]) and val (fp16 or fp32 [N, K], one dtype
        for all layers); x [T, B, I]; h0s: None or one [B, N] (or None) per
        layer.  Returns the list of every layer's H [T, B, N]."""
        L = len(layers)
        T, B, I = x.shape
        N, K = layers[0]["col"].shape
        vdt = layers[0]["val"].dtype
        _need(x, "x", (torch.float32, torch.float16), (T, B, I))
        for l, ly in enumerate(layers):
            _need(ly["U"], f"layers[{l}].U", (torch.float16,), (N, I if l == 0 else N))
            _need(ly["col"], f"layers[{l}].col", (torch.int16,), (N, K))
            _need(ly["val"], f"layers[{l}].val", (vdt,), (N, K))
            if ly.get("bias") is not None:
                _need(ly["bias"], f"layers[{l}].bias", (torch.float32,), (N,))
            if h0s is not None and h0s[l] is not None:
                _need(h0s[l], f"h0s[{l}]", (torch.float32,), (B, N))
        if workspace is None:
            workspace = torch.empty((T, B, N), dtype=torch.float32, device=x.device)
        _need(workspace, "workspace", (torch.float32,), (T, B, N))
        if outs is None:
            outs = [torch.empty((T, B, N), dtype=torch.float32, device=x.device) for _ in range(L)]
        for l, o in enumerate(outs):
            _need(o, f"outs[{l}]", (torch.float32,), (T, B, N))
        ptrs = lambda ts: (ctypes.c_void_p * L)(*[(t.data_ptr() if t is not None else None) for t in ts])
        Up, Cp, Vp, Hp = (ptrs([ly["U"] for ly in layers]), ptrs([ly["col"] for ly in layers]),
                          ptrs([ly["val"] for ly in layers]), ptrs(outs))
        bp = ptrs([ly.get("bias") for ly in layers])
        hp = ptrs(h0s) if h0s is not None else None
        xt = DATA_FLOAT if x.dtype == torch.float32 else DATA_HALF
        vt = DATA_FLOAT if vdt == torch.float32 else DATA_HALF
        st = self._lib.prnn_forward_stack_sparse(self._h, L, N, I, B, T, K, xt, x.data_ptr(), Up, bp, Cp, vt, Vp, hp,
                                                 workspace.data_ptr(), Hp, _stream_ptr(stream))
        _check("prnn_forward_stack_sparse", st)
        return outs

    # -- linear attention with a decay for each head -------------------------
    # (The checks are written for few Python calls: a step's kernel takes a
    # few microseconds.)
    def _stream(self, stream):
        return _stream_ptr(stream) if stream is not None else _current_raw_stream(self._index)

    def _strided(self, t, name, dtype, shape):
        """t's strides, once it is what it should be."""
        if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != self._index
                or (t.stride(-1) != 1 and shape[-1] > 1)):
            _need_strided(t, name, self.device, (dtype,), shape)
        return t.stride()

    def _dense(self, t, name, dtype, shape):
        if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != self._index
                or not t.is_contiguous()):
            _need(t, name, (dtype,), shape)
            _need_strided(t, name, self.device, (dtype,), shape)  # another GPU's
        return t.data_ptr()

    def _attention(self, q, k, v, log_decay, scale, offsets, lengths, max_len, step, more):
        """Checks the inputs, writes the descriptors of the attention, of q, k
        and v and of the sequences in `more` (heads, head size, dtype, tensor
        or None for a new one, name, stream), and returns those tensors and the
        shape of the states."""
        lead = 1 if step or offsets is not None else 2
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or t.dim() != lead + 2:
                raise ValueError(f"{name} must have {lead + 2} axes")
        dtype = q.dtype
        code = SEQUENCE_TYPES.get(dtype)
        if code is None:
            raise TypeError(f"q must have dtype in {tuple(SEQUENCE_TYPES)}, got {dtype}")
        *rows, H, Dk = q.shape
        Hkv, Dv = v.shape[-2:]
        rows = tuple(rows)
        total, at_lengths, at_offsets = 0, None, None
        if step:
            B, T, axes = rows[0], 1, (None, 0)
        elif offsets is not None:
            if lengths is not None:
                raise ValueError("give offsets (packed sequences) or lengths, not both")
            if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
                raise ValueError("offsets must be [B + 1]")
            B, total, axes = offsets.shape[0] - 1, rows[0], (0, None)
            T = total if max_len is None else max(-1, min(int(max_len), total))  # (longer than the rows: as long)
            at_offsets = self._dense(offsets, "offsets", torch.int32, (B + 1,))
        else:
            (T, B), axes = rows, (0, 1)
            if lengths is not None:
                at_lengths = self._dense(lengths, "lengths", torch.int32, (B,))
        _ATTENTION.pack_into(self._desc, 0, B, min(T, 0x7fffffff), H, Hkv, Dk, Dv, code, Dk ** -0.5 if scale is None else scale,
                             self._dense(log_decay, "log_decay", torch.float32, (H,)), at_lengths or 0,
                             at_offsets or 0, total)
        at = _ATTENTION.size
        outs = []
        token, batch = axes
        shapes = {"H": H, "Hkv": Hkv, "Dk": Dk, "Dv": Dv}
        for t, name, heads, size, stream in (
                (q, "q", "H", "Dk", 0), (k, "k", "Hkv", "Dk", 0), (v, "v", "Hkv", "Dv", 0), *more):
            shape = (*rows, shapes[heads], shapes[size])
            if t is None:
                t = _empty(q, shape, dtype, stream)
                strides = t.stride()
            else:
                strides = self._strided(t, name, dtype, shape)
            _SEQUENCE.pack_into(self._desc, at, t.data_ptr(),
                                strides[token] if token is not None and shape[token] > 1 else 0,
                                strides[batch] if batch is not None and shape[batch] > 1 else 0,
                                strides[-2] if shape[-2] > 1 else 0)
            at += _SEQUENCE.size
            outs.append(t)
        return outs[3:], (B, H, Dk, Dv)

    def _state(self, t, name, shape):
        return self._dense(t, name, torch.float32, shape) if t is not None else None

    def linear_attention(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                         scale: Optional[float] = None, initial_state: Optional[torch.Tensor] = None,
                         final_state: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                         lengths: Optional[torch.Tensor] = None, max_len: Optional[int] = None,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """S[t] = exp(log_decay) S[t-1] + k[t] v[t]^T, o[t] = scale S[t]^T q[t] for whole sequences.

        q [T, B, H, Dk], k [T, B, Hkv, Dk], v [T, B, Hkv, Dv] (fp32, fp16 or
        bf16; any strides with a contiguous last axis) give o [T, B, H, Dv];
        log_decay fp32 [H]; scale None: Dk ** -0.5.  Sequences of unequal length:
        ``lengths`` int32 [B] (rows of o past them are zeros), or packed
        sequences, the tensors [rows, heads, D], with ``offsets`` int32 [B + 1]
        and max_len the longest sequence's tokens (None: rows, at some cost).
        initial_state (None: zeros) and final_state (written, may be the
        initial one) are fp32 [B, H, Dk, Dv]."""
        (out,), state = self._attention(q, k, v, log_decay, scale, offsets, lengths, max_len, False,
                                        ((out, "out", "H", "Dv", stream),))
        a = self._desc_at
        s = a + _ATTENTION.size
        _check("prnn_linear_attention", self._lib.prnn_linear_attention(
            self._h, a, s, s + 32, s + 64, self._state(initial_state, "initial_state", state), s + 96,
            self._state(final_state, "final_state", state), self._stream(stream)))
        return out

    def linear_attention_backward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                                  grad_out: torch.Tensor, *, scale: Optional[float] = None,
                                  initial_state: Optional[torch.Tensor] = None,
                                  grad_final_state: Optional[torch.Tensor] = None,
                                  grad_initial_state: Optional[torch.Tensor] = None,
                                  offsets: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                                  max_len: Optional[int] = None, grad_q: Optional[torch.Tensor] = None,
                                  grad_k: Optional[torch.Tensor] = None, grad_v: Optional[torch.Tensor] = None,
                                  stream=None):
        """Gradients of linear_attention: (dq, dk, dv), and into grad_initial_state
        where it is given.  The inputs are those of the forward call; the decays
        are constants."""
        if grad_out is None:
            raise TypeError("grad_out must be a torch tensor")
        (_, *grads), state = self._attention(
            q, k, v, log_decay, scale, offsets, lengths, max_len, False,
            ((grad_out, "grad_out", "H", "Dv", None), (grad_q, "grad_q", "H", "Dk", stream),
             (grad_k, "grad_k", "Hkv", "Dk", stream), (grad_v, "grad_v", "Hkv", "Dv", stream)))
        a = self._desc_at
        s = a + _ATTENTION.size
        _check("prnn_linear_attention_backward", self._lib.prnn_linear_attention_backward(
            self._h, a, s, s + 32, s + 64, self._state(initial_state, "initial_state", state), s + 96,
            self._state(grad_final_state, "grad_final_state", state), s + 128, s + 160, s + 192,
            self._state(grad_initial_state, "grad_initial_state", state), self._stream(stream)))
        return tuple(grads)

    def linear_attention_step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                              state: torch.Tensor, *, scale: Optional[float] = None,
                              new_state: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
        """One new token of every sequence: q [B, H, Dk], k [B, Hkv, Dk], v [B, Hkv,
        Dv] give o [B, H, Dv].  state fp32 [B, H, Dk, Dv] is updated in place, or
        left as it is and the new one written to new_state."""
        (out,), shape = self._attention(q, k, v, log_decay, scale, None, None, None, True,
                                        ((out, "out", "H", "Dv", stream),))
        a = self._desc_at
        s = a + _ATTENTION.size
        s0 = self._dense(state, "state", torch.float32, shape)
        s1 = s0 if new_state is None else self._dense(new_state, "new_state", torch.float32, shape)
        _check("prnn_linear_attention_step", self._lib.prnn_linear_attention_step(
            self._h, a, s, s + 32, s + 64, s0, s + 96, s1, self._stream(stream)))
        return out

    # -- the gated delta rule -----------------------------------------------
    def _delta_rule(self, q, k, v, log_decay, beta, scale, offsets, lengths, max_len, step, outs):
        """As _attention: writes the descriptors of the rule, of q, k, v, log_decay
        and beta and of the sequences in `outs` (heads as q's or v's, head size or
        None for one fp32 value a head, tensor or None for a new one, name, stream, or
        ABSENT), and returns those tensors, the shape of the states and whether
        there is a log_decay."""
        lead = 1 if step or offsets is not None else 2
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor) or t.dim() != lead + 2:
                raise ValueError(f"{name} must have {lead + 2} axes")
        if not isinstance(beta, torch.Tensor):
            raise TypeError("beta must be a torch tensor")
        dtype = q.dtype
        code = SEQUENCE_TYPES.get(dtype)
        if code is None:
            raise TypeError(f"q must have dtype in {tuple(SEQUENCE_TYPES)}, got {dtype}")
        q_shape, v_shape = q.shape, v.shape
        Hk, Dk = q_shape[-2:]
        H, Dv = v_shape[-2:]
        n = q_shape[0]
        rows = q_shape[:-2]
        total, at_lengths, at_offsets = 0, 0, 0
        if step:
            B, T, token, batch = n, 1, -1, 0
        elif offsets is not None:
            if lengths is not None:
                raise ValueError("give offsets (packed sequences) or lengths, not both")
            if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
                raise ValueError("offsets must be [B + 1]")
            B, total, token, batch = offsets.shape[0] - 1, n, 0, -1
            T = total if max_len is None else max(-1, min(int(max_len), total))  # (longer than the rows: as long)
            at_offsets = self._dense(offsets, "offsets", torch.int32, (B + 1,))
        else:
            T, B, token, batch = n, q_shape[1], 0, 1
            if lengths is not None:
                at_lengths = self._dense(lengths, "lengths", torch.int32, (B,))
        rule = [B, min(T, 0x7fffffff), H, Hk, Dk, Dv, code, Dk ** -0.5 if scale is None else scale, at_lengths, at_offsets, total]
        wide, per_head = (*rows, H, Dv), (*rows, H)
        more_tokens, more_batch = token >= 0 and rows[token] > 1, batch >= 0 and rows[batch] > 1
        index, made = self._index, []

        def vectors(t, name, shape, heads):
            if (t.dtype != dtype or t.shape != shape or t.get_device() != index or (t.stride(-1) != 1 and shape[-1] > 1)):
                _need_strided(t, name, self.device, (dtype,), shape)
            s = t.stride()
            rule.extend((t.data_ptr(), s[token] if more_tokens else 0, s[batch] if more_batch else 0, s[-2] if heads > 1 else 0))

        def values(t, name):  # (one a token and head, at any strides)
            if (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.shape != per_head
                    or t.get_device() != index):
                _need_strided(t, name, self.device, (torch.float32,), per_head)
            s = t.stride()
            rule.extend((t.data_ptr(), s[token] if more_tokens else 0, s[batch] if more_batch else 0, s[-1] if H > 1 else 0))

        vectors(q, "q", q_shape, Hk)
        vectors(k, "k", q_shape, Hk)
        vectors(v, "v", wide, H)
        if log_decay is None:
            rule.extend(_NO_SEQUENCE)
        else:
            values(log_decay, "log_decay")
        values(beta, "beta")
        for kind, t, name, stream in outs:
            if kind == "values":
                if t is None:
                    if stream is ABSENT:
                        rule.extend(_NO_SEQUENCE)
                        made.append(None)
                        continue
                    t = _empty(q, per_head, torch.float32, stream)
                values(t, name)
            else:
                shape = q_shape if kind == "keys" else wide
                if t is None:
                    t = _empty(q, shape, dtype, stream)
                elif not isinstance(t, torch.Tensor):
                    raise TypeError(f"{name} must be a torch tensor")
                vectors(t, name, shape, shape[-2])
            made.append(t)
        (_DELTA_FORWARD if len(made) == 1 else _DELTA_BACKWARD).pack_into(self._desc, 0, *rule)
        return made, (B, H, Dk, Dv), log_decay is not None

    def gated_delta_rule(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: Optional[torch.Tensor],
                         beta: torch.Tensor, *, scale: Optional[float] = None,
                         initial_state: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                         offsets: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                         max_len: Optional[int] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Sd = exp(log_decay[t]) S[t-1], S[t] = Sd + beta[t] k[t] (v[t] - Sd^T k[t])^T, o[t] = scale S[t]^T q[t] for
        whole sequences.

        q and k [T, B, Hk, Dk], v [T, B, H, Dv] (fp32, fp16 or bf16; any strides
        with a contiguous last axis), log_decay (or None: no decay) and beta
        fp32 [T, B, H] (any strides) give o [T, B, H, Dv]; scale None: Dk **
        -0.5.  Sequences of unequal length (offsets, lengths, max_len) and states
        fp32 [B, H, Dk, Dv] as in linear_attention."""
        (out,), state, decays = self._delta_rule(q, k, v, log_decay, beta, scale, offsets, lengths, max_len, False,
                                                 (("rows", out, "out", stream),))
        a = self._desc_at
        s = a + _DELTA_RULE.size
        _check("prnn_gated_delta_rule", self._lib.prnn_gated_delta_rule(
            self._h, a, s, s + 32, s + 64, s + 96 if decays else None, s + 128,
            self._state(initial_state, "initial_state", state), s + 160,
            self._state(final_state, "final_state", state), self._stream(stream)))
        return out

    def gated_delta_rule_backward(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                  log_decay: Optional[torch.Tensor], beta: torch.Tensor, grad_out: torch.Tensor, *,
                                  scale: Optional[float] = None, initial_state: Optional[torch.Tensor] = None,
                                  grad_final_state: Optional[torch.Tensor] = None,
                                  grad_initial_state: Optional[torch.Tensor] = None,
                                  offsets: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                                  max_len: Optional[int] = None, grad_q: Optional[torch.Tensor] = None,
                                  grad_k: Optional[torch.Tensor] = None, grad_v: Optional[torch.Tensor] = None,
                                  grad_log_decay: Optional[torch.Tensor] = None,
                                  grad_beta: Optional[torch.Tensor] = None, stream=None):
        """Gradients of gated_delta_rule: (dq, dk, dv, dlog_decay, dbeta), and into
        grad_initial_state where it is given.  The inputs are those of the
        forward call; dlog_decay is None without a log_decay (unless
        grad_log_decay is given)."""
        if grad_out is None:
            raise TypeError("grad_out must be a torch tensor")
        (_, *grads), state, decays = self._delta_rule(
            q, k, v, log_decay, beta, scale, offsets, lengths, max_len, False,
            (("rows", grad_out, "grad_out", None), ("keys", grad_q, "grad_q", stream), ("keys", grad_k, "grad_k", stream),
             ("rows", grad_v, "grad_v", stream),
             ("values", grad_log_decay, "grad_log_decay", ABSENT if log_decay is None else stream),
             ("values", grad_beta, "grad_beta", stream)))
        a = self._desc_at
        s = a + _DELTA_RULE.size
        _check("prnn_gated_delta_rule_backward", self._lib.prnn_gated_delta_rule_backward(
            self._h, a, s, s + 32, s + 64, s + 96 if decays else None, s + 128,
            self._state(initial_state, "initial_state", state), s + 160,
            self._state(grad_final_state, "grad_final_state", state), s + 192, s + 224, s + 256,
            s + 288 if grads[3] is not None else None, s + 320,
            self._state(grad_initial_state, "grad_initial_state", state), self._stream(stream)))
        return tuple(grads)

    def gated_delta_rule_step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              log_decay: Optional[torch.Tensor], beta: torch.Tensor, state: torch.Tensor, *,
                              scale: Optional[float] = None, new_state: Optional[torch.Tensor] = None,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One new token of every sequence: q and k [B, Hk, Dk], v [B, H, Dv],
        log_decay (or None) and beta [B, H] give o [B, H, Dv].  state fp32 [B, H,
        Dk, Dv] is updated in place, or left as it is and the new one written
        to new_state."""
        (out,), shape, decays = self._delta_rule(q, k, v, log_decay, beta, scale, None, None, None, True,
                                                 (("rows", out, "out", stream),))
        a = self._desc_at
        s = a + _DELTA_RULE.size
        s0 = self._dense(state, "state", torch.float32, shape)
        s1 = s0 if new_state is None else self._dense(new_state, "new_state", torch.float32, shape)
        _check("prnn_gated_delta_rule_step", self._lib.prnn_gated_delta_rule_step(
            self._h, a, s, s + 32, s + 64, s + 96 if decays else None, s + 128, s0, s + 160, s1, self._stream(stream)))
        return out

    # -- layer norm -------------------------------------------------------------
    def _norm_rows(self, t, name, dtype, shape):
        """The rows of t [..., N]: how many, and the elements from one to the next."""
        strides = self._strided(t, name, dtype, shape)
        N = shape[-1]
        if len(shape) == 2:
            return (shape[0], strides[0]) if shape[0] > 1 else (shape[0], N)
        M, ld = 1, N
        for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
            if size == 1:
                continue
            if M == 1:
                ld = stride
            elif stride != ld * M and t.numel() > 0:
                raise ValueError(f"the rows of {name} must lie at one stride")
            M *= size
        return M, max(ld, N) if M <= 1 else ld

    def _norm_params(self, params, dtype, N):
        """Pointers of [N] parameters (None where absent), and their type's code."""
        ptype = None
        for p, name in params:
            if p is not None:
                ptype = p.dtype if ptype is None else ptype
                if ptype != dtype and ptype != torch.float32:
                    raise TypeError(f"{name} must have dtype in {(torch.float32, dtype)}, got {ptype}")
        ptype = torch.float32 if ptype is None else ptype
        return [None if p is None else self._dense(p, name, ptype, (N,)) for p, name in params], SEQUENCE_TYPES[ptype]

    def _norm_type(self, x):
        if not isinstance(x, torch.Tensor) or x.dtype not in SEQUENCE_TYPES or x.dim() < 1:
            raise TypeError(f"x must be a tensor with dtype in {tuple(SEQUENCE_TYPES)}")
        return SEQUENCE_TYPES[x.dtype]

    def layer_norm(self, x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, *, out: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """(x - mean) * rstd * weight + bias over the last axis of x (fp32, fp16 or
        bf16); weight and bias [N], fp32 or x's dtype, or None.  mean and rstd
        (fp32, x's shape without its last axis) are written where given, for
        the backward pass; out may be x."""
        code, shape = self._norm_type(x), x.shape
        M, ldx = self._norm_rows(x, "x", x.dtype, shape)
        (w, b), pcode = self._norm_params(((weight, "weight"), (bias, "bias")), x.dtype, shape[-1])
        m = None if mean is None else self._dense(mean, "mean", torch.float32, shape[:-1])
        r = None if rstd is None else self._dense(rstd, "rstd", torch.float32, shape[:-1])
        if out is None:
            out = _empty(x, shape, x.dtype, stream)
            ldy = shape[-1]
        else:
            _, ldy = self._norm_rows(out, "out", x.dtype, shape)
        _check("prnn_layer_norm", self._lib.prnn_layer_norm(
            self._h, M, shape[-1], code, x.data_ptr(), ldx, pcode, w, b, eps, out.data_ptr(), ldy, m, r,
            self._stream(stream)))
        return out

    def layer_norm_backward(self, grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                            weight: Optional[torch.Tensor] = None, *, grad_x: Optional[torch.Tensor] = None,
                            grad_weight: Optional[torch.Tensor] = None, grad_bias: Optional[torch.Tensor] = None,
                            stream=None):
        """Gradients of layer_norm: (dx, dweight, dbias).  dweight and dbias have
        weight's dtype; without a weight they are computed only into the
        buffers given, and are None otherwise."""
        code, shape = self._norm_type(x), x.shape
        N = shape[-1]
        M, ldx = self._norm_rows(x, "x", x.dtype, shape)
        _, lddy = self._norm_rows(grad_out, "grad_out", x.dtype, shape)
        m = self._dense(mean, "mean", torch.float32, shape[:-1])
        r = self._dense(rstd, "rstd", torch.float32, shape[:-1])
        if weight is not None:
            grad_weight = _empty(x, (N,), weight.dtype, stream) if grad_weight is None else grad_weight
            grad_bias = _empty(x, (N,), weight.dtype, stream) if grad_bias is None else grad_bias
        (w, dw, db), pcode = self._norm_params(
            ((weight, "weight"), (grad_weight, "grad_weight"), (grad_bias, "grad_bias")), x.dtype, N)
        if grad_x is None:
            grad_x = _empty(x, shape, x.dtype, stream)
            lddx = N
        else:
            _, lddx = self._norm_rows(grad_x, "grad_x", x.dtype, shape)
        _check("prnn_layer_norm_backward", self._lib.prnn_layer_norm_backward(
            self._h, M, N, code, grad_out.data_ptr(), lddy, x.data_ptr(), ldx, m, r, pcode, w, grad_x.data_ptr(), lddx,
            dw, db, self._stream(stream)))
        return grad_x, grad_weight, grad_bias

    # -- rms norm ---------------------------------------------------------------
    def _rms_norm(self, x, weight, eps, residual, sum_out, rstd, out_type, out_code, out, scales, group, stream):
        code, shape = self._norm_type(x), x.shape
        M, ldx = self._norm_rows(x, "x", x.dtype, shape)
        (w,), pcode = self._norm_params(((weight, "weight"),), x.dtype, shape[-1])
        ldr = lds = 0
        if residual is not None:
            _, ldr = self._norm_rows(residual, "residual", x.dtype, shape)
        if sum_out is not None:
            _, lds = self._norm_rows(sum_out, "sum_out", x.dtype, shape)
        r = None if rstd is None else self._dense(rstd, "rstd", torch.float32, shape[:-1])
        if out is None:
            out = _empty(x, shape, out_type, stream)
            ldy = shape[-1]
        else:
            _, ldy = self._norm_rows(out, "out", out_type, shape)
        _check("prnn_rms_norm", self._lib.prnn_rms_norm(
            self._h, M, shape[-1], code, x.data_ptr(), ldx, _ptr(residual), ldr, pcode, w, eps, _ptr(sum_out), lds,
            out_code if out_code is not None else code, out.data_ptr(), ldy, _ptr(scales), group, r, self._stream(stream)))
        return out

    def rms_norm(self, x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                 residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """s * rstd * weight with s = x + residual over the last axis of x (fp32, fp16
        or bf16); weight [N], fp32 or x's dtype, or None.  sum_out (of x's shape
        and dtype; may be x or residual) receives s, rstd (fp32, x's shape
        without its last axis) is written for the backward pass; out may be x
        or residual."""
        return self._rms_norm(x, weight, eps, residual, sum_out, rstd, x.dtype if isinstance(x, torch.Tensor) else None,
                              None, out, None, 0, stream)

    def rms_norm_e4m3(self, x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                      residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                      group: Optional[int] = None, out: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, stream=None):
        """rms_norm with an output in 8 bits: (out, scales), out torch.float8_e4m3fn
        of x's shape, to be multiplied by scales fp32, one for each row (x's
        shape without its last axis) or, with group=128, for each 128 columns (x's
        leading axes, then ceil(N / 128))."""
        if group not in (None, RMS_GROUP):
            raise ValueError(f"group must be None or {RMS_GROUP}, got {group}")
        self._norm_type(x)
        shape = x.shape[:-1] if group is None else (*x.shape[:-1], -(-x.shape[-1] // RMS_GROUP))
        if scales is None:
            scales = _empty(x, shape, torch.float32, stream)
        self._dense(scales, "scales", torch.float32, shape)
        return self._rms_norm(x, weight, eps, residual, sum_out, rstd, torch.float8_e4m3fn, DATA_E4M3, out, scales,
                              group or 0, stream), scales

    def rms_norm_backward(self, grad_out: torch.Tensor, x: torch.Tensor, rstd: torch.Tensor,
                          weight: Optional[torch.Tensor] = None, *, grad_sum: Optional[torch.Tensor] = None,
                          grad_x: Optional[torch.Tensor] = None, grad_weight: Optional[torch.Tensor] = None,
                          stream=None):
        """Gradients of rms_norm: (dx, dweight).  x is the sum that it stored (its x,
        without a residual), grad_sum the gradient that reaches that sum itself;
        dx is the gradient of x and of the residual.  dweight has weight's
        dtype; without a weight it is computed only into the buffer given, and
        is None otherwise."""
        code, shape = self._norm_type(x), x.shape
        N = shape[-1]
        M, ldx = self._norm_rows(x, "x", x.dtype, shape)
        _, lddy = self._norm_rows(grad_out, "grad_out", x.dtype, shape)
        ldds = self._norm_rows(grad_sum, "grad_sum", x.dtype, shape)[1] if grad_sum is not None else 0
        r = self._dense(rstd, "rstd", torch.float32, shape[:-1])
        if weight is not None and grad_weight is None:
            grad_weight = _empty(x, (N,), weight.dtype, stream)
        (w, dw), pcode = self._norm_params(((weight, "weight"), (grad_weight, "grad_weight")), x.dtype, N)
        if grad_x is None:
            grad_x = _empty(x, shape, x.dtype, stream)
            lddx = N
        else:
            _, lddx = self._norm_rows(grad_x, "grad_x", x.dtype, shape)
        _check("prnn_rms_norm_backward", self._lib.prnn_rms_norm_backward(
            self._h, M, N, code, grad_out.data_ptr(), lddy, x.data_ptr(), ldx, r, pcode, w, _ptr(grad_sum), ldds,
            grad_x.data_ptr(), lddx, dw, self._stream(stream)))
        return grad_x, grad_weight

    def sync_floor(self, N: int, B: int, T: int, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
        """The exchange/step protocol of a dense call without arithmetic."""
        if out is None:
            out = torch.empty((T, B, N), dtype=torch.float32, device=self.device)
        _need(out, "out", (torch.float32,), (T, B, N))
        _check("prnn_sync_floor", self._lib.prnn_sync_floor(self._h, N, B, T, out.data_ptr(), _stream_ptr(stream)))
        return out


_default_handles = {}


@atexit.register
def _close_default_handles():
    """Destroys the module's default handles at interpreter exit, before the
    HIP runtime and torch tear down (handlers run in reverse order of
    registration, and torch registers its own when it is imported, before
    this module's)."""
    while _default_handles:
        _, h = _default_handles.popitem()
        try:
            h.close()
        except Exception:
            pass


def default_handle() -> Handle:
    dev = torch.cuda.current_device()
    h = _default_handles.get(dev)
    if h is None:
        h = _default_handles[dev] = Handle()
    return h


def forward_dense(W, X, h0=None, out=None, stream=None):
    return default_handle().forward_dense(W, X, h0, out, stream)


def forward_sparse(col, val, X, h0=None, out=None, stream=None):
    return default_handle().forward_sparse(col, val, X, h0, out, stream)


NOALLOC_MAX_N = 2560  # PRNN_NOALLOC_MAX_N


def forward_dense_noalloc(W: torch.Tensor, X: torch.Tensor, h0: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """prnn_forward_dense_noalloc: the dense recurrence without a handle, on the
    library's fixed device array (nothing allocated by the library).  status:
    None or a one-element int32/uint32 device tensor, 0 after a good run."""
    lib = load_library()
    T, B, N = X.shape
    _need(W, "W", (torch.float32, torch.float16), (N, N))
    _need(X, "X", (torch.float32,), (T, B, N))
    if h0 is not None:
        _need(h0, "h0", (torch.float32,), (B, N))
    if out is None:
        out = torch.empty((T, B, N), dtype=torch.float32, device=X.device)
    _need(out, "out", (torch.float32,), (T, B, N))
    if status is not None:
        _need(status, "status", (torch.int32, torch.uint32), (1,))
    wt = DATA_FLOAT if W.dtype == torch.float32 else DATA_HALF
    st = lib.prnn_forward_dense_noalloc(N, B, T, wt, W.data_ptr(), X.data_ptr(),
                                        h0.data_ptr() if h0 is not None else None, out.data_ptr(),
                                        status.data_ptr() if status is not None else None, _stream_ptr(stream))
    _check("prnn_forward_dense_noalloc", st)
    return out
