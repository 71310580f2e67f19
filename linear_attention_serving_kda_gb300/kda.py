"""Python binding of the C ABI in include/kda.h (ctypes; marshalling only).

Each function has the name of its C entry point and passes device pointers
of torch tensors straight through; every step of the layer runs in the CUDA
library.  Loading fails loudly when the library has not been built: there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARGUMENT = 1
KDA_ERR_UNSUPPORTED_GEOMETRY = 2
KDA_ERR_INVALID_BOUND = 3
KDA_ERR_WORKSPACE = 4
KDA_ERR_LAUNCH = 5
KDA_ERR_DEVICE = 6
KDA_DEV_BAD_SEQLENS = 1
KDA_DEV_BAD_SLOT = 2
KDA_DEV_BAD_ACCEPTED = 4
KDA_DEV_TIMEOUT = 8
KDA_ACT_EXP = 0
KDA_ACT_RCP = 1
KDA_ACT_SIGMOID = 2
KDA_ACT_SILU = 3
KDA_DTYPE_F32 = 0
KDA_DTYPE_BF16 = 1
KDA_GATE_SOFTPLUS = 0
KDA_GATE_SAFE = 1
KDA_NORM_GATE_NONE = 0
KDA_NORM_GATE_SIGMOID = 1
KDA_NORM_GATE_SILU = 2
KDA_MAX_POOL_SLOTS = 262144
KDA_MAX_ROWS = 2147483000


class kda_params(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32), ("head_dim_k", ctypes.c_int32),
        ("head_dim_v", ctypes.c_int32), ("conv_kernel", ctypes.c_int32),
        ("gate_mode", ctypes.c_int32), ("gate_lower_bound", ctypes.c_float),
        ("l2_eps", ctypes.c_float), ("norm_eps", ctypes.c_float),
        ("scale", ctypes.c_float), ("io_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32), ("num_slots", ctypes.c_int32),
        ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
        ("conv_weight", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p),
    ]


class kda_gdn_params(ctypes.Structure):
    _fields_ = [
        ("num_heads_k", ctypes.c_int32), ("num_heads_v", ctypes.c_int32),
        ("head_dim_k", ctypes.c_int32), ("head_dim_v", ctypes.c_int32),
        ("l2_norm", ctypes.c_int32), ("l2_eps", ctypes.c_float), ("scale", ctypes.c_float),
        ("io_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("num_slots", ctypes.c_int32),
        ("q_row_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64), ("v_row_stride", ctypes.c_int64),
        ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
    ]


class kda_conv_params(ctypes.Structure):
    _fields_ = [
        ("channels", ctypes.c_int32), ("conv_kernel", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
        ("num_slots", ctypes.c_int32), ("conv_weight", ctypes.c_void_p),
    ]


class kda_norm_params(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32), ("post_norm", ctypes.c_int32), ("gate_act", ctypes.c_int32),
        ("residual_scale", ctypes.c_float), ("norm_eps", ctypes.c_float), ("io_dtype", ctypes.c_int32),
        ("res_dtype", ctypes.c_int32), ("post_weight", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
    ]


class kda_slot_pool(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p), ("layer_stride_bytes", ctypes.c_int64), ("slot_bytes", ctypes.c_int64),
        ("num_layers", ctypes.c_int32), ("num_slots", ctypes.c_int32),
    ]


_VP = ctypes.c_void_p
_I32 = ctypes.c_int32
_SIG = {
    "kda_prefill_varlen": (ctypes.c_int, [ctypes.POINTER(kda_params), _VP, _I32, _I32, _VP, _VP, _VP, _VP,
                                          _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP, _VP]),
    "kda_prefill_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(kda_params), _I32, _I32]),
    "kda_prefill_varlen_static_ws": (ctypes.c_int, [ctypes.POINTER(kda_params), _VP, _I32, _I32, _VP, _VP, _VP,
                                                    _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "kda_prefill_static_workspace_capacity": (ctypes.c_size_t, []),
    "kda_prefill_scan": (ctypes.c_int, [ctypes.POINTER(kda_params), _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP,
                                        _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _I32, _VP, _VP]),
    "kda_prefill_scan_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(kda_params), _I32, _I32, _I32]),
    "kda_debug_split_chains_only": (ctypes.c_int, [ctypes.POINTER(kda_params), _VP, _I32, _I32, _VP, _VP, _VP,
                                                   _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t,
                                                   _VP, ctypes.c_uint32, _VP]),
    "kda_debug_activations": (ctypes.c_int, [_I32, _VP, _VP, _I32, _VP]),
    "kda_decode": (ctypes.c_int, [ctypes.POINTER(kda_params), _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                  _VP, _VP, _VP, _VP, _VP]),
    "kda_verify_window": (ctypes.c_int, [ctypes.POINTER(kda_params), _I32, _I32, _VP, _VP, _VP, _VP, _VP,
                                         _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "kda_verify_log_bytes": (ctypes.c_size_t, [ctypes.POINTER(kda_params), _I32, _I32]),
    "kda_commit_verify": (ctypes.c_int, [ctypes.POINTER(kda_params), _I32, _I32] + [_VP] * 14 + [_VP]),
    "kda_commit": (ctypes.c_int, [ctypes.POINTER(kda_params), _I32, _I32, _VP, _VP, _VP, _VP, _VP,
                                  _VP, _VP]),
    "kda_gdn_prefill_varlen": (ctypes.c_int, [ctypes.POINTER(kda_gdn_params), _VP, _I32, _I32] + [_VP] * 9 +
                               [ctypes.c_size_t, _VP, _VP]),
    "kda_gdn_prefill_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(kda_gdn_params), _I32, _I32]),
    "kda_gdn_decode": (ctypes.c_int, [ctypes.POINTER(kda_gdn_params), _I32] + [_VP] * 9 + [_VP]),
    "kda_conv_varlen": (ctypes.c_int, [ctypes.POINTER(kda_conv_params), _VP, _I32, _I32] + [_VP] * 6),
    "kda_conv_decode": (ctypes.c_int, [ctypes.POINTER(kda_conv_params), _I32] + [_VP] * 6),
    "kda_block_norm": (ctypes.c_int, [ctypes.POINTER(kda_norm_params), ctypes.c_int64] + [_VP] * 6),
    "kda_slots_copy": (ctypes.c_int, [ctypes.POINTER(kda_slot_pool), _I32] + [_VP] * 4),
    "kda_slots_zero": (ctypes.c_int, [ctypes.POINTER(kda_slot_pool), _I32] + [_VP] * 3),
    "kda_slots_compact_plan": (ctypes.c_int, [ctypes.POINTER(kda_slot_pool)] + [_VP] * 5),
    "kda_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kda_abi_version": (ctypes.c_int, []),
}

_lib = None


def load(path: Optional[str] = None):
    """Load libkda.so (raises if it is missing)."""
    global _lib
    if _lib is None:
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"KDA CUDA library not built: {p} is missing "
                               "(run linear_attention_serving_kda_gb300.build.build())")
        lib = ctypes.CDLL(p)
        for name, (res, args) in _SIG.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


class KdaError(RuntimeError):
    def __init__(self, rc: int):
        super().__init__(f"{status_string(rc)} ({rc})")
        self.rc = rc


def status_string(rc: int) -> str:
    return load().kda_status_string(rc).decode()


def check(rc: int) -> None:
    if rc != KDA_OK:
        raise KdaError(rc)


@dataclass
class Params:
    """Layer configuration; the four parameter tensors live on the device."""

    num_heads: int
    head_dim: int
    conv_kernel: int
    gate_mode: int
    A_log: object
    dt_bias: object
    conv_weight: object
    norm_weight: object = None
    gate_lower_bound: float = -5.0
    l2_eps: float = 1e-6
    norm_eps: float = 1e-6
    scale: float = 1.0
    io_dtype: int = KDA_DTYPE_BF16
    out_dtype: int = KDA_DTYPE_BF16
    num_slots: int = 1
    head_dim_v: Optional[int] = None

    def c_struct(self) -> kda_params:
        return kda_params(
            num_heads=self.num_heads, head_dim_k=self.head_dim,
            head_dim_v=self.head_dim if self.head_dim_v is None else self.head_dim_v,
            conv_kernel=self.conv_kernel, gate_mode=self.gate_mode,
            gate_lower_bound=self.gate_lower_bound, l2_eps=self.l2_eps,
            norm_eps=self.norm_eps, scale=self.scale, io_dtype=self.io_dtype,
            out_dtype=self.out_dtype, num_slots=self.num_slots,
            A_log=_ptr(self.A_log), dt_bias=_ptr(self.dt_bias),
            conv_weight=_ptr(self.conv_weight), norm_weight=_ptr(self.norm_weight))


@dataclass
class GdnParams:
    """Heads of the gated delta rule with one decay per head (kda_gdn_params)."""

    num_heads_k: int
    num_heads_v: int
    head_dim_k: int
    head_dim_v: int
    A_log: object
    dt_bias: object
    l2_norm: bool = True
    l2_eps: float = 1e-6
    scale: float = 1.0
    io_dtype: int = KDA_DTYPE_BF16
    out_dtype: int = KDA_DTYPE_BF16
    num_slots: int = 1
    q_row_stride: int = 0
    k_row_stride: int = 0
    v_row_stride: int = 0

    def c_struct(self) -> kda_gdn_params:
        return kda_gdn_params(
            num_heads_k=self.num_heads_k, num_heads_v=self.num_heads_v, head_dim_k=self.head_dim_k,
            head_dim_v=self.head_dim_v, l2_norm=int(self.l2_norm), l2_eps=self.l2_eps, scale=self.scale,
            io_dtype=self.io_dtype, out_dtype=self.out_dtype, num_slots=self.num_slots,
            q_row_stride=self.q_row_stride, k_row_stride=self.k_row_stride, v_row_stride=self.v_row_stride,
            A_log=_ptr(self.A_log), dt_bias=_ptr(self.dt_bias))


@dataclass
class ConvParams:
    """A causal depthwise convolution with SiLU (kda_conv_params)."""

    channels: int
    conv_kernel: int
    conv_weight: object
    io_dtype: int = KDA_DTYPE_BF16
    num_slots: int = 1

    def c_struct(self) -> kda_conv_params:
        return kda_conv_params(channels=self.channels, conv_kernel=self.conv_kernel, io_dtype=self.io_dtype,
                               num_slots=self.num_slots, conv_weight=_ptr(self.conv_weight))


@dataclass
class NormParams:
    """The norms around a block (kda_norm_params)."""

    dim: int
    post_norm: bool = True
    gate_act: int = KDA_NORM_GATE_NONE
    residual_scale: float = 1.0
    norm_eps: float = 1e-6
    post_weight: object = None
    pre_weight: object = None
    io_dtype: int = KDA_DTYPE_BF16
    res_dtype: int = KDA_DTYPE_BF16

    def c_struct(self) -> kda_norm_params:
        return kda_norm_params(
            dim=self.dim, post_norm=int(self.post_norm), gate_act=self.gate_act, residual_scale=self.residual_scale,
            norm_eps=self.norm_eps, io_dtype=self.io_dtype, res_dtype=self.res_dtype,
            post_weight=_ptr(self.post_weight), pre_weight=_ptr(self.pre_weight))


@dataclass
class SlotPool:
    """A pool of state slots over layers (kda_slot_pool)."""

    pool: object
    num_layers: int
    num_slots: int
    slot_bytes: int
    layer_stride_bytes: int

    def c_struct(self) -> kda_slot_pool:
        return kda_slot_pool(pool=_ptr(self.pool), layer_stride_bytes=self.layer_stride_bytes,
                             slot_bytes=self.slot_bytes, num_layers=self.num_layers, num_slots=self.num_slots)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def kda_prefill_workspace_bytes(params: Params, N: int, T: int) -> int:
    return load().kda_prefill_workspace_bytes(ctypes.byref(params.c_struct()), N, T)


def kda_verify_log_bytes(params: Params, B: int, W: int) -> int:
    return load().kda_verify_log_bytes(ctypes.byref(params.c_struct()), B, W)


def kda_prefill_varlen(params: Params, cu_seqlens, N: int, T: int, q, k, v, gate, beta, out_gate,
                       slots, conv_state, rec_state, out, workspace=None, ws_bytes: int = 0,
                       dev_status=None, stream=None) -> int:
    return load().kda_prefill_varlen(
        ctypes.byref(params.c_struct()), _ptr(cu_seqlens), N, T, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
        _ptr(beta), _ptr(out_gate), _ptr(slots), _ptr(conv_state), _ptr(rec_state), _ptr(out),
        _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))


def kda_prefill_varlen_static_ws(params: Params, cu_seqlens, N: int, T: int, q, k, v, gate, beta, out_gate,
                                 slots, conv_state, rec_state, out, dev_status=None, stream=None) -> int:
    """kda_prefill_varlen with the library's built-in scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    return load().kda_prefill_varlen_static_ws(
        ctypes.byref(params.c_struct()), _ptr(cu_seqlens), N, T, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
        _ptr(beta), _ptr(out_gate), _ptr(slots), _ptr(conv_state), _ptr(rec_state), _ptr(out),
        _ptr(dev_status), _stream(stream))


def kda_prefill_scan(params: Params, cu_seqlens, N: int, T: int, q, k, v, gate, beta, out_gate, slots,
                     conv_state, rec_state, out, workspace, ws_bytes: int, segments: int, dev_status=None,
                     stream=None) -> int:
    return load().kda_prefill_scan(
        ctypes.byref(params.c_struct()), _ptr(cu_seqlens), N, T, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
        _ptr(beta), _ptr(out_gate), _ptr(slots), _ptr(conv_state), _ptr(rec_state), _ptr(out),
        _ptr(workspace), ws_bytes, segments, _ptr(dev_status), _stream(stream))


def kda_prefill_scan_workspace_bytes(params: Params, N: int, T: int, segments: int) -> int:
    return load().kda_prefill_scan_workspace_bytes(ctypes.byref(params.c_struct()), N, T, segments)


def kda_debug_split_chains_only(params: Params, cu_seqlens, N: int, T: int, q, k, v, gate, beta, out_gate,
                                slots, conv_state, rec_state, out, workspace, ws_bytes: int, dev_status,
                                poll_limit: int, stream=None) -> int:
    """Test hook: the split path's chains without producers, flag waits
    limited to poll_limit polls (they run out and report KDA_DEV_TIMEOUT)."""
    return load().kda_debug_split_chains_only(
        ctypes.byref(params.c_struct()), _ptr(cu_seqlens), N, T, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
        _ptr(beta), _ptr(out_gate), _ptr(slots), _ptr(conv_state), _ptr(rec_state), _ptr(out),
        _ptr(workspace), ws_bytes, _ptr(dev_status), poll_limit, _stream(stream))


def kda_debug_activations(which: int, x, y, n: int, stream=None) -> int:
    """Test hook: y[i] = f(x[i]) with the kernels' shared activation f
    (KDA_ACT_EXP, KDA_ACT_RCP, KDA_ACT_SIGMOID, KDA_ACT_SILU)."""
    return load().kda_debug_activations(which, _ptr(x), _ptr(y), n, _stream(stream))


def kda_prefill_static_workspace_capacity() -> int:
    return load().kda_prefill_static_workspace_capacity()


def kda_decode(params: Params, B: int, q, k, v, gate, beta, out_gate, slots, conv_state, rec_state,
               out, dev_status=None, stream=None) -> int:
    return load().kda_decode(
        ctypes.byref(params.c_struct()), B, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta),
        _ptr(out_gate), _ptr(slots), _ptr(conv_state), _ptr(rec_state), _ptr(out), _ptr(dev_status),
        _stream(stream))


def kda_verify_window(params: Params, B: int, W: int, q, k, v, gate, beta, out_gate, slots,
                      conv_state, rec_state, log, out, dev_status=None, stream=None) -> int:
    return load().kda_verify_window(
        ctypes.byref(params.c_struct()), B, W, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta),
        _ptr(out_gate), _ptr(slots), _ptr(conv_state), _ptr(rec_state), _ptr(log), _ptr(out),
        _ptr(dev_status), _stream(stream))


def kda_commit(params: Params, B: int, W: int, accepted, slots, log, conv_state, rec_state,
               dev_status=None, stream=None) -> int:
    return load().kda_commit(
        ctypes.byref(params.c_struct()), B, W, _ptr(accepted), _ptr(slots), _ptr(log),
        _ptr(conv_state), _ptr(rec_state), _ptr(dev_status), _stream(stream))


def kda_commit_verify(params: Params, B: int, W: int, accepted, log_prev, q, k, v, gate, beta, out_gate,
                      slots, conv_state, rec_state, log, out, dev_status=None, stream=None) -> int:
    """Commit the previous window's accepted rows, then verify a new window."""
    return load().kda_commit_verify(
        ctypes.byref(params.c_struct()), B, W, _ptr(accepted), _ptr(log_prev), _ptr(q), _ptr(k), _ptr(v),
        _ptr(gate), _ptr(beta), _ptr(out_gate), _ptr(slots), _ptr(conv_state), _ptr(rec_state), _ptr(log),
        _ptr(out), _ptr(dev_status), _stream(stream))


def kda_gdn_prefill_workspace_bytes(params: GdnParams, N: int, T: int) -> int:
    return load().kda_gdn_prefill_workspace_bytes(ctypes.byref(params.c_struct()), N, T)


def kda_gdn_prefill_varlen(params: GdnParams, cu_seqlens, N: int, T: int, q, k, v, gate, beta, slots, rec_state, out,
                           workspace=None, ws_bytes: int = 0, dev_status=None, stream=None) -> int:
    """Prompt rows through the gated delta rule with one decay per head."""
    return load().kda_gdn_prefill_varlen(
        ctypes.byref(params.c_struct()), _ptr(cu_seqlens), N, T, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta),
        _ptr(slots), _ptr(rec_state), _ptr(out), _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))


def kda_gdn_decode(params: GdnParams, B: int, q, k, v, gate, beta, slots, rec_state, out, dev_status=None,
                   stream=None) -> int:
    """One row per sequence through the gated delta rule with one decay per head."""
    return load().kda_gdn_decode(
        ctypes.byref(params.c_struct()), B, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(slots),
        _ptr(rec_state), _ptr(out), _ptr(dev_status), _stream(stream))


def kda_conv_varlen(params: ConvParams, cu_seqlens, N: int, T: int, x, slots, conv_state, y, dev_status=None,
                    stream=None) -> int:
    """Causal depthwise convolution with carried state and SiLU over prompt rows."""
    return load().kda_conv_varlen(ctypes.byref(params.c_struct()), _ptr(cu_seqlens), N, T, _ptr(x), _ptr(slots),
                                  _ptr(conv_state), _ptr(y), _ptr(dev_status), _stream(stream))


def kda_conv_decode(params: ConvParams, B: int, x, slots, conv_state, y, dev_status=None, stream=None) -> int:
    """The same for one row per sequence."""
    return load().kda_conv_decode(ctypes.byref(params.c_struct()), B, _ptr(x), _ptr(slots), _ptr(conv_state), _ptr(y),
                                  _ptr(dev_status), _stream(stream))


def kda_block_norm(params: NormParams, rows: int, y, gate=None, residual=None, h_out=None, x_out=None,
                   stream=None) -> int:
    """Norm after a block with its gate, scaled residual, norm before the next block."""
    return load().kda_block_norm(ctypes.byref(params.c_struct()), rows, _ptr(y), _ptr(gate), _ptr(residual),
                                 _ptr(h_out), _ptr(x_out), _stream(stream))


def kda_slots_copy(pool: SlotPool, n: int, src, dst, dev_status=None, stream=None) -> int:
    """Copies slot src[i] to slot dst[i] in every layer of the pool."""
    return load().kda_slots_copy(ctypes.byref(pool.c_struct()), n, _ptr(src), _ptr(dst), _ptr(dev_status),
                                 _stream(stream))


def kda_slots_zero(pool: SlotPool, n: int, slots, dev_status=None, stream=None) -> int:
    """Zeroes slots in every layer of the pool."""
    return load().kda_slots_zero(ctypes.byref(pool.c_struct()), n, _ptr(slots), _ptr(dev_status), _stream(stream))


def kda_slots_compact_plan(pool: SlotPool, live, src, dst, remap, stream=None) -> int:
    """The moves (for kda_slots_copy) that close the holes of a pool."""
    return load().kda_slots_compact_plan(ctypes.byref(pool.c_struct()), _ptr(live), _ptr(src), _ptr(dst), _ptr(remap),
                                         _stream(stream))


class Prepared:
    """A call of one entry point with its arguments marshalled once.

    ``Prepared("kda_decode", params, B, q, ...)()`` calls the C function with
    the same pointers every time (the tensors must stay alive and in place).
    """

    def __init__(self, name: str, params, *args, stream=None):
        self.fn = getattr(load(), name)
        self.pstruct = params.c_struct()
        conv = []
        for a in args:
            if a is None or isinstance(a, int):
                conv.append(a)
            else:
                conv.append(a.data_ptr())
        self.args = (ctypes.byref(self.pstruct), *conv, _stream(stream))

    def __call__(self) -> int:
        return self.fn(*self.args)
