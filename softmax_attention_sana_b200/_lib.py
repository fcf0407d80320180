"""ctypes binding of libsana (include/sana.h).

Argument marshalling only: every step of the attention path runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  If libsana.so is missing the import fails loudly; there is no
fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
from ctypes import (POINTER, Structure, c_char_p, c_double, c_float, c_int, c_longlong, c_size_t,
                    c_void_p)

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsana.so")

SANA_OK, SANA_ERR_INVALID_ARG, SANA_ERR_UNSUPPORTED, SANA_ERR_WORKSPACE, SANA_ERR_CUDA, \
    SANA_ERR_TIMEOUT = range(6)
SANA_F32, SANA_BF16 = 0, 1
EPI_NONE, EPI_SILU, EPI_RESIDUAL = 0, 1, 2
STATUS_NAMES = {0: "SANA_OK", 1: "SANA_ERR_INVALID_ARG", 2: "SANA_ERR_UNSUPPORTED",
                3: "SANA_ERR_WORKSPACE", 4: "SANA_ERR_CUDA", 5: "SANA_ERR_TIMEOUT"}


class SanaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Shape(Structure):
    _fields_ = [("B", c_int), ("T", c_int), ("H", c_int), ("W", c_int), ("heads", c_int),
                ("head_dim", c_int), ("t_offset", c_int)]


class RopeStruct(Structure):
    _fields_ = [("cos_t", c_void_p), ("sin_t", c_void_p), ("cos_h", c_void_p), ("sin_h", c_void_p),
                ("cos_w", c_void_p), ("sin_w", c_void_p), ("n_t", c_int), ("n_h", c_int),
                ("n_w", c_int), ("T_total", c_int), ("H", c_int), ("W", c_int)]


class StackConfig(Structure):
    _fields_ = [("layers", c_int), ("block_span", c_int), ("ratio", c_int), ("use_attnres", c_int),
                ("ffn_mult", c_int), ("eps", c_float), ("rms_eps", c_float),
                ("anchor_scale", c_float), ("anchor_keep_tiles", c_int),
                ("mx_projections", c_int)]


class StackWeights(Structure):
    _fields_ = [("w_qkvg", POINTER(c_void_p)), ("w_o", POINTER(c_void_p)),
                ("w_up", POINTER(c_void_p)), ("w_down", POINTER(c_void_p)),
                ("w_attn", c_void_p), ("w_ffn", c_void_p),
                ("mx_qkvg", POINTER(c_void_p)), ("mx_qkvg_scales", POINTER(c_void_p)),
                ("mx_o", POINTER(c_void_p)), ("mx_o_scales", POINTER(c_void_p)),
                ("mx_up", POINTER(c_void_p)), ("mx_up_scales", POINTER(c_void_p)),
                ("mx_down", POINTER(c_void_p)), ("mx_down_scales", POINTER(c_void_p))]


class StackWsLayout(Structure):
    _fields_ = [("x_hat", c_size_t), ("q", c_size_t), ("k", c_size_t), ("v", c_size_t),
                ("g", c_size_t), ("attn", c_size_t), ("ffn", c_size_t), ("num_blocks", c_int),
                ("blocks", c_size_t * 16)]


class RotaryScaling(Structure):
    _fields_ = [("kind", c_int), ("factor", c_double), ("original", c_int), ("beta_fast", c_double),
                ("beta_slow", c_double), ("attention_factor", c_double)]


class RotaryStruct(Structure):
    _fields_ = [("table", c_void_p), ("max_positions", c_int), ("rotary_dim", c_int),
                ("layout", c_int)]


class QkShape(Structure):
    _fields_ = [("B", c_int), ("N", c_int), ("heads", c_int), ("kv_heads", c_int),
                ("head_dim", c_int), ("q_stride", c_longlong), ("k_stride", c_longlong)]


class QkPositions(Structure):
    _fields_ = [("rotary", POINTER(RotaryStruct)), ("rope", POINTER(RopeStruct)), ("T", c_int),
                ("H", c_int), ("W", c_int), ("positions", c_void_p), ("offset", c_int)]


class WindowShape(Structure):
    _fields_ = [("B", c_int), ("N", c_int), ("N_keys", c_int), ("heads", c_int), ("kv_heads", c_int),
                ("head_dim", c_int), ("q_stride", c_longlong), ("k_stride", c_longlong),
                ("v_stride", c_longlong), ("gate_stride", c_longlong), ("window", c_int),
                ("sinks", c_int), ("block", c_int), ("lengths", c_void_p), ("scale", c_float)]


class WindowDecodeShape(Structure):
    _fields_ = [("B", c_int), ("N", c_int), ("heads", c_int), ("kv_heads", c_int),
                ("head_dim", c_int), ("capacity", c_int), ("window", c_int), ("sinks", c_int),
                ("scale", c_float)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libsana.so not built ({LIB_PATH}); run softmax_attention_sana_b200/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "sana_version": (c_char_p, []),
        "sana_last_error_string": (c_char_p, []),
        "sana_rope_tables_count": (c_size_t, [c_int] * 6),
        "sana_rope_tables_host": (c_int, [c_int] * 6 + [c_double, c_void_p]),
        "sana_rope_bind": (c_int, [c_void_p] + [c_int] * 6 + [POINTER(RopeStruct)]),
        "sana_linattn_workspace_size": (c_size_t, [POINTER(Shape), c_int]),
        "sana_linattn_fwd": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                     POINTER(RopeStruct), c_float, c_void_p, c_void_p, c_size_t,
                                     c_void_p]),
        "sana_linattn_state_workspace_size": (c_size_t, [POINTER(Shape), c_int]),
        "sana_linattn_state": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p,
                                       POINTER(RopeStruct), c_void_p, c_void_p, c_void_p, c_size_t,
                                       c_void_p]),
        "sana_linattn_apply": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p,
                                       POINTER(RopeStruct), c_void_p, c_void_p, c_float, c_void_p,
                                       c_void_p]),
        "sana_linattn_block_causal_step": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p,
                                                   c_void_p, c_void_p, POINTER(RopeStruct), c_float,
                                                   c_void_p, c_void_p, c_int, c_void_p, c_void_p,
                                                   c_size_t, c_void_p]),
        "sana_linattn_block_causal_scan_workspace_size": (c_size_t, [POINTER(Shape), c_int, c_int]),
        "sana_linattn_block_causal_scan": (c_int, [POINTER(Shape), c_int, c_int, c_void_p, c_void_p,
                                                   c_void_p, c_void_p, POINTER(RopeStruct),
                                                   c_float, c_void_p, c_void_p, c_int, c_void_p,
                                                   c_void_p, c_size_t, c_void_p]),
        "sana_linattn_bwd_workspace_size": (c_size_t, [POINTER(Shape), c_int]),
        "sana_linattn_bwd": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                     POINTER(RopeStruct), c_float, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
        "sana_linattn_bwd_saved_state": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p,
                                                 c_void_p, c_void_p, POINTER(RopeStruct), c_float,
                                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                                 c_void_p, c_void_p, c_void_p, c_size_t,
                                                 c_void_p]),
        "sana_softmax_anchor_workspace_size": (c_size_t, [POINTER(Shape), c_int]),
        "sana_softmax_anchor_fwd": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p, c_void_p,
                                            c_void_p, POINTER(RopeStruct), c_float, c_void_p,
                                            c_void_p, c_size_t, c_void_p]),
        "sana_rope_apply": (c_int, [POINTER(Shape), c_int, c_void_p, POINTER(RopeStruct), c_float,
                                    c_void_p, c_void_p]),
        "sana_softmax_anchor_rotated_fwd": (c_int, [POINTER(Shape), c_void_p, c_void_p, c_void_p,
                                                    c_void_p, c_void_p, c_void_p]),
        "sana_softmax_anchor_sparse_workspace_size": (c_size_t, [POINTER(Shape), c_int]),
        "sana_softmax_anchor_sparse_fwd": (c_int, [POINTER(Shape), c_int, c_void_p, c_void_p,
                                                   c_void_p, c_void_p, POINTER(RopeStruct),
                                                   c_float, c_int, c_void_p, c_int, c_void_p,
                                                   c_void_p, c_size_t, c_void_p]),
        "sana_attnres_route": (c_int, [c_int, c_longlong, c_int, c_int, POINTER(c_void_p), c_int,
                                       c_void_p, c_float, c_void_p, c_void_p, c_void_p]),
        "sana_attnres_route_bwd_workspace_size": (c_size_t, [c_int, c_longlong, c_int]),
        "sana_attnres_route_bwd": (c_int, [c_int, c_longlong, c_int, c_int, POINTER(c_void_p),
                                           c_int, c_void_p, c_float, c_void_p, POINTER(c_void_p),
                                           c_void_p, c_void_p, c_size_t, c_void_p]),
        "sana_gemm_bf16": (c_int, [c_longlong, c_int, c_int, c_void_p, c_longlong, c_void_p,
                                   c_void_p, c_longlong, c_int, c_void_p]),
        "sana_rmsnorm": (c_int, [c_longlong, c_int, c_int, c_void_p, c_float, c_void_p, c_void_p]),
        "sana_hybrid_stack_workspace_size": (c_size_t, [POINTER(Shape), POINTER(StackConfig)]),
        "sana_hybrid_stack_workspace_layout": (c_int, [POINTER(Shape), POINTER(StackConfig),
                                                       POINTER(StackWsLayout)]),
        "sana_hybrid_stack_fwd": (c_int, [POINTER(Shape), POINTER(StackConfig),
                                          POINTER(StackWeights), POINTER(RopeStruct), c_void_p,
                                          c_void_p, c_void_p, c_size_t, c_void_p]),
        "sana_mx_scale_bytes": (c_size_t, [c_longlong, c_int]),
        "sana_mx_quantize": (c_int, [c_void_p, c_longlong, c_int, c_int, c_void_p, c_void_p,
                                     c_void_p]),
        "sana_mx_gemm": (c_int, [c_longlong, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_longlong, c_int, c_void_p]),
        "sana_mx_linear_workspace_size": (c_size_t, [c_longlong, c_int]),
        "sana_mx_linear": (c_int, [c_longlong, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_longlong, c_int, c_void_p, c_size_t, c_void_p]),
        "sana_rotary_table": (c_int, [c_int, c_int, c_double, POINTER(RotaryScaling), c_void_p,
                                      c_void_p]),
        "sana_rotary_apply": (c_int, [POINTER(QkShape), c_int, POINTER(QkPositions), c_int, c_void_p,
                                      c_void_p, c_float, c_void_p, c_void_p, c_void_p]),
        "sana_qk_norm_rope": (c_int, [POINTER(QkShape), c_int, POINTER(QkPositions), c_void_p,
                                      c_void_p, c_void_p, c_void_p, c_float, c_float, c_void_p,
                                      c_void_p, c_void_p]),
        "sana_qk_norm_rope_bwd_workspace_size": (c_size_t, [POINTER(QkShape)]),
        "sana_qk_norm_rope_bwd": (c_int, [POINTER(QkShape), c_int, POINTER(QkPositions), c_void_p,
                                          c_void_p, c_void_p, c_void_p, c_float, c_float, c_void_p,
                                          c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                          c_void_p, c_size_t, c_void_p]),
        "sana_window_anchor_fwd": (c_int, [POINTER(WindowShape), c_void_p, c_void_p, c_void_p,
                                           c_void_p, c_void_p, c_void_p, c_void_p]),
        "sana_window_anchor_bwd_workspace_size": (c_size_t, [POINTER(WindowShape), c_int]),
        "sana_window_anchor_bwd": (c_int, [POINTER(WindowShape)] + [c_void_p] * 12 + [c_size_t,
                                                                                      c_void_p]),
        "sana_window_anchor_decode_workspace_size": (c_size_t, [POINTER(WindowDecodeShape)]),
        "sana_window_anchor_decode": (c_int, [POINTER(WindowDecodeShape)] + [c_void_p] * 9 +
                                      [c_size_t, c_void_p]),
        "sana_sync_status": (c_int, [c_void_p]),
        "sana_selftest_bounded_wait": (c_int, [ctypes.c_uint, c_void_p]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def last_error() -> str:
    return lib.sana_last_error_string().decode()


def check(status: int):
    if status != SANA_OK:
        raise SanaError(status, last_error())


# ---------------------------------------------------------------- helpers

def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream():
    return c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SANA_BF16
    if t.dtype == torch.float32:
        return SANA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def make_shape(B, grid, heads, head_dim, t_offset=0) -> Shape:
    T, H, W = grid
    return Shape(B, T, H, W, heads, head_dim, t_offset)


class Rope:
    """Device copy of the 3D RoPE tables for frames [0, T_total) of an H x W grid."""

    def __init__(self, T_total, H, W, split, theta=10000.0, device="cuda"):
        n_t, n_h, n_w = split
        n = lib.sana_rope_tables_count(T_total, H, W, n_t, n_h, n_w)
        host = torch.empty(max(n, 1), dtype=torch.float32)
        check(lib.sana_rope_tables_host(T_total, H, W, n_t, n_h, n_w, theta, c_void_p(host.data_ptr())))
        self.host = host
        self.tables = host.to(device)
        self.struct = RopeStruct()
        check(lib.sana_rope_bind(c_void_p(self.tables.data_ptr()), T_total, H, W, n_t, n_h, n_w,
                                 ctypes.byref(self.struct)))
        self.T_total, self.H, self.W, self.split = T_total, H, W, tuple(split)


def host_rope_tables(T_total, H, W, split, theta=10000.0) -> torch.Tensor:
    """The six fp32 tables as the library computes them on the host."""
    n_t, n_h, n_w = split
    n = lib.sana_rope_tables_count(T_total, H, W, n_t, n_h, n_w)
    host = torch.empty(max(n, 1), dtype=torch.float32)
    check(lib.sana_rope_tables_host(T_total, H, W, n_t, n_h, n_w, theta, c_void_p(host.data_ptr())))
    return host[:n]


# ---------------------------------------------------------------- linear attention

def linattn_workspace_size(B, grid, heads, head_dim, dtype_code) -> int:
    s = make_shape(B, grid, heads, head_dim)
    return lib.sana_linattn_workspace_size(ctypes.byref(s), dtype_code)


def linattn_state_workspace_size(B, grid, heads, head_dim, dtype_code) -> int:
    s = make_shape(B, grid, heads, head_dim)
    return lib.sana_linattn_state_workspace_size(ctypes.byref(s), dtype_code)


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def linattn_fwd(q, k, v, gate, rope: Rope, grid, heads, eps=1e-6, out=None, ws=None):
    """Gated bidirectional ReLU linear attention with RoPE after the ReLU."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n)
    if gate is not None:
        _need(gate, "gate")
    B, N, C = q.shape
    D = C // heads
    dt = _dtype_code(q)
    s = make_shape(B, grid, heads, D)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = _ws(lib.sana_linattn_workspace_size(ctypes.byref(s), dt), q.device)
    check(lib.sana_linattn_fwd(ctypes.byref(s), dt, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
                               ctypes.byref(rope.struct), eps, _ptr(out), _ptr(ws), ws.numel(),
                               _stream()))
    return out


def linattn_state(k, v, rope: Rope, grid, heads, S=None, z=None, ws=None):
    """S = sum_j RoPE(phi K_j)^T V_j (B, heads, D, D) and z = sum_j phi K_j (B, heads, D), fp32."""
    _need(k, "k")
    _need(v, "v")
    B, N, C = k.shape
    D = C // heads
    dt = _dtype_code(k)
    s = make_shape(B, grid, heads, D)
    if S is None:
        S = torch.empty(B, heads, D, D, dtype=torch.float32, device=k.device)
    if z is None:
        z = torch.empty(B, heads, D, dtype=torch.float32, device=k.device)
    if ws is None:
        ws = _ws(lib.sana_linattn_state_workspace_size(ctypes.byref(s), dt), k.device)
    check(lib.sana_linattn_state(ctypes.byref(s), dt, _ptr(k), _ptr(v), ctypes.byref(rope.struct),
                                 _ptr(S), _ptr(z), _ptr(ws), ws.numel(), _stream()))
    return S, z


def linattn_apply(q, gate, rope: Rope, grid, heads, S, z, eps=1e-6, out=None):
    """Y = sigmoid(G) * RoPE(phi Q) S / (phi Q . z + eps) for a given state."""
    _need(q, "q")
    B, N, C = q.shape
    D = C // heads
    s = make_shape(B, grid, heads, D)
    if out is None:
        out = torch.empty_like(q)
    check(lib.sana_linattn_apply(ctypes.byref(s), _dtype_code(q), _ptr(q), _ptr(gate),
                                 ctypes.byref(rope.struct), _ptr(S), _ptr(z), eps, _ptr(out),
                                 _stream()))
    return out


def linattn_block_causal_step(q, k, v, gate, rope: Rope, grid, t_offset, heads, state_S, state_z,
                              commit=True, eps=1e-6, out=None, ws=None):
    """One block-causal chunk; state_S (B, heads, D, D) / state_z (B, heads, D) fp32 in place."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (state_S, "state_S"), (state_z, "state_z")):
        _need(t, n)
    B, N, C = q.shape
    D = C // heads
    dt = _dtype_code(q)
    s = make_shape(B, grid, heads, D, t_offset)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = _ws(lib.sana_linattn_workspace_size(ctypes.byref(s), dt), q.device)
    check(lib.sana_linattn_block_causal_step(
        ctypes.byref(s), dt, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), ctypes.byref(rope.struct), eps,
        _ptr(state_S), _ptr(state_z), int(bool(commit)), _ptr(out), _ptr(ws), ws.numel(), _stream()))
    return out


def linattn_bwd(q, k, v, gate, rope: Rope, grid, heads, dy, eps=1e-6, ws=None, S=None, z=None):
    """Gradients (dq, dk, dv, dgate) of the gated linear-attention layer for dY
    (dgate is None for the ungated layer).  bf16.  S, z: the forward's state
    as linattn_state returned it for these k, v (then it is not rebuilt)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dy, "dy")):
        _need(t, n)
    if (S is None) != (z is None):
        raise ValueError("linattn_bwd: give both S and z or neither")
    B, N, C = q.shape
    D = C // heads
    dt = _dtype_code(q)
    s = make_shape(B, grid, heads, D)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = None if gate is None else torch.empty_like(gate)
    if ws is None:
        ws = _ws(lib.sana_linattn_bwd_workspace_size(ctypes.byref(s), dt), q.device)
    if S is None:
        check(lib.sana_linattn_bwd(
            ctypes.byref(s), dt, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), ctypes.byref(rope.struct),
            eps, _ptr(dy), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ws), ws.numel(), _stream()))
    else:
        check(lib.sana_linattn_bwd_saved_state(
            ctypes.byref(s), dt, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), ctypes.byref(rope.struct),
            eps, _ptr(S), _ptr(z), _ptr(dy), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ws),
            ws.numel(), _stream()))
    return dq, dk, dv, dg


def linattn_block_causal_scan_workspace_size(B, grid, heads, D, chunk_frames, dtype_code,
                                             t_offset=0) -> int:
    s = make_shape(B, grid, heads, D, t_offset)
    return lib.sana_linattn_block_causal_scan_workspace_size(ctypes.byref(s), chunk_frames,
                                                             dtype_code)


def linattn_block_causal_scan(q, k, v, gate, rope: Rope, grid, t_offset, heads, chunk_frames,
                              state_S, state_z, commit=True, eps=1e-6, out=None, ws=None):
    """A whole sequence of blocks of chunk_frames frames (the last block takes the
    remaining frames); state_S / state_z fp32 in place as for the block step."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (state_S, "state_S"), (state_z, "state_z")):
        _need(t, n)
    B, N, C = q.shape
    D = C // heads
    dt = _dtype_code(q)
    s = make_shape(B, grid, heads, D, t_offset)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = _ws(lib.sana_linattn_block_causal_scan_workspace_size(ctypes.byref(s), chunk_frames,
                                                                   dt), q.device)
    check(lib.sana_linattn_block_causal_scan(
        ctypes.byref(s), chunk_frames, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
        ctypes.byref(rope.struct), eps, _ptr(state_S), _ptr(state_z), int(bool(commit)), _ptr(out),
        _ptr(ws), ws.numel(), _stream()))
    return out


# ---------------------------------------------------------------- anchor

def softmax_anchor_fwd(q, k, v, gate, rope, grid, heads, scale=0.0, out=None, ws=None):
    """Gated bidirectional softmax attention with 3D RoPE on Q, K (rope may be None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n)
    B, N, C = q.shape
    D = C // heads
    dt = _dtype_code(q)
    s = make_shape(B, grid, heads, D)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = _ws(lib.sana_softmax_anchor_workspace_size(ctypes.byref(s), dt), q.device)
    check(lib.sana_softmax_anchor_fwd(
        ctypes.byref(s), dt, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
        None if rope is None else ctypes.byref(rope.struct), scale, _ptr(out), _ptr(ws), ws.numel(),
        _stream()))
    return out


def rope_apply(x, rope, grid, heads, mul=1.0, out=None):
    """out = mul * RoPE(x) for a (B, N, C) tensor (rope may be None: no rotation)."""
    _need(x, "x")
    B, N, C = x.shape
    s = make_shape(B, grid, heads, C // heads)
    if out is None:
        out = torch.empty_like(x)
    check(lib.sana_rope_apply(ctypes.byref(s), _dtype_code(x), _ptr(x),
                              None if rope is None else ctypes.byref(rope.struct), mul, _ptr(out),
                              _stream()))
    return out


def softmax_anchor_rotated_fwd(q_rot, k_rot, v, gate, grid, heads, out=None):
    """The anchor's attention phase on rotated operands (bf16): Q' = scale *
    log2(e) * RoPE(Q), K' = RoPE(K) as rope_apply writes them."""
    for t, n in ((q_rot, "q_rot"), (k_rot, "k_rot"), (v, "v")):
        _need(t, n)
    B, N, C = q_rot.shape
    s = make_shape(B, grid, heads, C // heads)
    if out is None:
        out = torch.empty_like(v)
    check(lib.sana_softmax_anchor_rotated_fwd(ctypes.byref(s), _ptr(q_rot), _ptr(k_rot), _ptr(v),
                                              _ptr(gate), _ptr(out), _stream()))
    return out


def anchor_tile_count(N: int) -> int:
    """Key tiles of 128 tokens; query blocks are pairs of them."""
    return (N + 127) // 128


def softmax_anchor_sparse_workspace_size(B, grid, heads, head_dim) -> int:
    s = make_shape(B, grid, heads, head_dim)
    return lib.sana_softmax_anchor_sparse_workspace_size(ctypes.byref(s), SANA_BF16)


def softmax_anchor_sparse_fwd(q, k, v, gate, rope, grid, heads, keep_tiles, tiles=None,
                              select=True, scale=0.0, out=None, ws=None):
    """Block-sparse gated softmax anchor (bf16).  With select, the library picks
    the keep_tiles key tiles of every 256-query block and writes them into
    `tiles` (allocated if None); without, the given int32 tiles
    [B, heads, n_blocks, keep_tiles] are used.  Returns (out, tiles)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n)
    B, N, C = q.shape
    D = C // heads
    dt = _dtype_code(q)
    s = make_shape(B, grid, heads, D)
    nt = anchor_tile_count(N)
    if tiles is None:
        tiles = torch.empty(B, heads, (nt + 1) // 2, keep_tiles, dtype=torch.int32, device=q.device)
    _need(tiles, "tiles")
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = _ws(lib.sana_softmax_anchor_sparse_workspace_size(ctypes.byref(s), dt), q.device)
    check(lib.sana_softmax_anchor_sparse_fwd(
        ctypes.byref(s), dt, _ptr(q), _ptr(k), _ptr(v), _ptr(gate),
        None if rope is None else ctypes.byref(rope.struct), scale, keep_tiles, _ptr(tiles),
        int(bool(select)), _ptr(out), _ptr(ws), ws.numel(), _stream()))
    return out, tiles


# ---------------------------------------------------------------- rotary positions, q/k norm

ROTARY_INTERLEAVED, ROTARY_HALF = 0, 1
_LAYOUTS = {"interleaved": ROTARY_INTERLEAVED, "half": ROTARY_HALF}
_SCALINGS = {"linear": 1, "ntk": 2, "yarn": 3}


def _c_int(*values):
    """Refuses what ctypes would cut to 32 bits."""
    for v in values:
        if not -0x80000000 <= v <= 0x7fffffff:
            raise ValueError(f"{v} does not fit a C int")


class Rotary:
    """Device table of rotary (cos, sin) for positions [0, max_positions): rotary_dim elements of a
    head are turned (the rest pass through), paired "interleaved" (2j, 2j + 1) or "half" (j, j +
    rotary_dim / 2).  scaling: None, ("linear", factor), ("ntk", factor) or ("yarn", factor,
    original_positions[, beta_fast, beta_slow, attention_factor]).  8 bytes a position and pair."""

    def __init__(self, max_positions, rotary_dim, theta=10000.0, layout="interleaved", scaling=None,
                 device="cuda"):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, not {layout!r}")
        sc = None
        if scaling is not None:
            kind, *rest = scaling
            if kind not in _SCALINGS or not 1 <= len(rest) <= (5 if kind == "yarn" else 1) or \
                    (kind == "yarn" and len(rest) < 2):
                raise ValueError(f"bad rotary scaling {scaling!r}")
            factor, original, fast, slow, att = (list(rest) + [0, 32.0, 1.0, 0.0][len(rest) - 1:])
            _c_int(original)
            sc = RotaryScaling(_SCALINGS[kind], factor, original, fast, slow, att)
        _c_int(max_positions, rotary_dim)
        self.max_positions, self.rotary_dim, self.layout = max_positions, rotary_dim, layout
        self.table = torch.empty(max(max_positions, 1), max(rotary_dim // 2, 1), 2,
                                 dtype=torch.float32, device=device)
        with torch.cuda.device(self.table.device):
            check(lib.sana_rotary_table(max_positions, rotary_dim, theta,
                                        None if sc is None else ctypes.byref(sc), _ptr(self.table),
                                        _stream()))
            if not torch.cuda.is_current_stream_capturing():  # any stream may use the table from here on
                torch.cuda.current_stream().synchronize()
        self.struct = RotaryStruct(self.table.data_ptr(), max_positions, rotary_dim, _LAYOUTS[layout])
        self.pointer = ctypes.pointer(self.struct)


def _same_device(first, *others):
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"tensors on {first.device} and {t.device} in one call")


def _call_on(t, fn, *args):
    """fn(*args, stream) on t's device and its current stream, checked."""
    index = t.get_device()
    if index == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != SANA_OK:
        raise SanaError(status, last_error())


def _addr(t):
    return None if t is None else t.data_ptr()


def _ws_args(ws, t):
    """Address and bytes of a caller's workspace for a call on t."""
    _need(ws, "ws")
    _same_device(t, ws)
    return ws.data_ptr(), ws.nbytes


def _token_stride(t, name, width):
    """Elements between the tokens of a (B, N, width) tensor whose rows are contiguous and whose
    sequences follow each other at the same stride (a slice of a packed projection is one)."""
    if not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a CUDA tensor (B, N, {width})")
    B, N, C = t.shape
    seq, step, unit = t.stride()
    if C != width or (unit != 1 and C > 1):
        raise ValueError(f"{name} must be a CUDA tensor (B, N, {width}) with contiguous rows")
    if B * N <= 1:
        return width
    if N > 1:
        if B > 1 and seq != N * step:
            raise ValueError(f"{name}: sequences must follow each other at the tokens' stride")
    else:
        step = seq
    if step < width:  # (0, of an expanded tensor, would stand for the row's width)
        raise ValueError(f"{name}: its tokens need rows of their own, {width} elements apart or more")
    return step


def _qk_call(q, k, rotary, heads, kv_heads, positions, offset, grid):
    """The shape and position structs of a call (and what they point to)."""
    if q.dim() != 3 or heads < 1 or q.shape[2] % heads:
        raise ValueError(f"q must be (B, N, heads * head_dim) with heads={heads}")
    B, N, C = q.shape
    D = C // heads
    if (k is None) != (kv_heads == 0):
        raise ValueError("k is None exactly where kv_heads is 0")
    k_stride = 0
    if k is not None:
        k_stride = _token_stride(k, "k", kv_heads * D)
        Bk, Nk, _ = k.shape
        if k.dtype is not q.dtype or Bk != B or Nk != N:
            raise ValueError("q and k must have one dtype and the same (B, N)")
    _c_int(offset, *(grid or ()))
    s = QkShape(B, N, heads, kv_heads, D, _token_stride(q, "q", C), k_stride)
    at_positions = None
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.shape != (B, N) or \
                not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int32 tensor (B, N)")
        at_positions = positions.data_ptr()
    if isinstance(rotary, Rotary):
        if grid is not None:
            raise ValueError("grid goes with a Rope")
        at, table = QkPositions(rotary.pointer, None, 0, 0, 0, at_positions, offset), rotary.table
    else:
        if grid is None:
            raise ValueError("a Rope needs the tokens' grid=(T, H, W)")
        at = QkPositions(None, ctypes.pointer(rotary.struct), *grid, at_positions, offset)
        table = rotary.tables
    _same_device(q, k, positions, table)
    return s, at


def _norm_weight(w, name, q, D):
    if w is None:
        return
    _need(w, name)
    if w.dtype != torch.float32 or w.shape != (D,):
        raise ValueError(f"{name} must be fp32 ({D},)")
    _same_device(q, w)


def _out_like(out, name, q, width):
    """A contiguous (B, N, width) tensor like q: `out`, checked, or a new one."""
    if out is None:
        if q.is_contiguous() and q.shape[2] == width:
            return torch.empty_like(q)
        return q.new_empty((*q.shape[:2], width))
    B, N, _ = q.shape
    _need(out, name)
    if out.dtype is not q.dtype or out.shape != (B, N, width):
        raise ValueError(f"{name} must be {q.dtype} {(B, N, width)}")
    _same_device(q, out)
    return out


def rotary_apply(q, k, rotary, heads, kv_heads, positions=None, offset=0, grid=None, inverse=False,
                 q_mul=1.0, q_out=None, k_out=None):
    """(q_mul * R q, R k): the rotation of every head at its token's position -- offset + n, offset +
    positions[b, n], or the (T, H, W) grid of a Rope.  inverse: the transposed rotation (the
    gradient).  k is None with kv_heads 0 (then k_out is None).  bf16 or fp32."""
    s, at = _qk_call(q, k, rotary, heads, kv_heads, positions, offset, grid)
    q_out = _out_like(q_out, "q_out", q, heads * s.head_dim)
    k_out = None if k is None else _out_like(k_out, "k_out", k, kv_heads * s.head_dim)
    _call_on(q, lib.sana_rotary_apply, s, _dtype_code(q), at, int(bool(inverse)), q.data_ptr(),
             _addr(k), q_mul, q_out.data_ptr(), _addr(k_out))
    return q_out, k_out


def qk_norm_rope(q, k, q_weight, k_weight, rotary, heads, kv_heads, positions=None, offset=0,
                 grid=None, eps=1e-6, q_mul=1.0, q_out=None, k_out=None):
    """RMS norm of every query and key head (weights fp32 (head_dim,), None = ones) and the rotation
    of rotary_apply, in one pass."""
    s, at = _qk_call(q, k, rotary, heads, kv_heads, positions, offset, grid)
    _norm_weight(q_weight, "q_weight", q, s.head_dim)
    _norm_weight(k_weight, "k_weight", q, s.head_dim)
    q_out = _out_like(q_out, "q_out", q, heads * s.head_dim)
    k_out = None if k is None else _out_like(k_out, "k_out", k, kv_heads * s.head_dim)
    _call_on(q, lib.sana_qk_norm_rope, s, _dtype_code(q), at, q.data_ptr(), _addr(k),
             _addr(q_weight), _addr(k_weight), eps, q_mul, q_out.data_ptr(), _addr(k_out))
    return q_out, k_out


def qk_norm_rope_bwd_workspace_size(B, N, head_dim) -> int:
    _c_int(B, N, head_dim)
    s = QkShape(B, N, 1, 0, head_dim, 0, 0)
    return lib.sana_qk_norm_rope_bwd_workspace_size(ctypes.byref(s))


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, rotary, heads, kv_heads,
                     positions=None, offset=0, grid=None, eps=1e-6, q_mul=1.0, ws=None):
    """Gradients (dq, dk, d_q_weight, d_k_weight) of qk_norm_rope for its outputs' gradients; a
    weight that is None has its gradient (that of ones) all the same, keys that are None none."""
    s, at = _qk_call(q, k, rotary, heads, kv_heads, positions, offset, grid)
    D = s.head_dim
    _norm_weight(q_weight, "q_weight", q, D)
    _norm_weight(k_weight, "k_weight", q, D)
    dq_out = _out_like(dq_out, "dq_out", q, heads * D)
    if (dk_out is None) != (k is None):
        raise ValueError("dk_out goes with k")
    dk_out = None if k is None else _out_like(dk_out, "dk_out", k, kv_heads * D)
    dq = _out_like(None, "dq", q, heads * D)
    dk = None if k is None else _out_like(None, "dk", k, kv_heads * D)
    dwq = torch.empty(D, dtype=torch.float32, device=q.device)
    dwk = None if k is None else torch.empty_like(dwq)
    if ws is None:
        ws = _ws(lib.sana_qk_norm_rope_bwd_workspace_size(ctypes.byref(s)), q.device)
    _call_on(q, lib.sana_qk_norm_rope_bwd, s, _dtype_code(q), at, q.data_ptr(), _addr(k),
             _addr(q_weight), _addr(k_weight), eps, q_mul, dq_out.data_ptr(), _addr(dk_out),
             dq.data_ptr(), _addr(dk), dwq.data_ptr(), _addr(dwk), *_ws_args(ws, q))
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------- windowed anchor

def _window_shape(q, k, v, gate, heads, kv_heads, window, sinks, block, lengths, scale):
    """The shape struct of a call on q, gate (B, N, heads * 128) and k, v (B, N_keys, kv_heads * 128)."""
    bf16 = torch.bfloat16
    if q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16 or \
            (gate is not None and gate.dtype is not bf16):
        raise TypeError("q, k, v and gate must be bfloat16")
    if q.dim() != 3 or k.dim() != 3 or heads < 1 or q.shape[2] % heads:
        raise ValueError(f"q must be (B, N, heads * head_dim) with heads={heads}, k (B, N_keys, ...)")
    B, N, C = q.shape
    D = C // heads
    ck = kv_heads * D
    strides = (_token_stride(q, "q", C), _token_stride(k, "k", ck), _token_stride(v, "v", ck),
               0 if gate is None else _token_stride(gate, "gate", C))
    if k.shape != v.shape or k.shape[0] != B:
        raise ValueError("q, k and v must have one batch size, k and v one length")
    if gate is not None and gate.shape != q.shape:
        raise ValueError("gate must have q's shape")
    at_lengths = None
    if lengths is not None:
        if lengths.dtype is not torch.int32 or lengths.shape != (B,) or not lengths.is_contiguous():
            raise ValueError("lengths must be a contiguous int32 tensor (B,)")
        at_lengths = lengths.data_ptr()
    _c_int(window, sinks, block)
    _same_device(q, k, v, gate, lengths)
    return WindowShape(B, N, k.shape[1], heads, kv_heads, D, *strides, window, sinks, block,
                       at_lengths, scale)


def window_anchor_fwd(q, k, v, gate, heads, kv_heads, window, sinks=0, block=1, lengths=None,
                      scale=0.0, out=None, lse=None, want_lse=False):
    """Gated softmax attention over a sliding window and the first `sinks` tokens (bf16, head_dim
    128; rotate q and k first).  The N queries are the last of k's N_keys positions; one at position
    p sees key j iff j < min(e, length) and (j >= e - window or j < sinks), e = (p // block + 1) *
    block; window 0: no limit.  gate may be None, lengths (B,) int32 or None.  Returns out, or (out,
    lse) with lse (B, heads, N) fp32."""
    s = _window_shape(q, k, v, gate, heads, kv_heads, window, sinks, block, lengths, scale)
    out = _out_like(out, "out", q, q.shape[2])
    if lse is None and want_lse:
        lse = torch.empty(s.B, heads, s.N, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse")
        _same_device(q, lse)
        if lse.dtype != torch.float32 or lse.shape != (s.B, heads, s.N):
            raise ValueError("lse must be fp32 (B, heads, N)")
    _call_on(q, lib.sana_window_anchor_fwd, s, q.data_ptr(), k.data_ptr(), v.data_ptr(),
             _addr(gate), out.data_ptr(), _addr(lse))
    return out if lse is None else (out, lse)


def window_anchor_bwd_workspace_size(B, N, N_keys, heads, kv_heads, window, sinks=0, block=1,
                                     gated=False, head_dim=128) -> int:
    _c_int(B, N, N_keys, heads, kv_heads, window, sinks, block, head_dim)
    s = WindowShape(B, N, N_keys, heads, kv_heads, head_dim, 0, 0, 0, 0, window, sinks, block, None, 0.0)
    return lib.sana_window_anchor_bwd_workspace_size(ctypes.byref(s), int(bool(gated)))


def window_anchor_bwd(q, k, v, gate, out, lse, dy, heads, kv_heads, window, sinks=0, block=1,
                      lengths=None, scale=0.0, ws=None):
    """Gradients (dq, dk, dv, dgate) of window_anchor_fwd for dY, given its inputs, out and lse
    (dgate is None without a gate)."""
    s = _window_shape(q, k, v, gate, heads, kv_heads, window, sinks, block, lengths, scale)
    out, dy = _out_like(out, "out", q, q.shape[2]), _out_like(dy, "dy", q, q.shape[2])
    _need(lse, "lse")
    _same_device(q, lse)
    if lse.dtype != torch.float32 or lse.shape != (s.B, heads, s.N):
        raise ValueError("lse must be fp32 (B, heads, N)")
    dq = _out_like(None, "dq", q, q.shape[2])
    dk, dv = _out_like(None, "dk", k, k.shape[2]), _out_like(None, "dv", v, v.shape[2])
    dg = None if gate is None else _out_like(None, "dgate", q, q.shape[2])
    if s.N == 0:  # no queries: nothing reaches the keys
        return dq, dk.zero_(), dv.zero_(), dg
    if ws is None:
        ws = _ws(lib.sana_window_anchor_bwd_workspace_size(ctypes.byref(s), int(gate is not None)), q.device)
    _call_on(q, lib.sana_window_anchor_bwd, s, q.data_ptr(), k.data_ptr(), v.data_ptr(),
             _addr(gate), out.data_ptr(), lse.data_ptr(), dy.data_ptr(), dq.data_ptr(),
             dk.data_ptr(), dv.data_ptr(), _addr(dg), *_ws_args(ws, q))
    return dq, dk, dv, dg


def window_anchor_decode_workspace_size(B, N, heads, kv_heads, capacity, window, sinks=0,
                                        head_dim=128) -> int:
    _c_int(B, N, heads, kv_heads, capacity, window, sinks, head_dim)
    s = WindowDecodeShape(B, N, heads, kv_heads, head_dim, capacity, window, sinks, 0.0)
    return lib.sana_window_anchor_decode_workspace_size(ctypes.byref(s))


def window_anchor_decode(q, k, v, gate, k_cache, v_cache, lengths, heads, kv_heads, window, sinks=0,
                         scale=0.0, out=None, ws=None):
    """One step of the N newest tokens of every sequence: writes k, v (B, N, kv_heads * 128) into the
    ring caches (B, capacity, kv_heads * 128) at positions lengths[b] + n and attends over the sinks
    and the window (bf16).  Position p lives in slot p while p < capacity, then in slot sinks + (p -
    sinks) % (capacity - sinks).  lengths (B,) int32 is left as it is; a negative one is an empty
    batch entry (nothing written, zeros out)."""
    for t in (q, k, v, gate, k_cache, v_cache):
        if t is not None:
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("q, k, v, gate and the caches must be contiguous CUDA tensors")
            if t.dtype is not torch.bfloat16:
                raise TypeError("q, k, v, gate and the caches must be bfloat16")
    if q.dim() != 3 or k_cache.dim() != 3 or heads < 1 or q.shape[2] % heads:
        raise ValueError(f"q must be (B, N, heads * head_dim) with heads={heads}, caches (B, capacity, ...)")
    B, N, C = q.shape
    D = C // heads
    ck = kv_heads * D
    if k.shape != (B, N, ck) or v.shape != k.shape or (gate is not None and gate.shape != q.shape):
        raise ValueError("k and v must be (B, N, kv_heads * head_dim), gate like q")
    capacity = k_cache.shape[1]
    if k_cache.shape != (B, capacity, ck) or v_cache.shape != k_cache.shape:
        raise ValueError("the caches must be (B, capacity, kv_heads * head_dim)")
    if lengths.dtype is not torch.int32 or lengths.shape != (B,) or not lengths.is_contiguous():
        raise ValueError("lengths must be a contiguous int32 tensor (B,)")
    _c_int(window, sinks)
    _same_device(q, k, v, gate, k_cache, v_cache, lengths)
    s = WindowDecodeShape(B, N, heads, kv_heads, D, capacity, window, sinks, scale)
    out = _out_like(out, "out", q, C)
    if ws is None:
        need = lib.sana_window_anchor_decode_workspace_size(s)
        ws = _ws(need, q.device) if need else None  # most steps of small batches need none
    _call_on(q, lib.sana_window_anchor_decode, s, q.data_ptr(), k.data_ptr(), v.data_ptr(),
             _addr(gate), k_cache.data_ptr(), v_cache.data_ptr(), lengths.data_ptr(),
             out.data_ptr(), *((None, 0) if ws is None else _ws_args(ws, q)))
    return out


# ---------------------------------------------------------------- AttnRes, norm, GEMM

def attnres_route(sources, w, rms_eps=1e-6, out=None, alpha=None, want_alpha=False):
    """h = sum_i softmax_i(w . RMSNorm(v_i)) v_i over (B, N, C) sources."""
    for i, t in enumerate(sources):
        _need(t, f"sources[{i}]")
    _need(w, "w")
    B, N, C = sources[0].shape
    dt = _dtype_code(sources[0])
    if out is None:
        out = torch.empty_like(sources[0])
    if want_alpha and alpha is None:
        alpha = torch.empty(B, N, len(sources), dtype=torch.float32, device=sources[0].device)
    arr = (c_void_p * len(sources))(*[t.data_ptr() for t in sources])
    check(lib.sana_attnres_route(B, N, C, dt, arr, len(sources), _ptr(w), rms_eps, _ptr(out),
                                 _ptr(alpha), _stream()))
    return (out, alpha) if want_alpha else out


def attnres_route_bwd(sources, w, dh, rms_eps=1e-6, ws=None):
    """Gradients (list of d sources, d w) of attnres_route for dh.  bf16 sources."""
    for i, t in enumerate(sources):
        _need(t, f"sources[{i}]")
    _need(w, "w")
    _need(dh, "dh")
    B, N, C = sources[0].shape
    dt = _dtype_code(sources[0])
    grads = [torch.empty_like(t) for t in sources]
    dw = torch.empty(C, dtype=torch.float32, device=w.device)
    if ws is None:
        ws = _ws(lib.sana_attnres_route_bwd_workspace_size(B, N, C), w.device)
    src = (c_void_p * len(sources))(*[t.data_ptr() for t in sources])
    dst = (c_void_p * len(grads))(*[t.data_ptr() for t in grads])
    check(lib.sana_attnres_route_bwd(B, N, C, dt, src, len(sources), _ptr(w), rms_eps, _ptr(dh),
                                     dst, _ptr(dw), _ptr(ws), ws.numel(), _stream()))
    return grads, dw


def rmsnorm(x, eps=1e-6, out=None):
    _need(x, "x")
    C = x.shape[-1]
    rows = x.numel() // C
    if out is None:
        out = torch.empty_like(x)
    check(lib.sana_rmsnorm(rows, C, _dtype_code(x), _ptr(x), eps, _ptr(out), _stream()))
    return out


def gemm_bf16(A, W, out=None, epilogue=EPI_NONE):
    """out = epilogue(A . W^T), A (M, K) bf16, W (N, K) bf16, fp32 accumulation."""
    M, K = A.shape[-2] if A.dim() == 2 else A.numel() // A.shape[-1], A.shape[-1]
    N = W.shape[0]
    if out is None:
        out = torch.empty(*A.shape[:-1], N, dtype=torch.bfloat16, device=A.device)
    check(lib.sana_gemm_bf16(M, N, K, _ptr(A), A.stride(-2) if A.dim() >= 2 else K, _ptr(W),
                             _ptr(out), out.stride(-2) if out.dim() >= 2 else N, epilogue, _stream()))
    return out


# ---------------------------------------------------------------- stack

def stack_config(layers, block_span=8, ratio=4, use_attnres=True, ffn_mult=3, eps=1e-6,
                 rms_eps=1e-6, anchor_scale=0.0, anchor_keep_tiles=0,
                 mx_projections=False) -> StackConfig:
    return StackConfig(layers, block_span, ratio, int(bool(use_attnres)), ffn_mult, eps, rms_eps,
                       anchor_scale, anchor_keep_tiles, int(bool(mx_projections)))


def mx_quantize_stack_weights(weights):
    """Per-layer weight dicts with the MX form of every projection weight added
    (keys '<name>_mxq' codes and '<name>_mxs' scales), as the stack reads them
    with mx_projections on."""
    out = []
    for d in weights:
        e = dict(d)
        for key in ("qkvg", "o", "up", "down"):
            if key in d:
                e[key + "_mxq"], e[key + "_mxs"] = mx_quantize(d[key], fp4=True)
        out.append(e)
    return out


def hybrid_stack_fwd(x, weights, w_attn, w_ffn, rope: Rope, grid, heads, cfg: StackConfig,
                     out=None, ws=None):
    _need(x, "x")
    B, N, C = x.shape
    s = make_shape(B, grid, heads, C // heads)
    L = cfg.layers

    def arr(key):
        if cfg.ffn_mult == 0 and key.split("_")[0] in ("up", "down"):
            return None
        if any(key not in weights[l] for l in range(L)):
            return None
        return (c_void_p * L)(*[weights[l][key].data_ptr() for l in range(L)])

    names = ("qkvg", "o", "up", "down")
    keep = {k: arr(k) for k in names + tuple(n + sfx for n in names for sfx in ("_mxq", "_mxs"))}
    p = lambda a: None if a is None else ctypes.cast(a, POINTER(c_void_p))
    sw = StackWeights(
        p(keep["qkvg"]), p(keep["o"]), p(keep["up"]), p(keep["down"]),
        None if w_attn is None else w_attn.data_ptr(), None if w_ffn is None else w_ffn.data_ptr(),
        p(keep["qkvg_mxq"]), p(keep["qkvg_mxs"]), p(keep["o_mxq"]), p(keep["o_mxs"]),
        p(keep["up_mxq"]), p(keep["up_mxs"]), p(keep["down_mxq"]), p(keep["down_mxs"]))
    if out is None:
        out = torch.empty_like(x)
    if ws is None:
        ws = _ws(lib.sana_hybrid_stack_workspace_size(ctypes.byref(s), ctypes.byref(cfg)), x.device)
    check(lib.sana_hybrid_stack_fwd(ctypes.byref(s), ctypes.byref(cfg), ctypes.byref(sw),
                                    ctypes.byref(rope.struct), _ptr(x), _ptr(out), _ptr(ws),
                                    ws.numel(), _stream()))
    return out


def hybrid_stack_workspace_size(B, grid, heads, cfg: StackConfig, head_dim=128) -> int:
    s = make_shape(B, grid, heads, head_dim)
    return lib.sana_hybrid_stack_workspace_size(ctypes.byref(s), ctypes.byref(cfg))


def hybrid_stack_workspace_views(ws, B, grid, heads, cfg: StackConfig, head_dim=128) -> dict:
    """Views of the stack's intermediates inside its workspace `ws` (a uint8
    tensor) after a call: keys x_hat, q, k, v, g, attn, ffn (absent when
    ffn_mult is 0) and blocks (list), each (B, N, width) bf16."""
    s = make_shape(B, grid, heads, head_dim)
    lay = StackWsLayout()
    check(lib.sana_hybrid_stack_workspace_layout(ctypes.byref(s), ctypes.byref(cfg),
                                                 ctypes.byref(lay)))
    N = grid[0] * grid[1] * grid[2]
    C = heads * head_dim

    def view(off, width):
        nbytes = B * N * width * 2
        return ws[off:off + nbytes].view(torch.bfloat16).view(B, N, width)

    out = {k: view(getattr(lay, k), C) for k in ("x_hat", "q", "k", "v", "g", "attn")}
    if cfg.ffn_mult > 0:
        out["ffn"] = view(lay.ffn, cfg.ffn_mult * C)
    out["blocks"] = [view(lay.blocks[i], C) for i in range(lay.num_blocks)]
    return out


# ---------------------------------------------------------------- MX projection GEMM

def mx_quantize(x, fp4=False):
    """MX quantisation of a bf16 (rows, K) tensor along K: returns (codes,
    scales) as uint8 tensors -- E4M3 codes (rows, K), or E2M1 codes packed two
    per byte (rows, K/2) with fp4, and the E8M0 scale atoms."""
    _need(x, "x")
    K = x.shape[-1]
    rows = x.numel() // K
    q = torch.empty(rows, K // 2 if fp4 else K, dtype=torch.uint8, device=x.device)
    sf = torch.empty(max(int(lib.sana_mx_scale_bytes(rows, K)), 16), dtype=torch.uint8,
                     device=x.device)
    check(lib.sana_mx_quantize(_ptr(x), rows, K, int(bool(fp4)), _ptr(q), _ptr(sf), _stream()))
    return q, sf


def mx_gemm(xq, x_scales, wq, w_scales, N, out=None, epilogue=EPI_NONE):
    """out = epilogue(Q8(x) . Q4(w)^T) from quantised operands (see mx_quantize)."""
    M, K = xq.shape
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=xq.device)
    check(lib.sana_mx_gemm(M, N, K, _ptr(xq), _ptr(x_scales), _ptr(wq), _ptr(w_scales), _ptr(out),
                           out.stride(0), epilogue, _stream()))
    return out


def mx_linear(x, wq, w_scales, N, out=None, epilogue=EPI_NONE, ws=None):
    """The quantised projection of bf16 activations x (M, K) against
    pre-quantised MXFP4 weights: activations quantised to MXFP8 on the fly."""
    _need(x, "x")
    M, K = x.shape
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = _ws(lib.sana_mx_linear_workspace_size(M, K), x.device)
    check(lib.sana_mx_linear(M, N, K, _ptr(x), _ptr(wq), _ptr(w_scales), _ptr(out), out.stride(0),
                             epilogue, _ptr(ws), ws.numel(), _stream()))
    return out


def selftest_bounded_wait(limit_ms=50):
    """Enqueue a kernel whose bounded wait runs out (see include/sana.h)."""
    check(lib.sana_selftest_bounded_wait(limit_ms, _stream()))


def sync_status():
    check(lib.sana_sync_status(_stream()))
