"""Chunked causal linear attention for GB300 (sm_103a): Python binding of liblinattn.

Argument marshalling only: every step of the computation runs in the CUDA
library (``_lib/liblinattn.so``, built in-tree by ``build.py``).  PyTorch is
used to allocate outputs and workspaces and to supply the current stream.
There is no fallback: if the library is missing, every call raises.

Low-level functions carry the C names (``linattn_fwd`` ...) and take raw
pointers; the helpers ``fwd``, ``bwd``, ``chunk_states`` and ``state_scan``
take torch tensors.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "liblinattn.so")

OK = 0
ERR_INVALID = -1
ERR_UNSUPPORTED = -2
ERR_ALIGN = -3
ERR_WORKSPACE = -4
ERR_CUDA = -5
ERR_DEVICE_TIMEOUT = -6
ERR_DEVICE = -7
ERR_SCRATCH_LIMIT = -8
NOALLOC_MAX_TILES = 65536
BF16, F32, E4M3 = 0, 1, 2
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}
MAX_NEW_TOKENS = 16  # of paged_decode_q8
OP_FWD, OP_BWD, OP_CHUNK_STATES, OP_CHECKPOINT = 1, 2, 3, 4
OP_FWD_GATED, OP_BWD_GATED, OP_CHECKPOINT_GATED = 5, 6, 7
OP_SOFTMAX_SEGMENT, OP_SOFTMAX_SEGMENT_BWD = 8, 9
OP_FWD_GATED_VEC, OP_BWD_GATED_VEC, OP_CHECKPOINT_GATED_VEC = 10, 11, 12
OP_FWD_DELTA, OP_BWD_DELTA, OP_CHECKPOINT_DELTA, OP_PAGED_DECODE = 13, 14, 15, 16
ABI_VERSION = 2


class LinattnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


class Shape(ctypes.Structure):
    """Mirror of ``linattn_shape`` in include/linattn.h."""
    _fields_ = [
        ("abi_version", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32),
        ("T", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("chunk", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64), ("stride_t", ctypes.c_int64),
        ("decay", ctypes.c_void_p),
    ]


_lock = threading.Lock()
_lib = None
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "linattn_abi_version": ([], _i32),
    "linattn_status_string": ([_i32], ctypes.c_char_p),
    "linattn_workspace_size": ([ctypes.POINTER(Shape), _i32, _i32, ctypes.POINTER(_sz)], _i32),
    "linattn_fwd": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_bwd": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_fwd_ckpt": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp], _i32),
    "linattn_bwd_ckpt": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp, _vp,
                          _sz, _vp], _i32),
    "linattn_chunk_states": ([ctypes.POINTER(Shape), _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_chunk_states_rev": ([ctypes.POINTER(Shape), _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_fwd_gated": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp], _i32),
    "linattn_bwd_gated": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp, _vp,
                           _vp, _vp, _sz, _vp], _i32),
    "linattn_fwd_gated_vec": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_bwd_gated_vec": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp, _sz, _vp], _i32),
    "linattn_fwd_gated_vec_ckpt": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _sz,
                                    _vp], _i32),
    "linattn_bwd_gated_vec_ckpt": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_decode": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "linattn_fwd_delta": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp, _sz,
                           _vp], _i32),
    "linattn_bwd_delta": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp, _vp,
                           _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_decode_delta": ([ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp], _i32),
    "linattn_paged_append": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp,
                              _vp, _vp, _vp], _i32),
    "linattn_paged_decode": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64,
                              _vp, ctypes.c_float, _vp, _sz, _vp], _i32),
    "linattn_paged_append_q8": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp,
                                 _i32, _i64, _vp, _vp, _vp, _vp], _i32),
    "linattn_paged_gather_q8": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _i64, _i64, _vp, _i32,
                                 _i64, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "linattn_paged_decode_q8": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp,
                                 _vp, _i32, _i64, _vp, ctypes.c_float, _vp, _sz, _vp], _i32),
    "linattn_rope_fwd": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                          ctypes.c_float, _vp, _i32, _vp], _i32),
    "linattn_rope_bwd": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                          ctypes.c_float, _vp, _i32, _vp], _i32),
    "linattn_rope_frequencies": ([_i32, ctypes.c_double, _i32, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                  ctypes.c_double, _vp], _i32),
    "linattn_state_scan_workspace_size": ([_i32, _i32, _i32, _i32, ctypes.POINTER(_sz)], _i32),
    "linattn_state_scan": ([_i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "linattn_device_status": ([_vp, _vp], _i32),
    "linattn_state_scan_noalloc": ([_i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "linattn_diag_mma": ([_i32, _vp, _vp, _vp, _vp], _i32),
    "linattn_diag_wait": ([_vp, _vp], _i32),
    "linattn_segment_decay": ([_vp, _i32, _i32, _i32, _vp, _vp], _i32),
    "linattn_softmax_segment_fwd": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp,
                                     ctypes.c_float, _vp, _sz, _vp], _i32),
    "linattn_softmax_segment_bwd": ([ctypes.POINTER(Shape), ctypes.POINTER(Shape), _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp, _vp, ctypes.c_float, _vp, _sz, _vp], _i32),
    "linattn_diag_scan_withhold": ([_i32, _i32, _i32, _i32, _vp, _vp, _i32, ctypes.c_double, _vp, _sz, _vp],
                                   _i32),
    "linattn_timing_enable": ([_i32], _i32),
    "linattn_timing_collect": ([_i32, ctypes.POINTER(_i32), ctypes.POINTER(ctypes.c_float)], _i32),
    "linattn_kernel_name": ([_i32], ctypes.c_char_p),
}
KERNEL_KINDS = 34


def lib():
    """The loaded ctypes library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m chunked_state_scan_causal_gb300.build`")
            l = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in _SIGS.items():
                f = getattr(l, name)
                f.argtypes = args
                f.restype = res
            _lib = l
    return _lib


_fast = None


class _NoModule:
    """Stands for the compiled marshalling where it was not built: no call is ordinary."""
    paged_append_q8 = paged_gather_q8 = paged_decode_q8 = rope = staticmethod(lambda *args: None)


def _bind():
    """The compiled marshalling of ordinary calls (csrc/bind.cpp): its functions return None for any other call."""
    global _fast
    if _fast is None:
        import importlib.util

        import torch  # noqa: F401 (its libraries are the module's)

        from . import build
        lib()
        path = build.bind_path()
        if not os.path.exists(path):
            _fast = _NoModule
            return _fast
        spec = importlib.util.spec_from_file_location("_bind", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _fast = module
    return _fast


def status_string(status: int) -> str:
    try:
        return lib().linattn_status_string(status).decode()
    except RuntimeError:
        return "?"


# ------------------------------------------------------------------ C names (raw pointers)
def linattn_status_string(status: int) -> str:
    return lib().linattn_status_string(status).decode()


def linattn_abi_version() -> int:
    return lib().linattn_abi_version()


def linattn_workspace_size(shape: Shape, op: int, seg_len: int = 0) -> tuple[int, int]:
    n = _sz(0)
    st = lib().linattn_workspace_size(ctypes.byref(shape), op, seg_len, ctypes.byref(n))
    return st, n.value


def linattn_fwd(shape, q, k, v, o, init_state, final_state, chunk_states, ws, ws_bytes, stream) -> int:
    return lib().linattn_fwd(ctypes.byref(shape), q, k, v, o, init_state, final_state, chunk_states,
                             ws, ws_bytes, stream)


def linattn_bwd(shape, q, k, v, dO, init_state, d_final, dq, dk, dv, d_init, ws, ws_bytes, stream) -> int:
    return lib().linattn_bwd(ctypes.byref(shape), q, k, v, dO, init_state, d_final, dq, dk, dv, d_init,
                             ws, ws_bytes, stream)


def linattn_decode(shape, q, k, v, o, state, stream) -> int:
    return lib().linattn_decode(ctypes.byref(shape), q, k, v, o, state, stream)


def linattn_fwd_ckpt(shape, q, k, v, o, init_state, final_state, ckpt, ckpt_bytes, ws, ws_bytes, stream) -> int:
    return lib().linattn_fwd_ckpt(ctypes.byref(shape), q, k, v, o, init_state, final_state, ckpt, ckpt_bytes,
                                  ws, ws_bytes, stream)


def linattn_bwd_ckpt(shape, q, k, v, dO, init_state, d_final, ckpt, ckpt_bytes, dq, dk, dv, d_init, ws, ws_bytes,
                     stream) -> int:
    return lib().linattn_bwd_ckpt(ctypes.byref(shape), q, k, v, dO, init_state, d_final, ckpt, ckpt_bytes, dq, dk,
                                  dv, d_init, ws, ws_bytes, stream)


def linattn_chunk_states(shape, seg_len, k, v, out, ws, ws_bytes, stream) -> int:
    return lib().linattn_chunk_states(ctypes.byref(shape), seg_len, k, v, out, ws, ws_bytes, stream)


def linattn_fwd_gated(shape, q, k, v, log_gate, o, init_state, final_state, ckpt, ckpt_bytes, ws, ws_bytes,
                      stream) -> int:
    return lib().linattn_fwd_gated(ctypes.byref(shape), q, k, v, log_gate, o, init_state, final_state, ckpt,
                                   ckpt_bytes, ws, ws_bytes, stream)


def linattn_bwd_gated(shape, q, k, v, dO, log_gate, init_state, d_final, ckpt, ckpt_bytes, dq, dk, dv, d_log_gate,
                      d_init, ws, ws_bytes, stream) -> int:
    return lib().linattn_bwd_gated(ctypes.byref(shape), q, k, v, dO, log_gate, init_state, d_final, ckpt,
                                   ckpt_bytes, dq, dk, dv, d_log_gate, d_init, ws, ws_bytes, stream)


def linattn_fwd_gated_vec(shape, q, k, v, log_gate, o, init_state, final_state, ws, ws_bytes, stream) -> int:
    return lib().linattn_fwd_gated_vec(ctypes.byref(shape), q, k, v, log_gate, o, init_state, final_state, ws,
                                       ws_bytes, stream)


def linattn_bwd_gated_vec(shape, q, k, v, dO, log_gate, init_state, d_final, dq, dk, dv, d_log_gate, d_init, ws,
                          ws_bytes, stream) -> int:
    return lib().linattn_bwd_gated_vec(ctypes.byref(shape), q, k, v, dO, log_gate, init_state, d_final, dq, dk, dv,
                                       d_log_gate, d_init, ws, ws_bytes, stream)


def linattn_fwd_gated_vec_ckpt(shape, q, k, v, log_gate, o, init_state, final_state, ckpt, ckpt_bytes, ws, ws_bytes,
                               stream) -> int:
    return lib().linattn_fwd_gated_vec_ckpt(ctypes.byref(shape), q, k, v, log_gate, o, init_state, final_state, ckpt,
                                            ckpt_bytes, ws, ws_bytes, stream)


def linattn_bwd_gated_vec_ckpt(shape, q, k, v, dO, log_gate, init_state, d_final, ckpt, ckpt_bytes, dq, dk, dv,
                               d_log_gate, d_init, ws, ws_bytes, stream) -> int:
    return lib().linattn_bwd_gated_vec_ckpt(ctypes.byref(shape), q, k, v, dO, log_gate, init_state, d_final, ckpt,
                                            ckpt_bytes, dq, dk, dv, d_log_gate, d_init, ws, ws_bytes, stream)


def linattn_chunk_states_rev(shape, seg_len, q, dO, out, ws, ws_bytes, stream) -> int:
    return lib().linattn_chunk_states_rev(ctypes.byref(shape), seg_len, q, dO, out, ws, ws_bytes, stream)


def linattn_state_scan_workspace_size(G, BH, dk, dv) -> tuple[int, int]:
    n = _sz(0)
    st = lib().linattn_state_scan_workspace_size(G, BH, dk, dv, ctypes.byref(n))
    return st, n.value


def linattn_state_scan(G, BH, dk, dv, seg_decay, local, init, out, total, ws, ws_bytes, stream) -> int:
    return lib().linattn_state_scan(G, BH, dk, dv, seg_decay, local, init, out, total, ws, ws_bytes, stream)


def linattn_state_scan_noalloc(G, BH, dk, dv, seg_decay, local, init, out, total, device_status, stream) -> int:
    """Allocation-free scan: no workspace; the library's fixed device scratch is used instead."""
    return lib().linattn_state_scan_noalloc(G, BH, dk, dv, seg_decay, local, init, out, total, device_status,
                                            stream)


def linattn_device_status(ws, stream) -> int:
    return lib().linattn_device_status(ws, stream)


def linattn_softmax_segment_fwd(q_shape, kv_shape, q, k, v, o, lse, softmax_scale, ws, ws_bytes, stream) -> int:
    return lib().linattn_softmax_segment_fwd(ctypes.byref(q_shape), ctypes.byref(kv_shape), q, k, v, o, lse,
                                             softmax_scale, ws, ws_bytes, stream)


def linattn_softmax_segment_bwd(q_shape, kv_shape, q, k, v, o, dO, lse, dq, dk, dv, softmax_scale, ws, ws_bytes,
                                stream) -> int:
    return lib().linattn_softmax_segment_bwd(ctypes.byref(q_shape), ctypes.byref(kv_shape), q, k, v, o, dO, lse, dq,
                                             dk, dv, softmax_scale, ws, ws_bytes, stream)


def linattn_fwd_delta(shape, q, k, v, log_gate, beta, gate_dtype, o, init_state, final_state, ckpt, ckpt_bytes, ws,
                      ws_bytes, stream) -> int:
    return lib().linattn_fwd_delta(ctypes.byref(shape), q, k, v, log_gate, beta, gate_dtype, o, init_state,
                                   final_state, ckpt, ckpt_bytes, ws, ws_bytes, stream)


def linattn_bwd_delta(shape, q, k, v, dO, log_gate, beta, gate_dtype, init_state, d_final, ckpt, ckpt_bytes, dq, dk,
                      dv, d_log_gate, d_beta, d_init, ws, ws_bytes, stream) -> int:
    return lib().linattn_bwd_delta(ctypes.byref(shape), q, k, v, dO, log_gate, beta, gate_dtype, init_state, d_final,
                                   ckpt, ckpt_bytes, dq, dk, dv, d_log_gate, d_beta, d_init, ws, ws_bytes, stream)


def linattn_decode_delta(shape, q, k, v, log_gate, beta, gate_dtype, o, state, stream) -> int:
    return lib().linattn_decode_delta(ctypes.byref(shape), q, k, v, log_gate, beta, gate_dtype, o, state, stream)


def linattn_paged_append(new_shape, cache_shape, k, v, k_cache, v_cache, block_table, max_blocks, table_stride, start,
                         new_lens, device_status, stream) -> int:
    return lib().linattn_paged_append(ctypes.byref(new_shape), ctypes.byref(cache_shape), k, v, k_cache, v_cache,
                                      block_table, max_blocks, table_stride, start, new_lens, device_status, stream)


def linattn_paged_decode(q_shape, cache_shape, q, k_cache, v_cache, o, lse, block_table, max_blocks, table_stride,
                         seq_lens, softmax_scale, ws, ws_bytes, stream) -> int:
    return lib().linattn_paged_decode(ctypes.byref(q_shape), ctypes.byref(cache_shape), q, k_cache, v_cache, o, lse,
                                      block_table, max_blocks, table_stride, seq_lens, softmax_scale, ws, ws_bytes,
                                      stream)


def _ref(shape):
    return None if shape is None else ctypes.byref(shape)


def linattn_paged_append_q8(new_shape, cache_shape, k, v, k_cache, v_cache, scales, scale_stride_p, scale_stride_h,
                            block_table, max_blocks, table_stride, start, new_lens, device_status, stream) -> int:
    return lib().linattn_paged_append_q8(ctypes.byref(new_shape), ctypes.byref(cache_shape), k, v, k_cache, v_cache,
                                         scales, scale_stride_p, scale_stride_h, block_table, max_blocks, table_stride,
                                         start, new_lens, device_status, stream)


def linattn_paged_gather_q8(out_shape, cache_shape, k_cache, v_cache, scales, scale_stride_p, scale_stride_h,
                            block_table, max_blocks, table_stride, seq_lens, start, k, v, device_status, stream) -> int:
    return lib().linattn_paged_gather_q8(ctypes.byref(out_shape), ctypes.byref(cache_shape), k_cache, v_cache, scales,
                                         scale_stride_p, scale_stride_h, block_table, max_blocks, table_stride,
                                         seq_lens, start, k, v, device_status, stream)


def linattn_paged_decode_q8(q_shape, cache_shape, q, k_cache, v_cache, scales, scale_stride_p, scale_stride_h, o, lse,
                            block_table, max_blocks, table_stride, seq_lens, softmax_scale, ws, ws_bytes,
                            stream) -> int:
    return lib().linattn_paged_decode_q8(ctypes.byref(q_shape), ctypes.byref(cache_shape), q, k_cache, v_cache, scales,
                                         scale_stride_p, scale_stride_h, o, lse, block_table, max_blocks, table_stride,
                                         seq_lens, softmax_scale, ws, ws_bytes, stream)


def linattn_rope_fwd(q_shape, k_shape, q, k, q_out, k_out, freqs, rot, layout, factor, positions, per_token,
                     stream) -> int:
    return lib().linattn_rope_fwd(ctypes.byref(q_shape), _ref(k_shape), q, k, q_out, k_out, freqs, rot, layout, factor,
                                  positions, per_token, stream)


def linattn_rope_bwd(q_shape, k_shape, dq_out, dk_out, dq, dk, freqs, rot, layout, factor, positions, per_token,
                     stream) -> int:
    return lib().linattn_rope_bwd(ctypes.byref(q_shape), _ref(k_shape), dq_out, dk_out, dq, dk, freqs, rot, layout,
                                  factor, positions, per_token, stream)


def linattn_rope_frequencies(rot, base, scaling, factor, trained_len, fast_turns, slow_turns, freqs) -> int:
    return lib().linattn_rope_frequencies(rot, base, scaling, factor, trained_len, fast_turns, slow_turns, freqs)


def linattn_segment_decay(decay, B, H, seg_len, out, stream) -> int:
    return lib().linattn_segment_decay(decay, B, H, seg_len, out, stream)


def linattn_diag_scan_withhold(G, BH, dk, dv, local, out, withhold_tile, wait_limit_ms, ws, ws_bytes,
                               stream) -> int:
    return lib().linattn_diag_scan_withhold(G, BH, dk, dv, local, out, withhold_tile, wait_limit_ms, ws,
                                            ws_bytes, stream)


def linattn_diag_mma(mode, A, B, D, stream) -> int:
    return lib().linattn_diag_mma(mode, A, B, D, stream)


def linattn_diag_wait(out, stream) -> int:
    return lib().linattn_diag_wait(out, stream)


def linattn_timing_enable(on: bool) -> int:
    return lib().linattn_timing_enable(1 if on else 0)


def linattn_timing_collect() -> dict:
    """{kernel name: (launches, total ms)} of the launches recorded since the last collect."""
    n = (_i32 * KERNEL_KINDS)()
    ms = (ctypes.c_float * KERNEL_KINDS)()
    st = lib().linattn_timing_collect(KERNEL_KINDS, n, ms)
    if st < 0:
        raise LinattnError(st, "linattn_timing_collect")
    return {linattn_kernel_name(k): (n[k], ms[k]) for k in range(KERNEL_KINDS) if n[k]}


def linattn_kernel_name(kind: int) -> str:
    return lib().linattn_kernel_name(kind).decode()


# ------------------------------------------------------------------ torch helpers
def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev, stream=None):
    import torch
    if stream is not None:
        return stream.cuda_stream
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not on {dev}")
    # (the raw handle: building the Stream object around it costs more than some of the kernels)
    return torch._C._cuda_getCurrentRawStream(dev.index)


def shape_of(q, decay=None, chunk: int = 64) -> Shape:
    """linattn_shape for a [B, H, T, d] tensor (last dim contiguous)."""
    import torch
    if q.dim() != 4 or q.stride(-1) != 1:
        raise ValueError("sequence tensors must be [B, H, T, d] with a contiguous last dimension")
    B, H, T, d = q.shape
    dt = BF16 if q.dtype == torch.bfloat16 else F32 if q.dtype == torch.float32 else None
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    sb, sh, st, _ = q.stride()
    return Shape(ABI_VERSION, B, H, T, d, d, chunk, dt, sb, sh, st, _ptr(decay))


def _same_layout(ref, *ts):
    shape, stride, dtype, device = ref.shape, ref.stride(), ref.dtype, ref.device
    for t in ts:
        if t is not None and (t.shape != shape or t.stride() != stride or t.dtype != dtype or t.device != device):
            raise ValueError("q, k, v (and dO, outputs) must share shape, strides, dtype and device")


def _check(st, what):
    if st != OK:
        raise LinattnError(st, what)


def workspace(q, op: int, decay=None, seg_len: int = 0):
    import torch
    st, n = linattn_workspace_size(shape_of(q, decay), op, seg_len)
    _check(st, "linattn_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def checkpoint(q, decay=None):
    """Buffer for the forward group states kept by fwd(..., ckpt=...) for bwd(..., ckpt=...)."""
    import torch
    st, n = linattn_workspace_size(shape_of(q, decay), OP_CHECKPOINT)
    _check(st, "linattn_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def fwd(q, k, v, decay=None, init_state=None, want_final=False, want_chunk_states=False,
        out=None, ws=None, stream=None, ckpt=None):
    """o (, final_state) (, chunk_states) for q, k, v [B, H, T, d] (bf16 or fp32).

    With ``ckpt`` (from ``checkpoint``) the forward group states are also stored for ``bwd(..., ckpt=)``."""
    import torch
    _same_layout(q, k, v, out)
    B, H, T, d = q.shape
    o = out if out is not None else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    fin = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if want_final else None
    nch = (T + 63) // 64
    cs = torch.empty((B, H, nch, d, d), dtype=torch.float32, device=q.device) if want_chunk_states else None
    shape = shape_of(q, decay)
    if ws is None:
        ws = workspace(q, OP_FWD, decay)
    if ckpt is not None:
        if cs is not None:
            raise ValueError("per-chunk states are not offered together with a checkpoint")
        st = linattn_fwd_ckpt(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(init_state), _ptr(fin),
                              _ptr(ckpt), ckpt.numel(), _ptr(ws), ws.numel(), _stream(q.device, stream))
        _check(st, "linattn_fwd_ckpt")
        return o, fin, cs
    st = linattn_fwd(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(init_state), _ptr(fin), _ptr(cs),
                     _ptr(ws), ws.numel(), _stream(q.device, stream))
    _check(st, "linattn_fwd")
    return o, fin, cs


def bwd(q, k, v, dO, decay=None, init_state=None, want_dinit=False, outs=None, ws=None, stream=None, ckpt=None,
        d_final=None):
    """(dq, dk, dv, d_init or None) for the upstream gradient dO (forward states from ``ckpt`` if given).

    ``d_final`` [B, H, d, d] fp32: gradient arriving at the final state (None: zero)."""
    import torch
    _same_layout(q, k, v, dO)
    B, H, T, d = q.shape
    if outs is None:
        outs = [torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device) for _ in range(3)]
    dq, dk, dv = outs
    dinit = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if want_dinit else None
    shape = shape_of(q, decay)
    if ws is None:
        ws = workspace(q, OP_BWD, decay)
    if ckpt is not None:
        st = linattn_bwd_ckpt(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(init_state), _ptr(d_final),
                              _ptr(ckpt), ckpt.numel(),
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dinit), _ptr(ws), ws.numel(),
                              _stream(q.device, stream))
        _check(st, "linattn_bwd_ckpt")
        return dq, dk, dv, dinit
    st = linattn_bwd(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(init_state), _ptr(d_final), _ptr(dq), _ptr(dk),
                     _ptr(dv), _ptr(dinit), _ptr(ws), ws.numel(), _stream(q.device, stream))
    _check(st, "linattn_bwd")
    return dq, dk, dv, dinit


def decode(q, k, v, state, decay=None, out=None, stream=None):
    """o for T new tokens [B, H, T, d]; `state` [B, H, d, d] fp32 is updated in place."""
    import torch
    _same_layout(q, k, v, out)
    if state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be contiguous fp32 [B, H, d, d]")
    o = out if out is not None else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    st = linattn_decode(shape_of(q, decay), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(state),
                        _stream(q.device, stream))
    _check(st, "linattn_decode")
    return o


def chunk_states(k, v, seg_len: int, decay=None, out=None, ws=None, stream=None):
    """Segment-local states [G, B, H, d, d] (fp32) for G = T / seg_len segments."""
    import torch
    _same_layout(k, v)
    B, H, T, d = k.shape
    G = T // seg_len if seg_len > 0 else 0
    out = out if out is not None else torch.empty((G, B, H, d, d), dtype=torch.float32, device=k.device)
    if ws is None:
        ws = workspace(k, OP_CHUNK_STATES, decay, seg_len)
    st = linattn_chunk_states(shape_of(k, decay), seg_len, _ptr(k), _ptr(v), _ptr(out), _ptr(ws), ws.numel(),
                              _stream(k.device, stream))
    _check(st, "linattn_chunk_states")
    return out


def chunk_states_rev(q, dO, seg_len: int, decay=None, out=None, ws=None, stream=None):
    """Segment-local gradient states [G, B, H, d, d] (fp32): sum_s lambda^{s - start + 1} q_s dO_s^T."""
    import torch
    _same_layout(q, dO)
    B, H, T, d = q.shape
    G = T // seg_len if seg_len > 0 else 0
    out = out if out is not None else torch.empty((G, B, H, d, d), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(q, OP_CHUNK_STATES, decay, seg_len)
    st = linattn_chunk_states_rev(shape_of(q, decay), seg_len, _ptr(q), _ptr(dO), _ptr(out), _ptr(ws), ws.numel(),
                                  _stream(q.device, stream))
    _check(st, "linattn_chunk_states_rev")
    return out


def checkpoint_gated(q):
    """Checkpoint buffer of fwd_gated for bwd_gated (group states and the final state)."""
    import torch
    st, n = linattn_workspace_size(shape_of(q, None), OP_CHECKPOINT_GATED)
    _check(st, "linattn_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def _gate_tensor(log_gate, q):
    import torch
    B, H, T, _ = q.shape
    if log_gate.dtype != torch.float32 or not log_gate.is_contiguous() or tuple(log_gate.shape) != (B, H, T):
        raise ValueError("log_gate must be contiguous fp32 [B, H, T]")
    return log_gate


def fwd_gated(q, k, v, log_gate, ckpt, init_state=None, want_final=False, out=None, ws=None, stream=None):
    """(o, final_state or None) with a gate per token: S_t = exp(log_gate_t) S_{t-1} + k_t v_t^T.
    ``ckpt`` (from checkpoint_gated) receives what bwd_gated needs."""
    import torch
    _same_layout(q, k, v, out)
    _gate_tensor(log_gate, q)
    B, H, T, d = q.shape
    o = out if out is not None else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    fin = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if want_final else None
    shape = shape_of(q, None)
    if ws is None:
        ws = workspace(q, OP_FWD_GATED)
    st = linattn_fwd_gated(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(o), _ptr(init_state), _ptr(fin),
                           _ptr(ckpt), ckpt.numel(), _ptr(ws), ws.numel(), _stream(q.device, stream))
    _check(st, "linattn_fwd_gated")
    return o, fin


def bwd_gated(q, k, v, dO, log_gate, ckpt, init_state=None, d_final=None, want_dinit=False, outs=None, ws=None,
              stream=None, dlg_out=None):
    """(dq, dk, dv, d_log_gate, d_init or None) of fwd_gated for the upstream gradient dO."""
    import torch
    _same_layout(q, k, v, dO)
    _gate_tensor(log_gate, q)
    B, H, T, d = q.shape
    if outs is None:
        outs = [torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device) for _ in range(3)]
    dq, dk, dv = outs
    dlg = dlg_out if dlg_out is not None else torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    dinit = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if want_dinit else None
    shape = shape_of(q, None)
    if ws is None:
        ws = workspace(q, OP_BWD_GATED)
    st = linattn_bwd_gated(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(log_gate), _ptr(init_state),
                           _ptr(d_final), _ptr(ckpt), ckpt.numel(), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlg),
                           _ptr(dinit), _ptr(ws), ws.numel(), _stream(q.device, stream))
    _check(st, "linattn_bwd_gated")
    return dq, dk, dv, dlg, dinit


def _gate_tensor_vec(log_gate, q):
    import torch
    B, H, T, d = q.shape
    if log_gate.dtype != torch.float32 or not log_gate.is_contiguous() or tuple(log_gate.shape) != (B, H, T, d):
        raise ValueError("log_gate must be contiguous fp32 [B, H, T, d]")
    return log_gate


def checkpoint_gated_vec(q):
    """Checkpoint buffer of fwd_gated_vec(..., ckpt=) for bwd_gated_vec(..., ckpt=) (the chunk
    groups' entering states and log-gate sums)."""
    import torch
    st, n = linattn_workspace_size(shape_of(q, None), OP_CHECKPOINT_GATED_VEC)
    _check(st, "linattn_workspace_size")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def fwd_gated_vec(q, k, v, log_gate, init_state=None, want_final=False, out=None, ws=None, stream=None, ckpt=None):
    """(o, final_state or None) with a gate per token and key dimension:
    S_t = diag(exp(log_gate_t)) S_{t-1} + k_t v_t^T (log_gate [B, H, T, d] fp32).  With ``ckpt``
    (from checkpoint_gated_vec) the groups' states are also kept for bwd_gated_vec(..., ckpt=)."""
    import torch
    _same_layout(q, k, v, out)
    _gate_tensor_vec(log_gate, q)
    B, H, T, d = q.shape
    o = out if out is not None else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    fin = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if want_final else None
    if ws is None:
        ws = workspace(q, OP_FWD_GATED_VEC)
    if ckpt is not None:
        st = linattn_fwd_gated_vec_ckpt(shape_of(q, None), _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(o),
                                        _ptr(init_state), _ptr(fin), _ptr(ckpt), ckpt.numel(), _ptr(ws), ws.numel(),
                                        _stream(q.device, stream))
        _check(st, "linattn_fwd_gated_vec_ckpt")
        return o, fin
    st = linattn_fwd_gated_vec(shape_of(q, None), _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(o),
                               _ptr(init_state), _ptr(fin), _ptr(ws), ws.numel(), _stream(q.device, stream))
    _check(st, "linattn_fwd_gated_vec")
    return o, fin


def bwd_gated_vec(q, k, v, dO, log_gate, init_state=None, d_final=None, want_dinit=False, outs=None, ws=None,
                  stream=None, ckpt=None):
    """(dq, dk, dv, d_log_gate [B, H, T, d], d_init or None) of fwd_gated_vec for the upstream gradient dO
    (the forward's group states from ``ckpt`` if given)."""
    import torch
    _same_layout(q, k, v, dO)
    _gate_tensor_vec(log_gate, q)
    B, H, T, d = q.shape
    if outs is None:
        outs = [torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device) for _ in range(3)]
    dq, dk, dv = outs
    dlg = torch.empty((B, H, T, d), dtype=torch.float32, device=q.device)
    dinit = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if want_dinit else None
    if ws is None:
        ws = workspace(q, OP_BWD_GATED_VEC)
    if ckpt is not None:
        st = linattn_bwd_gated_vec_ckpt(shape_of(q, None), _ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(log_gate),
                                        _ptr(init_state), _ptr(d_final), _ptr(ckpt), ckpt.numel(), _ptr(dq), _ptr(dk),
                                        _ptr(dv), _ptr(dlg), _ptr(dinit), _ptr(ws), ws.numel(),
                                        _stream(q.device, stream))
        _check(st, "linattn_bwd_gated_vec_ckpt")
        return dq, dk, dv, dlg, dinit
    st = linattn_bwd_gated_vec(shape_of(q, None), _ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(log_gate),
                               _ptr(init_state), _ptr(d_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlg), _ptr(dinit),
                               _ptr(ws), ws.numel(), _stream(q.device, stream))
    _check(st, "linattn_bwd_gated_vec")
    return dq, dk, dv, dlg, dinit


def state_scan(local, seg_decay=None, init=None, want_total=False, out=None, ws=None, stream=None):
    """Exclusive scan over the leading axis of local [G, *BH, dk, dv] (fp32)."""
    import torch
    G, dk, dv = local.shape[0], local.shape[-2], local.shape[-1]
    BH = local[0].numel() // (dk * dv)
    if not local.is_contiguous() or local.dtype != torch.float32:
        raise ValueError("local states must be contiguous fp32")
    out = out if out is not None else torch.empty_like(local)
    total = torch.empty(local.shape[1:], dtype=torch.float32, device=local.device) if want_total else None
    if ws is None:
        st, n = linattn_state_scan_workspace_size(G, BH, dk, dv)
        _check(st, "linattn_state_scan_workspace_size")
        ws = torch.empty(n, dtype=torch.uint8, device=local.device)
    st = linattn_state_scan(G, BH, dk, dv, _ptr(seg_decay), _ptr(local), _ptr(init), _ptr(out), _ptr(total),
                            _ptr(ws), ws.numel(), _stream(local.device, stream))
    _check(st, "linattn_state_scan")
    return out, total


def segment_decay(decay, B: int, seg_len: int, out=None, stream=None):
    """Per-(b, h) scan multiplier decay[h]^seg_len, [B*H] fp32 (None for decay None)."""
    import torch
    if decay is None:
        return None
    H = decay.numel()
    out = out if out is not None else torch.empty(B * H, dtype=torch.float32, device=decay.device)
    st = linattn_segment_decay(_ptr(decay), B, H, seg_len, _ptr(out), _stream(decay.device, stream))
    _check(st, "linattn_segment_decay")
    return out


def softmax_segment_fwd(q, k, v, scale: float = 0.0, want_lse: bool = False, out=None, ws=None, stream=None):
    """(o, lse or None): causal softmax attention of q [B,H,Tq,128] (the last Tq positions)
    over the prefix k, v [B,H,Tk,128] (bf16; scale 0 means 1/sqrt(128))."""
    import torch
    _same_layout(q, out)
    _same_layout(k, v)
    B, H, Tq, d = q.shape
    o = out if out is not None else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, H, Tq), dtype=torch.float32, device=q.device) if want_lse else None
    if ws is None:
        ws = workspace(q, OP_SOFTMAX_SEGMENT)
    st = linattn_softmax_segment_fwd(shape_of(q), shape_of(k), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), scale,
                                     _ptr(ws), ws.numel(), _stream(q.device, stream))
    _check(st, "linattn_softmax_segment_fwd")
    return o, lse


def softmax_segment_bwd(q, k, v, o, dO, lse, scale: float = 0.0, outs=None, ws=None, stream=None):
    """(dq, dk, dv): gradients of the causal softmax attention segment for the output
    gradient dO, from the forward's o and lse (bf16 q, o, dO, dq with q's layout; k, v,
    dk, dv with k's layout; scale 0 means 1/sqrt(128))."""
    import torch
    _same_layout(q, o)
    _same_layout(q, dO)
    _same_layout(k, v)
    if outs is None:
        outs = (torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device),
                torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device),
                torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device=v.device))
    dq, dk, dv = outs
    _same_layout(q, dq)
    _same_layout(k, dk)
    _same_layout(k, dv)
    if ws is None:
        ws = workspace(q, OP_SOFTMAX_SEGMENT_BWD)
    st = linattn_softmax_segment_bwd(shape_of(q), shape_of(k), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO),
                                     _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), scale, _ptr(ws), ws.numel(),
                                     _stream(q.device, stream))
    _check(st, "linattn_softmax_segment_bwd")
    return dq, dk, dv


_paged_ws = {}  # workspace bytes of paged_decode by (device, head dimension): they depend on nothing else


def _paged_workspace(q):
    import torch
    n = _paged_ws.get((q.device, q.shape[-1]))
    if n is None:
        st, n = linattn_workspace_size(shape_of(q), OP_PAGED_DECODE)
        _check(st, "linattn_workspace_size")
        _paged_ws[(q.device, q.shape[-1])] = n
    return q.new_empty(n, dtype=torch.uint8)


@functools.lru_cache(maxsize=1024)
def _delta_bytes(op, B, H, T, d, dtype, device):
    st, n = linattn_workspace_size(Shape(ABI_VERSION, B, H, T, d, d, 64, dtype, H * T * d, T * d, d, None), op)
    _check(st, "linattn_workspace_size")
    return max(n, 256)


def _delta_buffer(op, sh, q):
    """A workspace or checkpoint: its size depends on the shape (and the device) alone, and is asked for once."""
    import torch
    return q.new_empty(_delta_bytes(op, sh.B, sh.H, sh.T, sh.dk, sh.dtype, q.device), dtype=torch.uint8)


def _under(stream, f, *args):
    """f with `stream` the current one, so that what it allocates belongs to that stream too (memory of another
    stream could be handed out again while the call still runs)."""
    import torch
    with torch.cuda.stream(stream):
        return f(*args)


def _buffers(q, *ts):
    """Workspaces and checkpoints that the caller brought: kernels write them."""
    for t in ts:
        if t is not None and (t.device != q.device or not t.is_contiguous()):
            raise ValueError("workspaces and checkpoints must be contiguous, on the inputs' device")


def _like(q):
    """An output with q's layout."""
    import torch
    return torch.empty_like(q) if q.is_contiguous() else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype,
                                                                            device=q.device)


def checkpoint_delta(q):
    """Checkpoint buffer of fwd_delta(..., ckpt=) for bwd_delta."""
    return _delta_buffer(OP_CHECKPOINT_DELTA, shape_of(q), q)


def _delta_gates(log_gate, beta, q):
    """The gate type of the C ABI, after checking both gates (log_gate may be None)."""
    import torch
    dt = BF16 if beta.dtype == torch.bfloat16 else F32 if beta.dtype == torch.float32 else None
    shape, device = q.shape[:3], q.device
    for g in (beta,) if log_gate is None else (beta, log_gate):
        if dt is None or g.dtype != beta.dtype or not g.is_contiguous() or g.shape != shape or g.device != device:
            raise ValueError("log_gate and beta must be contiguous [B, H, T], both fp32 or both bf16, on q's device")
    return dt


def _states(q, *ts):
    import torch
    B, H, _, d = q.shape
    for t in ts:
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.shape != (B, H, d, d)
                              or t.device != q.device):
            raise ValueError("states must be contiguous fp32 [B, H, d, d] on q's device")


def fwd_delta(q, k, v, log_gate, beta, init_state=None, want_final=False, out=None, ws=None, stream=None, ckpt=None):
    """(o, final_state or None) of the gated delta rule: S_t = S' + beta_t k_t (v_t - S'^T k_t)^T with
    S' = exp(log_gate_t) S_{t-1}, o_t = S_t^T q_t (log_gate None: no decay; log_gate and beta [B, H, T],
    both fp32 or both bf16).  With ``ckpt`` (from checkpoint_delta) what bwd_delta needs is kept."""
    if stream is not None:
        return _under(stream, fwd_delta, q, k, v, log_gate, beta, init_state, want_final, out, ws, None, ckpt)
    import torch
    _same_layout(q, k, v, out)
    gdt = _delta_gates(log_gate, beta, q)
    _states(q, init_state)
    _buffers(q, ws, ckpt)
    o = out if out is not None else _like(q)
    B, H, T, d = q.shape
    fin = q.new_empty((B, H, d, d), dtype=torch.float32) if want_final else None
    sh = shape_of(q)
    if ws is None:
        # (with a checkpoint only its status word is used)
        ws = _delta_buffer(OP_FWD_DELTA, sh, q) if ckpt is None else q.new_empty(256, dtype=torch.uint8)
    st = linattn_fwd_delta(sh, _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(beta), gdt, _ptr(o),
                           _ptr(init_state), _ptr(fin), _ptr(ckpt), 0 if ckpt is None else ckpt.numel(), _ptr(ws),
                           ws.numel(), _stream(q.device))
    _check(st, "linattn_fwd_delta")
    return o, fin


def bwd_delta(q, k, v, dO, log_gate, beta, ckpt, init_state=None, d_final=None, want_dinit=False, outs=None, ws=None,
              stream=None):
    """(dq, dk, dv, d_log_gate or None, d_beta, d_init or None) of fwd_delta for the upstream gradient dO
    (the gates' gradients in the gates' type).  v and init_state are the forward's: what they add is in the checkpoint,
    and they are only checked."""
    if stream is not None:
        return _under(stream, bwd_delta, q, k, v, dO, log_gate, beta, ckpt, init_state, d_final, want_dinit, outs, ws)
    import torch
    _same_layout(q, k, v, dO)
    gdt = _delta_gates(log_gate, beta, q)
    _states(q, init_state, d_final)
    _buffers(q, ws, ckpt)
    B, H, T, d = q.shape
    if outs is None:
        dq, dk, dv = _like(q), _like(q), _like(q)
    else:
        dq, dk, dv = outs
        _same_layout(q, dq, dk, dv)
    dlg = None if log_gate is None else torch.empty_like(log_gate)
    db = torch.empty_like(beta)
    dinit = q.new_empty((B, H, d, d), dtype=torch.float32) if want_dinit else None
    sh = shape_of(q)
    if ws is None:
        ws = _delta_buffer(OP_BWD_DELTA, sh, q)
    st = linattn_bwd_delta(sh, _ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(log_gate), _ptr(beta), gdt,
                           _ptr(init_state), _ptr(d_final), _ptr(ckpt), ckpt.numel(), _ptr(dq), _ptr(dk), _ptr(dv),
                           _ptr(dlg), _ptr(db), _ptr(dinit), _ptr(ws), ws.numel(), _stream(q.device))
    _check(st, "linattn_bwd_delta")
    return dq, dk, dv, dlg, db, dinit


def decode_delta(q, k, v, log_gate, beta, state, out=None, stream=None):
    """o of the gated delta rule for T new tokens [B, H, T, d]; `state` [B, H, d, d] fp32 is updated in place."""
    if stream is not None:
        return _under(stream, decode_delta, q, k, v, log_gate, beta, state, out)
    _same_layout(q, k, v, out)
    gdt = _delta_gates(log_gate, beta, q)
    _states(q, state)
    o = out if out is not None else _like(q)
    st = linattn_decode_delta(shape_of(q), _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(beta), gdt, _ptr(o),
                              _ptr(state), _stream(q.device))
    _check(st, "linattn_decode_delta")
    return o


def _int_rows(q, B, *ts):
    import torch
    for t in ts:
        if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (B,) or not t.is_contiguous()
                              or t.device != q.device):
            raise ValueError("lengths and positions must be contiguous int32 [B] on the cache's device")


def _table(q, block_table):
    import torch
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != q.shape[0] \
            or block_table.stride(1) != 1 or block_table.device != q.device:
        raise ValueError("block_table must be int32 [B, max_blocks] with contiguous rows on the cache's device")
    n = block_table.shape[1]
    stride = block_table.stride(0) if block_table.shape[0] > 1 else n
    if stride < n:  # (one row expanded over the batch, say: its storage does not hold B rows)
        raise ValueError("block_table's rows must not overlap")
    return _ptr(block_table), n, stride


def paged_append(k, v, k_cache, v_cache, block_table, start, new_lens=None, device_status=None, stream=None):
    """Writes new tokens k, v [B, Hkv, T, d] into a paged cache [pages, Hkv, page, d] (any strides): token t of
    sequence b at position start[b] + t, in page block_table[b, position // page].  new_lens [B]: only the first
    new_lens[b] tokens of a padded batch.  device_status: int32 tensor for LINATTN_ERR_INVALID (bad pages)."""
    if stream is not None:
        return _under(stream, paged_append, k, v, k_cache, v_cache, block_table, start, new_lens, device_status)
    import torch
    _same_layout(k, v)
    _same_layout(k_cache, v_cache)
    if k_cache.device != k.device:
        raise ValueError("the new tokens and the cache must be on one device")
    _int_rows(k, k.shape[0], start, new_lens)
    if device_status is not None and (device_status.dtype != torch.int32 or device_status.numel() < 1
                                      or device_status.device != k.device):
        raise ValueError("device_status must be an int32 tensor on the cache's device")
    tab, n, stride = _table(k, block_table)
    st = linattn_paged_append(shape_of(k), shape_of(k_cache), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), tab, n,
                              stride, _ptr(start), _ptr(new_lens), _ptr(device_status), _stream(k.device))
    _check(st, "linattn_paged_append")


def paged_decode(q, k_cache, v_cache, block_table, seq_lens, scale: float = 0.0, want_lse: bool = False, out=None,
                 ws=None, stream=None):
    """(o, lse or None): softmax attention of one new token per sequence, q [B, Hq, 1, d], over the first
    seq_lens[b] tokens of its pages (scale 0 means 1/sqrt(d); lse [B, Hq, 1] fp32).  Page ids outside the cache count
    as absent tokens: pass ws= (workspace(q, OP_PAGED_DECODE)) to read of them with device_status(ws)."""
    if stream is not None:
        return _under(stream, paged_decode, q, k_cache, v_cache, block_table, seq_lens, scale, want_lse, out, ws)
    import torch
    _same_layout(q, out)
    _same_layout(k_cache, v_cache)
    if k_cache.device != q.device:
        raise ValueError("q and the cache must be on one device")
    _int_rows(q, q.shape[0], seq_lens)
    _buffers(q, ws)
    tab, n, stride = _table(q, block_table)
    o = out if out is not None else _like(q)
    lse = q.new_empty(q.shape[:3], dtype=torch.float32) if want_lse else None
    if ws is None:
        ws = _paged_workspace(q)
    st = linattn_paged_decode(shape_of(q), shape_of(k_cache), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o),
                              _ptr(lse), tab, n, stride, _ptr(seq_lens), scale, _ptr(ws), ws.numel(),
                              _stream(q.device))
    _check(st, "linattn_paged_decode")
    return o, lse


# ------------------------------------------------------------------ the paged cache in 8 bits
# (Ordinary calls go through _bind(), which takes a third of the time; what follows is the same for every other call.)
def _elsewhere(device, stream):
    """Whether a call on `device` needs another current device or stream than the caller's (see _over_there)."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not on {device}")
    return stream is not None or torch._C._cuda_getDevice() != device.index


def _over_there(device, stream, f, *args):
    """f with `device` the current one, and `stream` (if any) its current stream: see _under."""
    import torch
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return f(*args)


def _codes(device, k_cache, v_cache, scales):
    """The cache's shape for the C ABI and the strides of its scales, after checking all three."""
    import torch
    shape, stride = k_cache.shape, k_cache.stride()
    if k_cache.dtype != torch.float8_e4m3fn or len(shape) != 4 or stride[3] != 1:
        raise ValueError("caches must be float8_e4m3fn [pages, Hkv, page, d] with a contiguous last dimension")
    if v_cache.dtype != torch.float8_e4m3fn or v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError("k_cache and v_cache must share shape, strides and dtype")
    P, H, page, d = shape
    n = page // 16
    strides = scales.stride()
    if scales.dtype != torch.float32 or scales.shape != (P, H, n, 2) or strides[3] != 1 or (strides[2] != 2 and n > 1):
        raise ValueError("scales must be fp32 [pages, Hkv, page / 16, 2], contiguous in the last two dimensions")
    if k_cache.device != device or v_cache.device != device or scales.device != device:
        raise ValueError("the tokens, the cache and its scales must be on one device")
    return (Shape(ABI_VERSION, P, H, page, d, d, 64, E4M3, *stride[:3], None), strides[0] if P > 1 else 2 * n * H,
            strides[1] if H > 1 else 2 * n)


def _status_word(device, device_status):
    import torch
    if device_status.dtype != torch.int32 or device_status.numel() < 1 or device_status.device != device:
        raise ValueError("device_status must be an int32 tensor on the cache's device")
    return device_status.data_ptr()


def paged_append_q8(k, v, k_cache, v_cache, scales, block_table, start, new_lens=None, device_status=None, stream=None):
    """paged_append into a cache in 8 bits: k_cache, v_cache [pages, Hkv, page, d] float8_e4m3fn (any strides, pages a
    multiple of 16 tokens) and scales [pages, Hkv, page / 16, 2] fp32 for every 16 tokens' keys and values.
    The scale is the smallest power of two that holds the block; a block that is already begun keeps its scale or, where the
    new tokens need a larger one, has its codes rounded again (not at once: order the call with readers of that block on other
    streams).  Values that are not finite become NaN.  Tokens behind the last new one of a block do not outlast the call."""
    if stream is None and device_status is None and (_fast or _bind()).paged_append_q8(
            k, v, k_cache, v_cache, scales, block_table, start, new_lens):
        return
    device = k.device
    if _elsewhere(device, stream):
        return _over_there(device, stream, paged_append_q8, k, v, k_cache, v_cache, scales, block_table, start, new_lens,
                           device_status)
    _same_layout(k, v)
    cache, sp, sh = _codes(device, k_cache, v_cache, scales)
    shape = shape_of(k)
    _int_rows(k, shape.B, start, new_lens)
    tab, n, stride = _table(k, block_table)
    st = lib().linattn_paged_append_q8(shape, cache, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                       scales.data_ptr(), sp, sh, tab, n, stride, start.data_ptr(),
                                       None if new_lens is None else new_lens.data_ptr(),
                                       None if device_status is None else _status_word(device, device_status),
                                       _stream(device))
    if st:
        _check(st, "linattn_paged_append_q8")


def paged_gather_q8(k_cache, v_cache, scales, block_table, seq_lens, T, dtype=None, start=None, out=None,
                    device_status=None, stream=None):
    """(k, v) [B, Hkv, T, d] in `dtype` (bf16 if None, or fp32): T cached tokens of every sequence from start[b] on (from
    the first if None); rows past its length are zero.  What softmax_segment_fwd takes as its prefix."""
    if stream is None and device_status is None and out is None:
        r = (_fast or _bind()).paged_gather_q8(k_cache, v_cache, scales, block_table, seq_lens, T, dtype, start)
        if r is not None:
            return r
    device = k_cache.device
    if _elsewhere(device, stream):
        return _over_there(device, stream, paged_gather_q8, k_cache, v_cache, scales, block_table, seq_lens, T, dtype,
                           start, out, device_status)
    import torch
    cache, sp, sh = _codes(device, k_cache, v_cache, scales)
    shape = (block_table.shape[0], cache.H, T, cache.dk)
    if out is None:
        dtype = dtype or torch.bfloat16
        k, v = torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device)
    else:
        k, v = out
        _same_layout(k, v)
        if k.shape != shape or (dtype or k.dtype) != k.dtype or k.device != device:
            raise ValueError("outputs must be [B, Hkv, T, d] in the type asked for, on the cache's device")
    _int_rows(k, shape[0], seq_lens, start)
    tab, n, stride = _table(k, block_table)
    st = lib().linattn_paged_gather_q8(shape_of(k), cache, k_cache.data_ptr(), v_cache.data_ptr(), scales.data_ptr(), sp,
                                       sh, tab, n, stride, seq_lens.data_ptr(),
                                       None if start is None else start.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       None if device_status is None else _status_word(device, device_status),
                                       _stream(device))
    if st:
        _check(st, "linattn_paged_gather_q8")
    return k, v


def paged_decode_q8(q, k_cache, v_cache, scales, block_table, seq_lens, scale: float = 0.0, want_lse: bool = False,
                    out=None, ws=None, stream=None):
    """(o, lse or None): softmax attention of the last T tokens of every sequence (1 to MAX_NEW_TOKENS), q [B, Hq, T, d],
    over its pages in 8 bits; query t sees the tokens before seq_lens[b] - T + 1 + t (scale 0 means 1/sqrt(d); lse
    [B, Hq, T] fp32).  Page ids outside the cache count as absent tokens: pass ws= (workspace(q, OP_PAGED_DECODE)) to read
    of them with device_status(ws)."""
    if stream is None:
        r = (_fast or _bind()).paged_decode_q8(q, k_cache, v_cache, scales, block_table, seq_lens, scale, want_lse, out, ws)
        if r is not None:
            return r
    device = q.device
    if _elsewhere(device, stream):
        return _over_there(device, stream, paged_decode_q8, q, k_cache, v_cache, scales, block_table, seq_lens, scale,
                           want_lse, out, ws)
    import torch
    cache, sp, sh = _codes(device, k_cache, v_cache, scales)
    shape = shape_of(q)
    _int_rows(q, shape.B, seq_lens)
    tab, n, stride = _table(q, block_table)
    if out is None:
        o = _like(q)
    else:
        _same_layout(q, out)
        o = out
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=device) if want_lse else None
    if ws is None:
        size = _paged_ws.get((device, shape.dk)) or _paged_workspace(q).numel()
        ws = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        _buffers(q, ws)
        size = ws.numel()
    st = lib().linattn_paged_decode_q8(shape, cache, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                       scales.data_ptr(), sp, sh, o.data_ptr(), None if lse is None else lse.data_ptr(),
                                       tab, n, stride, seq_lens.data_ptr(), scale, ws.data_ptr(), size, _stream(device))
    if st:
        _check(st, "linattn_paged_decode_q8")
    return o, lse


# ------------------------------------------------------------------ rotary positions
def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained_len: float = 0.0, fast_turns: float = 32.0, slow_turns: float = 1.0, device=None):
    """Radians per position of the rot / 2 pairs of rope_fwd, [rot / 2] fp64: base^(-2 i / rot), for a context `factor`
    times as long as trained: "linear" (all divided by factor), "base" (of a larger base: the slowest pair slowed factor
    times, the fastest not) or "parts" (pairs with more than fast_turns turns in trained_len positions stay, those with less
    than slow_turns are slowed, a ramp between; attention is commonly sharpened with it by rope_fwd's
    factor = 1 + 0.1 log(factor))."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    f = torch.empty(max(rot // 2, 1), dtype=torch.float64)
    st = linattn_rope_frequencies(rot, base, ROPE_SCALINGS[scaling], factor, trained_len, fast_turns, slow_turns,
                                  _ptr(f))
    _check(st, "linattn_rope_frequencies")
    return f if device is None else f.to(device)


def _rope(name, q, k, freqs, positions, layout, factor, outs, stream):
    if stream is None and layout in ROPE_LAYOUTS:
        qo, ko = outs or (None, None)
        r = (_fast or _bind()).rope(name == "linattn_rope_bwd", q, k, freqs, positions, ROPE_LAYOUTS[layout], factor, qo, ko)
        if r is not None:
            return r
    device = q.device
    if _elsewhere(device, stream):
        return _over_there(device, stream, _rope, name, q, k, freqs, positions, layout, factor, outs, None)
    import torch
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or freqs.stride(0) != 1 or freqs.device != device:
        raise ValueError("freqs must be contiguous fp64 [rot / 2] on q's device")
    shape = shape_of(q)
    per_token = positions.dim() == 2
    if positions.dtype != torch.int32 or positions.shape != ((shape.B, shape.T) if per_token else (shape.B,)) \
            or not positions.is_contiguous() or positions.device != device:
        raise ValueError("positions must be contiguous int32 [B] (of the first tokens) or [B, T] on q's device")
    qo, ko = outs if outs is not None else (_like(q), None if k is None else _like(k))
    if outs is not None:
        _same_layout(q, qo)
    kshape = kp = kop = None
    if k is not None:
        kshape = shape_of(k)
        if kshape.B != shape.B or kshape.T != shape.T or kshape.dk != shape.dk or kshape.dtype != shape.dtype \
                or k.device != device:
            raise ValueError("q and k must share B, T, d, dtype and device")
        if outs is not None:
            if ko is None:
                raise ValueError("outs must hold an output for k")
            _same_layout(k, ko)
        kp, kop = k.data_ptr(), ko.data_ptr()
    elif ko is not None:
        raise ValueError("an output for k without k")
    st = getattr(lib(), name)(shape, kshape, q.data_ptr(), kp, qo.data_ptr(), kop, freqs.data_ptr(), 2 * freqs.shape[0],
                              ROPE_LAYOUTS[layout], factor, positions.data_ptr(), per_token, _stream(device))
    if st:
        _check(st, name)
    return qo, ko


def rope_fwd(q, k, freqs, positions, layout: str = "half", factor: float = 1.0, outs=None, stream=None):
    """(q', k' or None): rotary positions on q [B, Hq, T, d] and k [B, Hkv, T, d] (or None): the pairs of the first
    2 len(freqs) dimensions, (i, i + rot / 2) ("half") or (2 i, 2 i + 1) ("interleaved"), are turned by position x
    freqs[i] (rope_frequencies) and multiplied by `factor`; the rest is copied.  positions int32: [B], the first
    token's (the others follow), or [B, T].  Outputs have their inputs' strides, so that those of slices of one
    projection span as much as it does; outs may be (q, k) themselves, which takes no memory (rope_bwd needs neither)."""
    return _rope("linattn_rope_fwd", q, k, freqs, positions, layout, factor, outs, stream)


def rope_bwd(dq_out, dk_out, freqs, positions, layout: str = "half", factor: float = 1.0, outs=None, stream=None):
    """(dq, dk or None): the gradients of rope_fwd's inputs from those of its outputs."""
    return _rope("linattn_rope_bwd", dq_out, dk_out, freqs, positions, layout, factor, outs, stream)


def device_status(ws, stream=None) -> int:
    return linattn_device_status(_ptr(ws), _stream(ws.device, stream))
