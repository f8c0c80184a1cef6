"""Thin Python binding of the C ABI in ``include/ts_hc.h`` (ctypes).

Two layers, both argument marshalling only -- every step of the computation
runs in the library's CUDA kernels:

* ``ts_hc_*``: the C entry points under their own names, taking raw device
  pointers (ints), a ``TsWeight`` struct and a CUDA stream handle; they return
  the ``ts_status`` code.
* ``hc_call`` / ``hc_inject_call`` / ``hc_mixer`` / ``hc_inject_add`` /
  ``hc_replicate_entry`` / ``hc_stack``, and for a speculative decoding step
  ``hc_rope`` / ``hc_kv_write`` / ``hc_kv_read`` / ``hc_kv_compact`` /
  ``hc_tree_build`` / ``hc_tree_attention`` / ``hc_verify``: the same calls
  for torch CUDA tensors. They allocate outputs/workspace with torch when not given, pass
  the current torch stream, and raise ``HCError`` on any error status.

There is no fallback: if the library is not built or cannot be loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

from .build import LIB_PATH

TS_OK, TS_ERR_INVALID_ARG, TS_ERR_UNSUPPORTED, TS_ERR_CUDA, TS_ERR_WORKSPACE, TS_ERR_TIMEOUT = range(6)
TS_W_BF16, TS_W_INT4_AFFINE = 0, 1
TS_KV_BF16, TS_KV_FP8, TS_KV_INT4 = range(3)
TS_ROPE_PLAIN, TS_ROPE_LINEAR, TS_ROPE_NTK, TS_ROPE_BY_PARTS = range(4)
RMS_EPS = 1e-6  # families/qwen4/mod.rs, RMS_EPS

EXPORTS = ("ts_hc_workspace_bytes", "ts_hc_workspace_layout", "ts_hc_call", "ts_hc_inject_add",
           "ts_hc_mixer", "ts_hc_call_debug", "ts_hc_inject_call", "ts_hc_entry_call", "ts_hc_exit_logits",
           "ts_hc_replicate_entry", "ts_hc_ple_workspace_bytes", "ts_hc_ple_workspace_layout", "ts_hc_ple",
           "ts_hc_last_error",
           "ts_hc_device_status", "ts_hc_call_noalloc", "ts_hc_stack_workspace_bytes", "ts_hc_stack",
           "ts_hc_stack_ple_workspace_bytes", "ts_hc_stack_ple", "ts_hc_selftest_timeout",
           "ts_hc_rope_table", "ts_hc_rope", "ts_hc_kv_write", "ts_hc_kv_read", "ts_hc_kv_compact", "ts_hc_tree_build",
           "ts_hc_tree_attention_workspace_bytes", "ts_hc_tree_attention", "ts_hc_verify")
TS_HC_STATIC_SCRATCH_BYTES = 64 * 1024 * 1024  # include/ts_hc.h


class HCError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"ts_hc status {status}: {message}")
        self.status = status


class TsWeight(ctypes.Structure):
    _fields_ = [
        ("type", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("data", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("biases", ctypes.c_void_p),
    ]


class TsHcModule(ctypes.Structure):
    """``ts_hc_module``: one hyper-connection module's hc_norm weight and linears."""
    _fields_ = [
        ("hc_norm_w", ctypes.c_void_p),
        ("down", TsWeight),
        ("up", TsWeight),
        ("inject", TsWeight),
    ]


class TsHcPleModule(ctypes.Structure):
    """``ts_hc_ple_module``: a stack's PLE tensors."""
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("n_rows", ctypes.c_long),
        ("key_proj", ctypes.c_void_p),
        ("value_proj", ctypes.c_void_p),
        ("norm_key_w", ctypes.c_void_p),
        ("norm_query_w", ctypes.c_void_p),
        ("norm_conv_w", ctypes.c_void_p),
        ("conv_w", ctypes.c_void_p),
    ]


class TsHcRopeScaling(ctypes.Structure):
    """``ts_hc_rope_scaling``: how a rotary table's frequencies are changed for long contexts."""
    _fields_ = [
        ("type", ctypes.c_int32),
        ("factor", ctypes.c_float),
        ("original_positions", ctypes.c_float),
        ("beta_fast", ctypes.c_float),
        ("beta_slow", ctypes.c_float),
        ("magnitude", ctypes.c_float),
    ]


class TsHcKvCache(ctypes.Structure):
    """``ts_hc_kv_cache``: a paged cache's format and tensors."""
    _fields_ = [
        ("type", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("n_pages", ctypes.c_long),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("k_biases", ctypes.c_void_p),
        ("v_biases", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
    ]


# ts_hc_sublayer_fn: (user, layer, which, t0, M, mixed, &out, stream) -> ts_status
SUBLAYER_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                               ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p)

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


def library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load ``libts_hc.so`` (once). Raises if it is missing: there is no fallback."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library {p} is not built; run hyper_connection_residual_call_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i, l, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_size_t, ctypes.c_float
        wp = ctypes.POINTER(TsWeight)
        lib.ts_hc_workspace_bytes.argtypes = [i, i, i, i]
        lib.ts_hc_workspace_bytes.restype = sz
        lib.ts_hc_workspace_layout.argtypes = [i, i, i, i, ctypes.POINTER(sz), ctypes.POINTER(sz)]
        lib.ts_hc_workspace_layout.restype = i
        lib.ts_hc_call.argtypes = [vp, vp, wp, wp, wp, vp, vp, l, i, i, i, i, f, vp, sz, vp]
        lib.ts_hc_call.restype = i
        lib.ts_hc_mixer.argtypes = [vp, vp, wp, wp, vp, i, i, i, i, f, vp, sz, vp]
        lib.ts_hc_mixer.restype = i
        lib.ts_hc_call_debug.argtypes = [vp, vp, wp, wp, wp, vp, vp, l, i, i, i, i, f, vp, sz, vp, vp]
        lib.ts_hc_call_debug.restype = i
        lib.ts_hc_inject_add.argtypes = [vp, vp, vp, l, i, i, i, vp]
        lib.ts_hc_inject_add.restype = i
        lib.ts_hc_inject_call.argtypes = [vp, vp, vp, l, vp, wp, wp, wp, vp, vp, l, i, i, i, i, f, vp, sz, vp]
        lib.ts_hc_inject_call.restype = i
        lib.ts_hc_entry_call.argtypes = [vp, vp, vp, wp, wp, wp, vp, vp, l, i, i, i, i, f, vp, sz, vp]
        lib.ts_hc_entry_call.restype = i
        lib.ts_hc_exit_logits.argtypes = [vp, vp, vp, l, vp, wp, wp, vp, i, vp, vp, i, i, i, i, f, vp, sz, vp]
        lib.ts_hc_exit_logits.restype = i
        lib.ts_hc_ple_workspace_bytes.argtypes = [i, i, i]
        lib.ts_hc_ple_workspace_bytes.restype = sz
        lib.ts_hc_ple_workspace_layout.argtypes = [i, i, i, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        lib.ts_hc_ple_workspace_layout.restype = i
        lib.ts_hc_ple.argtypes = [vp, vp, vp, l, vp, vp, vp, vp, vp, vp, vp, i, i, i, f, vp, sz, vp]
        lib.ts_hc_ple.restype = i
        lib.ts_hc_call_noalloc.argtypes = [vp, vp, wp, wp, wp, vp, vp, l, i, i, i, i, f, vp]
        lib.ts_hc_call_noalloc.restype = i
        lib.ts_hc_replicate_entry.argtypes = [vp, vp, i, i, i, vp]
        lib.ts_hc_replicate_entry.restype = i
        mp = ctypes.POINTER(TsHcModule)
        lib.ts_hc_stack_workspace_bytes.argtypes = [i, i, i, i]
        lib.ts_hc_stack_workspace_bytes.restype = sz
        lib.ts_hc_stack.argtypes = [vp, i, mp, mp, i, mp, SUBLAYER_FN, vp, vp, i, i, i, i, f, vp, sz, vp]
        lib.ts_hc_stack.restype = i
        lib.ts_hc_stack_ple_workspace_bytes.argtypes = [i, i, i, i]
        lib.ts_hc_stack_ple_workspace_bytes.restype = sz
        lib.ts_hc_stack_ple.argtypes = [vp, i, mp, mp, i, mp, ctypes.POINTER(TsHcPleModule), vp, vp, SUBLAYER_FN,
                                        vp, vp, i, i, i, i, f, vp, sz, vp]
        lib.ts_hc_stack_ple.restype = i
        cp = ctypes.POINTER(TsHcKvCache)
        lib.ts_hc_rope_table.argtypes = [vp, i, i, ctypes.c_double, ctypes.POINTER(TsHcRopeScaling), vp]
        lib.ts_hc_rope_table.restype = i
        lib.ts_hc_rope.argtypes = [vp, l, vp, l, vp, vp, i, vp, l, vp, l, i, i, i, i, i, i, i, vp]
        lib.ts_hc_rope.restype = i
        lib.ts_hc_kv_write.argtypes = [vp, l, vp, l, cp, vp, i, i, vp]
        lib.ts_hc_kv_write.restype = i
        lib.ts_hc_kv_read.argtypes = [cp, vp, vp, vp, i, i, vp]
        lib.ts_hc_kv_read.restype = i
        lib.ts_hc_kv_compact.argtypes = [cp, vp, vp, vp, vp, i, i, vp]
        lib.ts_hc_kv_compact.restype = i
        lib.ts_hc_tree_build.argtypes = [vp, l, vp, vp, vp, i, i, vp]
        lib.ts_hc_tree_build.restype = i
        lib.ts_hc_tree_attention_workspace_bytes.argtypes = [i, i, i, cp]
        lib.ts_hc_tree_attention_workspace_bytes.restype = sz
        lib.ts_hc_tree_attention.argtypes = [vp, l, cp, vp, vp, l, vp, vp, i, i, i, f, vp, sz, vp]
        lib.ts_hc_tree_attention.restype = i
        lib.ts_hc_verify.argtypes = [vp, vp, vp, vp, l, vp, vp, vp, vp, vp, vp, i, i, i, vp]
        lib.ts_hc_verify.restype = i
        lib.ts_hc_selftest_timeout.argtypes = [vp]
        lib.ts_hc_selftest_timeout.restype = i
        lib.ts_hc_last_error.argtypes = []
        lib.ts_hc_last_error.restype = ctypes.c_char_p
        lib.ts_hc_device_status.argtypes = [vp, ctypes.POINTER(i)]
        lib.ts_hc_device_status.restype = i
        if path is None:
            _lib = lib
        return lib


# ------------------------------------------------------------- C names

def ts_hc_workspace_bytes(M: int, H: int, C: int, lowrank: int) -> int:
    return library().ts_hc_workspace_bytes(M, H, C, lowrank)


def ts_hc_workspace_layout(M: int, H: int, C: int, lowrank: int) -> Tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    st = library().ts_hc_workspace_layout(M, H, C, lowrank, ctypes.byref(a), ctypes.byref(b))
    _check(st)
    return a.value, b.value


def ts_hc_call(raw, hc_norm_w, down, up, inject, mixed, inject_w, inject_stride, M, H, C, lowrank,
               eps, workspace, workspace_bytes, stream) -> int:
    return library().ts_hc_call(raw, hc_norm_w, _wref(down), _wref(up), _wref(inject), mixed, inject_w,
                                inject_stride, M, H, C, lowrank, eps, workspace, workspace_bytes, stream)


def ts_hc_mixer(raw, hc_norm_w, down, up, mixed, M, H, C, lowrank, eps, workspace, workspace_bytes,
                stream) -> int:
    return library().ts_hc_mixer(raw, hc_norm_w, _wref(down), _wref(up), mixed, M, H, C, lowrank, eps,
                                 workspace, workspace_bytes, stream)


def ts_hc_call_debug(raw, hc_norm_w, down, up, inject, mixed, inject_w, inject_stride, M, H, C, lowrank,
                     eps, workspace, workspace_bytes, w_out, stream) -> int:
    """ts_hc_call (ts_hc_mixer when ``inject`` is None) that also writes w = sigmoid(up(act))."""
    return library().ts_hc_call_debug(raw, hc_norm_w, _wref(down), _wref(up), _wref(inject), mixed, inject_w,
                                      inject_stride, M, H, C, lowrank, eps, workspace, workspace_bytes, w_out,
                                      stream)


def ts_hc_inject_add(raw, out, inject_w, inject_stride, M, H, C, stream) -> int:
    return library().ts_hc_inject_add(raw, out, inject_w, inject_stride, M, H, C, stream)


def ts_hc_inject_call(raw, out, prev_inject_w, prev_inject_stride, hc_norm_w, down, up, inject, mixed,
                      inject_w, inject_stride, M, H, C, lowrank, eps, workspace, workspace_bytes,
                      stream) -> int:
    return library().ts_hc_inject_call(raw, out, prev_inject_w, prev_inject_stride, hc_norm_w, _wref(down),
                                       _wref(up), _wref(inject), mixed, inject_w, inject_stride, M, H, C,
                                       lowrank, eps, workspace, workspace_bytes, stream)


def ts_hc_entry_call(emb, raw, hc_norm_w, down, up, inject, mixed, inject_w, inject_stride, M, H, C, lowrank,
                     eps, workspace, workspace_bytes, stream) -> int:
    """Entry replication fused into the first call: raw = repeat(emb, C), then the call on it."""
    return library().ts_hc_entry_call(emb, raw, hc_norm_w, _wref(down), _wref(up), _wref(inject), mixed, inject_w,
                                      inject_stride, M, H, C, lowrank, eps, workspace, workspace_bytes, stream)


def ts_hc_exit_logits(raw, out, prev_inject_w, prev_inject_stride, hc_norm_w, down, up, lm_head, V, mixed, logits,
                      M, H, C, lowrank, eps, workspace, workspace_bytes, stream) -> int:
    """The exit: (inject-add,) hyper_connection_mixer, then lm_head into fp32 logits."""
    return library().ts_hc_exit_logits(raw, out, prev_inject_w, prev_inject_stride, hc_norm_w, _wref(down), _wref(up),
                                       lm_head, V, mixed, logits, M, H, C, lowrank, eps, workspace, workspace_bytes,
                                       stream)


def ts_hc_ple_workspace_bytes(M: int, H: int, C: int) -> int:
    return library().ts_hc_ple_workspace_bytes(M, H, C)


def ts_hc_ple_workspace_layout(M: int, H: int, C: int) -> Tuple[int, int, int]:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(library().ts_hc_ple_workspace_layout(M, H, C, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def ts_hc_ple(hidden, rows, table, n_rows, key_proj, value_proj, norm_key_w, norm_query_w, norm_conv_w, conv_w,
              conv_state, M, H, C, eps, workspace, workspace_bytes, stream) -> int:
    """The PLE gate added to the wide residual (in place), for M consecutive tokens."""
    return library().ts_hc_ple(hidden, rows, table, n_rows, key_proj, value_proj, norm_key_w, norm_query_w,
                               norm_conv_w, conv_w, conv_state, M, H, C, eps, workspace, workspace_bytes, stream)


def ts_hc_call_noalloc(raw, hc_norm_w, down, up, inject, mixed, inject_w, inject_stride, M, H, C, lowrank,
                       eps, stream) -> int:
    """ts_hc_call with its scratch in the library's own device array (no workspace argument),
    for callers that cannot allocate device memory."""
    return library().ts_hc_call_noalloc(raw, hc_norm_w, _wref(down), _wref(up), _wref(inject), mixed,
                                        inject_w, inject_stride, M, H, C, lowrank, eps, stream)


def ts_hc_replicate_entry(emb, raw, M, H, C, stream) -> int:
    return library().ts_hc_replicate_entry(emb, raw, M, H, C, stream)


def ts_hc_stack_workspace_bytes(max_chunk: int, H: int, C: int, lowrank: int) -> int:
    return library().ts_hc_stack_workspace_bytes(max_chunk, H, C, lowrank)


def ts_hc_stack(emb, T, attn, mlp, n_layers, final_mixer, sublayer, user, mixed_out, max_chunk, H, C, lowrank,
                eps, workspace, workspace_bytes, stream) -> int:
    """``attn`` / ``mlp``: ctypes arrays of ``TsHcModule`` (or None); ``final_mixer``: a
    ``TsHcModule`` (or None); ``sublayer``: a ``SUBLAYER_FN`` (or None)."""
    return library().ts_hc_stack(emb, T, attn, mlp, n_layers, _wref(final_mixer),
                                 sublayer if sublayer is not None else SUBLAYER_FN(), user, mixed_out,
                                 max_chunk, H, C, lowrank, eps, workspace, workspace_bytes, stream)


def ts_hc_stack_ple_workspace_bytes(max_chunk: int, H: int, C: int, lowrank: int) -> int:
    return library().ts_hc_stack_ple_workspace_bytes(max_chunk, H, C, lowrank)


def ts_hc_stack_ple(emb, T, attn, mlp, n_layers, final_mixer, ple, ple_rows, ple_conv_state, sublayer, user,
                    mixed_out, max_chunk, H, C, lowrank, eps, workspace, workspace_bytes, stream) -> int:
    """As ``ts_hc_stack``, with ``ple`` a ``TsHcPleModule`` (or None) and the row ids and
    conv state as device pointers."""
    return library().ts_hc_stack_ple(emb, T, attn, mlp, n_layers, _wref(final_mixer),
                                     None if ple is None else ctypes.byref(ple), ple_rows, ple_conv_state,
                                     sublayer if sublayer is not None else SUBLAYER_FN(), user, mixed_out,
                                     max_chunk, H, C, lowrank, eps, workspace, workspace_bytes, stream)


def ts_hc_rope_table(table, max_pos, rot, theta, scaling, stream) -> int:
    """``scaling``: a ``TsHcRopeScaling`` or None."""
    return library().ts_hc_rope_table(table, max_pos, rot, theta, _wref(scaling), stream)


def ts_hc_rope(q, q_stride, k, k_stride, positions, table, max_pos, q_out, q_out_stride, k_out, k_out_stride, N, q_heads,
               k_heads, D, rot, interleaved, inverse, stream) -> int:
    return library().ts_hc_rope(q, q_stride, k, k_stride, positions, table, max_pos, q_out, q_out_stride, k_out,
                                k_out_stride, N, q_heads, k_heads, D, rot, interleaved, inverse, stream)


def ts_hc_kv_write(k, k_stride, v, v_stride, cache, ctx_len, B, T, stream) -> int:
    """``cache``: a ``TsHcKvCache`` (here and below)."""
    return library().ts_hc_kv_write(k, k_stride, v, v_stride, _wref(cache), ctx_len, B, T, stream)


def ts_hc_kv_read(cache, start, k_out, v_out, B, n, stream) -> int:
    return library().ts_hc_kv_read(_wref(cache), start, k_out, v_out, B, n, stream)


def ts_hc_kv_compact(cache, ctx_len, path, n_accepted, new_len, B, T, stream) -> int:
    return library().ts_hc_kv_compact(_wref(cache), ctx_len, path, n_accepted, new_len, B, T, stream)


def ts_hc_tree_build(parents, parents_stride, ctx_len, mask, positions, B, T, stream) -> int:
    return library().ts_hc_tree_build(parents, parents_stride, ctx_len, mask, positions, B, T, stream)


def ts_hc_tree_attention_workspace_bytes(B: int, T: int, q_heads: int, cache) -> int:
    return library().ts_hc_tree_attention_workspace_bytes(B, T, q_heads, _wref(cache))


def ts_hc_tree_attention(q, q_stride, cache, ctx_len, mask, mask_stride, out, lse, B, T, q_heads, scale, workspace,
                         workspace_bytes, stream) -> int:
    return library().ts_hc_tree_attention(q, q_stride, _wref(cache), ctx_len, mask, mask_stride, out, lse, B, T, q_heads,
                                          scale, workspace, workspace_bytes, stream)


def ts_hc_verify(logits, draft_probs, tokens, parents, parents_stride, temperature, u, noise, n_accepted, path,
                 next_token, B, T, V, stream) -> int:
    return library().ts_hc_verify(logits, draft_probs, tokens, parents, parents_stride, temperature, u, noise, n_accepted,
                                  path, next_token, B, T, V, stream)


def ts_hc_selftest_timeout(stream) -> int:
    """Launches the failure-path self-test (a bounded wait that must give up)."""
    return library().ts_hc_selftest_timeout(stream)


def ts_hc_last_error() -> str:
    return library().ts_hc_last_error().decode()


def ts_hc_device_status(stream) -> Tuple[int, int]:
    v = ctypes.c_int()
    st = library().ts_hc_device_status(stream, ctypes.byref(v))
    return st, v.value


def _wref(w: Optional[TsWeight]):
    return None if w is None else ctypes.byref(w)


def _check(st: int) -> None:
    if st != TS_OK:
        raise HCError(st, ts_hc_last_error())


# ------------------------------------------------------------- torch layer

def _torch():
    import torch
    return torch


def _stream_handle(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def weight_struct(w) -> TsWeight:
    """A ``TsWeight`` for a weight with attributes kind, data, scale, bias, group
    (tensors already on the device)."""
    s = TsWeight()
    if w.kind == "bf16":
        s.type, s.group = TS_W_BF16, 0
        s.data = w.data.data_ptr()
    elif w.kind == "int4":
        s.type, s.group = TS_W_INT4_AFFINE, int(w.group)
        s.data, s.scales, s.biases = w.data.data_ptr(), w.scale.data_ptr(), w.bias.data_ptr()
    else:
        raise ValueError(f"unknown weight kind {w.kind!r}")
    return s


def _need(t, name, dtype, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise HCError(TS_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise HCError(TS_ERR_INVALID_ARG, f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise HCError(TS_ERR_INVALID_ARG, f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise HCError(TS_ERR_INVALID_ARG, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def workspace(M: int, H: int, C: int, L: int, device=None):
    torch = _torch()
    n = max(ts_hc_workspace_bytes(M, H, C, L), 256)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def hc_call(raw, weights, *, H: int, C: int, mixed=None, inject_w=None, inject_stride: Optional[int] = None,
            eps: float = RMS_EPS, ws=None, stream=None):
    """attn_hc / mlp_hc on raw [M, C*H] bf16 with ``weights`` (g, down, up, inject).

    Returns (mixed [M, H] bf16, inject_w fp32). With a caller-given ``inject_w``
    buffer and ``inject_stride``, token t's gates land at element t*inject_stride.
    """
    torch = _torch()
    M = raw.shape[0]
    L = weights.down.rows
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    _need(weights.g, "hc_norm_w", torch.bfloat16, (C * H,))
    if mixed is None:
        mixed = torch.empty((M, H), dtype=torch.bfloat16, device=raw.device)
    _need(mixed, "mixed", torch.bfloat16, (M, H))
    if inject_w is None:
        inject_stride = C
        inject_w = torch.empty((max(M, 1), C), dtype=torch.float32, device=raw.device)
    if inject_stride is None:
        raise HCError(TS_ERR_INVALID_ARG, "inject_stride is required with a caller-given inject_w")
    if ws is None:
        ws = workspace(M, H, C, L, raw.device)
    st = ts_hc_call(raw.data_ptr(), weights.g.data_ptr(), weight_struct(weights.down),
                    weight_struct(weights.up), weight_struct(weights.inject), mixed.data_ptr(),
                    inject_w.data_ptr(), inject_stride, M, H, C, L, eps, ws.data_ptr(),
                    ws.numel() * ws.element_size(), _stream_handle(stream))
    _check(st)
    return mixed, inject_w


def hc_mixer(raw, weights, *, H: int, C: int, mixed=None, eps: float = RMS_EPS, ws=None, stream=None):
    """The final hyper_connection_mixer on raw [M, C*H] bf16; returns mixed [M, H] bf16."""
    torch = _torch()
    M = raw.shape[0]
    L = weights.down.rows
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    _need(weights.g, "hc_norm_w", torch.bfloat16, (C * H,))
    if mixed is None:
        mixed = torch.empty((M, H), dtype=torch.bfloat16, device=raw.device)
    _need(mixed, "mixed", torch.bfloat16, (M, H))
    if ws is None:
        ws = workspace(M, H, C, L, raw.device)
    st = ts_hc_mixer(raw.data_ptr(), weights.g.data_ptr(), weight_struct(weights.down),
                     weight_struct(weights.up), mixed.data_ptr(), M, H, C, L, eps, ws.data_ptr(),
                     ws.numel() * ws.element_size(), _stream_handle(stream))
    _check(st)
    return mixed


def hc_call_debug(raw, weights, *, H: int, C: int, mixed=None, inject_w=None, inject_stride: Optional[int] = None,
                  eps: float = RMS_EPS, ws=None, w_out=None, stream=None):
    """``hc_call`` (or the mixer when ``weights.inject`` is None) through ``ts_hc_call_debug``.

    Returns (mixed, inject_w or None, w) with w = sigmoid(up(act)) fp32 [M, C*H].
    """
    torch = _torch()
    M = raw.shape[0]
    L = weights.down.rows
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    _need(weights.g, "hc_norm_w", torch.bfloat16, (C * H,))
    if mixed is None:
        mixed = torch.empty((M, H), dtype=torch.bfloat16, device=raw.device)
    _need(mixed, "mixed", torch.bfloat16, (M, H))
    has_inject = weights.inject is not None
    if has_inject and inject_w is None:
        inject_stride = C
        inject_w = torch.empty((max(M, 1), C), dtype=torch.float32, device=raw.device)
    if has_inject and inject_stride is None:
        raise HCError(TS_ERR_INVALID_ARG, "inject_stride is required with a caller-given inject_w")
    if w_out is None:
        w_out = torch.empty((max(M, 1), C * H), dtype=torch.float32, device=raw.device)
    _need(w_out, "w_out", torch.float32)
    if ws is None:
        ws = workspace(M, H, C, L, raw.device)
    st = ts_hc_call_debug(raw.data_ptr(), weights.g.data_ptr(), weight_struct(weights.down),
                          weight_struct(weights.up), weight_struct(weights.inject) if has_inject else None,
                          mixed.data_ptr(), inject_w.data_ptr() if has_inject else None, inject_stride or 0, M, H,
                          C, L, eps, ws.data_ptr(), ws.numel() * ws.element_size(), w_out.data_ptr(),
                          _stream_handle(stream))
    _check(st)
    return mixed, (inject_w if has_inject else None), w_out[:M]


def hc_inject_add(raw, out, inject_w, *, H: int, C: int, inject_stride: Optional[int] = None, stream=None):
    """raw[m, c*H+h] += out[m, h] * inject_w[m*stride + c], in place; returns raw."""
    torch = _torch()
    M = raw.shape[0]
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    _need(out, "out", torch.bfloat16, (M, H))
    if not inject_w.is_cuda or inject_w.dtype != torch.float32:
        raise HCError(TS_ERR_INVALID_ARG, "inject_w must be a CUDA float32 tensor")
    st = ts_hc_inject_add(raw.data_ptr(), out.data_ptr(), inject_w.data_ptr(),
                          C if inject_stride is None else inject_stride, M, H, C, _stream_handle(stream))
    _check(st)
    return raw


def hc_inject_call(raw, out, prev_inject_w, weights, *, H: int, C: int, prev_inject_stride: Optional[int] = None,
                   mixed=None, inject_w=None, inject_stride: Optional[int] = None, eps: float = RMS_EPS,
                   ws=None, stream=None):
    """The previous sublayer's inject-add fused into the next call: raw += out * prev gates
    (in place), then attn_hc / mlp_hc on it -- or the exit mixer when weights.inject is None.
    Returns (mixed, inject_w); inject_w is None for the mixer."""
    torch = _torch()
    M = raw.shape[0]
    L = weights.down.rows
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    _need(out, "out", torch.bfloat16, (M, H))
    _need(weights.g, "hc_norm_w", torch.bfloat16, (C * H,))
    if not prev_inject_w.is_cuda or prev_inject_w.dtype != torch.float32:
        raise HCError(TS_ERR_INVALID_ARG, "prev_inject_w must be a CUDA float32 tensor")
    if mixed is None:
        mixed = torch.empty((M, H), dtype=torch.bfloat16, device=raw.device)
    _need(mixed, "mixed", torch.bfloat16, (M, H))
    has_inject = weights.inject is not None
    if has_inject and inject_w is None:
        inject_stride = C
        inject_w = torch.empty((max(M, 1), C), dtype=torch.float32, device=raw.device)
    if has_inject and inject_stride is None:
        raise HCError(TS_ERR_INVALID_ARG, "inject_stride is required with a caller-given inject_w")
    if ws is None:
        ws = workspace(M, H, C, L, raw.device)
    st = ts_hc_inject_call(raw.data_ptr(), out.data_ptr(), prev_inject_w.data_ptr(),
                           C if prev_inject_stride is None else prev_inject_stride, weights.g.data_ptr(),
                           weight_struct(weights.down), weight_struct(weights.up),
                           weight_struct(weights.inject) if has_inject else None, mixed.data_ptr(),
                           inject_w.data_ptr() if has_inject else None, inject_stride or 0, M, H, C, L, eps,
                           ws.data_ptr(), ws.numel() * ws.element_size(), _stream_handle(stream))
    _check(st)
    return mixed, (inject_w if has_inject else None)


def hc_entry_call(emb, weights, *, C: int, raw=None, mixed=None, inject_w=None, inject_stride: Optional[int] = None,
                  eps: float = RMS_EPS, ws=None, stream=None):
    """The entry replication fused into the first call: raw [M, C*H] = emb [M, H] repeated C
    times (written), then attn_hc on it -- or the mixer when weights.inject is None.
    Returns (raw, mixed, inject_w or None)."""
    torch = _torch()
    M, H = emb.shape
    L = weights.down.rows
    _need(emb, "emb", torch.bfloat16, (M, H))
    _need(weights.g, "hc_norm_w", torch.bfloat16, (C * H,))
    if raw is None:
        raw = torch.empty((M, C * H), dtype=torch.bfloat16, device=emb.device)
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    if mixed is None:
        mixed = torch.empty((M, H), dtype=torch.bfloat16, device=emb.device)
    _need(mixed, "mixed", torch.bfloat16, (M, H))
    has_inject = weights.inject is not None
    if has_inject and inject_w is None:
        inject_stride = C
        inject_w = torch.empty((max(M, 1), C), dtype=torch.float32, device=emb.device)
    if has_inject and inject_stride is None:
        raise HCError(TS_ERR_INVALID_ARG, "inject_stride is required with a caller-given inject_w")
    if ws is None:
        ws = workspace(M, H, C, L, emb.device)
    st = ts_hc_entry_call(emb.data_ptr(), raw.data_ptr(), weights.g.data_ptr(), weight_struct(weights.down),
                          weight_struct(weights.up), weight_struct(weights.inject) if has_inject else None,
                          mixed.data_ptr(), inject_w.data_ptr() if has_inject else None, inject_stride or 0, M, H, C,
                          L, eps, ws.data_ptr(), ws.numel() * ws.element_size(), _stream_handle(stream))
    _check(st)
    return raw, mixed, (inject_w if has_inject else None)


def hc_exit_logits(raw, weights, lm_head, *, H: int, C: int, out=None, prev_inject_w=None,
                   prev_inject_stride: Optional[int] = None, mixed=None, logits=None, eps: float = RMS_EPS, ws=None,
                   stream=None):
    """The decoder's exit: with ``out`` given, raw += out * prev gates (in place) first; then the
    mixer (``weights``: g, down, up) and lm_head [V, H] bf16. Returns (mixed [M, H] bf16,
    logits [M, V] fp32)."""
    torch = _torch()
    M = raw.shape[0]
    L = weights.down.rows
    V = lm_head.shape[0]
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    _need(weights.g, "hc_norm_w", torch.bfloat16, (C * H,))
    _need(lm_head, "lm_head", torch.bfloat16, (V, H))
    if mixed is None:
        mixed = torch.empty((M, H), dtype=torch.bfloat16, device=raw.device)
    _need(mixed, "mixed", torch.bfloat16, (M, H))
    if logits is None:
        logits = torch.empty((M, V), dtype=torch.float32, device=raw.device)
    _need(logits, "logits", torch.float32, (M, V))
    if out is not None:
        _need(out, "out", torch.bfloat16, (M, H))
        if prev_inject_w is None or not prev_inject_w.is_cuda or prev_inject_w.dtype != torch.float32:
            raise HCError(TS_ERR_INVALID_ARG, "prev_inject_w must be a CUDA float32 tensor with out")
    if ws is None:
        ws = workspace(M, H, C, L, raw.device)
    st = ts_hc_exit_logits(raw.data_ptr(), out.data_ptr() if out is not None else None,
                           prev_inject_w.data_ptr() if out is not None else None,
                           (C if prev_inject_stride is None else prev_inject_stride) if out is not None else 0,
                           weights.g.data_ptr(), weight_struct(weights.down), weight_struct(weights.up),
                           lm_head.data_ptr(), V, mixed.data_ptr(), logits.data_ptr(), M, H, C, L, eps, ws.data_ptr(),
                           ws.numel() * ws.element_size(), _stream_handle(stream))
    _check(st)
    return mixed, logits


def hc_ple(hidden, rows, weights, conv_state, *, C: int, eps: float = RMS_EPS, ws=None, stream=None):
    """The PLE gate on hidden [M, C*H] bf16 (in place) for M consecutive tokens of one
    sequence. ``rows`` int32 [M, 16] table row ids; ``weights`` has table, key_proj,
    value_proj, norm_key, norm_query, norm_conv, conv_w; ``conv_state`` fp32 [9, C*H]
    (updated). Returns (hidden, the workspace)."""
    torch = _torch()
    M = hidden.shape[0]
    H = weights.value_proj.shape[0]
    W = C * H
    _need(hidden, "hidden", torch.bfloat16, (M, W))
    _need(rows, "rows", torch.int32, (M, 16))
    _need(weights.table, "table", torch.bfloat16)
    _need(weights.key_proj, "key_proj", torch.bfloat16, (W, H))
    _need(weights.value_proj, "value_proj", torch.bfloat16, (H, H))
    for name in ("norm_key", "norm_query", "norm_conv"):
        _need(getattr(weights, name), name, torch.bfloat16, (W,))
    _need(weights.conv_w, "conv_w", torch.bfloat16, (W, 4))
    _need(conv_state, "conv_state", torch.float32, (9, W))
    if ws is None:
        ws = torch.empty(max(ts_hc_ple_workspace_bytes(M, H, C), 256), dtype=torch.uint8, device=hidden.device)
    st = ts_hc_ple(hidden.data_ptr(), rows.data_ptr(), weights.table.data_ptr(), weights.table.shape[0],
                   weights.key_proj.data_ptr(), weights.value_proj.data_ptr(), weights.norm_key.data_ptr(),
                   weights.norm_query.data_ptr(), weights.norm_conv.data_ptr(), weights.conv_w.data_ptr(),
                   conv_state.data_ptr(), M, H, C, eps, ws.data_ptr(), ws.numel() * ws.element_size(),
                   _stream_handle(stream))
    _check(st)
    return hidden, ws


def hc_replicate_entry(emb, *, C: int, raw=None, stream=None):
    """raw [M, C*H] bf16 with every stream equal to emb [M, H] (repeat, not pad)."""
    torch = _torch()
    M, H = emb.shape
    _need(emb, "emb", torch.bfloat16, (M, H))
    if raw is None:
        raw = torch.empty((M, C * H), dtype=torch.bfloat16, device=emb.device)
    _need(raw, "raw", torch.bfloat16, (M, C * H))
    _check(ts_hc_replicate_entry(emb.data_ptr(), raw.data_ptr(), M, H, C, _stream_handle(stream)))
    return raw


def device_status(stream=None) -> int:
    st, v = ts_hc_device_status(_stream_handle(stream))
    _check(st)
    return v


def module_struct(w) -> TsHcModule:
    """A ``TsHcModule`` for weights with attributes g, down, up, inject (inject may be None)."""
    m = TsHcModule()
    m.hc_norm_w = w.g.data_ptr()
    m.down, m.up = weight_struct(w.down), weight_struct(w.up)
    if w.inject is not None:
        m.inject = weight_struct(w.inject)
    return m


def stack_workspace(max_chunk: int, H: int, C: int, L: int, device=None, with_ple: bool = False):
    torch = _torch()
    n = (ts_hc_stack_ple_workspace_bytes if with_ple else ts_hc_stack_workspace_bytes)(max_chunk, H, C, L)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def ple_module_struct(w) -> TsHcPleModule:
    """A ``TsHcPleModule`` for PLE weights with attributes table, key_proj, value_proj,
    norm_key, norm_query, norm_conv, conv_w."""
    m = TsHcPleModule()
    m.table = w.table.data_ptr()
    m.n_rows = w.table.shape[0]
    m.key_proj, m.value_proj = w.key_proj.data_ptr(), w.value_proj.data_ptr()
    m.norm_key_w, m.norm_query_w = w.norm_key.data_ptr(), w.norm_query.data_ptr()
    m.norm_conv_w, m.conv_w = w.norm_conv.data_ptr(), w.conv_w.data_ptr()
    return m


def hc_stack(emb, layers, final, sublayer, *, C: int, max_chunk: Optional[int] = None, mixed_out=None,
             eps: float = RMS_EPS, ws=None, stream=None, ple=None, ple_rows=None, ple_state=None):
    """The decoder stack's hyper-connection path on T tokens through ``ts_hc_stack``
    (``ts_hc_stack_ple`` when ``ple`` is given).

    ``emb`` [T, H] bf16; ``layers``: a sequence of (attn, mlp) weights (g, down, up,
    inject); ``final``: the exit mixer's weights. ``sublayer(layer, which, t0, mixed)``
    gets the call's output ``mixed`` ([M, H] bf16, a view into the workspace) and
    returns the sublayer output, a CUDA bf16 tensor [M, H] that it may compute on the
    current stream; the driver injects it with the call's gates. ``ple``: PLE weights
    (table, key_proj, value_proj, norm_key, norm_query, norm_conv, conv_w) applied
    before layer 1's attn_hc, with ``ple_rows`` int32 [T, 16] and ``ple_state`` fp32
    [9, C*H] (updated). Returns (mixed_out [T, H], the last chunk's residual
    [M, C*H] -- a view into ``ws``).
    """
    torch = _torch()
    T, H = emb.shape
    L = final.down.rows
    _need(emb, "emb", torch.bfloat16, (T, H))
    max_chunk = max(T, 1) if max_chunk is None else max_chunk
    if mixed_out is None:
        mixed_out = torch.empty((T, H), dtype=torch.bfloat16, device=emb.device)
    _need(mixed_out, "mixed_out", torch.bfloat16, (T, H))
    if ple is not None:
        _need(ple_rows, "ple_rows", torch.int32, (T, 16))
        _need(ple_state, "ple_state", torch.float32, (9, C * H))
    if ws is None:
        ws = stack_workspace(max_chunk, H, C, L, emb.device, with_ple=ple is not None)
    n = len(layers)
    attn = (TsHcModule * max(n, 1))(*[module_struct(a) for a, _ in layers])
    mlp = (TsHcModule * max(n, 1))(*[module_struct(m) for _, m in layers])
    fin = module_struct(final)
    keep, errors = [], []
    base = ws.data_ptr()

    def trampoline(user, layer, which, t0, M, mixed_ptr, out_pp, stream_h):
        try:
            off = mixed_ptr - base
            mixed = ws[off:off + 2 * M * H].view(torch.bfloat16).view(M, H)
            out = sublayer(layer, which, t0, mixed)
            _need(out, "sublayer output", torch.bfloat16, (M, H))
            if stream is not None:  # the caching allocator must not hand it out before the driver's stream used it
                out.record_stream(stream)
            keep.append(out)
            out_pp[0] = out.data_ptr()
            return TS_OK
        except Exception as e:  # reported after the C call returns
            errors.append(e)
            return TS_ERR_INVALID_ARG

    fn = SUBLAYER_FN(trampoline)
    if ple is None:
        st = ts_hc_stack(emb.data_ptr(), T, attn, mlp, n, fin, fn, None, mixed_out.data_ptr(), max_chunk, H, C,
                         L, eps, base, ws.numel() * ws.element_size(), _stream_handle(stream))
    else:
        st = ts_hc_stack_ple(emb.data_ptr(), T, attn, mlp, n, fin, ple_module_struct(ple), ple_rows.data_ptr(),
                             ple_state.data_ptr(), fn, None, mixed_out.data_ptr(), max_chunk, H, C, L, eps, base,
                             ws.numel() * ws.element_size(), _stream_handle(stream))
    if errors:
        raise errors[0]
    _check(st)
    M_last = T - (max(T, 1) - 1) // max_chunk * max_chunk if T else 0
    raw_last = ws[:2 * M_last * C * H].view(torch.bfloat16).view(M_last, C * H)
    return mixed_out, raw_last


# ------------------------------------------------------------- a speculative decoding step

# These calls run once per layer and step on a few rows, where their host time is what counts: what is
# checked for every tensor is checked here with a few attribute reads, and the errors are worded elsewhere.

def _rows(t, name):
    """(tokens, heads, D, token stride) of bf16 rows [N, heads, D] or [B, T, heads, D]: each token's
    heads side by side, the tokens at one stride (a slice of a projection's output will do)."""
    torch = _torch()
    try:
        ok = t.dtype is torch.bfloat16 and t.is_cuda
        shape, stride = t.shape, t.stride()
    except AttributeError:
        ok = False
    if not ok:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise HCError(TS_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
        raise HCError(TS_ERR_INVALID_ARG, f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if len(shape) == 3:
        n, h, d = shape
        step = stride[0]
    elif len(shape) == 4:
        b, n, h, d = shape
        step = stride[1] if n != 1 else stride[0]
        if b > 1 and n > 1 and stride[0] != n * step:
            raise HCError(TS_ERR_INVALID_ARG, f"{name}: its sequences' tokens are not at one stride: {tuple(stride)}")
        n *= b
    else:
        raise HCError(TS_ERR_INVALID_ARG, f"{name} has shape {tuple(shape)}, expected [tokens, heads, D] or [B, T, heads, D]")
    if (stride[-1] != 1 and d > 1) or (stride[-2] != d and h > 1):
        raise HCError(TS_ERR_INVALID_ARG, f"{name}: a token's heads must lie side by side, strides are {tuple(stride)}")
    return n, h, d, step if n > 1 else h * d


def _is(t, name, dtype, shape=None):
    """``_need`` with its common answer found first; returns the address."""
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous() and (shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtype, shape)
    return t.data_ptr()


def _stream_of(stream, t) -> int:
    """The handle of ``stream``, or of the stream that is current on ``t``'s device."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(t.get_device())  # current_stream() without its object: 0.1 us for 3


def _made(t, stream):
    """A tensor that this module allocated, about to be used on ``stream`` (None: the current one)."""
    if stream is not None:
        t.record_stream(stream)
    return t


def rope_table(max_pos: int, rot: int, theta: float, *, scaling: Optional[TsHcRopeScaling] = None, device=None, stream=None):
    """The rotary table fp32 [max_pos, rot/2, 2] of (cos, sin) for ``hc_rope``."""
    torch = _torch()
    table = _made(torch.empty((max_pos, max(rot // 2, 0), 2), dtype=torch.float32, device=device or "cuda"), stream)
    _check(ts_hc_rope_table(table.data_ptr(), max_pos, rot, theta, scaling, _stream_handle(stream)))
    return table


def hc_rope(q, k, positions, table, *, interleaved: bool = False, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions of ``q`` [N, q_heads, D] and ``k`` [N, k_heads, D] (or [B, T, heads, D]; k may be
    None) bf16 at ``positions`` int32 (N of them), by ``table`` [max_pos, rot/2, 2]. ``inverse`` turns back
    (the gradient). Returns (q_out, k_out); passing q and k as them turns in place."""
    torch = _torch()
    n, hq, d, sq = _rows(q, "q")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        if stream is not None:
            q_out.record_stream(stream)
        so = hq * d
    else:
        no, ho, do, so = _rows(q_out, "q_out")
        if (no, ho, do) != (n, hq, d):
            raise HCError(TS_ERR_INVALID_ARG, f"q_out has shape {tuple(q_out.shape)}, expected {tuple(q.shape)}")
    hk, sk, sko, kp, kop = 0, 0, 0, None, None
    if k is not None:
        nk, hk, dk, sk = _rows(k, "k")
        if nk != n or dk != d:
            raise HCError(TS_ERR_INVALID_ARG, f"k has shape {tuple(k.shape)}, q has {tuple(q.shape)}")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=q.device)
            if stream is not None:
                k_out.record_stream(stream)
            sko = hk * d
        else:
            no, ho, do, sko = _rows(k_out, "k_out")
            if (no, ho, do) != (n, hk, d):
                raise HCError(TS_ERR_INVALID_ARG, f"k_out has shape {tuple(k_out.shape)}, expected {tuple(k.shape)}")
        kp, kop = k.data_ptr(), k_out.data_ptr()
    pp = _is(positions, "positions", torch.int32)
    if positions.numel() != n:
        raise HCError(TS_ERR_INVALID_ARG, f"positions has {positions.numel()} entries for {n} tokens")
    tp = _is(table, "table", torch.float32)
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2:
        raise HCError(TS_ERR_INVALID_ARG, f"table has shape {tuple(shape)}, expected [max_pos, rot/2, 2]")
    st = (_lib or library()).ts_hc_rope(q.data_ptr(), sq, kp, sk, pp, tp, shape[0], q_out.data_ptr(), so, kop, sko, n, hq, hk, d,
                                        2 * shape[1], interleaved, inverse, _stream_of(stream, q))
    if st:
        _check(st)
    return q_out, k_out


class KVCache:
    """A paged cache of one layer's keys and values: the caller's tensors and their format.

    ``kind`` "bf16": k, v bf16 [pages, heads, page_size, D]; "fp8": uint8 (e4m3 codes) of that shape and
    k_scale, v_scale uint8 [pages, heads, page_size]; "int4": uint8 [pages, heads, page_size, D/2] and
    k_scale, v_scale, k_bias, v_bias fp16 [pages, heads, page_size, D/group]. ``page_table`` int32
    [B, max_pages]. The tensors are read and written where they are; replacing one makes a new KVCache.
    """

    def __init__(self, kind: str, k, v, page_table, *, k_scale=None, v_scale=None, k_bias=None, v_bias=None, group: int = 0):
        torch = _torch()
        kinds = {"bf16": TS_KV_BF16, "fp8": TS_KV_FP8, "int4": TS_KV_INT4}
        if kind not in kinds:
            raise HCError(TS_ERR_INVALID_ARG, f"unknown cache kind {kind!r}")
        dtype = torch.bfloat16 if kind == "bf16" else torch.uint8
        _need(k, "cache.k", dtype)
        if k.dim() != 4:
            raise HCError(TS_ERR_INVALID_ARG, f"cache.k has shape {tuple(k.shape)}, expected [pages, heads, page_size, row]")
        _need(v, "cache.v", dtype, k.shape)
        pages, heads, size, row = k.shape
        d = row * 2 if kind == "int4" else row
        _need(page_table, "cache.page_table", torch.int32)
        if page_table.dim() != 2:
            raise HCError(TS_ERR_INVALID_ARG, f"cache.page_table has shape {tuple(page_table.shape)}, expected [B, max_pages]")
        if kind == "fp8":
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                _need(t, "cache." + name, torch.uint8, (pages, heads, size))
        if kind == "int4":
            if group not in (32, 64, 128) or d % group:
                raise HCError(TS_ERR_UNSUPPORTED, f"cache.group = {group}: INT4 groups of 32, 64 or 128 and at most head_dim = {d} are supported")
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale), ("k_bias", k_bias), ("v_bias", v_bias)):
                _need(t, "cache." + name, torch.float16, (pages, heads, size, d // group))
        self.kind, self.group, self.page_size, self.heads, self.head_dim = kind, group, size, heads, d
        self.batch, self.max_pages = page_table.shape
        self.lengths = (self.batch,)
        self.tensors = (k, v, page_table, k_scale, v_scale, k_bias, v_bias)  # kept alive with the struct
        self.struct = TsHcKvCache(kinds[kind], group, size, heads, d, self.max_pages, pages, k.data_ptr(), v.data_ptr(),
                                  *(t.data_ptr() if t is not None else None for t in (k_scale, v_scale, k_bias, v_bias)),
                                  page_table.data_ptr())
        self.ref = ctypes.byref(self.struct)


def kv_cache(kind: str, pages: int, heads: int, page_size: int, head_dim: int, page_table, *, group: int = 64) -> KVCache:
    """A ``KVCache`` over newly allocated, zeroed tensors."""
    torch = _torch()
    dev, lead = page_table.device, (pages, heads, page_size)
    zeros = lambda *shape, dtype: torch.zeros(shape, dtype=dtype, device=dev)  # noqa: E731
    if kind == "bf16":
        return KVCache(kind, *(zeros(*lead, head_dim, dtype=torch.bfloat16) for _ in range(2)), page_table)
    if kind == "fp8":
        k, v = (zeros(*lead, head_dim, dtype=torch.uint8) for _ in range(2))
        ks, vs = (zeros(*lead, dtype=torch.uint8) for _ in range(2))
        return KVCache(kind, k, v, page_table, k_scale=ks, v_scale=vs)
    k, v = (zeros(*lead, head_dim // 2, dtype=torch.uint8) for _ in range(2))
    ks, vs, kb, vb = (zeros(*lead, head_dim // max(group, 1), dtype=torch.float16) for _ in range(4))
    return KVCache(kind, k, v, page_table, k_scale=ks, v_scale=vs, k_bias=kb, v_bias=vb, group=group)


def hc_kv_write(k, v, cache: KVCache, ctx_len, *, stream=None):
    """Stores ``k``, ``v`` [B, T, heads, D] bf16 at positions ctx_len[b] .. ctx_len[b] + T - 1, quantised to
    the cache's kind; ``ctx_len`` int32 [B]. Returns the cache."""
    _, h, d, sk = _rows(k, "k")
    _, _, _, sv = _rows(v, "v")
    shape = k.shape
    if len(shape) != 4 or shape[0] != cache.batch or h != cache.heads or d != cache.head_dim:
        raise HCError(TS_ERR_INVALID_ARG, f"k has shape {tuple(shape)}, expected [{cache.batch}, T, {cache.heads}, {cache.head_dim}]")
    if v.shape != shape:
        raise HCError(TS_ERR_INVALID_ARG, f"v has shape {tuple(v.shape)}, k has {tuple(shape)}")
    st = (_lib or library()).ts_hc_kv_write(k.data_ptr(), sk, v.data_ptr(), sv, cache.ref,
                                            _is(ctx_len, "ctx_len", _torch().int32, cache.lengths), cache.batch, shape[1],
                                            _stream_of(stream, k))
    if st:
        _check(st)
    return cache


def hc_kv_read(cache: KVCache, start, n: int, *, k_out=None, v_out=None, stream=None):
    """Positions start[b] .. start[b] + n - 1 of each sequence as bf16 [B, n, heads, D]; ``start`` int32 [B].
    Returns (k, v)."""
    torch = _torch()
    shape = (cache.batch, n, cache.heads, cache.head_dim)
    sp = _is(start, "start", torch.int32, cache.lengths)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=start.device)
        if stream is not None:
            k_out.record_stream(stream)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=start.device)
        if stream is not None:
            v_out.record_stream(stream)
    st = (_lib or library()).ts_hc_kv_read(cache.ref, sp, _is(k_out, "k_out", torch.bfloat16, shape),
                                           _is(v_out, "v_out", torch.bfloat16, shape), cache.batch, n, _stream_of(stream, start))
    if st:
        _check(st)
    return k_out, v_out


def hc_kv_compact(cache: KVCache, ctx_len, path, n_accepted, *, new_len=None, stream=None):
    """Moves the accepted nodes' rows (``path`` int32 [B, T] and ``n_accepted`` int32 [B] of ``hc_verify``)
    to the positions after ``ctx_len``; returns new_len int32 [B] = ctx_len + n_accepted + 1. A path that is
    refused at a step (recorded, see ``device_status``) counts the steps before it."""
    torch = _torch()
    cp = _is(ctx_len, "ctx_len", torch.int32, cache.lengths)
    np_ = _is(n_accepted, "n_accepted", torch.int32, cache.lengths)
    pp = _is(path, "path", torch.int32)
    if path.dim() != 2 or path.shape[0] != cache.batch:
        raise HCError(TS_ERR_INVALID_ARG, f"path has shape {tuple(path.shape)}, expected [{cache.batch}, T]")
    if new_len is None:
        new_len = _made(torch.empty_like(ctx_len), stream)
    st = (_lib or library()).ts_hc_kv_compact(cache.ref, cp, pp, np_, _is(new_len, "new_len", torch.int32, cache.lengths), cache.batch,
                                              path.shape[1], _stream_of(stream, ctx_len))
    if st:
        _check(st)
    return new_len


def hc_tree_build(parents, ctx_len=None, *, batch: Optional[int] = None, mask=None, positions=None, stream=None):
    """(mask int32 [B, T, ceil(T/32)], positions int32 [B, T]) of trees given by ``parents`` int32 [B, T], or
    [T] for one tree that ``batch`` sequences (or ctx_len's) share."""
    torch = _torch()
    _need(parents, "parents", torch.int32)
    t = parents.shape[-1]
    if parents.dim() == 1:
        b, step = (ctx_len.shape[0] if ctx_len is not None else batch or 1), 0
    else:
        b, step = parents.shape[0], t
    if parents.dim() > 2 or (batch is not None and batch != b):
        raise HCError(TS_ERR_INVALID_ARG, f"parents has shape {tuple(parents.shape)}, expected [B, T] or [T]")
    if ctx_len is not None:
        _need(ctx_len, "ctx_len", torch.int32, (b,))
    if mask is None:
        mask = _made(torch.empty((b, t, (t + 31) // 32), dtype=torch.int32, device=parents.device), stream)
    _need(mask, "mask", torch.int32, (b, t, (t + 31) // 32))
    if positions is None:
        positions = _made(torch.empty((b, t), dtype=torch.int32, device=parents.device), stream)
    _need(positions, "positions", torch.int32, (b, t))
    _check(ts_hc_tree_build(parents.data_ptr(), step, None if ctx_len is None else ctx_len.data_ptr(), mask.data_ptr(),
                            positions.data_ptr(), b, t, _stream_of(stream, parents)))
    return mask, positions


def tree_attention_workspace(B: int, T: int, q_heads: int, cache: KVCache, device=None):
    torch = _torch()
    n = ts_hc_tree_attention_workspace_bytes(B, T, q_heads, cache.struct)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or cache.tensors[0].device)


def hc_tree_attention(q, cache: KVCache, ctx_len, *, mask=None, scale: Optional[float] = None, out=None, lse=None, ws=None,
                      stream=None):
    """Attention of ``q`` [B, T, q_heads, D] bf16, the nodes at ctx_len[b] .. ctx_len[b] + T - 1, over the cache.
    ``mask`` int32 [B, T, ceil(T/32)] (or [T, ceil(T/32)] for one tree) of ``hc_tree_build``; None: a chain.
    ``scale`` defaults to D ** -0.5. Returns (out bf16 [B, T, q_heads, D], lse fp32 [B, T, q_heads])."""
    torch = _torch()
    _, h, d, sq = _rows(q, "q")
    shape = q.shape
    if len(shape) != 4 or shape[0] != cache.batch or d != cache.head_dim:
        raise HCError(TS_ERR_INVALID_ARG, f"q has shape {tuple(shape)}, expected [{cache.batch}, T, heads, {cache.head_dim}]")
    b, t = shape[0], shape[1]
    mp, step = None, 0
    if mask is not None:
        words = (t + 31) // 32
        if mask.dim() == 2:
            mp = _is(mask, "mask", torch.int32, (t, words))
        else:
            mp, step = _is(mask, "mask", torch.int32, (b, t, words)), t * words
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
        if stream is not None:
            out.record_stream(stream)
        op = out.data_ptr()
    else:
        op = _is(out, "out", torch.bfloat16, shape)
    if lse is None:
        lse = torch.empty((b, t, h), dtype=torch.float32, device=q.device)
        if stream is not None:
            lse.record_stream(stream)
        lp = lse.data_ptr()
    else:
        lp = _is(lse, "lse", torch.float32, (b, t, h))
    if ws is None:
        ws = _made(tree_attention_workspace(b, t, h, cache, q.device), stream)
    st = (_lib or library()).ts_hc_tree_attention(q.data_ptr(), sq, cache.ref, _is(ctx_len, "ctx_len", torch.int32, cache.lengths), mp,
                                                  step, op, lp, b, t, h, d ** -0.5 if scale is None else scale, ws.data_ptr(), ws.nbytes,
                                                  _stream_of(stream, q))
    if st:
        _check(st)
    return out, lse


def hc_verify(logits, tokens, parents=None, temperature=None, *, draft_probs=None, u=None, noise=None, n_accepted=None, path=None,
              next_token=None, stream=None):
    """Which of the drafted ``tokens`` int32 [B, T] hold, given the target's ``logits`` fp32 [B, T, V] and the
    draft's ``draft_probs`` fp32 [B, T, V]; ``parents`` int32 [B, T], [T] or None (a chain); ``temperature``
    fp32 [B]; ``u`` fp32 [B, T] in [0, 1) and ``noise`` fp32 [B, V] exponential variates. Without draft_probs, u
    and noise every sequence is greedy. Returns (n_accepted [B], path [B, T], next_token [B]), int32. A walk
    ends, with next token 0, at logits that are no distribution (recorded, see ``device_status``)."""
    torch = _torch()
    i32, f32 = torch.int32, torch.float32
    lp = _is(logits, "logits", f32)
    shape = logits.shape
    if len(shape) != 3:
        raise HCError(TS_ERR_INVALID_ARG, f"logits has shape {tuple(shape)}, expected [B, T, V]")
    b, t, v = shape
    tp = _is(tokens, "tokens", i32, (b, t))
    step, pp, dp, up, np_, cp = 0, None, None, None, None, None
    if parents is not None:
        if parents.dim() == 1:
            pp = _is(parents, "parents", i32, (t,))
        else:
            pp, step = _is(parents, "parents", i32, (b, t)), t
    if draft_probs is not None:
        dp, up = _is(draft_probs, "draft_probs", f32, shape), _is(u, "u", f32, (b, t))
        np_, cp = _is(noise, "noise", f32, (b, v)), _is(temperature, "temperature", f32, (b,))
    elif u is not None or noise is not None:
        raise HCError(TS_ERR_INVALID_ARG, "draft_probs, u and noise are given together, or none of them (greedy)")
    if n_accepted is None:
        n_accepted = _made(torch.empty(b, dtype=i32, device=logits.device), stream)
    if path is None:
        path = _made(torch.empty((b, t), dtype=i32, device=logits.device), stream)
    if next_token is None:
        next_token = _made(torch.empty(b, dtype=i32, device=logits.device), stream)
    st = (_lib or library()).ts_hc_verify(lp, dp, tp, pp, step, cp, up, np_, _is(n_accepted, "n_accepted", i32, (b,)),
                                          _is(path, "path", i32, (b, t)), _is(next_token, "next_token", i32, (b,)), b, t, v,
                                          _stream_of(stream, logits))
    if st:
        _check(st)
    return n_accepted, path, next_token
