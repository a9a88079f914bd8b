"""Thin Python binding over libminf.so: argument marshalling only.

Every function has the C ABI's name and argument order (include/minf.h), takes
torch CUDA tensors in place of device pointers, and raises MinfError on a
non-zero status.  All arithmetic runs in the library's kernels; there is no
CPU path.  If the library is missing, the first call raises -- nothing falls
back to another implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

MINF_OK = 0
MINF_ERR_ARG = 1
MINF_ERR_GEOMETRY = 2
MINF_ERR_UNSUPPORTED = 3
MINF_ERR_WORKSPACE = 5
MINF_ERR_CUDA = 6
ERRBIT_STORE_POS = 0x1
ERRBIT_ROPE_POS = 0x2
ERRBIT_ATTN_POS = 0x4
ERRBIT_TIMEOUT = 0x8
ERRBIT_BLOCK = 0x10
ERRBIT_WORKSPACE = 0x20
ERRBIT_CHUNK = 0x40

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_I64 = ctypes.c_int64

_SIGS = {
    "minf_status_string": ([_I], ctypes.c_char_p),
    "minf_version": ([], _I),
    "minf_rope_freqs": ([_P, _I, _F, _F], _I),
    "minf_rms_norm": ([_P, _P, _P, _I, _I, _F, _P], _I),
    "minf_rope": ([_P, _P, _I, _I, _I, _F, _F, _I, _P, _P], _I),
    "minf_kv_append": ([_P, _P, _I, _I, _P, _P, _P, _I, _P, _P], _I),
    "minf_rope_kv_append": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _I, _P, _P], _I),
    "minf_attn_decode_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "minf_attn_prefill_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "minf_gqa_attn_decode": ([_P, _P, _P, _P, _P, _P, _I, _I64, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P], _I),
    "minf_gqa_attn_decode_static_ws": ([_P, _P, _P, _P, _P, _P, _I, _I64, _P, _I, _I, _I, _I, _I, _F, _P, _P], _I),
    "minf_gqa_attn_prefill": ([_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                              _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    # the same step with early start (the launch before writes neither pos nor cached rows)
    "minf_layer_attn_step_chained": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                      _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_chained_f16": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                          _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_chained_q8": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                         _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_batched": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I64,
                                      _I, _I, _I, _I, _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_silu_mul": ([_P, _P, _P, _I64, _P], _I),
    # binary16 regions (torch.float16 tensors): the same arguments as the fp32 entry points
    "minf_kv_append_f16": ([_P, _P, _I, _I, _P, _P, _P, _I, _P, _P], _I),
    "minf_rope_kv_append_f16": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _I, _P, _P], _I),
    "minf_gqa_attn_decode_f16": ([_P, _P, _P, _P, _P, _P, _I, _I64, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P,
                                  _P], _I),
    "minf_gqa_attn_prefill_f16": ([_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_f16": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                  _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_batched_f16": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I64,
                                          _I, _I, _I, _I, _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    # Q8_0 regions (torch.uint8 tensors of rows of minf_q8_row_bytes(W) bytes)
    "minf_q8_row_bytes": ([_I], _SZ),
    "minf_kv_append_q8": ([_P, _P, _I, _I, _P, _P, _P, _I, _P, _P], _I),
    "minf_rope_kv_append_q8": ([_P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _I, _P, _P], _I),
    "minf_gqa_attn_decode_q8": ([_P, _P, _P, _P, _P, _P, _I, _I64, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P],
                                _I),
    "minf_gqa_attn_prefill_q8": ([_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_q8": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                 _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_batched_q8": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I64,
                                         _I, _I, _I, _I, _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_kv_append_paged_q8": ([_P, _P, _I64, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P], _I),
    "minf_gqa_attn_decode_paged_q8": ([_P, _P, _P, _P, _I64, _P, _I, _I, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P,
                                       _P], _I),
    "minf_layer_attn_step_paged_q8": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I64, _P, _I, _I, _I, _I,
                                       _I, _I, _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    # Q4 rows (torch.uint8 tensors of rows of minf_q4_row_bytes(W) bytes)
    "minf_q4_row_bytes": ([_I], _SZ),
    "minf_kv_append_q4": ([_P, _P, _I, _I, _P, _P, _P, _I, _P, _P], _I),
    # the fused QKV decode op
    "minf_fused_qkv": ([_P, _P, _P, _F, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _F, _I, _P,
                        _P], _I),
    "minf_layer_attn_step_qkv": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _F,
                                  _I, _P, _P, _SZ, _P, _P], _I),
    # paged regions: a pool of blocks and a block table per sequence
    "minf_kv_append_paged": ([_P, _P, _I64, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P], _I),
    "minf_kv_append_paged_f16": ([_P, _P, _I64, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P], _I),
    "minf_gqa_attn_decode_paged": ([_P, _P, _P, _P, _I64, _P, _I, _I, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P, _P],
                                   _I),
    "minf_gqa_attn_decode_paged_f16": ([_P, _P, _P, _P, _I64, _P, _I, _I, _P, _I, _I, _I, _I, _I, _F, _P, _SZ, _P,
                                        _P], _I),
    "minf_layer_attn_step_paged": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I64, _P, _I, _I, _I, _I, _I,
                                    _I, _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    "minf_layer_attn_step_paged_f16": ([_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _I64, _P, _I, _I, _I, _I,
                                        _I, _I, _F, _F, _I, _P, _P, _SZ, _P, _P], _I),
    # chunks of new tokens: several-axis RoPE, RoPE + store into paged regions, read back, attention
    "minf_rope_axes": ([_P, _P, _P, _I, _I, _P, _I, _I, _F, _F, _I, _P, _P], _I),
    "minf_attn_chunk_workspace_bytes": ([_I, _I, _I, _I, _I, _I], _SZ),
    # block tables from lengths, blocks given back
    "minf_block_table_grow": ([_P, _I, _I, _I64, _P, _P, _I, _P, _I, _P, _P, _P, _P, _P, _I, _P, _P], _I),
    "minf_block_table_release": ([_P, _I, _I, _I64, _P, _P, _I, _P, _I, _P, _P, _P, _P], _I),
}
for _end in ("", "_f16", "_q8", "_q4"):
    _SIGS["minf_rope_kv_append_chunk_paged" + _end] = (
        [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _I64, _P, _I, _I, _P, _P],
        _I)
    _SIGS["minf_kv_read_chunk_paged" + _end] = (
        [_P, _P, _I, _P, _P, _I64, _I, _P, _I, _I, _P, _P, _I, _I, _P, _P], _I)
    _SIGS["minf_gqa_attn_chunk_paged" + _end] = (
        [_P, _P, _P, _P, _I64, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P, _P], _I)
    _SIGS["minf_gqa_attn_window" + _end] = (
        [_P, _P, _P, _P, _P, _P, _I, _I64, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P, _P], _I)
    _SIGS["minf_layer_attn_step_chunk_paged" + _end] = (
        [_P, _P, _P, _F, _I, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _P, _P, _I64, _P, _I, _I, _I, _I, _I, _I, _F,
         _F, _I, _I, _I, _P, _P, _SZ, _P, _P], _I)


class MinfError(RuntimeError):
    def __init__(self, status: int, name: str):
        msg = lib().minf_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{name}: status {status} ({msg})")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def lib():
    """The loaded library (ctypes).  Raises if libminf.so has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"libminf.so is not built ({path}); run "
                                   "`python -c 'import __graft_entry__ as g; g.build()'` first")
            handle = ctypes.CDLL(path)
            for name, (args, res) in _SIGS.items():
                fn = getattr(handle, name)
                fn.argtypes = args
                fn.restype = res
            _lib = handle
    return _lib


def _check(status: int, name: str):
    if status != MINF_OK:
        raise MinfError(status, name)


def _dev(t, dtype=torch.float32, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _q8_rows(w, k_reg, v_reg):
    """Q8_0 and Q4 rows are both held as bytes, so the type does not tell them apart: regions that are too small for rows of
    w Q8_0 values are refused."""
    need = k_reg.shape[0] * (w + ((w // 32) * 2 + 15) // 16 * 16)
    for name, t in (("K", k_reg), ("V", v_reg)):
        if isinstance(t, torch.Tensor) and t.numel() < need:
            raise ValueError(f"the {name} regions (pools) must hold {k_reg.shape[0]} Q8_0 rows of {w} values, {need} bytes, "
                             f"they are {tuple(t.shape)}")


# The current stream's handle without a Stream object around it (which takes 3 us of a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# The current device without the check that CUDA is up (tensors on a device are proof of that; 87 ns against 243).
_here = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_here())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def minf_rope_freqs(hd: int, theta: float, freq_scale: float = 1.0) -> list[float]:
    import array

    buf = (ctypes.c_float * max(hd // 2, 1))()
    _check(lib().minf_rope_freqs(ctypes.cast(buf, _P), hd, theta, freq_scale), "minf_rope_freqs")
    return array.array("f", buf[: hd // 2])


def minf_rms_norm(y, x, w, eps: float, stream=None):
    rows, n = x.shape
    _check(lib().minf_rms_norm(_dev(y, name="y"), _dev(x, name="x"), _dev(w, name="w"), rows, n, eps,
                               _stream(stream)), "minf_rms_norm")


def minf_rope(x, pos, n_head: int, hd: int, theta: float, freq_scale: float, style: int, err,
              stream=None):
    nt = pos.numel()
    _check(lib().minf_rope(_dev(x, name="x"), _dev(pos, torch.int32, "pos"), nt, n_head, hd, theta,
                           freq_scale, style, _dev(err, torch.int32, "err"), _stream(stream)),
           "minf_rope")


def minf_kv_append(k_reg, v_reg, k_rows, v_rows, pos, err, stream=None):
    cap, W = k_reg.shape
    _check(lib().minf_kv_append(_dev(k_reg, name="k_reg"), _dev(v_reg, name="v_reg"), cap, W,
                                _dev(k_rows, name="k_rows"), _dev(v_rows, name="v_rows"),
                                _dev(pos, torch.int32, "pos"), pos.numel(),
                                _dev(err, torch.int32, "err"), _stream(stream)), "minf_kv_append")


def minf_rope_kv_append(q, k, v, pos, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, k_reg,
                        v_reg, err, stream=None):
    cap = k_reg.shape[0]
    _check(lib().minf_rope_kv_append(_dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"),
                                     _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head,
                                     hd, hd_kv, theta, freq_scale, style, _dev(k_reg, name="k_reg"),
                                     _dev(v_reg, name="v_reg"), cap, _dev(err, torch.int32, "err"),
                                     _stream(stream)), "minf_rope_kv_append")


def minf_attn_decode_workspace_bytes(n_seq, n_head, n_kv_head, hd_kv, max_cap) -> int:
    return int(lib().minf_attn_decode_workspace_bytes(n_seq, n_head, n_kv_head, hd_kv, max_cap))


def minf_attn_prefill_workspace_bytes(nt, n_head, n_kv_head, hd_kv, cap) -> int:
    return int(lib().minf_attn_prefill_workspace_bytes(nt, n_head, n_kv_head, hd_kv, cap))


def minf_gqa_attn_decode(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, pos, n_head, n_kv_head,
                         hd, hd_kv, scale, ws, err, stream=None):
    """k_reg/v_reg: the [rows, W] arena (or one sequence's [cap, W] regions)."""
    _check(lib().minf_gqa_attn_decode(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_reg, name="k_reg"), _dev(v_reg, name="v_reg"),
        _dev(seq_row_off, torch.int64, "seq_row_off"), _dev(seq_cap, torch.int32, "seq_cap"), max_cap,
        k_reg.shape[0], _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv, scale,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_gqa_attn_decode")


def minf_gqa_attn_decode_static_ws(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, pos, n_head,
                                   n_kv_head, hd, hd_kv, scale, err, stream=None):
    """minf_gqa_attn_decode for callers that cannot allocate: the library's own fixed device
    scratch replaces the workspace argument (see include/minf.h for its limits)."""
    _check(lib().minf_gqa_attn_decode_static_ws(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_reg, name="k_reg"), _dev(v_reg, name="v_reg"),
        _dev(seq_row_off, torch.int64, "seq_row_off"), _dev(seq_cap, torch.int32, "seq_cap"), max_cap,
        k_reg.shape[0], _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv, scale,
        _dev(err, torch.int32, "err"), _stream(stream)), "minf_gqa_attn_decode_static_ws")


def minf_gqa_attn_prefill(out, q, k_reg, v_reg, pos, n_head, n_kv_head, hd, hd_kv, scale, ws, err,
                          stream=None):
    cap = k_reg.shape[0]
    _check(lib().minf_gqa_attn_prefill(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_reg, name="k_reg"), _dev(v_reg, name="v_reg"),
        cap, _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv, scale,
        _dev(ws, torch.uint8, "ws"), _nbytes(ws), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_gqa_attn_prefill")


def _layer_step(name, reg_dtype, xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv,
                theta, freq_scale, style, out, ws, err, stream):
    nt, n_embd = h.shape
    cap = k_reg.shape[0]
    if reg_dtype is torch.uint8:
        _q8_rows(n_kv_head * hd_kv, k_reg, v_reg)
    _check(getattr(lib(), name)(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd,
        _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), _dev(pos, torch.int32, "pos"), nt,
        _dev(k_reg, reg_dtype, "k_reg"), _dev(v_reg, reg_dtype, "v_reg"), cap, n_head, n_kv_head, hd, hd_kv,
        theta, freq_scale, style, _dev(out, name="out"), _dev(ws, torch.uint8, "ws"), _nbytes(ws),
        _dev(err, torch.int32, "err"), _stream(stream)), name)


def minf_layer_attn_step(xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv,
                         theta, freq_scale, style, out, ws, err, stream=None):
    _layer_step("minf_layer_attn_step", torch.float32, xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head,
                n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream)


def minf_layer_attn_step_chained(xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv,
                                 theta, freq_scale, style, out, ws, err, stream=None):
    _layer_step("minf_layer_attn_step_chained", torch.float32, xn, h, gain, eps, q, k, v, pos, k_reg, v_reg,
                n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream)


def minf_layer_attn_step_chained_f16(xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv,
                                     theta, freq_scale, style, out, ws, err, stream=None):
    _layer_step("minf_layer_attn_step_chained_f16", torch.float16, xn, h, gain, eps, q, k, v, pos, k_reg, v_reg,
                n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream)


def minf_layer_attn_step_chained_q8(xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv,
                                    theta, freq_scale, style, out, ws, err, stream=None):
    _layer_step("minf_layer_attn_step_chained_q8", torch.uint8, xn, h, gain, eps, q, k, v, pos, k_reg, v_reg,
                n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream)


def minf_layer_attn_step_batched(xn, h, gain, eps, q, k, v, pos, k_arena, v_arena, seq_row_off, seq_cap,
                                 max_cap, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out,
                                 ws, err, stream=None):
    n_seq, n_embd = h.shape
    _check(lib().minf_layer_attn_step_batched(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd,
        _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), _dev(pos, torch.int32, "pos"), n_seq,
        _dev(k_arena, name="k_arena"), _dev(v_arena, name="v_arena"),
        _dev(seq_row_off, torch.int64, "seq_row_off"), _dev(seq_cap, torch.int32, "seq_cap"), max_cap,
        k_arena.shape[0], n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, _dev(out, name="out"),
        _dev(ws, torch.uint8, "ws"), ws.numel(), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_layer_attn_step_batched")


def minf_silu_mul(y, gate, up, stream=None):
    _check(lib().minf_silu_mul(_dev(y, name="y"), _dev(gate, name="gate"), _dev(up, name="up"),
                               gate.numel(), _stream(stream)), "minf_silu_mul")


# ----------------------------------------------------------------------------- binary16 regions
# The regions (or arena) are torch.float16 tensors; everything else is as for fp32 regions.
_H = torch.float16


def minf_kv_append_f16(k_reg, v_reg, k_rows, v_rows, pos, err, stream=None):
    cap, W = k_reg.shape
    _check(lib().minf_kv_append_f16(_dev(k_reg, _H, "k_reg"), _dev(v_reg, _H, "v_reg"), cap, W,
                                    _dev(k_rows, name="k_rows"), _dev(v_rows, name="v_rows"),
                                    _dev(pos, torch.int32, "pos"), pos.numel(),
                                    _dev(err, torch.int32, "err"), _stream(stream)), "minf_kv_append_f16")


def minf_rope_kv_append_f16(q, k, v, pos, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, k_reg,
                            v_reg, err, stream=None):
    cap = k_reg.shape[0]
    _check(lib().minf_rope_kv_append_f16(_dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"),
                                         _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head,
                                         hd, hd_kv, theta, freq_scale, style, _dev(k_reg, _H, "k_reg"),
                                         _dev(v_reg, _H, "v_reg"), cap, _dev(err, torch.int32, "err"),
                                         _stream(stream)), "minf_rope_kv_append_f16")


def minf_gqa_attn_decode_f16(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, pos, n_head, n_kv_head,
                             hd, hd_kv, scale, ws, err, stream=None):
    _check(lib().minf_gqa_attn_decode_f16(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_reg, _H, "k_reg"), _dev(v_reg, _H, "v_reg"),
        _dev(seq_row_off, torch.int64, "seq_row_off"), _dev(seq_cap, torch.int32, "seq_cap"), max_cap,
        k_reg.shape[0], _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv, scale,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_gqa_attn_decode_f16")


def minf_gqa_attn_prefill_f16(out, q, k_reg, v_reg, pos, n_head, n_kv_head, hd, hd_kv, scale, ws, err,
                              stream=None):
    cap = k_reg.shape[0]
    _check(lib().minf_gqa_attn_prefill_f16(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_reg, _H, "k_reg"), _dev(v_reg, _H, "v_reg"),
        cap, _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv, scale,
        _dev(ws, torch.uint8, "ws"), _nbytes(ws), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_gqa_attn_prefill_f16")


def minf_layer_attn_step_f16(xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv,
                             theta, freq_scale, style, out, ws, err, stream=None):
    nt, n_embd = h.shape
    cap = k_reg.shape[0]
    _check(lib().minf_layer_attn_step_f16(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd,
        _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), _dev(pos, torch.int32, "pos"), nt,
        _dev(k_reg, _H, "k_reg"), _dev(v_reg, _H, "v_reg"), cap, n_head, n_kv_head, hd, hd_kv,
        theta, freq_scale, style, _dev(out, name="out"), _dev(ws, torch.uint8, "ws"), _nbytes(ws),
        _dev(err, torch.int32, "err"), _stream(stream)), "minf_layer_attn_step_f16")


def minf_layer_attn_step_batched_f16(xn, h, gain, eps, q, k, v, pos, k_arena, v_arena, seq_row_off, seq_cap,
                                     max_cap, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out,
                                     ws, err, stream=None):
    n_seq, n_embd = h.shape
    _check(lib().minf_layer_attn_step_batched_f16(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd,
        _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), _dev(pos, torch.int32, "pos"), n_seq,
        _dev(k_arena, _H, "k_arena"), _dev(v_arena, _H, "v_arena"),
        _dev(seq_row_off, torch.int64, "seq_row_off"), _dev(seq_cap, torch.int32, "seq_cap"), max_cap,
        k_arena.shape[0], n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, _dev(out, name="out"),
        _dev(ws, torch.uint8, "ws"), ws.numel(), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_layer_attn_step_batched_f16")


# ----------------------------------------------------------------------------- paged regions
# k_pool/v_pool: [pool_rows, W] (float32, or float16 for the _f16 forms); block_table: int32
# [n_seq, max_blocks] on the device; block_rows: rows per block.
def _pool_dtype(name):
    return _H if name.endswith("_f16") else (torch.uint8 if name.endswith("_q8") else torch.float32)


def _kv_append_paged(name, k_pool, v_pool, block_table, block_rows, k_rows, v_rows, pos, err, stream):
    dt = _pool_dtype(name)
    n_seq, max_blocks = block_table.shape
    _check(getattr(lib(), name)(
        _dev(k_pool, dt, "k_pool"), _dev(v_pool, dt, "v_pool"), k_pool.shape[0], k_pool.shape[1],
        _dev(block_table, torch.int32, "block_table"), max_blocks, block_rows, _dev(k_rows, name="k_rows"),
        _dev(v_rows, name="v_rows"), _dev(pos, torch.int32, "pos"), n_seq, _dev(err, torch.int32, "err"),
        _stream(stream)), name)


def minf_kv_append_paged(k_pool, v_pool, block_table, block_rows, k_rows, v_rows, pos, err, stream=None):
    _kv_append_paged("minf_kv_append_paged", k_pool, v_pool, block_table, block_rows, k_rows, v_rows, pos, err,
                     stream)


def minf_kv_append_paged_f16(k_pool, v_pool, block_table, block_rows, k_rows, v_rows, pos, err, stream=None):
    _kv_append_paged("minf_kv_append_paged_f16", k_pool, v_pool, block_table, block_rows, k_rows, v_rows, pos, err,
                     stream)


def _decode_paged(name, out, q, k_pool, v_pool, block_table, block_rows, pos, n_head, n_kv_head, hd, hd_kv, scale,
                  ws, err, stream):
    dt = _pool_dtype(name)
    n_seq, max_blocks = block_table.shape
    if dt is torch.uint8:
        _q8_rows(n_kv_head * hd_kv, k_pool, v_pool)
    _check(getattr(lib(), name)(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_pool, dt, "k_pool"), _dev(v_pool, dt, "v_pool"),
        k_pool.shape[0], _dev(block_table, torch.int32, "block_table"), max_blocks, block_rows,
        _dev(pos, torch.int32, "pos"), n_seq, n_head, n_kv_head, hd, hd_kv, scale, _dev(ws, torch.uint8, "ws"),
        ws.numel(), _dev(err, torch.int32, "err"), _stream(stream)), name)


def minf_gqa_attn_decode_paged(out, q, k_pool, v_pool, block_table, block_rows, pos, n_head, n_kv_head, hd, hd_kv,
                               scale, ws, err, stream=None):
    _decode_paged("minf_gqa_attn_decode_paged", out, q, k_pool, v_pool, block_table, block_rows, pos, n_head,
                  n_kv_head, hd, hd_kv, scale, ws, err, stream)


def minf_gqa_attn_decode_paged_f16(out, q, k_pool, v_pool, block_table, block_rows, pos, n_head, n_kv_head, hd,
                                   hd_kv, scale, ws, err, stream=None):
    _decode_paged("minf_gqa_attn_decode_paged_f16", out, q, k_pool, v_pool, block_table, block_rows, pos, n_head,
                  n_kv_head, hd, hd_kv, scale, ws, err, stream)


def _step_paged(name, xn, h, gain, eps, q, k, v, pos, k_pool, v_pool, block_table, block_rows, n_head, n_kv_head,
                hd, hd_kv, theta, freq_scale, style, out, ws, err, stream):
    dt = _pool_dtype(name)
    n_seq, n_embd = h.shape
    max_blocks = block_table.shape[1]
    if dt is torch.uint8:
        _q8_rows(n_kv_head * hd_kv, k_pool, v_pool)
    _check(getattr(lib(), name)(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd,
        _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), _dev(pos, torch.int32, "pos"), n_seq,
        _dev(k_pool, dt, "k_pool"), _dev(v_pool, dt, "v_pool"), k_pool.shape[0],
        _dev(block_table, torch.int32, "block_table"), max_blocks, block_rows, n_head, n_kv_head, hd, hd_kv, theta,
        freq_scale, style, _dev(out, name="out"), _dev(ws, torch.uint8, "ws"), ws.numel(),
        _dev(err, torch.int32, "err"), _stream(stream)), name)


def minf_layer_attn_step_paged(xn, h, gain, eps, q, k, v, pos, k_pool, v_pool, block_table, block_rows, n_head,
                               n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream=None):
    _step_paged("minf_layer_attn_step_paged", xn, h, gain, eps, q, k, v, pos, k_pool, v_pool, block_table,
                block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream)


def minf_layer_attn_step_paged_f16(xn, h, gain, eps, q, k, v, pos, k_pool, v_pool, block_table, block_rows, n_head,
                                   n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream=None):
    _step_paged("minf_layer_attn_step_paged_f16", xn, h, gain, eps, q, k, v, pos, k_pool, v_pool, block_table,
                block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream)


def minf_kv_append_paged_q8(k_pool, v_pool, block_table, block_rows, k_rows, v_rows, pos, err, stream=None):
    """Pools [pool_rows, minf_q8_row_bytes(W)] uint8; W is taken from k_rows."""
    n_seq, max_blocks = block_table.shape
    _q8_rows(k_rows.shape[-1], k_pool, v_pool)
    _check(lib().minf_kv_append_paged_q8(
        _dev(k_pool, torch.uint8, "k_pool"), _dev(v_pool, torch.uint8, "v_pool"), k_pool.shape[0], k_rows.shape[-1],
        _dev(block_table, torch.int32, "block_table"), max_blocks, block_rows, _dev(k_rows, name="k_rows"),
        _dev(v_rows, name="v_rows"), _dev(pos, torch.int32, "pos"), n_seq, _dev(err, torch.int32, "err"),
        _stream(stream)), "minf_kv_append_paged_q8")


def minf_gqa_attn_decode_paged_q8(out, q, k_pool, v_pool, block_table, block_rows, pos, n_head, n_kv_head, hd, hd_kv,
                                  scale, ws, err, stream=None):
    _decode_paged("minf_gqa_attn_decode_paged_q8", out, q, k_pool, v_pool, block_table, block_rows, pos, n_head,
                  n_kv_head, hd, hd_kv, scale, ws, err, stream)


def minf_layer_attn_step_paged_q8(xn, h, gain, eps, q, k, v, pos, k_pool, v_pool, block_table, block_rows, n_head,
                                  n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream=None):
    _step_paged("minf_layer_attn_step_paged_q8", xn, h, gain, eps, q, k, v, pos, k_pool, v_pool, block_table,
                block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err, stream)


# ----------------------------------------------------------------------------- Q8_0 regions
# The regions (or arena) are torch.uint8 tensors [rows, minf_q8_row_bytes(W)]; the row width W
# (values) comes from the fp32 rows or the head geometry.
_U8 = torch.uint8


def minf_q8_row_bytes(row_width: int) -> int:
    return int(lib().minf_q8_row_bytes(row_width))


def minf_kv_append_q8(k_reg, v_reg, k_rows, v_rows, pos, err, stream=None):
    _q8_rows(k_rows.shape[-1], k_reg, v_reg)
    _check(lib().minf_kv_append_q8(_dev(k_reg, _U8, "k_reg"), _dev(v_reg, _U8, "v_reg"), k_reg.shape[0],
                                   k_rows.shape[-1], _dev(k_rows, name="k_rows"), _dev(v_rows, name="v_rows"),
                                   _dev(pos, torch.int32, "pos"), pos.numel(), _dev(err, torch.int32, "err"),
                                   _stream(stream)), "minf_kv_append_q8")


def minf_rope_kv_append_q8(q, k, v, pos, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, k_reg, v_reg, err,
                           stream=None):
    _q8_rows(n_kv_head * hd_kv, k_reg, v_reg)
    _check(lib().minf_rope_kv_append_q8(_dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"),
                                        _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv,
                                        theta, freq_scale, style, _dev(k_reg, _U8, "k_reg"), _dev(v_reg, _U8, "v_reg"),
                                        k_reg.shape[0], _dev(err, torch.int32, "err"), _stream(stream)),
           "minf_rope_kv_append_q8")


def minf_gqa_attn_decode_q8(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, pos, n_head, n_kv_head, hd, hd_kv,
                            scale, ws, err, stream=None):
    _q8_rows(n_kv_head * hd_kv, k_reg, v_reg)
    _check(lib().minf_gqa_attn_decode_q8(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_reg, _U8, "k_reg"), _dev(v_reg, _U8, "v_reg"),
        _dev(seq_row_off, torch.int64, "seq_row_off"), _dev(seq_cap, torch.int32, "seq_cap"), max_cap,
        k_reg.shape[0], _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv, scale,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_gqa_attn_decode_q8")


def minf_gqa_attn_prefill_q8(out, q, k_reg, v_reg, pos, n_head, n_kv_head, hd, hd_kv, scale, ws, err, stream=None):
    _q8_rows(n_kv_head * hd_kv, k_reg, v_reg)
    _check(lib().minf_gqa_attn_prefill_q8(
        _dev(out, name="out"), _dev(q, name="q"), _dev(k_reg, _U8, "k_reg"), _dev(v_reg, _U8, "v_reg"),
        k_reg.shape[0], _dev(pos, torch.int32, "pos"), pos.numel(), n_head, n_kv_head, hd, hd_kv, scale,
        _dev(ws, torch.uint8, "ws"), _nbytes(ws), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_gqa_attn_prefill_q8")


def minf_layer_attn_step_q8(xn, h, gain, eps, q, k, v, pos, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv, theta,
                            freq_scale, style, out, ws, err, stream=None):
    _q8_rows(n_kv_head * hd_kv, k_reg, v_reg)
    nt, n_embd = h.shape
    _check(lib().minf_layer_attn_step_q8(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd,
        _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), _dev(pos, torch.int32, "pos"), nt,
        _dev(k_reg, _U8, "k_reg"), _dev(v_reg, _U8, "v_reg"), k_reg.shape[0], n_head, n_kv_head, hd, hd_kv,
        theta, freq_scale, style, _dev(out, name="out"), _dev(ws, torch.uint8, "ws"), _nbytes(ws),
        _dev(err, torch.int32, "err"), _stream(stream)), "minf_layer_attn_step_q8")


def minf_layer_attn_step_batched_q8(xn, h, gain, eps, q, k, v, pos, k_arena, v_arena, seq_row_off, seq_cap, max_cap,
                                    n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, out, ws, err,
                                    stream=None):
    _q8_rows(n_kv_head * hd_kv, k_arena, v_arena)
    n_seq, n_embd = h.shape
    _check(lib().minf_layer_attn_step_batched_q8(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd,
        _dev(q, name="q"), _dev(k, name="k"), _dev(v, name="v"), _dev(pos, torch.int32, "pos"), n_seq,
        _dev(k_arena, _U8, "k_arena"), _dev(v_arena, _U8, "v_arena"),
        _dev(seq_row_off, torch.int64, "seq_row_off"), _dev(seq_cap, torch.int32, "seq_cap"), max_cap,
        k_arena.shape[0], n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style, _dev(out, name="out"),
        _dev(ws, torch.uint8, "ws"), ws.numel(), _dev(err, torch.int32, "err"), _stream(stream)),
        "minf_layer_attn_step_batched_q8")


# ----------------------------------------------------------------------------- Q4 regions
# torch.uint8 tensors [rows, minf_q4_row_bytes(W)]; the chunk and window operators take them too.
def minf_q4_row_bytes(row_width: int) -> int:
    return int(lib().minf_q4_row_bytes(row_width))


def minf_kv_append_q4(k_reg, v_reg, k_rows, v_rows, pos, err, stream=None):
    """Row t of k_rows, v_rows [nt, W] to row pos[t] of the regions (or of the pools, with a slot map as pos; in an arena
    of a sequence's own rows, KvArena.seq_view, whose capacity the positions are checked against)."""
    w, here = k_rows.shape[-1], _here()
    _chunk_pool("_q4", k_reg, v_reg, None, 0, w)
    for name, t in (("k_rows", k_rows), ("v_rows", v_rows)):
        _size(name, t, pos.numel() * w)
    _check(lib().minf_kv_append_q4(_ptr(k_reg, _U8, "k_reg", here), _ptr(v_reg, _U8, "v_reg", here), k_reg.shape[0], w,
                                   _ptr(k_rows, _F32, "k_rows", here), _ptr(v_rows, _F32, "v_rows", here),
                                   _ptr(pos, _I32, "pos", here), pos.numel(), _ptr(err, _I32, "err", here),
                                   _stream(stream)), "minf_kv_append_q4")


# ----------------------------------------------------------------------------- fused QKV op
def minf_fused_qkv(xn, h, gain, eps, w_qkv, b_qkv, pos, q, k, v, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv, theta,
                   freq_scale, style, err, stream=None):
    nt, n_embd = h.shape
    _check(lib().minf_fused_qkv(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd, _dev(w_qkv, name="w_qkv"),
        _dev(b_qkv, name="b_qkv"), _dev(pos, torch.int32, "pos"), nt, _dev(q, name="q"), _dev(k, name="k"),
        _dev(v, name="v"), _dev(k_reg, name="k_reg"), _dev(v_reg, name="v_reg"), k_reg.shape[0], n_head, n_kv_head,
        hd, hd_kv, theta, freq_scale, style, _dev(err, torch.int32, "err"), _stream(stream)), "minf_fused_qkv")


def minf_layer_attn_step_qkv(xn, h, gain, eps, w_qkv, b_qkv, pos, q, k, v, k_reg, v_reg, n_head, n_kv_head, hd, hd_kv,
                             theta, freq_scale, style, out, ws, err, stream=None):
    n_embd = h.shape[-1]
    _check(lib().minf_layer_attn_step_qkv(
        _dev(xn, name="xn"), _dev(h, name="h"), _dev(gain, name="gain"), eps, n_embd, _dev(w_qkv, name="w_qkv"),
        _dev(b_qkv, name="b_qkv"), _dev(pos, torch.int32, "pos"), _dev(q, name="q"), _dev(k, name="k"),
        _dev(v, name="v"), _dev(k_reg, name="k_reg"), _dev(v_reg, name="v_reg"), k_reg.shape[0], n_head, n_kv_head,
        hd, hd_kv, theta, freq_scale, style, _dev(out, name="out"), _dev(ws, torch.uint8, "ws"), ws.numel(),
        _dev(err, torch.int32, "err"), _stream(stream)), "minf_layer_attn_step_qkv")


# ----------------------------------------------------------------------------- chunks of new tokens
# chunk_off: int32 [n_seq + 1] on the device (None: one token a sequence); n_past: int32 [n_seq];
# pair_axis: the axis of each of the hd/2 pairs, as bytes or a sequence of ints (None: one axis).
# These check sizes too (the library sees only pointers), and that every tensor is on the current
# device, whose stream the call goes to.
_F32, _I32, _Tensor = torch.float32, torch.int32, torch.Tensor
_CHUNK_DTYPE = {"": torch.float32, "_f16": torch.float16, "_q8": torch.uint8, "_q4": torch.uint8}


def _ptr(t, dtype, name, here, n=None):
    """Address of a contiguous tensor of this type (and of n elements) on the current device (None stays None)."""
    if (t.__class__ is _Tensor and t.dtype is dtype and t.get_device() == here and t.is_contiguous()
            and (n is None or t.numel() == n)):
        return t.data_ptr()
    if t is None:
        return None
    if t.__class__ is not torch.Tensor and not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != here:
        raise ValueError(f"{name} must be on the current device (cuda:{here}), it is on {t.device}")
    if n is not None:
        _size(name, t, n)
    return t.data_ptr()


def _size(name, t, n):
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")


def _axis_bytes(pair_axis, hd):
    if pair_axis is None:
        return None
    pair_axis = bytes(pair_axis)
    if len(pair_axis) != hd // 2:
        raise ValueError(f"pair_axis must have hd/2 = {hd // 2} entries, got {len(pair_axis)}")
    return pair_axis


def _chunk_seqs(chunk_off, n_past, nt):
    n_seq = n_past.numel()
    if chunk_off is not None:
        _size("chunk_off", chunk_off, n_seq + 1)
    elif nt != n_seq:
        raise ValueError(f"without chunk_off there is one token a sequence: {nt} tokens for {n_seq} sequences")
    return n_seq


def _chunk_pool(end, k_pool, v_pool, block_table, n_seq, row_width):
    """(rows of the pools, columns of block_table)"""
    cols = row_width
    if end in ("_q8", "_q4"):
        if row_width % 32:
            raise ValueError("Q8_0 and Q4 rows hold whole 32-value blocks")
        cols = (row_width if end == "_q8" else row_width // 2) + ((row_width // 32) * 2 + 15) // 16 * 16
    shape = k_pool.shape
    if len(shape) != 2 or shape[1] != cols or v_pool.shape != shape:
        raise ValueError(f"the pools (regions) must both be [rows, {cols}], got {tuple(shape)} and {tuple(v_pool.shape)}")
    if block_table is None:
        return shape[0], 0
    table = block_table.shape
    if len(table) != 2 or table[0] != n_seq:
        raise ValueError(f"block_table must be [{n_seq}, max_blocks], got {tuple(table)}")
    return shape[0], table[1]


def minf_rope_axes(y, x, pos, pair_axis, n_head, hd, theta, freq_scale, style, err, stream=None):
    """pos: int32 [n_axis, nt] (or [nt] for one axis); y may be x."""
    n_axis, nt = pos.shape if pos.dim() == 2 else (1, pos.numel())
    here = _here()
    _size("x", x, nt * n_head * hd)
    _size("y", y, nt * n_head * hd)
    _check(lib().minf_rope_axes(_ptr(y, _F32, "y", here), _ptr(x, _F32, "x", here), _ptr(pos, _I32, "pos", here), nt,
                                n_axis, _axis_bytes(pair_axis, hd), n_head, hd, theta, freq_scale, style,
                                _ptr(err, _I32, "err", here), _stream(stream)), "minf_rope_axes")


def _rope_kv_append_chunk_paged(end, q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head, n_kv_head,
                                hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table, block_rows, err,
                                stream):
    dt, w = _CHUNK_DTYPE[end], n_kv_head * hd_kv
    nt = v.numel() // w
    n_axis = 1 if rope_pos is None or rope_pos.dim() == 1 else rope_pos.shape[0]
    here = _here()
    n_seq = _chunk_seqs(chunk_off, n_past, nt)
    rows, blocks = _chunk_pool(end, k_pool, v_pool, block_table, n_seq, w)
    nq, nk = nt * n_head * hd, nt * w
    axes = _axis_bytes(pair_axis, hd)
    if rope_pos is None and axes is not None:  # one position for every axis
        axes = None
    name = "minf_rope_kv_append_chunk_paged" + end
    _check(getattr(lib(), name)(
        _ptr(q_out, _F32, "q_out", here, nq), _ptr(k_out, _F32, "k_out", here, nk), _ptr(q, _F32, "q", here, nq),
        _ptr(k, _F32, "k", here, nk), _ptr(v, _F32, "v", here, nk),
        _ptr(rope_pos, _I32, "rope_pos", here, nt * n_axis), n_axis, axes, _ptr(chunk_off, _I32, "chunk_off", here),
        _ptr(n_past, _I32, "n_past", here), nt, n_seq, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style,
        _ptr(k_pool, dt, "k_pool", here), _ptr(v_pool, dt, "v_pool", here), rows,
        _ptr(block_table, _I32, "block_table", here), blocks, block_rows, _ptr(err, _I32, "err", here),
        _stream(stream)), name)


def minf_rope_kv_append_chunk_paged(q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head, n_kv_head, hd,
                                    hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table, block_rows, err,
                                    stream=None):
    _rope_kv_append_chunk_paged("", q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head, n_kv_head,
                                hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table, block_rows, err,
                                stream)


def minf_rope_kv_append_chunk_paged_f16(q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head, n_kv_head,
                                        hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table, block_rows,
                                        err, stream=None):
    _rope_kv_append_chunk_paged("_f16", q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head,
                                n_kv_head, hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table,
                                block_rows, err, stream)


def minf_rope_kv_append_chunk_paged_q8(q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head, n_kv_head,
                                       hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table, block_rows,
                                       err, stream=None):
    _rope_kv_append_chunk_paged("_q8", q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head,
                                n_kv_head, hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table,
                                block_rows, err, stream)


def minf_rope_kv_append_chunk_paged_q4(q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head, n_kv_head,
                                       hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table, block_rows,
                                       err, stream=None):
    _rope_kv_append_chunk_paged("_q4", q_out, k_out, q, k, v, rope_pos, pair_axis, chunk_off, n_past, n_head,
                                n_kv_head, hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, block_table,
                                block_rows, err, stream)


def _kv_read_chunk_paged(end, k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err, stream):
    dt, w = _CHUNK_DTYPE[end], k_rows.shape[-1]
    nt = k_rows.numel() // w
    here = _here()
    n_seq = _chunk_seqs(chunk_off, n_past, nt)
    pool_rows, blocks = _chunk_pool(end, k_pool, v_pool, block_table, n_seq, w)
    rows = torch.float16 if k_rows.dtype == torch.float16 else torch.float32
    name = "minf_kv_read_chunk_paged" + end
    _check(getattr(lib(), name)(
        _ptr(k_rows, rows, "k_rows", here), _ptr(v_rows, rows, "v_rows", here, nt * w), rows == torch.float16,
        _ptr(k_pool, dt, "k_pool", here),
        _ptr(v_pool, dt, "v_pool", here), pool_rows, w, _ptr(block_table, _I32, "block_table", here),
        blocks, block_rows, _ptr(chunk_off, _I32, "chunk_off", here),
        _ptr(n_past, _I32, "n_past", here), nt, n_seq, _ptr(err, _I32, "err", here), _stream(stream)), name)


def minf_kv_read_chunk_paged(k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err,
                             stream=None):
    """k_rows, v_rows: [nt, W] float32 or float16 (both the same)."""
    _kv_read_chunk_paged("", k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err, stream)


def minf_kv_read_chunk_paged_f16(k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err,
                                 stream=None):
    _kv_read_chunk_paged("_f16", k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err,
                         stream)


def minf_kv_read_chunk_paged_q8(k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err,
                                stream=None):
    _kv_read_chunk_paged("_q8", k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err,
                         stream)


def minf_kv_read_chunk_paged_q4(k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err,
                                stream=None):
    _kv_read_chunk_paged("_q4", k_rows, v_rows, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, err,
                         stream)


def minf_attn_chunk_workspace_bytes(nt, n_seq, n_head, n_kv_head, hd_kv, max_chunk) -> int:
    return int(lib().minf_attn_chunk_workspace_bytes(nt, n_seq, n_head, n_kv_head, hd_kv, max_chunk))


def _attn_rows(out, q, n_head, hd, hd_kv):
    nt = out.numel() // (n_head * hd_kv)
    _size("q", q, nt * n_head * hd)
    _size("out", out, nt * n_head * hd_kv)
    return nt


def _gqa_attn_chunk_paged(end, out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                          n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream):
    dt = _CHUNK_DTYPE[end]
    nt = _attn_rows(out, q, n_head, hd, hd_kv)
    here = _here()
    n_seq = _chunk_seqs(chunk_off, n_past, nt)
    rows, blocks = _chunk_pool(end, k_pool, v_pool, block_table, n_seq, n_kv_head * hd_kv)
    name = "minf_gqa_attn_chunk_paged" + end
    _check(getattr(lib(), name)(
        _ptr(out, _F32, "out", here), _ptr(q, _F32, "q", here), _ptr(k_pool, dt, "k_pool", here),
        _ptr(v_pool, dt, "v_pool", here), rows, _ptr(block_table, _I32, "block_table", here), blocks, block_rows,
        _ptr(chunk_off, _I32, "chunk_off", here), _ptr(n_past, _I32, "n_past", here), nt, n_seq, max_chunk, n_head,
        n_kv_head, hd, hd_kv, scale, window, n_sink, _ptr(ws, _U8, "ws", here), _nbytes(ws),
        _ptr(err, _I32, "err", here), _stream(stream)), name)


def minf_gqa_attn_chunk_paged(out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                              n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    _gqa_attn_chunk_paged("", out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                          n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def minf_gqa_attn_chunk_paged_f16(out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                                  n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    _gqa_attn_chunk_paged("_f16", out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                          n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def minf_gqa_attn_chunk_paged_q8(out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                                 n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    _gqa_attn_chunk_paged("_q8", out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                          n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def minf_gqa_attn_chunk_paged_q4(out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                                 n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    _gqa_attn_chunk_paged("_q4", out, q, k_pool, v_pool, block_table, block_rows, chunk_off, n_past, max_chunk, n_head,
                          n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def _gqa_attn_window(end, out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                     n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream):
    dt = _CHUNK_DTYPE[end]
    nt = _attn_rows(out, q, n_head, hd, hd_kv)
    here = _here()
    n_seq = _chunk_seqs(chunk_off, n_past, nt)
    rows, _ = _chunk_pool(end, k_reg, v_reg, None, n_seq, n_kv_head * hd_kv)
    if seq_row_off is None and rows < max_cap:
        raise ValueError(f"the regions have {rows} rows, max_cap is {max_cap}")
    name = "minf_gqa_attn_window" + end
    _check(getattr(lib(), name)(
        _ptr(out, _F32, "out", here), _ptr(q, _F32, "q", here), _ptr(k_reg, dt, "k_reg", here),
        _ptr(v_reg, dt, "v_reg", here), _ptr(seq_row_off, torch.int64, "seq_row_off", here, n_seq),
        _ptr(seq_cap, _I32, "seq_cap", here, n_seq), max_cap, rows,
        _ptr(chunk_off, _I32, "chunk_off", here), _ptr(n_past, _I32, "n_past", here), nt, n_seq, max_chunk, n_head,
        n_kv_head, hd, hd_kv, scale, window, n_sink, _ptr(ws, _U8, "ws", here), _nbytes(ws),
        _ptr(err, _I32, "err", here), _stream(stream)), name)


def minf_gqa_attn_window(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                         n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    """k_reg/v_reg: the [rows, W] arena (or one sequence's [cap, W] regions, with seq_row_off None)."""
    _gqa_attn_window("", out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                     n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def minf_gqa_attn_window_f16(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                             n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    _gqa_attn_window("_f16", out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                     n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def minf_gqa_attn_window_q8(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                            n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    _gqa_attn_window("_q8", out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                     n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def minf_gqa_attn_window_q4(out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                            n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream=None):
    _gqa_attn_window("_q4", out, q, k_reg, v_reg, seq_row_off, seq_cap, max_cap, chunk_off, n_past, max_chunk, n_head,
                     n_kv_head, hd, hd_kv, scale, window, n_sink, ws, err, stream)


def _layer_step_chunk_paged(end, xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk, k_pool,
                            v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style,
                            window, n_sink, out, ws, err, stream):
    dt, w = _CHUNK_DTYPE[end], n_kv_head * hd_kv
    nt, n_embd = h.shape
    n_axis = 1 if rope_pos is None or rope_pos.dim() == 1 else rope_pos.shape[0]
    here = _here()
    n_seq = _chunk_seqs(chunk_off, n_past, nt)
    _chunk_pool(end, k_pool, v_pool, block_table, n_seq, w)
    for name, t, n in (("xn", xn, nt * n_embd), ("gain", gain, n_embd), ("q", q, nt * n_head * hd), ("k", k, nt * w),
                       ("v", v, nt * w), ("rope_pos", rope_pos, nt * n_axis), ("out", out, nt * n_head * hd_kv)):
        if t is not None:
            _size(name, t, n)
    axes = _axis_bytes(pair_axis, hd)
    if rope_pos is None:
        axes = None
    name = "minf_layer_attn_step_chunk_paged" + end
    _check(getattr(lib(), name)(
        _ptr(xn, _F32, "xn", here), _ptr(h, _F32, "h", here), _ptr(gain, _F32, "gain", here), eps, n_embd,
        _ptr(q, _F32, "q", here), _ptr(k, _F32, "k", here), _ptr(v, _F32, "v", here),
        _ptr(rope_pos, _I32, "rope_pos", here), n_axis, axes,
        _ptr(chunk_off, _I32, "chunk_off", here), _ptr(n_past, _I32, "n_past", here), nt, n_seq, max_chunk,
        _ptr(k_pool, dt, "k_pool", here), _ptr(v_pool, dt, "v_pool", here), k_pool.shape[0],
        _ptr(block_table, _I32, "block_table", here), block_table.shape[1], block_rows, n_head, n_kv_head, hd, hd_kv,
        theta, freq_scale, style, window, n_sink, _ptr(out, _F32, "out", here), _ptr(ws, _U8, "ws", here), _nbytes(ws),
        _ptr(err, _I32, "err", here), _stream(stream)), name)


def minf_layer_attn_step_chunk_paged(xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk,
                                     k_pool, v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta,
                                     freq_scale, style, window, n_sink, out, ws, err, stream=None):
    _layer_step_chunk_paged("", xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk, k_pool,
                            v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale, style,
                            window, n_sink, out, ws, err, stream)


def minf_layer_attn_step_chunk_paged_f16(xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk,
                                         k_pool, v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta,
                                         freq_scale, style, window, n_sink, out, ws, err, stream=None):
    _layer_step_chunk_paged("_f16", xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk,
                            k_pool, v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale,
                            style, window, n_sink, out, ws, err, stream)


def minf_layer_attn_step_chunk_paged_q8(xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk,
                                        k_pool, v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta,
                                        freq_scale, style, window, n_sink, out, ws, err, stream=None):
    _layer_step_chunk_paged("_q8", xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk,
                            k_pool, v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale,
                            style, window, n_sink, out, ws, err, stream)


def minf_layer_attn_step_chunk_paged_q4(xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk,
                                        k_pool, v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta,
                                        freq_scale, style, window, n_sink, out, ws, err, stream=None):
    _layer_step_chunk_paged("_q4", xn, h, gain, eps, q, k, v, rope_pos, pair_axis, chunk_off, n_past, max_chunk,
                            k_pool, v_pool, block_table, block_rows, n_head, n_kv_head, hd, hd_kv, theta, freq_scale,
                            style, window, n_sink, out, ws, err, stream)


# ----------------------------------------------------------------------------- block tables
# block_table: int32 [n_seq, max_blocks]; free_ids: int32, the list of blocks that no table has, of which n_free (int32
# [1]) are there; n_free_out may be n_free.
def minf_block_table_grow(block_table, block_rows, pool_rows, n_past, n_new, free_ids, n_free, n_free_out, chunk_off,
                          pos, slot, err, stream=None):
    """pos, slot: int32 [nt] (None: not wanted; rows behind the last token become -1); without both, any number of
    tokens."""
    n_seq, max_blocks = block_table.shape
    here = _here()
    nt = pos.numel() if pos is not None else slot.numel() if slot is not None else 0x7fffffff - 65536
    _check(lib().minf_block_table_grow(
        _ptr(block_table, _I32, "block_table", here), max_blocks, block_rows, pool_rows, _ptr(n_past, _I32, "n_past", here, n_seq),
        _ptr(n_new, _I32, "n_new", here, n_seq), n_seq, _ptr(free_ids, _I32, "free_ids", here), free_ids.numel(),
        _ptr(n_free, _I32, "n_free", here, 1), _ptr(n_free_out, _I32, "n_free_out", here, 1),
        _ptr(chunk_off, _I32, "chunk_off", here, n_seq + 1), _ptr(pos, _I32, "pos", here), _ptr(slot, _I32, "slot", here, nt), nt,
        _ptr(err, _I32, "err", here, 1), _stream(stream)), "minf_block_table_grow")


def minf_block_table_release(block_table, block_rows, pool_rows, row_lo, row_hi, free_ids, n_free, n_free_out, err,
                             stream=None):
    n_seq, max_blocks = block_table.shape
    here = _here()
    _check(lib().minf_block_table_release(
        _ptr(block_table, _I32, "block_table", here), max_blocks, block_rows, pool_rows, _ptr(row_lo, _I32, "row_lo", here, n_seq),
        _ptr(row_hi, _I32, "row_hi", here, n_seq), n_seq, _ptr(free_ids, _I32, "free_ids", here), free_ids.numel(),
        _ptr(n_free, _I32, "n_free", here, 1), _ptr(n_free_out, _I32, "n_free_out", here, 1),
        _ptr(err, _I32, "err", here, 1), _stream(stream)), "minf_block_table_release")
