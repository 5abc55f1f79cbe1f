"""MI355X (gfx950) BitNet b1.58 BitLinear: thin Python binding of libbitlinear.so.

Every function here only marshals torch tensors (device memory) and the current
HIP stream into the C ABI declared in include/bitlinear.h (through ctypes, the
attention calls through csrc/binding.cpp); all arithmetic runs in the library's
HIP kernels. If the library is not built, importing works but every
call raises -- there is no fallback.

Functions mirror the C entry points:
  pack_weights(w)                      -> (packed uint8 [n][k/4], gamma fp32 [1])
  pack_weights_threshold(w, factor)    -> (packed uint8 [n][k/4], alpha fp32 [1], delta fp32 [1])
  quant_act(x)                         -> (q int8 [m][k], scale fp32 [m])
  quant_act_norm(x, gain=None)         -> the same for the RMS-normalized x
  forward_norm(x, packed, gamma, gain=None) -> y fp32 [m][n] of the RMS-normalized x
  quant_act_a4(x, keep=None)           -> (q int8 [m][k] doubled E2M1 codes, scale fp32 [m])
  forward_a4(x, packed, gamma, keep=None) -> y fp32 [m][n] of the W1.58A4 product
  forward(x, packed, gamma)            -> y fp32 [m][n]        (return_acc=True adds acc)
  ffn(x, gate, up, down)               -> y fp32 [m][hidden]   (return_hq=True adds qh, sh)
  pack_kmajor(packed)                  -> input-major copy [k][n/4] of packed [n][k/4]
  ffn_sparse(x, gate, up, down_t)      -> ffn() for m <= 4 with an input-major down matrix
  gemm_i32(q, packed)                  -> acc int32 [m][n]
  workspace_size(op, m, k, n)          -> bytes
  attention(q, k, v, cu_seqlens)       -> out [m][q_heads * head_dim]: causal attention over packed prompts
  cache_alloc(pages, kv_heads, head_dim) -> KVCache: int8 codes and fp32 scales of 64-token pages
  cache_append(cache, k, v, block_table, lens, cu_seqlens=None)   quantizes new tokens into the cache
  cache_read(cache, block_table, begin, cu_seqlens, m) -> (k, v) [m][kv_heads][head_dim]
  attention_cached(q, cache, block_table, lens, cu_seqlens=None, weights=None) -> out of new tokens over the cache
  cache_evict(block_table, lens, weights, keep) -> (block_table, lens, weights, evicted, evicted_count)
  rotary_frequencies(rotary_dim, base)  -> fp32 [rotary_dim / 2] angles per position, scaled for long contexts if asked
  rotate(q, k, inv_freq, begin, cu_seqlens=None) -> (q, k) rotated by their tokens' positions, each head normed before if asked
  attention_shared(q, cache, prefix_table, prefix_len, block_table, lens) -> attention_cached behind a prefix all sequences share
  bounds_alloc(cache), cache_bounds(cache, bounds, block_table, lens, cu_seqlens, m)   the extremes of every block's keys
  block_select(q, bounds, k_scale, block_table, lens, keep) -> selected int32 [m][kv_heads][keep] by an upper bound of the scores
  attention_selected(q, cache, block_table, lens, selected) -> attention_cached over the selected blocks
Activations may be float32 or bfloat16 CUDA (HIP) tensors, contiguous, [m][k]; q, k and v are
[m][heads][head_dim] and may be slices of a fused projection's rows (any stride between tokens).
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

import torch

__all__ = ["pack_weights", "pack_weights_threshold", "quant_act", "quant_act_norm", "forward_norm", "forward", "ffn", "gemm_i32", "workspace_size",
           "library_path", "load_library", "BitLinearError", "OP_FORWARD", "OP_FFN", "OP_PACK",
           "OP_GEMM_I32", "OP_PACK_THRESHOLD", "OP_FORWARD_NORM", "OP_FFN_SPARSE", "OP_FORWARD_A4",
           "pack_kmajor", "ffn_sparse", "quant_act_a4", "forward_a4",
           "attention", "attention_cached", "KVCache", "cache_alloc", "cache_append", "cache_read", "cache_evict",
           "attention_workspace_size", "attention_cached_workspace_size", "CACHE_BLOCK",
           "rotary_frequencies", "rotate", "attention_shared", "attention_shared_workspace_size", "bounds_alloc", "cache_bounds",
           "block_select", "block_select_workspace_size", "attention_selected", "attention_selected_workspace_size"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libbitlinear.so")

(OP_FORWARD, OP_FFN, OP_PACK, OP_GEMM_I32, OP_PACK_THRESHOLD, OP_FORWARD_NORM, OP_FFN_SPARSE,
 OP_FORWARD_A4) = range(8)  # bl_op in include/bitlinear.h
_F32, _BF16 = 0, 1

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_size = ctypes.c_size_t

_SIGNATURES = {
    "bitlinear_workspace_size": (_c_size, [_c_int, _c_i64, _c_i64, _c_i64]),
    "bitlinear_status_string": (ctypes.c_char_p, [_c_int]),
    "bitlinear_pack_weights": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_size, _c_p]),
    "bitlinear_pack_weights_threshold": (_c_int, [_c_p, _c_i64, _c_i64, ctypes.c_float, _c_p, _c_p, _c_p,
                                                  _c_p, _c_size, _c_p]),
    "bitlinear_quant_act": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "bitlinear_quant_act_norm": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p]),
    "bitlinear_forward_norm": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p,
                                        _c_p, _c_size, _c_p]),
    "bitlinear_forward": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_p,
                                   _c_p, _c_size, _c_p]),
    "bitlinear_ffn": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p,
                               _c_p, _c_p, _c_p, _c_p, _c_p, _c_size, _c_p]),
    "bitlinear_quant_act_a4": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "bitlinear_forward_a4": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_p,
                                      _c_p, _c_size, _c_p]),
    "bitlinear_pack_kmajor": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p]),
    "bitlinear_ffn_sparse": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p,
                                      _c_p, _c_p, _c_p, _c_p, _c_p, _c_size, _c_p]),
    "bitlinear_gemm_i32": (_c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_size, _c_p]),
    "bitlinear_attention_workspace_size": (_c_size, [_c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64]),
    "bitlinear_attention": (_c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_i64,
                                     _c_p, _c_i64, ctypes.c_float, _c_p, _c_p, _c_size, _c_p]),
    "bitlinear_cache_append": (_c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64,
                                        _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_p]),
    "bitlinear_cache_read": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_i64, _c_int, _c_i64,
                                      _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "bitlinear_attention_cached_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_int]),
    "bitlinear_attention_cached": (_c_int, [_c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64,
                                            _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64, ctypes.c_float, _c_p, _c_p,
                                            _c_p, _c_size, _c_p]),
    "bitlinear_cache_evict": (_c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                       _c_p, _c_p, _c_p]),
    "bitlinear_rotate": (_c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p,
                                  _c_i64, _c_int, ctypes.c_float, _c_p, _c_p, ctypes.c_float, _c_p, _c_i64, _c_p, _c_i64, _c_p]),
    "bitlinear_attention_shared_workspace_size": (_c_size, [_c_i64] * 7),
    "bitlinear_attention_shared": (_c_int, [_c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_p,
                                            _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64, ctypes.c_float, _c_p, _c_p,
                                            _c_size, _c_p]),
    "bitlinear_cache_bounds": (_c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_i64, _c_p, _c_p]),
    "bitlinear_block_select_workspace_size": (_c_size, [_c_i64] * 3),
    "bitlinear_block_select": (_c_int, [_c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_i64,
                                        _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_size, _c_p]),
    "bitlinear_attention_selected_workspace_size": (_c_size, [_c_i64] * 5),
    "bitlinear_attention_selected": (_c_int, [_c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_i64,
                                              _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64, ctypes.c_float, _c_p, _c_p, _c_size,
                                              _c_p]),
}

_lib = None


class BitLinearError(RuntimeError):
    pass


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libbitlinear.so (built by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise BitLinearError(f"{_LIB_PATH} is not built; run __graft_entry__.build() "
                             "(hipcc --offload-arch=gfx950) first")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        msg = load_library().bitlinear_status_string(status).decode()
        raise BitLinearError(f"{what}: {msg}")


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise BitLinearError(f"{name} must be a device (HIP) tensor")
    if not t.is_contiguous():
        raise BitLinearError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise BitLinearError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _act_dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return _F32
    if x.dtype == torch.bfloat16:
        return _BF16
    raise BitLinearError(f"activations must be float32 or bfloat16, got {x.dtype}")


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(op: int, m: int, k: int, n: int, device) -> torch.Tensor | None:
    nbytes = workspace_size(op, m, k, n)
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _ws_args(ws):
    return (ws.data_ptr(), ws.numel() * ws.element_size()) if ws is not None else (None, 0)


def _caller_workspace(ws: torch.Tensor, op: int, m: int, k: int, n: int) -> torch.Tensor | None:
    """A caller-supplied workspace must be a contiguous device tensor of at least
    workspace_size() bytes (the C ABI trusts the size it is given)."""
    need = workspace_size(op, m, k, n)
    if need == 0:
        return None
    _dev(ws, "workspace")
    if ws.numel() * ws.element_size() < need:
        raise BitLinearError(f"workspace holds {ws.numel() * ws.element_size()} bytes, {need} needed")
    return ws


def _check_out(out: torch.Tensor, shape, dtype, name: str):
    _dev(out, name, dtype)
    if tuple(out.shape) != tuple(shape):
        raise BitLinearError(f"{name} must have shape {tuple(shape)}, got {tuple(out.shape)}")


def workspace_size(op: int, m: int, k: int, n: int) -> int:
    return int(load_library().bitlinear_workspace_size(op, m, k, n))


def pack_weights(w: torch.Tensor):
    """fp32 weights [n][k] -> (packed uint8 [n][k/4], gamma fp32 [1])."""
    lib = load_library()
    n, k = w.shape
    packed = torch.empty((n, k // 4), dtype=torch.uint8, device=w.device)
    gamma = torch.empty(1, dtype=torch.float32, device=w.device)
    ws = _workspace(OP_PACK, 0, k, n, w.device)
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_pack_weights(_dev(w, "w", torch.float32), n, k, packed.data_ptr(),
                                      gamma.data_ptr(), wp, wn, _stream(w.device)),
           "bitlinear_pack_weights")
    return packed, gamma


def pack_weights_threshold(w: torch.Tensor, factor: float = 0.7):
    """fp32 weights [n][k] -> (packed uint8 [n][k/4], alpha fp32 [1], delta fp32 [1]) of the
    threshold quantizer; (packed, alpha) is used like (packed, gamma)."""
    lib = load_library()
    n, k = w.shape
    packed = torch.empty((n, k // 4), dtype=torch.uint8, device=w.device)
    alpha = torch.empty(1, dtype=torch.float32, device=w.device)
    delta = torch.empty(1, dtype=torch.float32, device=w.device)
    ws = _workspace(OP_PACK_THRESHOLD, 0, k, n, w.device)
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_pack_weights_threshold(_dev(w, "w", torch.float32), n, k, float(factor),
                                                packed.data_ptr(), alpha.data_ptr(), delta.data_ptr(), wp, wn,
                                                _stream(w.device)), "bitlinear_pack_weights_threshold")
    return packed, alpha, delta


def quant_act(x: torch.Tensor):
    """activations [m][k] -> (q int8 [m][k], scale fp32 [m])."""
    lib = load_library()
    m, k = x.shape
    q = torch.empty((m, k), dtype=torch.int8, device=x.device)
    s = torch.empty(m, dtype=torch.float32, device=x.device)
    _check(lib.bitlinear_quant_act(_dev(x, "x"), _act_dtype(x), m, k, q.data_ptr(), s.data_ptr(),
                                   _stream(x.device)), "bitlinear_quant_act")
    return q, s


def _gain(gain, k: int):
    if gain is None:
        return None
    if gain.numel() != k:
        raise BitLinearError(f"gain must have {k} entries, got {gain.numel()}")
    return _dev(gain, "gain", torch.float32)


def quant_act_norm(x: torch.Tensor, gain: torch.Tensor | None = None):
    """RMS-normalized activations [m][k] -> (q int8 [m][k], scale fp32 [m])."""
    lib = load_library()
    m, k = x.shape
    q = torch.empty((m, k), dtype=torch.int8, device=x.device)
    s = torch.empty(m, dtype=torch.float32, device=x.device)
    _check(lib.bitlinear_quant_act_norm(_dev(x, "x"), _act_dtype(x), m, k, _gain(gain, k), q.data_ptr(),
                                        s.data_ptr(), _stream(x.device)), "bitlinear_quant_act_norm")
    return q, s


def forward_norm(x: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor, gain: torch.Tensor | None = None,
                 *, return_acc: bool = False, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """BitLinear forward of the RMS-normalized x (the normalization fused into the quantization)."""
    lib = load_library()
    m, k = x.shape
    n = packed.shape[0]
    if packed.shape[1] * 4 != k:
        raise BitLinearError("packed weights do not match the activation width")
    if out is not None:
        _check_out(out, (m, n), torch.float32, "out")
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if return_acc else None
    ws = (_caller_workspace(workspace, OP_FORWARD_NORM, m, k, n) if workspace is not None
          else _workspace(OP_FORWARD_NORM, m, k, n, x.device))
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_forward_norm(_dev(x, "x"), _act_dtype(x), m, k, _gain(gain, k),
                                      _dev(packed, "packed", torch.uint8), _dev(gamma, "gamma", torch.float32), n,
                                      _dev(y, "y", torch.float32), acc.data_ptr() if acc is not None else None,
                                      wp, wn, _stream(x.device)), "bitlinear_forward_norm")
    return (y, acc) if return_acc else y


def quant_act_a4(x: torch.Tensor, keep: int | None = None):
    """4-bit activations [m][k] -> (q int8 [m][k] holding 2e, scale fp32 [m]); keep defaults to ceil(k / 2)."""
    lib = load_library()
    m, k = x.shape
    keep = (k + 1) // 2 if keep is None else int(keep)
    q = torch.empty((m, k), dtype=torch.int8, device=x.device)
    s = torch.empty(m, dtype=torch.float32, device=x.device)
    _check(lib.bitlinear_quant_act_a4(_dev(x, "x"), _act_dtype(x), m, k, keep, q.data_ptr(), s.data_ptr(),
                                      _stream(x.device)), "bitlinear_quant_act_a4")
    return q, s


def forward_a4(x: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor, keep: int | None = None,
               *, return_acc: bool = False, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None):
    """W1.58A4 forward: 4-bit top-K activations times the ternary weights."""
    lib = load_library()
    m, k = x.shape
    n = packed.shape[0]
    keep = (k + 1) // 2 if keep is None else int(keep)
    if packed.shape[1] * 4 != k:
        raise BitLinearError("packed weights do not match the activation width")
    if out is not None:
        _check_out(out, (m, n), torch.float32, "out")
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if return_acc else None
    ws = (_caller_workspace(workspace, OP_FORWARD_A4, m, k, n) if workspace is not None
          else _workspace(OP_FORWARD_A4, m, k, n, x.device))
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_forward_a4(_dev(x, "x"), _act_dtype(x), m, k, keep, _dev(packed, "packed", torch.uint8),
                                    _dev(gamma, "gamma", torch.float32), n, _dev(y, "y", torch.float32),
                                    acc.data_ptr() if acc is not None else None, wp, wn, _stream(x.device)),
           "bitlinear_forward_a4")
    return (y, acc) if return_acc else y


def forward(x: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor, *, return_acc: bool = False,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """BitLinear forward. x [m][k] (fp32/bf16), packed uint8 [n][k/4], gamma fp32 [1]."""
    lib = load_library()
    m, k = x.shape
    n = packed.shape[0]
    if packed.shape[1] * 4 != k:
        raise BitLinearError("packed weights do not match the activation width")
    if out is not None:
        _check_out(out, (m, n), torch.float32, "out")
    y = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=x.device)
    acc = torch.empty((m, n), dtype=torch.int32, device=x.device) if return_acc else None
    ws = (_caller_workspace(workspace, OP_FORWARD, m, k, n) if workspace is not None
          else _workspace(OP_FORWARD, m, k, n, x.device))
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_forward(_dev(x, "x"), _act_dtype(x), m, k, _dev(packed, "packed", torch.uint8),
                                 _dev(gamma, "gamma", torch.float32), n, _dev(y, "y", torch.float32),
                                 acc.data_ptr() if acc is not None else None, wp, wn,
                                 _stream(x.device)), "bitlinear_forward")
    return (y, acc) if return_acc else y


def ffn(x: torch.Tensor, gate, up, down, *, return_hq: bool = False,
        workspace: torch.Tensor | None = None):
    """Squared-ReLU gated FFN. gate/up/down are (packed, gamma) pairs:
    gate/up packed [ffn][hidden/4], down packed [hidden][ffn/4]."""
    lib = load_library()
    m, hidden = x.shape
    ffn_dim = gate[0].shape[0]
    if gate[0].shape[1] * 4 != hidden or up[0].shape != gate[0].shape or \
            down[0].shape != (hidden, ffn_dim // 4):
        raise BitLinearError("FFN weight shapes do not match")
    y = torch.empty((m, hidden), dtype=torch.float32, device=x.device)
    hq = torch.empty((m, ffn_dim), dtype=torch.int8, device=x.device) if return_hq else None
    hs = torch.empty(m, dtype=torch.float32, device=x.device) if return_hq else None
    ws = (_caller_workspace(workspace, OP_FFN, m, hidden, ffn_dim) if workspace is not None
          else _workspace(OP_FFN, m, hidden, ffn_dim, x.device))
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_ffn(_dev(x, "x"), _act_dtype(x), m, hidden, ffn_dim,
                             _dev(gate[0], "gate_packed", torch.uint8),
                             _dev(gate[1], "gate_gamma", torch.float32),
                             _dev(up[0], "up_packed", torch.uint8), _dev(up[1], "up_gamma", torch.float32),
                             _dev(down[0], "down_packed", torch.uint8),
                             _dev(down[1], "down_gamma", torch.float32),
                             y.data_ptr(), hq.data_ptr() if hq is not None else None,
                             hs.data_ptr() if hs is not None else None, wp, wn, _stream(x.device)),
           "bitlinear_ffn")
    return (y, hq, hs) if return_hq else y


def pack_kmajor(packed: torch.Tensor):
    """packed [n][k/4] -> the input-major packing [k][n/4] of the same codes (n % 4 == 0)."""
    lib = load_library()
    n, kb = packed.shape
    out = torch.empty((4 * kb, n // 4), dtype=torch.uint8, device=packed.device)
    _check(lib.bitlinear_pack_kmajor(_dev(packed, "packed", torch.uint8), n, 4 * kb, out.data_ptr(),
                                     _stream(packed.device)), "bitlinear_pack_kmajor")
    return out


def ffn_sparse(x: torch.Tensor, gate, up, down_t, *, return_hq: bool = False,
               workspace: torch.Tensor | None = None):
    """Decode FFN (m <= 4) skipping the zero channels of h in the down projection.
    gate/up are (packed [ffn][hidden/4], gamma); down_t is (pack_kmajor(down packed), gamma)."""
    lib = load_library()
    m, hidden = x.shape
    ffn_dim = gate[0].shape[0]
    if gate[0].shape[1] * 4 != hidden or up[0].shape != gate[0].shape or \
            down_t[0].shape != (ffn_dim, hidden // 4):
        raise BitLinearError("FFN weight shapes do not match")
    y = torch.empty((m, hidden), dtype=torch.float32, device=x.device)
    hq = torch.empty((m, ffn_dim), dtype=torch.int8, device=x.device) if return_hq else None
    hs = torch.empty(m, dtype=torch.float32, device=x.device) if return_hq else None
    ws = (_caller_workspace(workspace, OP_FFN_SPARSE, m, hidden, ffn_dim) if workspace is not None
          else _workspace(OP_FFN_SPARSE, m, hidden, ffn_dim, x.device))
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_ffn_sparse(_dev(x, "x"), _act_dtype(x), m, hidden, ffn_dim,
                                    _dev(gate[0], "gate_packed", torch.uint8),
                                    _dev(gate[1], "gate_gamma", torch.float32),
                                    _dev(up[0], "up_packed", torch.uint8), _dev(up[1], "up_gamma", torch.float32),
                                    _dev(down_t[0], "down_packed_t", torch.uint8),
                                    _dev(down_t[1], "down_gamma", torch.float32),
                                    y.data_ptr(), hq.data_ptr() if hq is not None else None,
                                    hs.data_ptr() if hs is not None else None, wp, wn, _stream(x.device)),
           "bitlinear_ffn_sparse")
    return (y, hq, hs) if return_hq else y


def gemm_i32(q: torch.Tensor, packed: torch.Tensor):
    """Bare int8 x ternary product: q int8 [m][k], packed [n][k/4] -> acc int32 [m][n]."""
    lib = load_library()
    m, k = q.shape
    n = packed.shape[0]
    acc = torch.empty((m, n), dtype=torch.int32, device=q.device)
    ws = _workspace(OP_GEMM_I32, m, k, n, q.device)
    wp, wn = _ws_args(ws)
    _check(lib.bitlinear_gemm_i32(_dev(q, "q", torch.int8), m, k, _dev(packed, "packed", torch.uint8), n,
                                  acc.data_ptr(), wp, wn, _stream(q.device)), "bitlinear_gemm_i32")
    return acc


# ---------------------------------------------------------------- attention and the 8-bit cache
CACHE_BLOCK = 64  # BL_CACHE_BLOCK in include/bitlinear.h


class KVCache(NamedTuple):
    """Pages of CACHE_BLOCK tokens: int8 codes [pages][kv_heads][64 * head_dim] in the order that
    include/bitlinear.h gives, and one fp32 scale per page and head [pages][kv_heads], for K and V."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def cache_alloc(pages: int, kv_heads: int, head_dim: int, device="cuda") -> KVCache:
    """An empty cache (head_dim 64 or 128)."""
    if head_dim not in (64, 128) or pages < 1 or kv_heads < 1:
        raise BitLinearError("a cache needs pages >= 1, kv_heads >= 1 and a head_dim of 64 or 128")
    codes = [torch.zeros((pages, kv_heads, CACHE_BLOCK * head_dim), dtype=torch.int8, device=device) for _ in range(2)]
    scales = [torch.zeros((pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(*codes, *scales)


# One token's calls take a few microseconds on the device, as long as it takes to look at their
# tensors from here: csrc/binding.cpp does that and calls the same C ABI. Its checks raise BitLinearError.
_native = None


def _attention_calls():
    global _native
    if _native is None:
        load_library()
        try:
            from . import _binding as module
        except ImportError as e:
            raise BitLinearError(f"the binding of the attention calls is not built ({e}); run __graft_entry__.build() first") from e
        module.bind(_LIB_PATH, BitLinearError)
        _native = module
    return _native


def attention_workspace_size(dtype: torch.dtype, m: int, q_heads: int, kv_heads: int, head_dim: int, seqs: int) -> int:
    code = _F32 if dtype == torch.float32 else _BF16 if dtype == torch.bfloat16 else -1
    return int(load_library().bitlinear_attention_workspace_size(code, m, q_heads, kv_heads, head_dim, seqs))


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
              scale: float | None = None, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Causal attention over packed prompts. q [m][q_heads][head_dim], k and v [m][kv_heads][head_dim]
    (fp32 or bf16, possibly slices of one projection's rows), cu_seqlens int32 [seqs + 1], not decreasing,
    -> [m][q_heads * head_dim] of q's type. Rows outside the sequences are not written."""
    return (_native or _attention_calls()).attention(q, k, v, cu_seqlens, scale, out, workspace)


def cache_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                 cu_seqlens: torch.Tensor | None = None) -> None:
    """Quantizes new tokens into the cache: row i of sequence s becomes token lens[s] + i. Without
    cu_seqlens, one row per sequence. lens is left as it is (a negative entry: an unused slot)."""
    (_native or _attention_calls()).cache_append(cache, k, v, block_table, lens, cu_seqlens)


def cache_read(cache: KVCache, block_table: torch.Tensor, begin: torch.Tensor, cu_seqlens: torch.Tensor | None, m: int,
               dtype: torch.dtype = torch.float32):
    """The values of tokens begin[s] + i of every sequence, as many as cu_seqlens gives rows (m in all;
    None: one each) -> (k, v) [m][kv_heads][head_dim]. Rows outside the sequences are not written."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise BitLinearError(f"dtype must be float32 or bfloat16, got {dtype}")
    return (_native or _attention_calls()).cache_read(cache, block_table, begin, cu_seqlens, m, dtype == torch.bfloat16)


def attention_cached_workspace_size(m: int, q_heads: int, kv_heads: int, head_dim: int, seqs: int, max_blocks: int,
                                    weights: bool = False) -> int:
    return int(load_library().bitlinear_attention_cached_workspace_size(m, q_heads, kv_heads, head_dim, seqs, max_blocks,
                                                                        int(weights)))


def attention_cached(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lens: torch.Tensor,
                     cu_seqlens: torch.Tensor | None = None, *, scale: float | None = None,
                     weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """Attention of new tokens, already appended, over the cache: row i of sequence s is token
    lens[s] + i and sees the tokens up to itself. q [m][q_heads][head_dim] -> [m][q_heads * head_dim]
    of q's type; weights fp32 [seqs][max_blocks] gets each block's attention weight added."""
    return (_native or _attention_calls()).attention_cached(q, cache, block_table, lens, cu_seqlens, scale, weights, out, workspace)


def cache_evict(block_table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor, keep: int, *, first: int = 0,
                recent: int = 1):
    """Chooses the blocks every sequence keeps: its first `first`, its last `recent` and, up to `keep`
    in all, those of the largest weight -> (block_table, lens, weights) of the kept blocks, and
    (evicted, evicted_count): the pages of the others (free now, unless sequences share them), -1 behind them."""
    return (_native or _attention_calls()).cache_evict(block_table, lens, weights, keep, first, recent)


# ---------------------------------------------------------------- positions, a shared prefix, chosen blocks

def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       length: int | None = None, low: float = 1.0, high: float = 32.0, device="cuda") -> torch.Tensor:
    """Angles per position of a head's rotated pairs, base^(-2 i / rotary_dim), fp32 [rotary_dim / 2] (computed in 64
    bits). For a context `factor` times the one a model was trained on (`length` tokens), scaling is
      "positions"  every angle divided by factor;
      "base"       the base raised to base * factor^(n / (n - 2)), n = rotary_dim: the slowest pair's angle divided by
                   factor, the fastest one's kept;
      "parts"      pairs that turn more than `high` times within `length` kept, those that turn less than `low` times
                   divided by factor, between the two linear in the number of turns. The attention's logits often
                   grow with it: rotate()'s magnitude, say 0.1 * log(factor) + 1."""
    if not (16 <= rotary_dim and rotary_dim % 16 == 0):
        raise BitLinearError(f"rotary_dim must be a multiple of 16, got {rotary_dim}")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor > 0):
        raise BitLinearError("base and factor must be finite and positive")
    if scaling not in (None, "positions", "base", "parts"):
        raise BitLinearError(f'scaling must be None, "positions", "base" or "parts", got {scaling!r}')
    if scaling == "base":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    if scaling == "positions":
        freq = freq / factor
    if scaling == "parts":
        if length is None or length < 1 or not 0 <= low < high:
            raise BitLinearError('scaling "parts" needs length >= 1 and 0 <= low < high')
        kept = ((length * freq / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        freq = freq * (kept + (1 - kept) / factor)
    return freq.to(torch.float32).to(device)


def rotate(q: torch.Tensor, k: torch.Tensor, inv_freq: torch.Tensor, begin: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *,
           interleaved: bool = False, q_gain: torch.Tensor | None = None, k_gain: torch.Tensor | None = None, eps: float = 1e-5,
           magnitude: float = 1.0, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """Rotates queries and keys by their tokens' positions, row i of sequence s standing at begin[s] + i (int32 [seqs];
    negative: an unused slot; without cu_seqlens one row per sequence), on the first 2 * len(inv_freq) elements of every
    head: pairs (i, i + len(inv_freq)), or (2i, 2i + 1) if interleaved. With a gain (fp32 [head_dim]) the head's RMS norm
    comes before. -> (q, k) dense, or `out`, which may be (q, k) themselves."""
    return (_native or _attention_calls()).rotate(q, k, inv_freq, begin, cu_seqlens, interleaved, q_gain, k_gain, eps, magnitude, out)


def attention_shared_workspace_size(m: int, q_heads: int, kv_heads: int, head_dim: int, seqs: int, max_blocks: int, prefix_blocks: int) -> int:
    return int(load_library().bitlinear_attention_shared_workspace_size(m, q_heads, kv_heads, head_dim, seqs, max_blocks, prefix_blocks))


def attention_shared(q: torch.Tensor, cache: KVCache, prefix_table: torch.Tensor, prefix_len: torch.Tensor, block_table: torch.Tensor,
                     lens: torch.Tensor, cu_seqlens: torch.Tensor | None = None, *, scale: float | None = None,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """attention_cached of a batch whose sequences share a prefix: every row sees the prefix's tokens (pages
    prefix_table int32 [prefix_blocks], prefix_len int32 [1] of them) and its own sequence's up to itself. lens and
    block_table count and hold the sequences' own tokens only. For bf16 queries the softmax weights over the prefix are
    rounded to fp16 (2^-11 of themselves; attention_cached holds 23 bits, as this call does for fp32)."""
    return (_native or _attention_calls()).attention_shared(q, cache, prefix_table, prefix_len, block_table, lens, cu_seqlens, scale,
                                                            out, workspace)


def bounds_alloc(cache: KVCache) -> torch.Tensor:
    """Bounds for every page of a cache: int8 [pages][kv_heads][2][head_dim]."""
    pages, heads, codes = cache.k.shape
    return torch.zeros((pages, heads, 2, codes // CACHE_BLOCK), dtype=torch.int8, device=cache.k.device)


def cache_bounds(cache: KVCache, bounds: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, cu_seqlens: torch.Tensor | None,
                 m: int) -> None:
    """The largest and the smallest K code of every dim, for the blocks that the m rows of a cache_append with the same
    tables reached (called after it, lens still as they were)."""
    (_native or _attention_calls()).cache_bounds(cache, bounds, block_table, lens, cu_seqlens, m)


def block_select_workspace_size(m: int, kv_heads: int, max_blocks: int) -> int:
    return int(load_library().bitlinear_block_select_workspace_size(m, kv_heads, max_blocks))


def block_select(q: torch.Tensor, bounds: torch.Tensor, k_scale: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, keep: int,
                 cu_seqlens: torch.Tensor | None = None, *, first: int = 0, recent: int = 1, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """Chooses the blocks of its sequence that every row and kv head attends to: the first `first`, the last `recent` (its
    own among them) and, up to `keep` in all, those whose keys may have the largest product with its queries by their
    bounds (k_scale: the cache's) -> int32 [m][kv_heads][keep], ascending, -1 behind them."""
    return (_native or _attention_calls()).block_select(q, bounds, k_scale, block_table, lens, keep, cu_seqlens, first, recent, out,
                                                        workspace)


def attention_selected_workspace_size(m: int, q_heads: int, kv_heads: int, head_dim: int, keep: int) -> int:
    return int(load_library().bitlinear_attention_selected_workspace_size(m, q_heads, kv_heads, head_dim, keep))


def attention_selected(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, lens: torch.Tensor, selected: torch.Tensor,
                       cu_seqlens: torch.Tensor | None = None, *, scale: float | None = None, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None):
    """attention_cached over the blocks that selected int32 [m][kv_heads][keep] lists for each row and kv head (entries
    that name no block are passed over, a block counts as often as it is listed)."""
    return (_native or _attention_calls()).attention_selected(q, cache, block_table, lens, selected, cu_seqlens, scale, out, workspace)
