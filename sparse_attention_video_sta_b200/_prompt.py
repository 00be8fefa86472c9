"""The prompt side of the binding: attention of packed sequences, and the 8-bit cache.

Same manner as the rest of the package (C names, argument checks, the current
CUDA stream); the package's namespace re-exports everything here.  The checks,
the outputs' and scratch's allocation and the calls into libsta are compiled
(``csrc/sta_torch.cpp``): a serving step makes these calls for every layer.  Tensors are
token-major, ``[tokens, heads, d]``, with free token and head strides
(multiples of 8 elements), so the parts of one fused projection are taken as
they are.

``stream`` (a ``torch.cuda.Stream`` or a raw handle; default the current one)
is the stream of a call's kernels and, for new tensors and scratch, of their
memory: the caller sees to it that this stream is behind what made the inputs
and in front of what reads the results.  New tensors may be dropped on the
current stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._build import torch_key


class _Missing:
    """Stands for a ``_sta_torch.so`` that is not there or is another PyTorch's or Python's: the calls of this part
    say so, the others need only libsta."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{self._why}; build _sta_torch.so with `python sparse_attention_video_sta_b200/_build.py`")


def _load():
    try:
        from . import _sta_torch
    except ImportError as e:
        return _Missing(str(e))
    built_for = getattr(_sta_torch, "built_for", "another version of this package")
    if built_for != torch_key():
        return _Missing(f"_sta_torch.so was built for {built_for}, this is {torch_key()}")
    return _sta_torch


_torch = _load()

__all__ = [
    "sta_packed_forward", "sta_packed_backward", "sta_packed_attention", "sta_packed_attention_backward",
    "StaPackedAttention", "sta_cache_append", "sta_cache_attention", "sta_cache_extend", "CacheStep",
    "sta_operator_status", "sta_debug_inject_operator_timeout", "SYMBOLS",
]

SYMBOLS = (
    "sta_packed_workspace", "sta_packed_forward", "sta_packed_backward", "sta_cache_append", "sta_cache_workspace",
    "sta_cache_attention", "sta_cache_extend", "sta_operator_status", "sta_debug_inject_operator_timeout",
)


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Packed(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("tokens_q", ctypes.c_int64), ("tokens_k", ctypes.c_int64),
                ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("causal", ctypes.c_int32),
                ("clear_tail", ctypes.c_int32), ("softmax_scale", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_int32), ("block_tokens", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


_lib = None
_check = None


def bind(lib, check) -> None:
    """Declare the C signatures on the loaded library (called by the package)."""
    global _lib, _check
    _lib, _check = lib, check
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    R, P, C, N = (ctypes.POINTER(t) for t in (_Rows, _Packed, _Cache, ctypes.c_int64))
    for name, args in {
        "sta_packed_workspace": [P, i32, N],
        "sta_packed_forward": [P, R, R, R, R, vp, vp, i64, vp],
        "sta_packed_backward": [P, R, R, R, R, R, vp, R, R, R, vp, i64, vp],
        "sta_cache_append": [C, R, R, i64, vp, vp],
        "sta_cache_workspace": [C, P, N],
        "sta_cache_attention": [C, P, vp, vp, i32, i64, R, R, vp, vp, i64, vp],
        "sta_cache_extend": [i32, i32, vp, vp, vp, vp, i32, i64, vp, i32, vp, vp, vp, i64, vp, vp, vp],
        "sta_operator_status": [vp],
        "sta_debug_inject_operator_timeout": [i32, i32],
    }.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ctypes.c_int
    if not isinstance(_torch, _Missing):
        _torch.bind({name: ctypes.cast(getattr(lib, name), vp).value for name in SYMBOLS}, check)


def _raw(stream) -> int:
    """The handle of a stream (a ``torch.cuda.Stream`` or a raw one); -1 is the current stream."""
    if stream is None:
        return -1
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


# ---------------------------------------------------------------- packed attention
def sta_packed_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                       cu_q: torch.Tensor, cu_k: torch.Tensor | None = None, causal: bool = True,
                       softmax_scale: float | None = None, clear_tail: bool = False, workspace=None, stream=None):
    """Attention of packed sequences into ``o`` (like ``q``) and ``lse`` (fp32 ``[heads, tokens]``).

    ``q`` ``[tokens, heads, d]`` and ``k``, ``v`` ``[tokens_k, kv_heads, d]`` in bf16; sequence ``b`` has the
    query rows ``cu_q[b] : cu_q[b + 1]`` and the key rows ``cu_k[b] : cu_k[b + 1]`` (``cu_k`` defaults to
    ``cu_q``; int32, on the device, read by the kernels).  With ``causal`` a sequence's last query sees
    every key.  Rows behind the last sequence are left as they were, or zeroed with ``clear_tail``; so are those
    before the first, though bounds that do not begin at 0 are reported (``sta_operator_status``)."""
    _torch.packed_forward(q, k, v, o, lse, cu_q, cu_k, causal, softmax_scale, clear_tail, workspace, _raw(stream))
    return o, lse


def sta_packed_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                        dout: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, cu_q: torch.Tensor,
                        cu_k: torch.Tensor | None = None, causal: bool = True, softmax_scale: float | None = None,
                        clear_tail: bool = False, workspace=None, stream=None):
    """Gradients of ``sta_packed_forward`` into ``dq`` (like ``q``), ``dk`` and ``dv`` (like ``k``); ``o`` and
    ``lse`` as the forward wrote them for the same problem."""
    _torch.packed_backward(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, causal, softmax_scale, clear_tail, workspace,
                           _raw(stream))
    return dq, dk, dv


def sta_packed_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                         cu_k: torch.Tensor | None = None, causal: bool = True, softmax_scale: float | None = None,
                         stream=None):
    """``sta_packed_forward`` into new tensors; rows behind the last sequence are zeros (``lse`` -inf).
    Returns ``(o bf16 [tokens, heads, d], lse fp32 [heads, tokens])``."""
    return _torch.packed_attention(q, k, v, cu_q, cu_k, causal, softmax_scale, _raw(stream))


def sta_packed_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                                  lse: torch.Tensor, dout: torch.Tensor, cu_q: torch.Tensor,
                                  cu_k: torch.Tensor | None = None, causal: bool = True,
                                  softmax_scale: float | None = None, stream=None):
    """``sta_packed_backward`` into new tensors ``(dq, dk, dv)``; rows behind the last sequence are zeros."""
    return _torch.packed_attention_backward(q, k, v, o, lse, dout, cu_q, cu_k, causal, softmax_scale, _raw(stream))


def _usable(t: torch.Tensor) -> torch.Tensor:
    """``t``, or a contiguous copy where its strides are not ones that the kernels take."""
    st, sh, sd = t.stride()
    fine = sd == 1 and (st > 0 and st % 8 == 0 or t.shape[0] <= 1) and (sh > 0 and sh % 8 == 0 or t.shape[1] == 1) and \
        t.data_ptr() % 16 == 0
    return t if fine else t.clone(memory_format=torch.contiguous_format)


class StaPackedAttention(torch.autograd.Function):
    """``O = StaPackedAttention.apply(q, k, v, cu_q, cu_k, causal, softmax_scale)`` on packed bf16 tensors,
    with gradients for q, k and v."""

    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k=None, causal=True, softmax_scale=None):
        q, k, v = _usable(q), _usable(k), _usable(v)
        o, lse = sta_packed_attention(q, k, v, cu_q, cu_k, causal, softmax_scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_q if cu_k is None else cu_k)
        ctx.causal, ctx.scale = causal, softmax_scale
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
        dq, dk, dv = sta_packed_attention_backward(q, k, v, o, lse, _usable(dout), cu_q, cu_k, ctx.causal, ctx.scale)
        return dq, dk, dv, None, None, None, None


# ---------------------------------------------------------------- cache
def sta_cache_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor, stream=None) -> None:
    """Write new tokens' ``k`` and ``v`` (bf16 ``[tokens, kv_heads, d]``) into the cache at ``slots`` (int64;
    negative: skipped), as ``sta_cache_extend`` gives them.

    ``k_cache``, ``v_cache``: e4m3 ``[blocks, kv_heads, block_tokens, d]``; ``k_scales``, ``v_scales``: fp32
    ``[blocks, kv_heads]``, a power of two for each block that grows with what the block holds."""
    _torch.cache_append(k, v, slots, k_cache, v_cache, k_scales, v_scales, _raw(stream))


def sta_cache_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                        v_scales: torch.Tensor, block_tables: torch.Tensor, lengths: torch.Tensor,
                        cu_q: torch.Tensor | None = None, softmax_scale: float | None = None, o=None, lse=None,
                        workspace=None, stream=None):
    """Causal attention of ``q`` (bf16 ``[tokens, heads, d]``) over the cache.

    ``lengths`` (int32): tokens of each sequence in the cache, its queries' own among them; ``block_tables``
    (int32 ``[batch, width]``): its blocks in order.  ``cu_q`` bounds each sequence's queries; without it there
    is one query for each sequence.  Returns ``(o, lse fp32 [heads, tokens])``; given tensors keep their rows
    behind the last sequence, new ones have zeros (-inf) there."""
    return _torch.cache_attention(q, k_cache, v_cache, k_scales, v_scales, block_tables, lengths, cu_q, softmax_scale, o,
                                  lse, workspace, _raw(stream))


class CacheStep(NamedTuple):
    """What ``sta_cache_extend`` gives a step."""
    slots: torch.Tensor       # int64 [max_slots]: the new tokens' slots, then -1
    cu_new: torch.Tensor      # int32 [batch + 1]: bounds of each request's new tokens
    lengths: torch.Tensor     # int32 [batch]: tokens held after the step
    free_count: torch.Tensor  # int32 [1]
    short: torch.Tensor       # int32 [1]: 0 done, n > 0 blocks missing, -1 out of range; unless 0 nothing changed


def sta_cache_extend(new_tokens: torch.Tensor, lengths: torch.Tensor, block_tables: torch.Tensor,
                     free_blocks: torch.Tensor, free_count: torch.Tensor, block_tokens: int, max_slots: int,
                     in_place: bool = False, stream=None) -> CacheStep:
    """Block tables and slots of a step, on the GPU: requests with ``new_tokens`` >= 0 get the blocks that
    their tokens need from the top of the free stack (``free_blocks[:free_count]``), after those with negative
    ``new_tokens`` (ended) have returned theirs.  ``block_tables`` and ``free_blocks`` are changed; ``lengths``
    and ``free_count`` too with ``in_place``, else new tensors hold what they become."""
    return CacheStep(*_torch.cache_extend(new_tokens, lengths, block_tables, free_blocks, free_count, block_tokens,
                                          max_slots, in_place, _raw(stream)))


def sta_operator_status(device=None, stream=None) -> int:
    """Synchronise and return (clearing it) the status of the calls of this part on ``device``: 0,
    ``STA_ERR_TIMEOUT`` or ``STA_ERR_BOUNDS`` (of both, the first; the next call then returns the other)."""
    with torch.cuda.device(device):
        s = torch.cuda.current_stream() if stream is None else stream
        h = s.cuda_stream if isinstance(s, torch.cuda.Stream) else int(s)
        return int(_lib.sta_operator_status(h))


def sta_debug_inject_operator_timeout(mode, limit_ms: int = 50) -> None:
    """Debug: make a device-side wait of the next packed or cache attention calls run out (``mode`` 0 off, 1 on)."""
    _check(_lib.sta_debug_inject_operator_timeout(int(mode), int(limit_ms)), "sta_debug_inject_operator_timeout")
