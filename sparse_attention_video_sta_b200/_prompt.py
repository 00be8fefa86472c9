"""The prompt side of the binding: attention of packed sequences, and the 8-bit cache.

Same manner as the rest of the package (C names, argument checks, the current
CUDA stream); the package's namespace re-exports everything here.  Tensors are
token-major, ``[tokens, heads, d]``, with free token and head strides
(multiples of 8 elements), so the parts of one fused projection are taken as
they are.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

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


# ---------------------------------------------------------------- arguments
# A serving step makes these calls for every layer, and the smallest kernels take a few
# microseconds: the checks below are written for few Python operations.
class _on:
    """The device and stream of one call: makes the tensors' device current, and hands the call's
    scratch and outputs to ``stream`` when that is not the current one."""

    __slots__ = ("device", "stream", "handle", "guard")

    def __init__(self, device: torch.device, stream):
        self.device, self.stream = device, stream

    def __enter__(self):
        self.guard = None
        index = self.device.index
        if index != torch._C._cuda_getDevice():
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        if self.stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(index)
        else:
            if not isinstance(self.stream, torch.cuda.Stream):
                self.stream = torch.cuda.ExternalStream(int(self.stream), device=self.device)
            self.handle = self.stream.cuda_stream
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def keep(self, *tensors):
        if self.stream is not None:
            for t in tensors:
                t.record_stream(self.stream)


def _rows(name: str, t: torch.Tensor, device, tokens: int, heads: int, d: int) -> _Rows:
    if t.dtype is not torch.bfloat16 or t.device != device:
        raise ValueError(f"{name} must be a bf16 tensor on {device}")
    if t.shape != (tokens, heads, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{tokens}, {heads}, {d}]")
    st, sh, sd = t.stride()
    if heads == 1:
        sh = d
    if tokens <= 1:
        st = heads * d
    p = t.data_ptr()
    if sd != 1 or st <= 0 or sh <= 0 or (st | sh) & 7 or p & 15:
        raise ValueError(f"{name}: the last dimension must be contiguous, the other strides positive multiples of 8 "
                         f"elements and the data 16-byte aligned (strides {t.stride()})")
    return _Rows(p, st, sh)


def _ints(name: str, t: torch.Tensor, device, size: int | None, dtype=torch.int32) -> int:
    if t.dtype is not dtype or t.device != device or t.dim() != 1 or not t.is_contiguous() or \
            (size is not None and t.shape[0] != size):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape [{'n' if size is None else size}] on {device}")
    return t.data_ptr()


def _problem(q, k, cu_q, cu_k, causal, clear_tail, softmax_scale) -> _Packed:
    if not q.is_cuda:
        raise ValueError("packed attention needs CUDA tensors")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, d]")
    if cu_k is None:
        cu_k = cu_q
    batch = cu_q.shape[0] - 1 if cu_q.dim() == 1 else -1
    if batch < 0:
        raise ValueError("cu_q must be [sequences + 1]")
    scale = 1.0 / math.sqrt(q.shape[2]) if softmax_scale is None else float(softmax_scale)
    return _Packed(batch, q.shape[1], k.shape[1], q.shape[2], q.shape[0], k.shape[0],
                   _ints("cu_q", cu_q, q.device, batch + 1), _ints("cu_k", cu_k, q.device, batch + 1),
                   1 if causal else 0, 1 if clear_tail else 0, scale)


def _lse_ptr(lse, q) -> int:
    if lse.dtype != torch.float32 or lse.device != q.device or not lse.is_contiguous() or \
            tuple(lse.shape) != (q.shape[1], q.shape[0]):
        raise ValueError(f"lse must be a contiguous fp32 tensor of shape [{q.shape[1]}, {q.shape[0]}] on {q.device}")
    return lse.data_ptr()


_sizes = {}  # workspace bytes by the sizes that they follow from


def _workspace(key, call, what, workspace, device, *args):
    """(tensor, pointer, bytes) of a call's scratch; allocated unless given."""
    need = _sizes.get(key)
    if need is None:
        n = ctypes.c_int64(0)
        _check(call(*args, ctypes.byref(n)), what)
        if len(_sizes) > 10000:
            _sizes.clear()
        need = _sizes[key] = n.value
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
            workspace.numel() < need:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {device}")
    return workspace, workspace.data_ptr(), workspace.numel()


def _packed_workspace(p, backward, workspace, device):
    key = (p.batch, p.heads, p.kv_heads, p.head_dim, p.tokens_q, p.tokens_k, backward, device.index)
    return _workspace(key, _lib.sta_packed_workspace, "sta_packed_workspace", workspace, device, ctypes.byref(p), backward)


def _empty_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


# ---------------------------------------------------------------- packed attention
def sta_packed_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                       cu_q: torch.Tensor, cu_k: torch.Tensor | None = None, causal: bool = True,
                       softmax_scale: float | None = None, clear_tail: bool = False, workspace=None, stream=None):
    """Attention of packed sequences into ``o`` (like ``q``) and ``lse`` (fp32 ``[heads, tokens]``).

    ``q`` ``[tokens, heads, d]`` and ``k``, ``v`` ``[tokens_k, kv_heads, d]`` in bf16; sequence ``b`` has the
    query rows ``cu_q[b] : cu_q[b + 1]`` and the key rows ``cu_k[b] : cu_k[b + 1]`` (``cu_k`` defaults to
    ``cu_q``; int32, on the device, read by the kernels).  With ``causal`` a sequence's last query sees
    every key.  Rows behind the last sequence are left as they were, or zeroed with ``clear_tail``."""
    p = _problem(q, k, cu_q, cu_k, causal, clear_tail, softmax_scale)
    dev = q.device
    with _on(dev, stream) as on:
        args = (ctypes.byref(p), _rows("q", q, dev, p.tokens_q, p.heads, p.head_dim),
                _rows("k", k, dev, p.tokens_k, p.kv_heads, p.head_dim),
                _rows("v", v, dev, p.tokens_k, p.kv_heads, p.head_dim),
                _rows("o", o, dev, p.tokens_q, p.heads, p.head_dim), _lse_ptr(lse, q))
        if q.shape[0] == 0:
            return o, lse
        w, wp, wn = _packed_workspace(p, 0, workspace, dev)
        _check(_lib.sta_packed_forward(*args, wp, wn, on.handle), "sta_packed_forward")
        if w is not None:
            on.keep(w)
    return o, lse


def sta_packed_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                        dout: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, cu_q: torch.Tensor,
                        cu_k: torch.Tensor | None = None, causal: bool = True, softmax_scale: float | None = None,
                        clear_tail: bool = False, workspace=None, stream=None):
    """Gradients of ``sta_packed_forward`` into ``dq`` (like ``q``), ``dk`` and ``dv`` (like ``k``); ``o`` and
    ``lse`` as the forward wrote them for the same problem."""
    p = _problem(q, k, cu_q, cu_k, causal, clear_tail, softmax_scale)
    dev = q.device
    with _on(dev, stream) as on:
        qs = [_rows(n, t, dev, p.tokens_q, p.heads, p.head_dim)
              for n, t in (("q", q), ("o", o), ("dout", dout), ("dq", dq))]
        ks = [_rows(n, t, dev, p.tokens_k, p.kv_heads, p.head_dim)
              for n, t in (("k", k), ("v", v), ("dk", dk), ("dv", dv))]
        lp = _lse_ptr(lse, q)
        if q.shape[0] == 0 and k.shape[0] == 0:
            return dq, dk, dv
        w, wp, wn = _packed_workspace(p, 1, workspace, dev)
        _check(_lib.sta_packed_backward(ctypes.byref(p), qs[0], ks[0], ks[1], qs[1], qs[2], lp, qs[3], ks[2], ks[3],
                                        wp, wn, on.handle), "sta_packed_backward")
        on.keep(w)
    return dq, dk, dv


def sta_packed_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                         cu_k: torch.Tensor | None = None, causal: bool = True, softmax_scale: float | None = None,
                         stream=None):
    """``sta_packed_forward`` into new tensors; rows behind the last sequence are zeros (``lse`` -inf).
    Returns ``(o bf16 [tokens, heads, d], lse fp32 [heads, tokens])``."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, d]")
    o = _empty_like(q)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    sta_packed_forward(q, k, v, o, lse, cu_q, cu_k, causal, softmax_scale, True, None, stream)
    _keep(stream, o, lse)
    return o, lse


def sta_packed_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                                  lse: torch.Tensor, dout: torch.Tensor, cu_q: torch.Tensor,
                                  cu_k: torch.Tensor | None = None, causal: bool = True,
                                  softmax_scale: float | None = None, stream=None):
    """``sta_packed_backward`` into new tensors ``(dq, dk, dv)``; rows behind the last sequence are zeros."""
    dq, dk, dv = _empty_like(q), _empty_like(k), _empty_like(v)
    sta_packed_backward(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, causal, softmax_scale, True, None, stream)
    _keep(stream, dq, dk, dv)
    return dq, dk, dv


def _keep(stream, *tensors):
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else \
            torch.cuda.ExternalStream(int(stream), device=tensors[0].device)
        for t in tensors:
            t.record_stream(s)


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
_CODES = (torch.float8_e4m3fn, torch.uint8)


def _cache(k_cache, v_cache, k_scales, v_scales) -> _Cache:
    if k_cache.dim() != 4 or not k_cache.is_cuda:
        raise ValueError("k_cache must be a CUDA tensor [blocks, kv_heads, block_tokens, d]")
    dev, shape = k_cache.device, k_cache.shape
    blocks, heads, bt, d = shape
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype not in _CODES or t.device != dev or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous e4m3 (or uint8) tensor of shape {tuple(shape)} on {dev}")
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t.dtype is not torch.float32 or t.device != dev or t.shape != (blocks, heads) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {tuple(shape[:2])} on {dev}")
    return _Cache(blocks, bt, heads, d, k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr())


def _tables(block_tables, batch, device):
    """(pointer, width, stride) of the block tables."""
    width = block_tables.shape[1] if block_tables.dim() == 2 else 0
    rows, cols = block_tables.stride() if width else (0, 0)
    if block_tables.dtype is not torch.int32 or block_tables.device != device or width == 0 or \
            block_tables.shape[0] != batch or (width > 1 and cols != 1) or (batch > 1 and rows < width):
        raise ValueError(f"block_tables must be an int32 tensor [{batch}, width] on {device} with contiguous rows")
    return block_tables.data_ptr(), width, rows if batch > 1 else width


def sta_cache_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor, stream=None) -> None:
    """Write new tokens' ``k`` and ``v`` (bf16 ``[tokens, kv_heads, d]``) into the cache at ``slots`` (int64;
    negative: skipped), as ``sta_cache_extend`` gives them.

    ``k_cache``, ``v_cache``: e4m3 ``[blocks, kv_heads, block_tokens, d]``; ``k_scales``, ``v_scales``: fp32
    ``[blocks, kv_heads]``, a power of two for each block that grows with what the block holds."""
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    dev = k_cache.device
    n = slots.shape[0] if slots.dim() == 1 else -1
    sp = _ints("slots", slots, dev, None, torch.int64)
    kr, vr = (_rows(name, t, dev, n, c.kv_heads, c.head_dim) for name, t in (("k", k), ("v", v)))
    with _on(dev, stream) as on:
        _check(_lib.sta_cache_append(ctypes.byref(c), kr, vr, n, sp, on.handle), "sta_cache_append")


def sta_cache_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                        v_scales: torch.Tensor, block_tables: torch.Tensor, lengths: torch.Tensor,
                        cu_q: torch.Tensor | None = None, softmax_scale: float | None = None, o=None, lse=None,
                        workspace=None, stream=None):
    """Causal attention of ``q`` (bf16 ``[tokens, heads, d]``) over the cache.

    ``lengths`` (int32): tokens of each sequence in the cache, its queries' own among them; ``block_tables``
    (int32 ``[batch, width]``): its blocks in order.  ``cu_q`` bounds each sequence's queries; without it there
    is one query for each sequence.  Returns ``(o, lse fp32 [heads, tokens])``; given tensors keep their rows
    behind the last sequence, new ones have zeros (-inf) there."""
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    dev = k_cache.device
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, d]")
    T, H, d = q.shape
    B = lengths.shape[0] if lengths.dim() == 1 else -1
    lp = _ints("lengths", lengths, dev, None)
    cp = None if cu_q is None else _ints("cu_q", cu_q, dev, B + 1)
    if cu_q is None and T != B:
        raise ValueError(f"{T} queries for {B} sequences: give cu_q")
    tp, width, stride = _tables(block_tables, B, dev)
    new = o is None
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    p = _Packed(B, H, c.kv_heads, d, T, 0, cp, None, 1, 1 if new else 0, scale)
    with _on(dev, stream) as on:
        if new:
            o = _empty_like(q)
            on.keep(o)
        if lse is None:
            lse = torch.empty((H, T), dtype=torch.float32, device=dev)
            on.keep(lse)
        qr, orow = _rows("q", q, dev, T, H, d), _rows("o", o, dev, T, H, d)
        lsp = _lse_ptr(lse, q)
        if T == 0 or B == 0:
            if new:
                o.zero_(), lse.fill_(-math.inf)
            return o, lse
        key = (c.block_tokens, c.kv_heads, d, B, H, T, dev.index)
        w, wp, wn = _workspace(key, _lib.sta_cache_workspace, "sta_cache_workspace", workspace, dev, ctypes.byref(c),
                               ctypes.byref(p))
        _check(_lib.sta_cache_attention(ctypes.byref(c), ctypes.byref(p), lp, tp, width, stride, qr, orow, lsp, wp, wn,
                                        on.handle), "sta_cache_attention")
        on.keep(w)
    return o, lse


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
    dev = lengths.device
    if not lengths.is_cuda:
        raise ValueError("sta_cache_extend needs CUDA tensors")
    B = lengths.shape[0] if lengths.dim() == 1 else -1
    lp, np_ = _ints("lengths", lengths, dev, None), _ints("new_tokens", new_tokens, dev, B)
    fp, cp = _ints("free_blocks", free_blocks, dev, None), _ints("free_count", free_count, dev, 1)
    tp, width, stride = _tables(block_tables, B, dev)
    max_slots = int(max_slots)
    with _on(dev, stream) as on:
        slots = torch.empty(max(max_slots, 0), dtype=torch.int64, device=dev)
        cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
        short = torch.empty_like(free_count)
        len_out = lengths if in_place else torch.empty_like(lengths)
        count_out = free_count if in_place else torch.empty_like(free_count)
        _check(_lib.sta_cache_extend(B, int(block_tokens), np_, lp, len_out.data_ptr(), tp, width, stride, fp,
                                     free_blocks.shape[0], cp, count_out.data_ptr(), slots.data_ptr(), max_slots,
                                     cu.data_ptr(), short.data_ptr(), on.handle), "sta_cache_extend")
        on.keep(slots, cu, short)
        if not in_place:
            on.keep(len_out, count_out)
    return CacheStep(slots, cu, len_out, count_out, short)


def sta_operator_status(device=None, stream=None) -> int:
    """Synchronise and return (clearing it) the status of the calls of this part on ``device``."""
    with torch.cuda.device(device):
        s = torch.cuda.current_stream() if stream is None else stream
        h = s.cuda_stream if isinstance(s, torch.cuda.Stream) else int(s)
        return int(_lib.sta_operator_status(h))


def sta_debug_inject_operator_timeout(mode, limit_ms: int = 50) -> None:
    """Debug: make a device-side wait of the next packed or cache attention calls run out (``mode`` 0 off, 1 on)."""
    _check(_lib.sta_debug_inject_operator_timeout(int(mode), int(limit_ms)), "sta_debug_inject_operator_timeout")
