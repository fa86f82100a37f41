"""The key / value cache in 8 bits: quantized as it is written, read back, and attended over.

Python binding of the fp4_kv_* calls of include/fp4.h (layouts, formulas and what the kernels check are
stated there). Argument marshalling only; like `fp4`, it raises if the library is missing.

    cache = kv.empty_cache(pages, kv_heads, page_tokens, head_dim, "cuda")
    batch = kv.Batch(cu_tokens, context, table)        # the step's rows and where they live
    kv.append(cache, k, v, batch)                      # [tokens, kv_heads, head_dim] -> E4M3 + E8M0
    o = kv.attention(q, cache, batch)                  # [tokens, q_heads, head_dim]
    k, v = kv.read(cache, batch, tokens)               # the same tokens back

A cache and a batch are checked once, when they are made, and describe their tensors to the library
from then on: a serving program keeps the cache for its life and one batch for the layers of a step
(whose tensors it may refill in place). K and queries may be rotated with fp4.hadamard before they get
here (a rotation of both leaves q.k as it is), which spreads outlier channels over the head.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import fp4
from .fp4 import DT_BF16, DT_F32, SCALE_E8M0_CEIL, SCALE_E8M0_FLOOR, Fp4Error, status_string

# The current stream's handle by device index; the public way to it makes a Stream object first, which
# takes a third of a small call's time on the host.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_NO_WINDOW = 2 ** 31 - 1  # no position is as far back: the same as any larger window
_CODES = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}


class CacheC(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class BatchC(ctypes.Structure):
    _fields_ = [("cu_tokens", ctypes.c_void_p), ("context", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("tokens", ctypes.c_int64), ("table_ld", ctypes.c_int64), ("seqs", ctypes.c_int32),
                ("table_pages", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("max_context", ctypes.c_int32)]


class AttnC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("ldq", ctypes.c_int64), ("ldq_head", ctypes.c_int64), ("ldo", ctypes.c_int64),
                ("ldo_head", ctypes.c_int64), ("dtype", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float)]


class PlanC(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("tile_rows", ctypes.c_int32), ("waves", ctypes.c_int32),
                ("workgroups", ctypes.c_int64)]


PLAN_ROWS, PLAN_ROWS_SPLIT, PLAN_ROWS_NEAR, PLAN_TILES = 1, 2, 3, 4

_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = fp4.lib()
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.fp4_kv_append.argtypes = [P, P, P, I64, I64, P, I64, I64, I32, I32, P]
        L.fp4_kv_append.restype = ctypes.c_int
        L.fp4_kv_read.argtypes = [P, P, P, I64, I64, P, I64, I64, I32, P]
        L.fp4_kv_read.restype = ctypes.c_int
        L.fp4_kv_attention_workspace_bytes.argtypes = [P, P, P]
        L.fp4_kv_attention_workspace_bytes.restype = I64
        L.fp4_kv_attention_plan.argtypes = [P, P, P, P]
        L.fp4_kv_attention_plan.restype = ctypes.c_int
        L.fp4_kv_attention.argtypes = [P, P, P, P, I64, P]
        L.fp4_kv_attention.restype = ctypes.c_int
        _lib = L
    return _lib


def _device_tensor(t, dtype, shape, name, contiguous=True) -> None:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class KVCache:
    """K and V of `pages` pages: k_codes uint8 [pages, kv_heads, page_tokens, head_dim], v_codes uint8
    [pages, kv_heads, head_dim, page_tokens], k_scales and v_scales uint8 [pages, kv_heads]."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, kv_heads, page_tokens, head_dim]")
        pages, heads, page, dim = k_codes.shape
        _device_tensor(k_codes, torch.uint8, (pages, heads, page, dim), "k_codes")
        _device_tensor(v_codes, torch.uint8, (pages, heads, dim, page), "v_codes")
        _device_tensor(k_scales, torch.uint8, (pages, heads), "k_scales")
        _device_tensor(v_scales, torch.uint8, (pages, heads), "v_scales")
        self.device = k_codes.device
        fp4._on(self.device, v_codes, k_scales, v_scales)
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = pages, heads, page, dim
        self._c = CacheC(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), pages,
                         heads, page, dim)
        self._p = ctypes.addressof(self._c)


def empty_cache(pages: int, kv_heads: int, page_tokens: int, head_dim: int, device) -> KVCache:
    """An empty cache: zero codes and scales (of no token: contexts say what a page holds)."""
    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.uint8, device=device)
    return KVCache(zeros(pages, kv_heads, page_tokens, head_dim), zeros(pages, kv_heads, head_dim, page_tokens),
                   zeros(pages, kv_heads), zeros(pages, kv_heads))


class Batch:
    """The rows of one step: cu_tokens int32 [seqs + 1], context int32 [seqs] (the new tokens included),
    table int32 [seqs, width] (rows may be strided). max_tokens / max_context: the largest number of
    rows and the largest context of any sequence where the program knows them (they only choose how
    work is split; without them a row count and the table's width are assumed)."""

    def __init__(self, cu_tokens: torch.Tensor, context: torch.Tensor, table: torch.Tensor,
                 max_tokens: int | None = None, max_context: int | None = None):
        if table.dim() != 2:
            raise ValueError("table must be [seqs, width]")
        seqs, width = table.shape
        _device_tensor(cu_tokens, torch.int32, (seqs + 1,), "cu_tokens")
        _device_tensor(context, torch.int32, (seqs,), "context")
        _device_tensor(table, torch.int32, (seqs, width), "table", contiguous=False)
        if width > 1 and table.stride(1) != 1:
            raise ValueError("table must be contiguous along its last axis")
        self.device = table.device
        fp4._on(self.device, cu_tokens, context)
        self.cu_tokens, self.context, self.table, self.seqs = cu_tokens, context, table, seqs
        self._last = self._make(0, cu_tokens.data_ptr(), context.data_ptr(), table.data_ptr(),
                                table.stride(0) if seqs > 1 else width, max_tokens or 0, max_context or 0)

    def _make(self, tokens, cu_tokens, context, table, table_ld, max_tokens, max_context):
        c = BatchC(cu_tokens, context, table, tokens, table_ld, self.seqs, self.table.shape[1], max_tokens, max_context)
        return tokens, ctypes.addressof(c), c

    def _at(self, tokens: int):
        """(tokens, address, struct) for calls of so many rows, never changed once made: threads may use
        one batch with different row counts. The last one is kept."""
        last = self._last
        if last[0] != tokens:
            c = last[2]
            last = self._last = self._make(tokens, c.cu_tokens, c.context, c.table, c.table_ld, c.max_tokens,
                                           c.max_context)
        return last


def _code(dtype, name: str) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {dtype}: float32 or bfloat16")
    return code


def _rows(t: torch.Tensor, heads, dim: int, dev, name: str) -> int:
    """Check [tokens, heads, dim] rows of bf16 / fp32 on dev; returns the dtype code."""
    code = _code(t.dtype, name)
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the cache on {dev}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {heads if heads is not None else 'heads'}, {dim}], not {tuple(shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return code


def _use(cache: KVCache, batch: Batch, tokens: int):
    if batch.device != cache.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    return batch._at(tokens)


def _stream(dev: torch.device) -> int:
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _check(status: int, what: str) -> None:
    if status != fp4.OK:
        raise Fp4Error(status, what)


def append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, batch: Batch, scale_mode: int = SCALE_E8M0_CEIL) -> None:
    """Quantize k and v [tokens, kv_heads, head_dim] (any token and head strides that are multiples of
    16 bytes) into the batch's pages. scale_mode: SCALE_E8M0_CEIL (nothing saturates) or _FLOOR."""
    dev = cache.device
    code = _rows(k, cache.kv_heads, cache.head_dim, dev, "k")
    if _rows(v, cache.kv_heads, cache.head_dim, dev, "v") != code or v.shape[0] != k.shape[0]:
        raise ValueError("k and v must have one dtype and one number of tokens")
    b = _use(cache, batch, k.shape[0])
    st = lib().fp4_kv_append(cache._p, b[1], k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                             v.stride(1), code, scale_mode, _stream(dev))
    _check(st, "fp4_kv_append")


def read(cache: KVCache, batch: Batch, tokens: int, dtype=torch.bfloat16, out=None):
    """(k, v), each [tokens, kv_heads, head_dim]: the last rows of each sequence as the cache holds them
    (rows of the batch that have no token keep what `out` held). out: a pair of tensors to write to."""
    dev = cache.device
    shape = (tokens, cache.kv_heads, cache.head_dim)
    if out is None:
        k, v = torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev)
    else:
        k, v = out
    code = _rows(k, cache.kv_heads, cache.head_dim, dev, "k")
    if _rows(v, cache.kv_heads, cache.head_dim, dev, "v") != code or k.shape[0] != tokens or v.shape[0] != tokens:
        raise ValueError(f"out must be two tensors of one dtype with {tokens} tokens")
    b = _use(cache, batch, tokens)
    st = lib().fp4_kv_read(cache._p, b[1], k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                           v.stride(1), code, _stream(dev))
    _check(st, "fp4_kv_read")
    return k, v


def attention_workspace_bytes(cache: KVCache, batch: Batch, tokens: int, q_heads: int, dtype=torch.bfloat16,
                              window: int = 0) -> int:
    """Bytes of workspace attention() needs for q [tokens, q_heads, head_dim]."""
    b = _use(cache, batch, tokens)
    a = AttnC(None, None, None, 0, 0, 0, 0, _code(dtype, "q"), q_heads, 1, min(window, _NO_WINDOW), 1.0)
    n = lib().fp4_kv_attention_workspace_bytes(cache._p, b[1], ctypes.addressof(a))
    if n < 0:
        raise Fp4Error(fp4.ERR_INVALID_ARG, "fp4_kv_attention_workspace_bytes")
    return n


def attention_plan(cache: KVCache, batch: Batch, tokens: int, q_heads: int, dtype=torch.bfloat16,
                   window: int = 0) -> PlanC:
    """How attention() of q [tokens, q_heads, head_dim] would be carried out: kernel (PLAN_...), tile_rows,
    waves, workgroups."""
    b = _use(cache, batch, tokens)
    a = AttnC(None, None, None, 0, 0, 0, 0, _code(dtype, "q"), q_heads, 1, min(window, _NO_WINDOW), 1.0)
    p = PlanC()
    _check(lib().fp4_kv_attention_plan(cache._p, b[1], ctypes.addressof(a), ctypes.addressof(p)),
           "fp4_kv_attention_plan")
    return p


def attention(q: torch.Tensor, cache: KVCache, batch: Batch, scale: float | None = None, causal: bool = True,
              window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """softmax(scale q K^T + mask) V of q [tokens, q_heads, head_dim] over each row's sequence in the
    cache; q_heads a multiple of kv_heads. scale: 1 / sqrt(head_dim) unless given. window: keys more
    than window - 1 tokens back are masked (0: none). lse: fp32 [tokens, q_heads], receives the log of
    each row's sum of exponentials. A row with no key gives zeros (lse -inf)."""
    dev = cache.device
    dim = cache.head_dim
    code = _rows(q, None, dim, dev, "q")
    tokens, heads = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif _rows(out, heads, dim, dev, "out") != code or out.shape[0] != tokens:
        raise ValueError("out must have q's shape and dtype")
    if lse is not None:
        _device_tensor(lse, torch.float32, (tokens, heads), "lse")
        fp4._on(dev, lse)
    b = _use(cache, batch, tokens)
    a = AttnC(q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None, q.stride(0), q.stride(1),
              out.stride(0), out.stride(1), code, heads, causal, min(window, _NO_WINDOW),
              scale if scale is not None else 1.0 / math.sqrt(dim))
    pa = ctypes.addressof(a)
    L = lib()
    need = L.fp4_kv_attention_workspace_bytes(cache._p, b[1], pa)
    ws = None
    if need > 0:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            fp4._ws_bytes(workspace, need, dev)
        ws = workspace.data_ptr()
    st = L.fp4_kv_attention(cache._p, b[1], pa, ws, need, _stream(dev))
    _check(st, "fp4_kv_attention")
    return out


__all__ = ["KVCache", "Batch", "empty_cache", "append", "read", "attention", "attention_plan", "attention_workspace_bytes",
           "SCALE_E8M0_CEIL", "SCALE_E8M0_FLOOR", "Fp4Error", "status_string"]
