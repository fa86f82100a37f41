"""What stands between a layer's block-scaled products: norm, rotary positions, gated feed-forward.

Python binding of fp4_rmsnorm, fp4_rope, fp4_gemm_gated and their backward passes of include/fp4.h (formulas,
layouts and limits are stated there). Argument marshalling only; like `fp4`, it raises if the library is missing.

    s = layer.rmsnorm(x, w, residual=r, out_q=params)         # s.sum the residual stream, s.q the product's operand
    q, k = layer.rope((q, k), rotary, batch)                  # positions of a kv.Batch, or int32 [tokens]
    h = layer.gated(s.q, layer.GatedWeights(w_gate, w_up), out_q=params)       # h.q: the down projection's operand

and for training

    y = layer.gated(s.q, weights, keep_gu=True)               # y.gu: what the backward pass reads
    d = layer.gated_backward(dh, y.gu, out_q=params)          # d.dgu, d.q
    dq, dk = layer.rope((dq, dk), rotary, positions, backward=True)
    dx, dw = layer.rmsnorm_backward(dy, s.sum, w, dsum=dr)    # dx: the gradient of x and of r alike
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import fp4, kv
from .fp4 import Fp4Error, Params, QTensor

SILU, GELU, GELU_TANH = 0, 1, 2
HALF, INTERLEAVED = 0, 1

_P, _I64, _I32, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class NormC(ctypes.Structure):
    _fields_ = [("x", _P), ("residual", _P), ("weight", _P), ("sum", _P), ("y", _P), ("rows", _I64), ("cols", _I64),
                ("ldx", _I64), ("ldr", _I64), ("lds", _I64), ("ldy", _I64), ("dtype", _I32), ("w_dtype", _I32), ("eps", _F)]


class NormGradC(ctypes.Structure):
    _fields_ = [("dy", _P), ("s", _P), ("dsum", _P), ("weight", _P), ("dx", _P), ("dweight", _P), ("rows", _I64),
                ("cols", _I64), ("lddy", _I64), ("lds", _I64), ("lddsum", _I64), ("lddx", _I64), ("dtype", _I32),
                ("w_dtype", _I32), ("eps", _F)]


class RopeC(ctypes.Structure):
    # the pairs of the C struct member by member: tuples take longer to convert than the rest of a call
    _fields_ = [("x0", _P), ("x1", _P), ("out0", _P), ("out1", _P), ("ldx0", _I64), ("ldx1", _I64), ("ldx_head0", _I64),
                ("ldx_head1", _I64), ("ldo0", _I64), ("ldo1", _I64), ("ldo_head0", _I64), ("ldo_head1", _I64),
                ("heads0", _I32), ("heads1", _I32), ("tokens", _I64), ("inv_freq", _P), ("positions", _P), ("batch", _P),
                ("scale", _F), ("dtype", _I32), ("head_dim", _I32), ("rotary_dim", _I32), ("layout", _I32), ("backward", _I32)]


class GatedC(ctypes.Structure):
    _fields_ = [("h", _P), ("gu", _P), ("ldh", _I64), ("ldgu", _I64), ("dtype", _I32), ("act", _I32)]


class GatedPlanC(ctypes.Structure):
    _fields_ = [("kernel", _I32), ("quantize_pass", _I32)]


PLAN_ROWS, PLAN_STREAM, PLAN_TILE128, PLAN_TILE128_DEEP, PLAN_TILE128_RAGGED, PLAN_TILE256 = range(1, 7)


class GatedGradC(ctypes.Structure):
    _fields_ = [("dh", _P), ("gu", _P), ("dgu", _P), ("rows", _I64), ("cols", _I64), ("lddh", _I64), ("ldgu", _I64),
                ("lddgu", _I64), ("dtype", _I32), ("act", _I32)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = fp4.lib()
        for name, args, res in (("fp4_rmsnorm", [_P, _P, _P, _P], ctypes.c_int),
                                ("fp4_rmsnorm_backward_workspace_bytes", [_P], _I64),
                                ("fp4_rmsnorm_backward", [_P, _P, _I64, _P], ctypes.c_int),
                                ("fp4_rope", [_P, _P], ctypes.c_int),
                                ("fp4_gemm_gated_workspace_bytes", [_P, _P, _P, _P, _P], _I64),
                                ("fp4_gemm_gated_plan", [_P, _P, _P, _P, _P, _P], ctypes.c_int),
                                ("fp4_gemm_gated", [_P, _P, _P, _P, _P, _P, _P, _I64, _P], ctypes.c_int),
                                ("fp4_gated_backward", [_P, _P, _P, _P], ctypes.c_int)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


_CODES = kv._CODES
_code, _check = kv._code, kv._check


def _stream_of(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


_stream = kv._raw_stream or _stream_of  # the current stream's handle by device index


# Small calls last as long as their host side, so a check first asks, in as few calls as there are, whether all is
# well; _refuse says what is not.

def _matrix(t: torch.Tensor, shape, dtype, index: int, name: str) -> int:
    """Check a row-major CUDA tensor of this shape and dtype on device `index`; returns its pitch."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == index and index >= 0:
        ld, step = t.stride()
        if step == 1 or shape[1] <= 1:
            return ld if shape[0] > 1 else shape[1]
    _refuse(t, shape, dtype, index, name)


def _refuse(t: torch.Tensor, shape, dtype, index: int, name: str):
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on {f'cuda:{index}' if index >= 0 else 'a CUDA device'}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    raise ValueError(f"{name} must be contiguous along its last axis")


def _first(t: torch.Tensor, name: str):
    """Shape, dtype code, device index and pitch of the matrix that the others of a call are held to."""
    code, shape, index = _CODES.get(t.dtype), t.shape, t.get_device()
    if code is not None and len(shape) == 2 and index >= 0:
        ld, step = t.stride()
        if step == 1 or shape[1] <= 1:
            return shape, code, index, ld if shape[0] > 1 else shape[1]
    _code(t.dtype, name)
    if len(shape) != 2:
        raise ValueError(f"{name} must be [rows, cols], not {list(shape)}")
    _refuse(t, shape, t.dtype, index, name)


def _vector(t: torch.Tensor, n: int, index: int, name: str) -> None:
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor, not {list(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")


def _new(rows: int, cols: int, dtype, dev) -> torch.Tensor:
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=dev)


def _params_c(p: Params):
    """The library's form of parameters, which are frozen: made once and kept with them."""
    c = p.__dict__.get("_c")
    if c is None:
        c = p.c()
        object.__setattr__(p, "_c", c)
    return c


# The current device's index; the public call initialises CUDA first if need be, which takes twice as long.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _there(index: int, call, *args, **kw):
    """The call with its tensors' device current: kernels and limits belong to the current device."""
    with torch.cuda.device(index):
        return call(*args, **kw)


def _codes(q: QTensor, rows: int, cols: int, params: Params, index: int, name: str) -> None:
    """Check that q's buffers hold a [rows, cols] tensor with one scale a block (of E8M0, the only ones here)."""
    n = rows * cols
    br, bc = params.block
    _bytes(q.codes, n >> 1 if params.elem == fp4.E2M1 else n, index, name)
    _bytes(q.scales, n // (br * bc), index, name)


def _bytes(t: torch.Tensor, need: int, index: int, name: str) -> None:
    if t.get_device() != index:
        raise ValueError(f"a buffer of {name} is on {t.device}, not on cuda:{index}")
    if t.nbytes < need or not t.is_contiguous():
        raise ValueError(f"a buffer of {name} must be contiguous and hold at least {need} bytes")


def _quant_out(rows: int, cols: int, params: Params, dev, index: int, q_out) -> QTensor:
    if q_out is not None:
        _codes(q_out, rows, cols, params, index, "q_out")
        return q_out
    if rows == 0:
        def none():
            return torch.empty(0, dtype=torch.uint8, device=dev)
        return QTensor(none(), none(), None, 0, cols, params)
    return fp4.empty_qtensor(rows, cols, params, dev)


def _quant_c(q: QTensor):
    """The library fills in the rest, and so does _describe here."""
    return fp4.QTensorC(q.codes.data_ptr(), q.scales.data_ptr())


def _describe(q: QTensor, rows: int, cols: int, params: Params) -> None:
    q.rows, q.cols, q.params, q.tensor_scale = rows, cols, params, None


def _workspace(workspace, need: int, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    fp4._ws_bytes(workspace, need, dev)
    return workspace


class Normed(NamedTuple):
    y: torch.Tensor | None    # the norm's output, None where only its codes are kept
    sum: torch.Tensor | None  # x + residual, what was normed; None without a residual
    q: QTensor | None         # y quantized


def rmsnorm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-5, residual: torch.Tensor | None = None,
            out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None, out_q: Params | None = None,
            q_out: QTensor | None = None, keep_y: bool = True) -> Normed:
    """The root-mean-square norm of the rows of x [rows, cols] (bf16 / fp32, any pitch of whole 16 bytes), or
    of x + residual, which is stored too (to sum_out: x or residual themselves, or a new tensor). weight [cols]
    bf16 / fp32. out_q: quantize the output (groups of 32, E8M0 scales; rotated with out_q.hadamard_n);
    keep_y=False then skips y itself."""
    shape, code, index, ldx = _first(x, "x")
    if index != _device():
        return _there(index, rmsnorm, x, weight, eps, residual, out, sum_out, out_q, q_out, keep_y)
    rows, cols = shape
    dtype, dev = x.dtype, x.device
    w_code = ldr = lds = ldy = 0
    w = r = s = y = None
    if weight is not None:
        _vector(weight, cols, index, "weight")
        w_code, w = _code(weight.dtype, "weight"), weight.data_ptr()
    if residual is not None:
        ldr, r = _matrix(residual, shape, dtype, index, "residual"), residual.data_ptr()
        if sum_out is None:
            sum_out, lds = _new(rows, cols, dtype, dev), cols
        else:
            lds = _matrix(sum_out, shape, dtype, index, "sum_out")
        s = sum_out.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    if out is not None:
        ldy, y = _matrix(out, shape, dtype, index, "out"), out.data_ptr()
    elif keep_y:
        out, ldy = _new(rows, cols, dtype, dev), cols
        y = out.data_ptr()
    elif out_q is None:
        raise ValueError("keep_y=False goes with out_q")
    c = NormC(x.data_ptr(), r, w, s, y, rows, cols, ldx, ldr, lds, ldy, code, w_code, eps)
    qp = qa = None
    if out_q is not None:
        q_out = _quant_out(rows, cols, out_q, dev, index, q_out)
        qp, qc = ctypes.addressof(_params_c(out_q)), _quant_c(q_out)
        qa = ctypes.addressof(qc)
    elif q_out is not None:
        raise ValueError("q_out goes with out_q")
    st = lib().fp4_rmsnorm(ctypes.addressof(c), qp, qa, _stream(index))
    if st:
        _check(st, "fp4_rmsnorm")
    if q_out is not None:
        _describe(q_out, rows, cols, out_q)
    return Normed(out, sum_out, q_out)


def rmsnorm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-5,
                     dsum: torch.Tensor | None = None, out: torch.Tensor | None = None, dweight=True,
                     workspace: torch.Tensor | None = None):
    """(dx, dweight) of y = rmsnorm(s) from dy, all [rows, cols] of one dtype: s is what was normed (Normed.sum,
    or x), dsum the gradient that reaches it from the residual stream. dx is the gradient of x and of the
    residual alike (out: dy or dsum themselves, or a new tensor). dweight: True for a new fp32 [cols], a tensor
    to write to, or False for none (a frozen weight)."""
    shape, code, index, lddy = _first(dy, "dy")
    if index != _device():
        return _there(index, rmsnorm_backward, dy, s, weight, eps, dsum, out, dweight, workspace)
    rows, cols = shape
    dtype, dev = dy.dtype, dy.device
    lds = _matrix(s, shape, dtype, index, "s")
    w_code = lddsum = 0
    w = ds = None
    if weight is not None:
        _vector(weight, cols, index, "weight")
        w_code, w = _code(weight.dtype, "weight"), weight.data_ptr()
    if dsum is not None:
        lddsum, ds = _matrix(dsum, shape, dtype, index, "dsum"), dsum.data_ptr()
    if out is None:
        out, lddx = _new(rows, cols, dtype, dev), cols
    else:
        lddx = _matrix(out, shape, dtype, index, "out")
    if dweight is True:
        dweight = torch.empty_strided((cols,), (1,), dtype=torch.float32, device=dev)
    elif dweight is False:
        dweight = None
    elif dweight is not None:
        _vector(dweight, cols, index, "dweight")
        if dweight.dtype is not torch.float32:
            raise TypeError("dweight must be float32")
    c = NormGradC(dy.data_ptr(), s.data_ptr(), ds, w, out.data_ptr(), None if dweight is None else dweight.data_ptr(), rows, cols,
                  lddy, lds, lddsum, lddx, code, w_code, eps)
    L, pc = lib(), ctypes.addressof(c)
    need, ws = L.fp4_rmsnorm_backward_workspace_bytes(pc), None
    if need > 0:
        workspace = _workspace(workspace, need, dev)
        ws = workspace.data_ptr()
    st = L.fp4_rmsnorm_backward(pc, ws, need, _stream(index))
    if st:
        _check(st, "fp4_rmsnorm_backward")
    return out, dweight


def rmsnorm_backward_workspace_bytes(rows: int, cols: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace rmsnorm_backward() with a dweight needs."""
    c = NormGradC(rows=rows, cols=cols, dtype=_code(dtype, "dy"), dweight=16)
    n = lib().fp4_rmsnorm_backward_workspace_bytes(ctypes.addressof(c))
    if n < 0:
        raise Fp4Error(fp4.ERR_INVALID_ARG, "fp4_rmsnorm_backward_workspace_bytes")
    return n


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_context: int = 0, low: float = 1.0, high: float = 4.0, fast: float = 32.0, slow: float = 1.0,
                       device=None):
    """(inv_freq, scale): the fp64 frequencies of each pair and the factor of the rotated values, for Rotary.
    Pair i of n = rotary_dim turns by f_i = base^(-2 i / n) a position. scaling, for contexts `factor` times
    as long as the model was trained on (`original_context`):
      None       f_i
      "linear"   f_i / factor: positions are squeezed
      "ntk"      base * factor^(n / (n - 2)): the slowest pair is squeezed by factor, the fastest not at all
      "bands"    pairs that turn more than `high` times in the original context keep f_i, less than `low` times take
                 f_i / factor, linear in the number of turns between
      "yarn"     the same with the blend linear in the pair's index between those of `fast` and `slow` turns, and
                 rotated values scaled by 0.1 ln(factor) + 1 (Peng et al., "YaRN: Efficient Context Window
                 Extension of Large Language Models", 2023)"""
    if rotary_dim <= 0 or rotary_dim % 2 or base <= 0 or factor <= 0:
        raise ValueError("rotary_dim must be even and positive, base and factor positive")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        if rotary_dim <= 2:
            raise ValueError("ntk scaling needs a rotary_dim above 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = float(base) ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling in ("bands", "yarn"):
        if original_context <= 0:
            raise ValueError(f"{scaling} scaling needs original_context")
        if scaling == "bands":
            turns = original_context * f / (2.0 * math.pi)
            keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        else:
            def index(turns):  # of the (fractional) pair that turns so often in the original context
                return rotary_dim * math.log(original_context / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
            lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rotary_dim - 1)
            keep = 1.0 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
            scale = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}: None, 'linear', 'ntk', 'bands' or 'yarn'")
    return f.to(device) if device is not None else f, scale


class Rotary:
    """What a model keeps of its positions: inv_freq fp64 [rotary_dim / 2] on the device, the layout of the
    pairs (HALF: channel i with i + rotary_dim / 2; INTERLEAVED: 2 i with 2 i + 1) and the rotated values' scale.
    All three may be assigned: a call takes them as they then are."""

    def __init__(self, inv_freq: torch.Tensor, layout: int = HALF, scale: float = 1.0):
        if layout not in (HALF, INTERLEAVED):
            raise ValueError("layout must be HALF or INTERLEAVED")
        self.inv_freq, self.layout, self.scale = inv_freq, layout, float(scale)

    @property
    def inv_freq(self) -> torch.Tensor:
        return self._inv_freq

    @inv_freq.setter
    def inv_freq(self, f: torch.Tensor) -> None:
        if f.dim() != 1 or f.dtype != torch.float64 or not f.is_cuda or not f.is_contiguous() or f.shape[0] == 0:
            raise ValueError("inv_freq must be a contiguous float64 CUDA vector (rotary_frequencies makes one)")
        self._inv_freq, self._device, self._dim = f, f.device, 2 * f.shape[0]
        self._ptr, self._index = f.data_ptr(), f.get_device()

    @property
    def device(self):
        return self._device

    @property
    def rotary_dim(self) -> int:
        return self._dim


def rope(x, rotary: Rotary, positions, out=None, backward: bool = False):
    """Rotary positions of x [tokens, heads, head_dim], or of a pair of such tensors (queries and keys, of one
    dtype and head_dim) in one launch; strides of whole 16 bytes. positions: int32 [tokens], or the kv.Batch of a cache (a
    sequence's rows are its last ones; rows with no token keep what `out` held). out: a tensor (pair) to write to,
    x itself for in place. backward=True turns the other way: the gradient of x from that of the result."""
    pair = not isinstance(x, torch.Tensor)
    a, b = x if pair else (x, None)
    f = rotary._inv_freq
    if f.data_ptr() != rotary._ptr:  # the tensor has been given other memory
        rotary.inv_freq = f
    index, dev = rotary._index, rotary._device
    if index != _device():
        return _there(index, rope, x, rotary, positions, out, backward)
    dtype = a.dtype
    code = _CODES.get(dtype)
    if code is None:
        _code(dtype, "x")
    tokens, heads, dim = _heads(a, tokens=None, dim=None, dtype=dtype, index=index, name="x")
    heads_b = _heads(b, tokens, dim, dtype, index, "x[1]")[1] if pair else 0
    if out is None:
        o = torch.empty_strided((tokens, heads, dim), (heads * dim, dim, 1), dtype=dtype, device=dev)
        p = torch.empty_strided((tokens, heads_b, dim), (heads_b * dim, dim, 1), dtype=dtype, device=dev) if pair else None
    else:
        o, p = out if pair else (out, None)
        for t, n in ((o, heads), (p, heads_b)):
            if t is not None and _heads(t, tokens, dim, dtype, index, "out")[1] != n:
                raise ValueError("out must have x's shape and dtype")
    pos = batch = None
    if isinstance(positions, kv.Batch):
        if positions.device != dev:
            raise ValueError(f"the batch is on {positions.device}, the rotary table on {dev}")
        held = positions._at(tokens)  # alive until the call has returned
        batch = held[1]
    else:
        _vector(positions, tokens, index, "positions")
        if positions.dtype is not torch.int32:
            raise TypeError("positions must be int32")
        pos = positions.data_ptr()
    x_ld, x_head, _ = a.stride()
    o_ld, o_head, _ = o.stride()
    if pair:
        x1, y1 = b.data_ptr(), p.data_ptr()
        x1_ld, x1_head, _ = b.stride()
        o1_ld, o1_head, _ = p.stride()
    else:
        x1 = y1 = None
        x1_ld = x1_head = o1_ld = o1_head = 0
    c = RopeC(a.data_ptr(), x1, o.data_ptr(), y1, x_ld, x1_ld, x_head, x1_head, o_ld, o1_ld, o_head, o1_head, heads, heads_b, tokens,
              rotary._ptr, pos, batch, rotary.scale, code, dim, rotary._dim, rotary.layout, backward)
    st = lib().fp4_rope(ctypes.addressof(c), _stream(index))
    if st:
        _check(st, "fp4_rope")
    return (o, p) if pair else o


def _heads(t: torch.Tensor, tokens, dim, dtype, index: int, name: str):
    """Check [tokens, heads, dim] rows (None: any) of dtype on device `index`; returns their shape."""
    shape = t.shape
    if len(shape) != 3 or (tokens is not None and shape[0] != tokens) or (dim is not None and shape[2] != dim):
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}, heads, {'head_dim' if dim is None else dim}], "
                         f"not {list(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the rotary table on cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return shape


class GatedWeights:
    """Gate and up projection [F, K], quantized alike (MXFP4 in groups of 32 or 32 x 32 tiles, or MXFP8), with the
    activation between them: checked and described to the library once, and again where one of the tensors has become
    another (quantized anew with out=, or assigned). up=None: gate is [2 F, K], the gate's rows first."""

    def __init__(self, gate: QTensor, up: QTensor | None = None, act: int = SILU):
        if act not in (SILU, GELU, GELU_TANH):
            raise ValueError("act must be SILU, GELU or GELU_TANH")
        self.act = act
        self._whole, self._whole_seen = (gate, None) if up is None else (None, None)
        self.gate, self.up = gate, up
        self._seen = None
        self._now()

    @property
    def device(self):
        return self.gate.codes.device

    @property
    def ff(self) -> int:
        return self.gate.rows

    @property
    def hidden(self) -> int:
        return self.gate.cols

    def _now(self):
        """(addresses of both descriptions, F, K, device index, device, the descriptions) of the tensors as they are."""
        if self._whole is not None and not _is(self._whole, self._whole_seen):
            self.gate, self.up = _halves(self._whole)
            self._whole_seen = _mark(self._whole)
        g, u, seen = self.gate, self.up, self._seen
        if seen is not None and _is(g, seen[0]) and _is(u, seen[1]):
            return seen[2]
        if (g.rows, g.cols) != (u.rows, u.cols):
            raise ValueError(f"gate is {(g.rows, g.cols)}, up {(u.rows, u.cols)}")
        dev = g.codes.device
        for q, name in ((g, "gate"), (u, "up")):
            fp4._check_q(q, q.rows, q.cols, q.params, dev, name)
        c = g.c(), u.c()
        p = ctypes.addressof(c[0]), ctypes.addressof(c[1])
        now = p, g.rows, g.cols, g.codes.get_device(), dev, c
        self._seen = _mark(g), _mark(u), now
        return now


def _mark(q: QTensor):
    return q, q.codes, q.scales, q.params, q.rows, q.cols, q.codes.data_ptr(), q.scales.data_ptr()


def _is(q: QTensor, mark) -> bool:
    """Whether q is what it was when it was marked, whatever its buffers hold."""
    if mark is None:
        return False
    was, codes, scales, params, rows, cols, codes_at, scales_at = mark
    return q is was and q.codes is codes and q.scales is scales and q.params is params and q.rows == rows and q.cols == cols \
        and codes.data_ptr() == codes_at and scales.data_ptr() == scales_at


def _halves(q: QTensor):
    """The upper and the lower half of a quantized tensor's rows (views)."""
    if q.rows % 2 or q.rows % (2 * q.params.block[0]):
        raise ValueError(f"a tensor of {q.rows} rows does not split into a gate and an up projection")
    fp4._check_q(q, q.rows, q.cols, q.params, q.codes.device, "gate")
    cb, sb, _ = fp4.buffer_sizes(q.rows // 2, q.cols, q.params)
    codes, scales = q.codes.view(-1).view(torch.uint8), q.scales.view(-1).view(torch.uint8)
    return tuple(QTensor(codes[i * cb:(i + 1) * cb], scales[i * sb:(i + 1) * sb], q.tensor_scale, q.rows // 2, q.cols, q.params)
                 for i in (0, 1))


class Gated(NamedTuple):
    h: torch.Tensor | None   # act(a gate^T) * (a up^T)
    q: QTensor | None        # h quantized
    gu: torch.Tensor | None  # the two products side by side [rows, 2 F], for gated_backward


def gated(a: QTensor, weights: GatedWeights, out_dtype=torch.bfloat16, out: torch.Tensor | None = None, keep_h: bool = True,
          keep_gu=False, out_q: Params | None = None, q_out: QTensor | None = None,
          workspace: torch.Tensor | None = None) -> Gated:
    """act(a gate^T) * (a up^T) of a [rows, K] in one pass (fp32 accumulation). keep_h=False skips h itself where
    out_q asks for its codes; keep_gu: True for a new [rows, 2 F] tensor of out_dtype with both products, or one to
    write to."""
    (pg, pu), ff, hidden, index, dev, _held = weights._now()  # alive until the call has returned
    rows, cols = a.rows, a.cols
    if index != _device():
        return _there(index, gated, a, weights, out_dtype, out, keep_h, keep_gu, out_q, q_out, workspace)
    if cols != hidden:
        raise ValueError(f"a has {cols} columns, the weights {hidden}")
    _codes(a, rows, cols, a.params, index, "a")
    dtype = out_dtype if out is None else out.dtype
    code = _CODES.get(dtype)
    if code is None:
        _code(dtype, "out")
    h = p = None
    ldh = ldgu = 0
    if out is not None:
        ldh, h = _matrix(out, (rows, ff), dtype, index, "out"), out.data_ptr()
    elif keep_h:
        out, ldh = _new(rows, ff, dtype, dev), ff
        h = out.data_ptr()
    gu = None
    if keep_gu is True:
        gu, ldgu = _new(rows, 2 * ff, dtype, dev), 2 * ff
        p = gu.data_ptr()
    elif keep_gu is not False and keep_gu is not None:
        gu = keep_gu
        ldgu, p = _matrix(gu, (rows, 2 * ff), dtype, index, "keep_gu"), gu.data_ptr()
    c = GatedC(h, p, ldh, ldgu, code, weights.act)
    ac = fp4.QTensorC(a.codes.data_ptr(), a.scales.data_ptr(), None, rows, cols, _params_c(a.params))
    L, pa, po = lib(), ctypes.addressof(ac), ctypes.addressof(c)
    qp = qa = ws = None
    need = 0
    if out_q is not None:
        q_out = _quant_out(rows, ff, out_q, dev, index, q_out)
        qp, qc = ctypes.addressof(_params_c(out_q)), _quant_c(q_out)
        qa = ctypes.addressof(qc)
        need = L.fp4_gemm_gated_workspace_bytes(pa, pg, pu, po, qp)  # there is none without out_q
        if need > 0:
            workspace = _workspace(workspace, need, dev)
            ws = workspace.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out goes with out_q")
    st = L.fp4_gemm_gated(pa, pg, pu, po, qp, qa, ws, need, _stream(index))
    if st:
        _check(st, "fp4_gemm_gated")
    if q_out is not None:
        _describe(q_out, rows, ff, out_q)
    return Gated(out, q_out, gu)


def gated_plan(rows: int, weights: GatedWeights, dtype=torch.bfloat16, out_q: Params | None = None) -> GatedPlanC:
    """How gated() of a [rows, K] would be carried out: kernel (PLAN_...), quantize_pass."""
    (pg, pu), _, hidden, _, _, _held = weights._now()
    p = weights.gate.params
    ac = fp4.QTensorC(None, None, None, rows, hidden, Params(elem=p.elem, hadamard_n=p.hadamard_n).c())
    c, plan = GatedC(dtype=_code(dtype, "out"), act=weights.act), GatedPlanC()
    _check(lib().fp4_gemm_gated_plan(ctypes.addressof(ac), pg, pu, ctypes.addressof(c),
                                     None if out_q is None else ctypes.addressof(_params_c(out_q)), ctypes.addressof(plan)),
           "fp4_gemm_gated_plan")
    return plan


def gated_workspace_bytes(rows: int, weights: GatedWeights, out_q: Params) -> int:
    """Bytes of workspace gated() of a [rows, K] with out_q needs."""
    return 4 * rows * weights.ff if gated_plan(rows, weights, out_q=out_q).quantize_pass else 0


class GatedGrad(NamedTuple):
    dgu: torch.Tensor | None  # gradients of both products side by side [rows, 2 F]
    q: QTensor | None         # dgu quantized along its rows


def gated_backward(dh: torch.Tensor, gu: torch.Tensor, act: int = SILU, out: torch.Tensor | None = None, keep: bool = True,
                   out_q: Params | None = None, q_out: QTensor | None = None) -> GatedGrad:
    """Gradients of gated()'s two products from dh [rows, F] and the gu [rows, 2 F] it kept (out: gu itself, or a
    new tensor). keep=False skips dgu itself where out_q asks for its codes."""
    shape, code, index, lddh = _first(dh, "dh")
    if index != _device():
        return _there(index, gated_backward, dh, gu, act, out, keep, out_q, q_out)
    rows, ff = shape
    dtype, dev, wide = dh.dtype, dh.device, (rows, 2 * ff)
    ldgu = _matrix(gu, wide, dtype, index, "gu")
    lddgu, p = 0, None
    if out is not None:
        lddgu, p = _matrix(out, wide, dtype, index, "out"), out.data_ptr()
    elif keep:
        out, lddgu = _new(rows, 2 * ff, dtype, dev), 2 * ff
        p = out.data_ptr()
    elif out_q is None:
        raise ValueError("keep=False goes with out_q")
    c = GatedGradC(dh.data_ptr(), gu.data_ptr(), p, rows, ff, lddh, ldgu, lddgu, code, act)
    qp = qa = None
    if out_q is not None:
        q_out = _quant_out(rows, 2 * ff, out_q, dev, index, q_out)
        qp, qc = ctypes.addressof(_params_c(out_q)), _quant_c(q_out)
        qa = ctypes.addressof(qc)
    elif q_out is not None:
        raise ValueError("q_out goes with out_q")
    st = lib().fp4_gated_backward(ctypes.addressof(c), qp, qa, _stream(index))
    if st:
        _check(st, "fp4_gated_backward")
    if q_out is not None:
        _describe(q_out, rows, 2 * ff, out_q)
    return GatedGrad(out, q_out)


__all__ = ["SILU", "GELU", "GELU_TANH", "HALF", "INTERLEAVED", "Normed", "Gated", "GatedGrad", "GatedWeights", "Rotary",
           "rmsnorm", "rmsnorm_backward", "rmsnorm_backward_workspace_bytes", "rotary_frequencies", "rope", "gated",
           "gated_plan", "gated_workspace_bytes", "gated_backward"]
