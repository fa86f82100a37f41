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
import functools
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
    _fields_ = [("x", _P * 2), ("out", _P * 2), ("ldx", _I64 * 2), ("ldx_head", _I64 * 2), ("ldo", _I64 * 2),
                ("ldo_head", _I64 * 2), ("heads", _I32 * 2), ("tokens", _I64), ("inv_freq", _P), ("positions", _P),
                ("batch", _P), ("scale", _F), ("dtype", _I32), ("head_dim", _I32), ("rotary_dim", _I32), ("layout", _I32),
                ("backward", _I32)]


class GatedC(ctypes.Structure):
    _fields_ = [("h", _P), ("gu", _P), ("ldh", _I64), ("ldgu", _I64), ("dtype", _I32), ("act", _I32)]


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
                                ("fp4_gemm_gated", [_P, _P, _P, _P, _P, _P, _P, _I64, _P], ctypes.c_int),
                                ("fp4_gated_backward", [_P, _P, _P, _P], ctypes.c_int)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


_code, _stream, _check = kv._code, kv._stream, kv._check


def _matrix(t: torch.Tensor, rows, cols, dtype, dev, name: str) -> None:
    """Check a row-major [rows, cols] CUDA tensor (None: any) of dtype on dev."""
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {'cols' if cols is None else cols}], not {tuple(shape)}")
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not on {dev if dev.type == 'cuda' else 'a CUDA device'}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")


def _pitch(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(t: torch.Tensor, n: int, dev, name: str) -> None:
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor, not {tuple(t.shape)}")
    fp4._on(dev, t)


@functools.lru_cache(maxsize=256)
def _params_c(p: Params):
    """The library's form of frozen parameters (read by it, never written) and its address; a call holds the pair."""
    c = p.c()
    return c, ctypes.addressof(c)


def _rows(t: torch.Tensor, heads, dim: int, dev, name: str) -> int:
    """Check [tokens, heads, dim] rows of bf16 / fp32 on dev; returns the dtype code."""
    code = _code(t.dtype, name)
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the rotary table on {dev}")
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {heads if heads is not None else 'heads'}, {dim}], not {tuple(t.shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return code


def _quant_out(rows: int, cols: int, params: Params, dev, q_out, name: str = "q_out") -> QTensor:
    if rows == 0:
        def none():
            return torch.empty(0, dtype=torch.uint8, device=dev)
        return q_out if q_out is not None else QTensor(none(), none(), None, 0, cols, params)
    if q_out is None:
        return fp4.empty_qtensor(rows, cols, params, dev)
    fp4._check_q(q_out, rows, cols, params, dev, name)
    return q_out


def _quant_c(q: QTensor):
    """The library fills in the rest, and so does _describe here."""
    return fp4.QTensorC(q.codes.data_ptr(), q.scales.data_ptr())


def _describe(q: QTensor, rows: int, cols: int, params: Params) -> None:
    q.rows, q.cols, q.params, q.tensor_scale = rows, cols, params, None


def _workspace(workspace, need: int, dev):
    if need <= 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        fp4._ws_bytes(workspace, need, dev)
    return workspace, need


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
    dev = x.device
    code = _code(x.dtype, "x")
    _matrix(x, None, None, x.dtype, dev, "x")
    rows, cols = x.shape
    w_code = 0
    if weight is not None:
        _vector(weight, cols, dev, "weight")
        w_code = _code(weight.dtype, "weight")
    if residual is not None:
        _matrix(residual, rows, cols, x.dtype, dev, "residual")
        if sum_out is None:
            sum_out = torch.empty((rows, cols), dtype=x.dtype, device=dev)
        else:
            _matrix(sum_out, rows, cols, x.dtype, dev, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    if out_q is None and not keep_y:
        raise ValueError("keep_y=False goes with out_q")
    if out is not None:
        _matrix(out, rows, cols, x.dtype, dev, "out")
    elif keep_y:
        out = torch.empty((rows, cols), dtype=x.dtype, device=dev)
    c = NormC(x.data_ptr(), None if residual is None else residual.data_ptr(), None if weight is None else weight.data_ptr(),
              None if sum_out is None else sum_out.data_ptr(), None if out is None else out.data_ptr(), rows, cols, _pitch(x),
              0 if residual is None else _pitch(residual), 0 if sum_out is None else _pitch(sum_out),
              0 if out is None else _pitch(out), code, w_code, eps)
    qp = qa = qc = None
    if out_q is not None:
        q_out = _quant_out(rows, cols, out_q, dev, q_out)
        held = _params_c(out_q)
        qp = held[1]
        qc = _quant_c(q_out)
        qa = ctypes.addressof(qc)
    elif q_out is not None:
        raise ValueError("q_out goes with out_q")
    _check(lib().fp4_rmsnorm(ctypes.addressof(c), qp, qa, _stream(dev)), "fp4_rmsnorm")
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
    dev = dy.device
    code = _code(dy.dtype, "dy")
    _matrix(dy, None, None, dy.dtype, dev, "dy")
    rows, cols = dy.shape
    _matrix(s, rows, cols, dy.dtype, dev, "s")
    w_code = 0
    if weight is not None:
        _vector(weight, cols, dev, "weight")
        w_code = _code(weight.dtype, "weight")
    if dsum is not None:
        _matrix(dsum, rows, cols, dy.dtype, dev, "dsum")
    if out is None:
        out = torch.empty((rows, cols), dtype=dy.dtype, device=dev)
    else:
        _matrix(out, rows, cols, dy.dtype, dev, "out")
    if dweight is True:
        dweight = torch.empty(cols, dtype=torch.float32, device=dev)
    elif dweight is False:
        dweight = None
    if dweight is not None:
        _vector(dweight, cols, dev, "dweight")
        if dweight.dtype != torch.float32:
            raise TypeError("dweight must be float32")
    c = NormGradC(dy.data_ptr(), s.data_ptr(), None if dsum is None else dsum.data_ptr(),
                  None if weight is None else weight.data_ptr(), out.data_ptr(), None if dweight is None else dweight.data_ptr(),
                  rows, cols, _pitch(dy), _pitch(s), 0 if dsum is None else _pitch(dsum), _pitch(out), code, w_code, eps)
    L, pc = lib(), ctypes.addressof(c)
    ws, need = _workspace(workspace, L.fp4_rmsnorm_backward_workspace_bytes(pc), dev)
    _check(L.fp4_rmsnorm_backward(pc, None if ws is None else ws.data_ptr(), need, _stream(dev)), "fp4_rmsnorm_backward")
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
    pairs (HALF: channel i with i + rotary_dim / 2; INTERLEAVED: 2 i with 2 i + 1) and the rotated values' scale."""

    def __init__(self, inv_freq: torch.Tensor, layout: int = HALF, scale: float = 1.0):
        if inv_freq.dim() != 1 or inv_freq.dtype != torch.float64 or not inv_freq.is_cuda or not inv_freq.is_contiguous() \
                or inv_freq.shape[0] == 0:
            raise ValueError("inv_freq must be a contiguous float64 CUDA vector (rotary_frequencies makes one)")
        if layout not in (HALF, INTERLEAVED):
            raise ValueError("layout must be HALF or INTERLEAVED")
        self.inv_freq, self.layout, self.scale, self.device = inv_freq, layout, float(scale), inv_freq.device
        self.rotary_dim = 2 * inv_freq.shape[0]
        self._ptr = inv_freq.data_ptr()


def rope(x, rotary: Rotary, positions, out=None, backward: bool = False):
    """Rotary positions of x [tokens, heads, head_dim], or of a pair of such tensors (queries and keys, of one
    dtype and head_dim) in one launch; strides of whole 16 bytes. positions: int32 [tokens], or the kv.Batch of a cache (a
    sequence's rows are its last ones; rows with no token keep what `out` held). out: a tensor (pair) to write to,
    x itself for in place. backward=True turns the other way: the gradient of x from that of the result."""
    pair = isinstance(x, (tuple, list))
    xs = x if pair else (x,)
    if pair and len(xs) != 2:
        raise ValueError("x must be a tensor or a pair of tensors")
    first, dev = xs[0], rotary.device
    tokens, dim = first.shape[0], first.shape[-1]
    code = _rows(first, None, dim, dev, "x")
    if pair and (_rows(xs[1], None, dim, dev, "x[1]") != code or xs[1].shape[0] != tokens):
        raise ValueError("both tensors must have one dtype and one number of tokens")
    if out is None:
        outs = tuple(torch.empty(t.shape, dtype=t.dtype, device=dev) for t in xs)
    else:
        outs = tuple(out) if pair else (out,)
        if len(outs) != len(xs):
            raise ValueError("out must be given like x")
        for t, o in zip(xs, outs):
            if _rows(o, t.shape[1], dim, dev, "out") != code or o.shape[0] != tokens:
                raise ValueError("out must have x's shape and dtype")
    pos = batch = None
    if isinstance(positions, kv.Batch):
        if positions.device != dev:
            raise ValueError(f"the batch is on {positions.device}, x on {dev}")
        held = positions._at(tokens)  # alive until the call has returned
        batch = held[1]
    else:
        if positions.dtype != torch.int32:
            raise TypeError("positions must be int32")
        _vector(positions, tokens, dev, "positions")
        pos = positions.data_ptr()
    a, o = xs[0], outs[0]
    if pair:
        b, p = xs[1], outs[1]
        c = RopeC((a.data_ptr(), b.data_ptr()), (o.data_ptr(), p.data_ptr()), (a.stride(0), b.stride(0)), (a.stride(1), b.stride(1)),
                  (o.stride(0), p.stride(0)), (o.stride(1), p.stride(1)), (a.shape[1], b.shape[1]), tokens, rotary._ptr, pos, batch,
                  rotary.scale, code, dim, rotary.rotary_dim, rotary.layout, backward)
    else:
        c = RopeC((a.data_ptr(),), (o.data_ptr(),), (a.stride(0),), (a.stride(1),), (o.stride(0),), (o.stride(1),), (a.shape[1],),
                  tokens, rotary._ptr, pos, batch, rotary.scale, code, dim, rotary.rotary_dim, rotary.layout, backward)
    _check(lib().fp4_rope(ctypes.addressof(c), _stream(dev)), "fp4_rope")
    return outs if pair else outs[0]


class GatedWeights:
    """Gate and up projection [F, K], quantized alike (MXFP4 in groups of 32 or 32 x 32 tiles, or MXFP8), with the
    activation between them: checked once, described to the library from then on. up=None: gate is [2 F, K],
    the gate's rows first."""

    def __init__(self, gate: QTensor, up: QTensor | None = None, act: int = SILU):
        if act not in (SILU, GELU, GELU_TANH):
            raise ValueError("act must be SILU, GELU or GELU_TANH")
        if up is None:
            gate, up = _halves(gate)
        if (gate.rows, gate.cols) != (up.rows, up.cols):
            raise ValueError(f"gate is {(gate.rows, gate.cols)}, up {(up.rows, up.cols)}")
        self.device = gate.codes.device
        for q, name in ((gate, "gate"), (up, "up")):
            fp4._check_q(q, q.rows, q.cols, q.params, self.device, name)
        self.gate, self.up, self.act, self.ff, self.hidden = gate, up, act, gate.rows, gate.cols
        self._c = gate.c(), up.c()
        self._p = tuple(ctypes.addressof(c) for c in self._c)


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
    dev, rows, ff = weights.device, a.rows, weights.ff
    if a.cols != weights.hidden:
        raise ValueError(f"a has {a.cols} columns, the weights {weights.hidden}")
    if rows > 0:
        fp4._check_q(a, rows, a.cols, a.params, dev, "a")
    code = _code(out_dtype if out is None else out.dtype, "out")
    dtype = out_dtype if out is None else out.dtype
    if out is not None:
        _matrix(out, rows, ff, dtype, dev, "out")
    elif keep_h:
        out = torch.empty((rows, ff), dtype=dtype, device=dev)
    gu = None
    if keep_gu is True:
        gu = torch.empty((rows, 2 * ff), dtype=dtype, device=dev)
    elif keep_gu is not False and keep_gu is not None:
        gu = keep_gu
        _matrix(gu, rows, 2 * ff, dtype, dev, "keep_gu")
    c = GatedC(None if out is None else out.data_ptr(), None if gu is None else gu.data_ptr(), 0 if out is None else _pitch(out),
               0 if gu is None else _pitch(gu), code, weights.act)
    qp = qa = qc = None
    if out_q is not None:
        q_out = _quant_out(rows, ff, out_q, dev, q_out)
        held = _params_c(out_q)
        qp = held[1]
        qc = _quant_c(q_out)
        qa = ctypes.addressof(qc)
    elif q_out is not None:
        raise ValueError("q_out goes with out_q")
    ac = fp4.QTensorC(a.codes.data_ptr(), a.scales.data_ptr(), None, rows, a.cols, _params_c(a.params)[0])
    L, pa, po, (pg, pu) = lib(), ctypes.addressof(ac), ctypes.addressof(c), weights._p
    ws, need = _workspace(workspace, L.fp4_gemm_gated_workspace_bytes(pa, pg, pu, po, qp), dev)
    _check(L.fp4_gemm_gated(pa, pg, pu, po, qp, qa, None if ws is None else ws.data_ptr(), need, _stream(dev)), "fp4_gemm_gated")
    if q_out is not None:
        _describe(q_out, rows, ff, out_q)
    return Gated(out, q_out, gu)


class GatedGrad(NamedTuple):
    dgu: torch.Tensor | None  # gradients of both products side by side [rows, 2 F]
    q: QTensor | None         # dgu quantized along its rows


def gated_backward(dh: torch.Tensor, gu: torch.Tensor, act: int = SILU, out: torch.Tensor | None = None, keep: bool = True,
                   out_q: Params | None = None, q_out: QTensor | None = None) -> GatedGrad:
    """Gradients of gated()'s two products from dh [rows, F] and the gu [rows, 2 F] it kept (out: gu itself, or a
    new tensor). keep=False skips dgu itself where out_q asks for its codes."""
    dev = dh.device
    code = _code(dh.dtype, "dh")
    _matrix(dh, None, None, dh.dtype, dev, "dh")
    rows, ff = dh.shape
    _matrix(gu, rows, 2 * ff, dh.dtype, dev, "gu")
    if out_q is None and not keep:
        raise ValueError("keep=False goes with out_q")
    if out is not None:
        _matrix(out, rows, 2 * ff, dh.dtype, dev, "out")
    elif keep:
        out = torch.empty((rows, 2 * ff), dtype=dh.dtype, device=dev)
    c = GatedGradC(dh.data_ptr(), gu.data_ptr(), None if out is None else out.data_ptr(), rows, ff, _pitch(dh), _pitch(gu),
                   0 if out is None else _pitch(out), code, act)
    qp = qa = qc = None
    if out_q is not None:
        q_out = _quant_out(rows, 2 * ff, out_q, dev, q_out)
        held = _params_c(out_q)
        qp = held[1]
        qc = _quant_c(q_out)
        qa = ctypes.addressof(qc)
    elif q_out is not None:
        raise ValueError("q_out goes with out_q")
    _check(lib().fp4_gated_backward(ctypes.addressof(c), qp, qa, _stream(dev)), "fp4_gated_backward")
    if q_out is not None:
        _describe(q_out, rows, 2 * ff, out_q)
    return GatedGrad(out, q_out)


__all__ = ["SILU", "GELU", "GELU_TANH", "HALF", "INTERLEAVED", "Normed", "Gated", "GatedGrad", "GatedWeights", "Rotary",
           "rmsnorm", "rmsnorm_backward", "rmsnorm_backward_workspace_bytes", "rotary_frequencies", "rope", "gated",
           "gated_backward"]
