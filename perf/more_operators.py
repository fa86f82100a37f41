"""Cases of the operators that stand between a decoder layer's block-scaled products: the root-mean-square
norm with the residual's addition and a low-bit output, rotary positions, and the gated feed-forward (both
projections, the activation and their product), each with its backward pass.

Low-bit outputs are MX groups of 32 along the rows (E2M1 or E4M3 elements, one power-of-two scale a group),
optionally of the values rotated by blocks of H_n / sqrt(n). They are returned as the elements' values (every
E2M1 value is an E4M3 one) and the scales' values.

`own` chooses between the plain torch form of each operator (elementary operations in 32 bits, angles in 64)
and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one user's single token through a serving layer: residual added, normed, rotated, 8-bit codes: latency
        dict(name="norm_one_token", op="norm", dtype="bf16", rows=1, cols=4096, residual=True, weight="bf16", y=False,
             q="e4m3", hn=128, rule="ceil"),
        # a batch of prompts, Llama-7B-shaped: bound by memory
        dict(name="norm_prompt", op="norm", dtype="bf16", rows=8192, cols=4096, residual=True, weight="bf16", y=False,
             q="e4m3", hn=128, rule="ceil"),
        # a final norm in fp32, an odd number of rows of a width off the powers of two, no low-bit output
        dict(name="norm_final_f32", op="norm", dtype="f32", rows=1003, cols=5120, residual=False, weight="f32", y=True,
             q="", hn=0, rule="ceil"),
        # a training step's backward of that norm: the gradient of the residual stream comes along
        dict(name="norm_backward", op="norm_grad", dtype="bf16", rows=8192, cols=4096, weight="bf16", stream=True),
        # the same in fp32 over a small ragged batch, where the weight's gradient is a larger share
        dict(name="norm_backward_f32", op="norm_grad", dtype="f32", rows=333, cols=1280, weight="f32", stream=False),
        # a decode step of a batch: queries and keys of one token a sequence, far positions, slices of one projection
        dict(name="rope_decode", op="rope", dtype="bf16", seqs=64, tokens=1, context=131072, q_heads=32, kv_heads=8,
             dim=128, rotary=128, layout="half", base=500000.0, stretch=8.0, given=False, backward=False),
        # gradients of prompts' queries and keys: part of each head, interleaved pairs
        dict(name="rope_backward", op="rope", dtype="bf16", seqs=4, tokens=4096, context=4096, q_heads=32, kv_heads=8,
             dim=128, rotary=64, layout="interleaved", base=10000.0, stretch=1.0, given=True, backward=True),
        # one user's single token through a Llama-7B-shaped feed-forward: bound by the weights' bytes
        dict(name="gated_one_token", op="gated", dtype="bf16", elem="e2m1", rows=1, hidden=4096, ff=11008, tile=False,
             act="silu", h=True, gu=False, q="", hn=0, rule="floor"),
        # a decode step of 48 sequences in 8 bits, the output coded and rotated for the down projection
        dict(name="gated_decode", op="gated", dtype="bf16", elem="e4m3", rows=48, hidden=4096, ff=11008, tile=False,
             act="silu", h=False, gu=False, q="e4m3", hn=128, rule="ceil"),
        # a training step's forward: 4096 tokens, the pre-activations kept for the backward pass
        dict(name="gated_train", op="gated", dtype="bf16", elem="e2m1", rows=4096, hidden=4096, ff=11008, tile=False,
             act="silu", h=True, gu=True, q="", hn=0, rule="floor"),
        # a chunk of uneven length: weights in 32 x 32 tiles, the other activation, coded in 4 bits beside the values
        dict(name="gated_chunk", op="gated", dtype="f32", elem="e2m1", rows=777, hidden=2048, ff=5504, tile=True,
             act="gelu_tanh", h=True, gu=False, q="e2m1", hn=64, rule="floor"),
        # its backward pass: gradients of both projections, coded along the rows for the product with the weights
        dict(name="gated_backward", op="gated_grad", dtype="bf16", rows=4096, ff=11008, act="silu", keep=True, q="e4m3",
             hn=128, rule="ceil"),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "rope", "gated", "gated", "gated_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, dtype=dtype)
    if op == "rope":
        dim = rng.choice([64, 80, 96, 112, 128, 192, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        c.update(seqs=spread(rng, 1, 128), tokens=rng.choice([1, spread(rng, 2, 4096)]), context=spread(rng, 4096, 1000000),
                 q_heads=kv_heads * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv_heads, dim=dim,
                 rotary=rng.choice([dim, dim, dim // 2, dim // 4]), layout=rng.choice(["half", "interleaved"]),
                 base=rng.choice([10000.0, 500000.0]), stretch=rng.choice([1.0, 1.0, 4.0, 32.0]), given=rng.random() < 0.5,
                 backward=rng.random() < 0.4)
    elif op == "gated_grad":
        c.update(rows=spread(rng, 1, 4096), ff=32 * spread(rng, 4, 448), act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                 keep=True)
        coding(rng, c, c["ff"])
    elif op == "gated":
        elem = rng.choice(["e2m1", "e2m1", "e4m3"])
        c.update(dtype="bf16" if elem == "e4m3" else dtype, elem=elem, rows=spread(rng, 1, 4096),
                 hidden=rng.choice([32, 128, 256, 256]) * spread(rng, 1, 32), ff=32 * spread(rng, 4, 448),
                 tile=elem == "e2m1" and rng.random() < 0.3, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                 h=True, gu=rng.random() < 0.4)
        coding(rng, c, c["ff"])
    else:
        c.update(rows=spread(rng, 1, 16384), cols=32 * spread(rng, 2, 512), weight=rng.choice(["bf16", "f32"]))
        if op == "norm":
            c.update(residual=rng.random() < 0.6, y=True)
            coding(rng, c, c["cols"])
            c["y"] = not c["q"] or rng.random() < 0.3
        else:
            c["stream"] = rng.random() < 0.5
    while cost(c) > 1:  # smaller until it costs no more than the largest listed cases do
        part = "seqs" if op == "rope" and c["seqs"] > 1 else "tokens" if op == "rope" else "rows"
        c[part] = (c[part] + 1) // 2
    return c


def coding(rng, c, cols):
    c["q"] = rng.choice(["", "e4m3", "e4m3", "e2m1"])
    c["hn"] = rng.choice([n for n in (0, 0, 16, 32, 64, 128) if n == 0 or cols % n == 0]) if c["q"] else 0
    c["rule"] = rng.choice(["ceil", "floor"])


def cost(c):
    """The drawn case's work over the largest listed one's of its operator."""
    largest = {"norm": 2.4e8, "norm_grad": 2.7e8, "rope": 3.4e8, "gated": 7.4e11, "gated_grad": 5.5e8}
    w = work(c)
    return (w["flops"] if c["op"] == "gated" else w["bytes"]) / largest[c["op"]]


def work(case):
    c, op = case, case["op"]
    esz = 2 if c["dtype"] == "bf16" else 4
    bits = {"": 0.0, "e2m1": 4.25, "e4m3": 8.25}
    if op == "norm":
        n = c["rows"] * c["cols"]
        return {"bytes": n * esz * (1 + 2 * c["residual"] + c["y"]) + n * bits[c["q"]] / 8 + c["cols"] * (2 if c["weight"] == "bf16" else 4),
                "flops": n * (6 + (2 * math.log2(c["hn"]) if c["hn"] else 0))}
    if op == "norm_grad":
        n = c["rows"] * c["cols"]
        return {"bytes": n * esz * (3 + c["stream"]) + c["cols"] * (4 + (2 if c["weight"] == "bf16" else 4)), "flops": 12 * n}
    if op == "rope":
        n = c["seqs"] * c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 2 * n * esz, "flops": 3 * n}
    if op == "gated_grad":
        n = c["rows"] * c["ff"]
        return {"bytes": n * esz * (3 + 2 * c["keep"]) + 2 * n * bits[c["q"]] / 8, "flops": 20 * n}
    m, k, f = c["rows"], c["hidden"], c["ff"]
    weights = 2 * f * k * bits[c["elem"]] / 8 if not c["tile"] else 2 * f * k * (0.5 + 1 / 1024)
    return {"bytes": weights + m * k * bits[c["elem"]] / 8 + m * f * (esz * (c["h"] + 2 * c["gu"]) + bits[c["q"]] / 8),
            "flops": 4 * m * f * k}


# ---- what a program has in hand ----

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c, op, dtype = case, case["op"], DTYPES[case["dtype"]]
    s = dict(case=c)

    def normal(*shape, size=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(size)

    def outliers(x, size):
        """A few channels larger than the others, as hidden states have them."""
        at = torch.randperm(x.shape[-1], generator=g, device=DEV)[: max(1, x.shape[-1] // 200)]
        x[..., at] *= size
        return x

    if c.get("hn"):
        s["hadamard"] = hadamard(c["hn"], torch.float32)
    if op == "norm":
        s["x"] = outliers(normal(c["rows"], c["cols"], size=0.7), 10.0).to(dtype)
        s["r"] = outliers(normal(c["rows"], c["cols"], size=2.0), 20.0).to(dtype) if c["residual"] else None
        s["w"] = (1.0 + normal(c["cols"], size=0.2)).to(DTYPES[c["weight"]])
    elif op == "norm_grad":
        s["s"] = outliers(normal(c["rows"], c["cols"], size=2.0), 20.0).to(dtype)
        s["dy"] = normal(c["rows"], c["cols"], size=1e-3).to(dtype)
        s["dsum"] = normal(c["rows"], c["cols"], size=1e-3).to(dtype) if c["stream"] else None
        s["w"] = (1.0 + normal(c["cols"], size=0.2)).to(DTYPES[c["weight"]])
    elif op == "rope":
        seqs, n, hq, hk, dim = c["seqs"], c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
        rows = seqs * n
        fused = normal(rows, hq + 2 * hk, dim).to(dtype)
        s["q"], s["k"] = fused[:, :hq], fused[:, hq: hq + hk]
        room = max(1, c["context"] - n)
        first = (torch.rand(seqs, generator=g, device=DEV, dtype=torch.float64) * room).long()
        s["positions"] = (first[:, None] + torch.arange(n, device=DEV)).reshape(-1).to(torch.int32)
        s["cu"] = torch.arange(seqs + 1, device=DEV, dtype=torch.int32) * n
        s["context"] = (first + n).to(torch.int32)
        i = torch.arange(c["rotary"] // 2, device=DEV, dtype=torch.float64)
        s["inv_freq"] = c["base"] ** (-2.0 * i / c["rotary"]) / c["stretch"]
        s["scale"] = 1.0 + 0.1 * math.log(c["stretch"])
    elif op == "gated_grad":
        s["dh"] = normal(c["rows"], c["ff"], size=1e-3).to(dtype)
        s["gu"] = normal(c["rows"], 2 * c["ff"], size=1.5).to(dtype)
    else:
        k = c["hidden"]
        s["a"], s["a_scales"] = coded(outliers(normal(c["rows"], k), 4.0), c["elem"], False)
        for name in ("gate", "up"):
            w = normal(c["ff"], k, size=1.5 / math.sqrt(k))
            w *= torch.exp(0.3 * torch.randn(c["ff"], 1, generator=g, device=DEV))
            s[name], s[name + "_scales"] = coded(w, c["elem"], c["tile"])
            del w
    if own:
        handles(s)
    return s


def handles(s):
    """What a program keeps from call to call of the library's: weights, tables, outputs of a serving step."""
    from bit_gemm_fwht_amd import fp4, kv, layer

    c, op = s["case"], s["case"]["op"]
    if c.get("q"):
        s["params"] = fp4.Params(elem=fp4.E2M1 if c["q"] == "e2m1" else fp4.E4M3, hadamard_n=c["hn"],
                                 scale_mode=fp4.SCALE_E8M0_CEIL if c["rule"] == "ceil" else fp4.SCALE_E8M0_FLOOR)
    if op == "rope":
        s["rotary_table"] = layer.Rotary(s["inv_freq"], layout=layer.HALF if c["layout"] == "half" else layer.INTERLEAVED,
                                         scale=s["scale"])
        if not c["given"]:
            table = torch.zeros(c["seqs"], -(-c["context"] // 32), dtype=torch.int32, device=DEV)
            s["batch"] = kv.Batch(s["cu"], s["context"], table)
    elif op == "gated":
        elem = fp4.E2M1 if c["elem"] == "e2m1" else fp4.E4M3
        row, tile = fp4.Params(elem=elem), fp4.Params(elem=elem, block=(32, 32) if c["tile"] else (1, 32))
        s["a_q"] = fp4.QTensor(s["a"], s["a_scales"], None, c["rows"], c["hidden"], row)
        gate, up = (fp4.QTensor(s[n], s[n + "_scales"], None, c["ff"], c["hidden"], tile) for n in ("gate", "up"))
        s["weights"] = layer.GatedWeights(gate, up, act=ACTS(layer)[c["act"]])
    if c.get("q") and c.get("rows", 0) <= 64:  # a serving step's outputs are kept
        s["q_out"] = fp4.empty_qtensor(c["rows"], 2 * c["ff"] if op == "gated_grad" else c.get("ff") or c["cols"], s["params"], DEV)


def ACTS(layer):
    return {"silu": layer.SILU, "gelu": layer.GELU, "gelu_tanh": layer.GELU_TANH}


def hadamard(n, dtype):
    """Sylvester's matrix of +-1, n a power of two: (-1)^(number of common bits of row and column)."""
    i = torch.arange(n, device=DEV)
    common = i[:, None] & i[None]
    for shift in (4, 2, 1):
        common = common ^ (common >> shift)
    return (1 - 2 * (common & 1)).to(dtype)


def coded(x, elem, tile):
    """fp32 [rows, cols] as MX codes and scales (bytes), nearest even, floor rule, one scale a group or 32 x 32 tile."""
    rows, cols = x.shape
    if tile:
        amax = x.abs().view(rows // 32, 32, cols // 32, 32).amax((1, 3))
        e = exponent(amax, elem, False)
        scale = e.repeat_interleave(32, 0).repeat_interleave(32, 1)
    else:
        e = exponent(x.abs().view(rows, cols // 32, 32).amax(2), elem, False)
        scale = e.repeat_interleave(32, 1)
    v = x * power(-scale)
    scales = (e + 127).to(torch.uint8).reshape(-1)
    if elem == "e4m3":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1), scales
    v = round4(v)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(rows, cols // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).reshape(-1), scales


# ---- the library's calls ----

def run(state):
    return (run_own if own else run_plain)(state)


def run_own(s):
    from bit_gemm_fwht_amd import layer

    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        r = layer.rmsnorm(s["x"], s["w"], eps=1e-5, residual=s["r"], out_q=s.get("params"), q_out=s.get("q_out"), keep_y=c["y"])
        return named(s, sum=r.sum, y=r.y, q=r.q)
    if op == "norm_grad":
        dx, dw = layer.rmsnorm_backward(s["dy"], s["s"], s["w"], eps=1e-5, dsum=s["dsum"])
        return {"dx": dx, "dw": dw}
    if op == "rope":
        q, k = layer.rope((s["q"], s["k"]), s["rotary_table"], s["positions"] if c["given"] else s["batch"],
                          backward=c["backward"])
        return {"q": q, "k": k}
    if op == "gated":
        r = layer.gated(s["a_q"], s["weights"], out_dtype=DTYPES[c["dtype"]], keep_h=c["h"], keep_gu=c["gu"],
                        out_q=s.get("params"), q_out=s.get("q_out"))
        return named(s, h=r.h, gu=r.gu, q=r.q)
    r = layer.gated_backward(s["dh"], s["gu"], act=ACTS(layer)[c["act"]], keep=c["keep"], out_q=s.get("params"),
                             q_out=s.get("q_out"))
    return named(s, dgu=r.dgu, q=r.q)


def named(s, q=None, **tensors):
    """The outputs that there are; a coded one as the values of its elements and scales."""
    out = {k: v for k, v in tensors.items() if v is not None}
    if q is not None:
        codes = q.codes
        if s["case"]["q"] == "e2m1":  # two E2M1 codes a byte, as two E4M3 ones
            if "pairs" not in s:
                byte = torch.arange(256, device=DEV)
                grid = torch.tensor(GRID + tuple(-v for v in GRID), device=DEV)
                pair = torch.stack([grid[byte & 15], grid[byte >> 4]], 1).to(torch.float8_e4m3fn)
                s["pairs"] = pair.view(torch.int16).reshape(-1)
            codes = s["pairs"][codes.int()]
        out["codes"] = codes.view(torch.float8_e4m3fn).view(q.rows, q.cols)
        out["scales"] = q.scales.view(torch.float8_e8m0fnu).view(q.rows, q.cols // 32)
    return out


# ---- the plain forms ----

def run_plain(s):
    op = s["case"]["op"]
    return {"norm": plain_norm, "norm_grad": plain_norm_grad, "rope": plain_rope, "gated": plain_gated,
            "gated_grad": plain_gated_grad}[op](s)


def exponent(amax, elem, ceil):
    """Of each block its exponent e: floor(log2 amax) less the element's own largest exponent, and with `ceil` one
    more where the largest element times 2^e is below amax."""
    m, ex = torch.frexp(amax)
    e = ex - (3 if elem == "e2m1" else 9)
    if ceil:
        e = e + (m > (0.75 if elem == "e2m1" else 0.875))
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def power(e):
    """2^e in fp32, exact (0 for e = -127, which stands for blocks of zeros)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def round4(v):
    """The E2M1 value nearest to v (ties to the even code), at most 6."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def quantized(s, x):
    """fp32 [rows, cols], rotated if the case says so, as the values of its elements and scales."""
    c = s["case"]
    rows, cols = x.shape
    if c["hn"]:
        x = ((x.view(-1, c["hn"]) @ s["hadamard"]) * (1.0 / math.sqrt(c["hn"]))).view(rows, cols)
    x = x.view(rows, cols // 32, 32)
    e = exponent(x.abs().amax(2), c["q"], c["rule"] == "ceil")
    v = x * power(-e)[..., None]
    v = round4(v) if c["q"] == "e2m1" else v.clamp(-448.0, 448.0)
    return {"codes": v.to(torch.float8_e4m3fn).view(rows, cols), "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def plain_norm(s):
    c = s["case"]
    dtype, out = DTYPES[c["dtype"]], {}
    x = s["x"].float()
    if c["residual"]:  # what the residual stream holds is what is normed
        out["sum"] = (x + s["r"].float()).to(dtype)
        x = out["sum"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * s["w"].float()
    if c["y"]:
        out["y"] = y.to(dtype)
    return {**out, **(quantized(s, y) if c["q"] else {})}


def plain_norm_grad(s):
    x, dy = s["s"].float(), s["dy"].float()
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5)
    n = x * rstd
    a = dy * s["w"].float()
    dx = rstd * (a - n * (a * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": (dy * n).sum(0)}


def turned(c, x, cos, sin):
    """Each pair (x1, x2) of the first `rotary` channels as (x1 cos - x2 sin, x2 cos + x1 sin)."""
    r = c["rotary"]
    x1, x2 = (x[..., : r // 2], x[..., r // 2: r]) if c["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.cat([y1, y2], -1) if c["layout"] == "half" else torch.stack([y1, y2], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1) if r < c["dim"] else y


def plain_rope(s):
    c = s["case"]
    if c["given"]:
        pos = s["positions"].double()
    else:
        row = torch.arange(s["q"].shape[0], device=DEV)
        seq = torch.searchsorted(s["cu"], row, right=True) - 1
        pos = (s["context"][seq] - s["cu"][seq + 1] + row).double()
    angle = pos[:, None, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()
    sin = -sin if c["backward"] else sin
    return {"q": turned(c, s["q"].float(), cos, sin).to(s["q"].dtype), "k": turned(c, s["k"].float(), cos, sin).to(s["k"].dtype)}


def values(codes, scales, rows, cols, elem, tile):
    """MX codes and scales as numbers."""
    if elem == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor(GRID + tuple(-x for x in GRID), device=DEV)
        v = grid[torch.stack([codes & 15, codes >> 4], -1).int()]
    f = power(scales.to(torch.int32) - 127)
    if tile:
        return (v.view(rows // 32, 32, cols // 32, 32) * f.view(rows // 32, 1, cols // 32, 1)).view(rows, cols)
    return (v.view(rows, cols // 32, 32) * f.view(rows, cols // 32, 1)).view(rows, cols)


def activation(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def slope(g, act):
    """The activation's derivative."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p * (1.0 + g * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    b = math.sqrt(2.0 / math.pi)
    t = torch.tanh(b * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * b * (1.0 + 3 * 0.044715 * g * g)


def plain_gated(s):
    c, out = s["case"], {}
    k, f = c["hidden"], c["ff"]
    a = values(s["a"], s["a_scales"], c["rows"], k, c["elem"], False)
    g = a @ values(s["gate"], s["gate_scales"], f, k, c["elem"], c["tile"]).T
    u = a @ values(s["up"], s["up_scales"], f, k, c["elem"], c["tile"]).T
    h = activation(g, c["act"]) * u
    if c["h"]:
        out["h"] = h.to(DTYPES[c["dtype"]])
    if c["gu"]:
        out["gu"] = torch.cat([g, u], 1).to(DTYPES[c["dtype"]])
    return {**out, **(quantized(s, h) if c["q"] else {})}


def plain_gated_grad(s):
    c = s["case"]
    dh, gu = s["dh"].float(), s["gu"].float()
    g, u = gu[:, : c["ff"]], gu[:, c["ff"]:]
    d = torch.cat([dh * u * slope(g, c["act"]), dh * activation(g, c["act"])], 1)
    out = {"dgu": d.to(s["dh"].dtype)} if c["keep"] else {}
    return {**out, **(quantized(s, d) if c["q"] else {})}


# ---- the definitions in 64 bits ----
# Codes of 8 bits are held to the quotient before its rounding, as values in bf16 are to the value before theirs.
# Scales and codes of 4 bits have no such value: a neighbour's is as near where fp32 cannot tell the two apart.

def number(codes, elem):
    """The values of element codes from their bits: (1 + m / 2^M) 2^(e - bias), or m 2^(1 - bias - M) where e is 0."""
    if elem == "e2m1":
        codes, man, bias = torch.stack([codes % 16, codes // 16], -1).reshape(-1), 1, 1
        sign, code = codes // 8, (codes % 8).long()
    else:
        sign, code, man, bias = codes // 128, (codes % 128).long(), 3, 7
    e, m = code // 2 ** man, (code % 2 ** man).double()
    v = torch.where(e > 0, (1.0 + m / 2 ** man) * torch.exp2(e.double() - bias), m * 2.0 ** (1 - bias - man))
    return v * (1.0 - 2.0 * sign)


def operand(codes, scales, rows, cols, elem, tile):
    f = torch.exp2(scales.double() - 127.0).view(-1, cols // 32).repeat_interleave(32, 1)
    return number(codes, elem).view(rows, cols) * (f.repeat_interleave(32, 0) if tile else f)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]

    def low(x):
        if c["hn"]:
            h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
            while h.shape[0] < c["hn"]:  # H_2n = [[H, H], [H, -H]]
                h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
            x = (x.reshape(-1, c["hn"]) @ h / math.sqrt(c["hn"])).view(x.shape)
        if c["q"] == "e2m1":
            return {"codes": None, "scales": None}
        x = x.view(x.shape[0], -1, 32)
        amax = x.abs().amax(2)
        e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140))) - 8.0
        if c["rule"] == "ceil":
            e = e + (448.0 * torch.exp2(e) < amax)
        e = torch.where(amax > 0, e, 0.0).clamp(-127.0, 127.0)
        return {"codes": (x / torch.exp2(e)[..., None]).clamp(-448.0, 448.0).view(x.shape[0], -1), "scales": None}

    if op == "norm":
        x, out = s["x"].double(), {}
        if c["residual"]:
            x = (x + s["r"].double()).to(DTYPES[c["dtype"]]).double()
            out["sum"] = x
        y = x / torch.sqrt((x ** 2).sum(1, keepdim=True) / c["cols"] + 1e-5) * s["w"].double()
        if c["y"]:
            out["y"] = y
        return {**out, **(low(y) if c["q"] else {})}
    if op == "norm_grad":
        # the derivative of sum_j dy_j w_j s_j (mean s^2 + eps)^(-1/2) by s_i, plus the stream's own
        x, dy, w = s["s"].double(), s["dy"].double(), s["w"].double()
        v = (x ** 2).sum(1, keepdim=True) / c["cols"] + 1e-5
        dot = (dy * w * x).sum(1, keepdim=True)
        dx = dy * w * v ** -0.5 - x * dot * v ** -1.5 / c["cols"]
        return {"dx": dx + s["dsum"].double() if c["stream"] else dx, "dw": (dy * x * v ** -0.5).sum(0)}
    if op == "rope":
        pos = torch.cat([torch.arange(int(n) - c["tokens"], int(n), device=DEV) for n in s["context"].tolist()]).double()
        turn = torch.polar(torch.full((1,), s["scale"], dtype=torch.float64, device=DEV), pos[:, None, None] * s["inv_freq"])
        turn = turn.conj() if c["backward"] else turn
        out = {}
        for name in ("q", "k"):
            x, r = s[name].double(), c["rotary"]
            pair = x[..., :r].reshape(*x.shape[:2], 2, r // 2).transpose(2, 3) if c["layout"] == "half" else x[..., :r].reshape(*x.shape[:2], r // 2, 2)
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            y = y.transpose(2, 3) if c["layout"] == "half" else y
            out[name] = torch.cat([y.reshape(*x.shape[:2], r), x[..., r:]], 2)
        return out
    act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda g: torch.nn.functional.gelu(g, approximate="tanh")}[c["act"]]
    if op == "gated":
        k, f = c["hidden"], c["ff"]
        a = operand(s["a"], s["a_scales"], c["rows"], k, c["elem"], False)
        g, u = (a @ operand(s[n], s[n + "_scales"], f, k, c["elem"], c["tile"]).T for n in ("gate", "up"))
        h = act(g) * u
        out = {"h": h} if c["h"] else {}
        if c["gu"]:
            out["gu"] = torch.cat([g, u], 1)
        return {**out, **(low(h) if c["q"] else {})}
    gu = s["gu"].double().requires_grad_()
    with torch.enable_grad():
        h = act(gu[:, : c["ff"]]) * gu[:, c["ff"]:]
        d, = torch.autograd.grad(h, gu, s["dh"].double())
    out = {"dgu": d} if c["keep"] else {}
    return {**out, **(low(d) if c["q"] else {})}
