"""A decoder layer of a model in low bits, served and trained, on synthetic weights.

Served (prompt, then single tokens), MXFP4 products rotated by H_128, keys and values in the 8-bit cache:

    norm (+ stream) -> q, k, v -> rope -> kv.append -> kv.attention -> product
    -> norm (+ stream) -> gated feed-forward -> product

every product's operand leaves the operator before it already rotated and quantized. Trained: a step of the
feed-forward half in MXFP8, forward and backward, with the gradients of its weights and inputs.

    python examples/decoder_layer.py [--hidden 4096] [--ff 11008] [--heads 32] [--kv-heads 8] [--tokens 1000] [--steps 8]

prints how far the layer's outputs and gradients are from the same layer in fp32 without quantization.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_gemm_fwht_amd import fp4, kv, layer  # noqa: E402


class DecoderLayer:
    """Weights bf16, in a dict: norms [hidden] "n1", "n2"; [out, in] "qkv", "out", "gate_up" (gate's rows first), "down"."""

    def __init__(self, w, heads, kv_heads, pages, rotary, page_tokens=32):
        self.params = fp4.Params(hadamard_n=128)
        self.heads, self.kv_heads, self.rotary = heads, kv_heads, rotary
        self.dim = w["out"].shape[1] // heads
        self.n1, self.n2 = w["n1"], w["n2"]
        self.qkv, self.out, gate_up, self.down = (fp4.quantize(w[n], self.params) for n in ("qkv", "out", "gate_up", "down"))
        self.gate_up = layer.GatedWeights(gate_up, act=layer.SILU)
        self.cache = kv.empty_cache(pages, kv_heads, page_tokens, self.dim, w["qkv"].device)

    def __call__(self, x, stream, batch):
        """x [tokens, hidden]: what the layer before adds to the stream (None before the first). Returns the same of
        this layer, and the stream that it goes to."""
        tokens, hidden = stream.shape
        if x is None:
            a = layer.rmsnorm(stream, self.n1, out_q=self.params, keep_y=False)
        else:
            a = layer.rmsnorm(x, self.n1, residual=stream, sum_out=stream, out_q=self.params, keep_y=False)
        fused = fp4.gemm(a.q, self.qkv).view(tokens, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = fused.split([self.heads, self.kv_heads, self.kv_heads], 1)  # slices: no copies
        layer.rope((q, k), self.rotary, batch, out=(q, k))
        kv.append(self.cache, k, v, batch)
        o = kv.attention(q, self.cache, batch)
        x = fp4.gemm(fp4.quantize(o.view(tokens, hidden), self.params), self.out)
        b = layer.rmsnorm(x, self.n2, residual=stream, sum_out=stream, out_q=self.params, keep_y=False)
        h = layer.gated(b.q, self.gate_up, out_q=self.params, keep_h=False)
        return fp4.gemm(h.q, self.down), stream


class FeedForward:
    """norm (+ stream) -> gated -> product in MXFP8: a training step's forward and backward pass. Each weight is
    quantized along both of its axes, as each of the passes contracts it."""

    def __init__(self, norm, gate_up, down):
        self.params = fp4.Params(elem=fp4.E4M3, scale_mode=fp4.SCALE_E8M0_CEIL)
        self.norm = norm
        self.gate_up, self.gate_up_t = fp4.quantize(gate_up, self.params), fp4.quantize_colwise(gate_up, self.params)
        self.down, self.down_t = fp4.quantize(down, self.params), fp4.quantize_colwise(down, self.params)
        self.weights = layer.GatedWeights(self.gate_up, act=layer.SILU)

    def forward(self, x, stream):
        a = layer.rmsnorm(x, self.norm, residual=stream, out_q=self.params)
        h = layer.gated(a.q, self.weights, keep_gu=True, out_q=self.params)
        self.kept = a, h
        return fp4.gemm(h.q, self.down), a.sum

    def backward(self, dy, dstream):
        """Gradients of x (and the stream alike), the norm's weight, gate_up and down from those of forward's results."""
        (a, h), p = self.kept, self.params
        dh = fp4.gemm(fp4.quantize(dy, p), self.down_t)
        d = layer.gated_backward(dh, h.gu, out_q=p)
        da = fp4.gemm(d.q, self.gate_up_t)
        dx, dnorm = layer.rmsnorm_backward(da, a.sum, self.norm, dsum=dstream)
        dgate_up = fp4.gemm(fp4.quantize_colwise(d.dgu, p), fp4.quantize_colwise(a.y, p))
        ddown = fp4.gemm(fp4.quantize_colwise(dy, p), fp4.quantize_colwise(h.h, p))
        return {"x": dx, "norm": dnorm, "gate_up": dgate_up, "down": ddown}


def plain_norm(s, w):
    return s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-5) * w.float()


def plain_feed_forward(s, w):
    g, u = (plain_norm(s, w["n2"]) @ w["gate_up"].float().T).chunk(2, 1)
    return (torch.nn.functional.silu(g) * u) @ w["down"].float().T


def plain_rope(x, pos, inv_freq):
    t = pos.double()[:, None, None] * inv_freq
    c, s = t.cos().float(), t.sin().float()
    a, b = x.chunk(2, 2)
    return torch.cat([a * c - b * s, b * c + a * s], 2)


def plain_layer(stream, w, heads, kv_heads, inv_freq, past):
    """The same in fp32 for one sequence; past: its keys and values so far, extended in place. Returns what is added."""
    n, hidden = stream.shape
    dim = hidden // heads
    q, k, v = (plain_norm(stream, w["n1"]) @ w["qkv"].float().T).view(n, -1, dim).split([heads, kv_heads, kv_heads], 1)
    pos = torch.arange(n, device=stream.device) + (past["k"].shape[0] if past else 0)
    q, k = plain_rope(q, pos, inv_freq), plain_rope(k, pos, inv_freq)
    past["k"] = torch.cat([past["k"], k]) if "k" in past else k
    past["v"] = torch.cat([past["v"], v]) if "v" in past else v
    k, v = (past[i].repeat_interleave(heads // kv_heads, 1).transpose(0, 1).contiguous() for i in "kv")
    s = q.transpose(0, 1) @ k.transpose(1, 2).contiguous() / math.sqrt(dim)
    s = s.masked_fill(torch.arange(k.shape[1], device=s.device) > pos[:, None], -math.inf)
    a = (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, hidden) @ w["out"].float().T
    return a + plain_feed_forward(stream + a, w)


def weights(hidden, ff, heads, kv_heads, g):
    def normal(*shape):
        return (torch.randn(*shape, generator=g, device=g.device) / math.sqrt(shape[-1])).bfloat16()
    dim = hidden // heads
    ones = [(1.0 + 0.1 * torch.randn(hidden, generator=g, device=g.device)).bfloat16() for _ in range(2)]
    return {"n1": ones[0], "n2": ones[1], "qkv": normal((heads + 2 * kv_heads) * dim, hidden), "out": normal(hidden, hidden),
            "gate_up": normal(2 * ff, hidden), "down": normal(hidden, ff)}


def relative(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


def serve(hidden=4096, ff=11008, heads=32, kv_heads=8, tokens=1000, steps=8, seed=0, device="cuda"):
    """A prompt of `tokens` tokens and one of a third of that, then `steps` single tokens of each. Returns the relative
    errors (2-norms) of what the layer adds to the stream, the prompt's and the single tokens' largest."""
    g = torch.Generator(device=device).manual_seed(seed)
    w = weights(hidden, ff, heads, kv_heads, g)
    page, lens = 32, [tokens, max(1, tokens // 3)]
    width = -(-(max(lens) + steps) // page)
    inv_freq, scale = layer.rotary_frequencies(hidden // heads, device=device)
    served = DecoderLayer(w, heads, kv_heads, 2 * width, layer.Rotary(inv_freq, scale=scale), page)
    table = torch.randperm(2 * width, generator=g, device=device).to(torch.int32).view(2, width)
    past, errors = [{}, {}], []
    for step in range(steps + 1):
        rows = lens if step == 0 else [1, 1]
        ctx = [n + step for n in lens]
        cu = torch.tensor([0, rows[0], sum(rows)], dtype=torch.int32, device=device)
        batch = kv.Batch(cu, torch.tensor(ctx, dtype=torch.int32, device=device), table, max_tokens=max(rows),
                         max_context=max(ctx))
        x = torch.randn(sum(rows), hidden, generator=g, device=device).bfloat16()
        y, stream = served(None, x.clone(), batch)
        got = y.float() + stream.float() - x.float()
        want = torch.cat([plain_layer(x[cu[i]:cu[i + 1]].float(), w, heads, kv_heads, inv_freq, past[i]) for i in range(2)])
        errors.append(relative(got, want))
    return errors[0], max(errors[1:]) if steps else None


def train(hidden=4096, ff=11008, tokens=1024, seed=0, device="cuda"):
    """One step of the feed-forward half. Returns the relative errors (2-norms) of its output and its gradients."""
    g = torch.Generator(device=device).manual_seed(seed)
    w = weights(hidden, ff, 1, 1, g)
    x, stream, dy, dstream = (torch.randn(tokens, hidden, generator=g, device=device).bfloat16() for _ in range(4))
    half = FeedForward(w["n2"], w["gate_up"], w["down"])
    y, s = half.forward(x, stream)
    got = half.backward(dy, dstream)
    leaf = {n: w[n].float().requires_grad_() for n in ("n2", "gate_up", "down")}
    s32 = (x.float() + stream.float()).requires_grad_()
    with torch.enable_grad():
        want_y = plain_feed_forward(s32, leaf)
        grads = torch.autograd.grad([want_y, s32 * 1.0], [s32, leaf["n2"], leaf["gate_up"], leaf["down"]],
                                    [dy.float(), dstream.float()])
    want = dict(zip(("x", "norm", "gate_up", "down"), grads))
    return {"y": relative(y, want_y), **{n: relative(got[n], want[n]) for n in want}}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("hidden", 4096), ("ff", 11008), ("heads", 32), ("kv-heads", 8), ("tokens", 1000), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    prompt, single = serve(a.hidden, a.ff, a.heads, a.kv_heads, a.tokens, a.steps)
    print(f"decoder layer, {a.tokens} tokens then {a.steps} single ones: relative error of its addition to the stream "
          f"{prompt:.4f} (prompt), {single:.4f} (single tokens, largest)")
    print("training step of its feed-forward, relative errors: " +
          ", ".join(f"{n} {e:.4f}" for n, e in train(a.hidden, a.ff).items()))
