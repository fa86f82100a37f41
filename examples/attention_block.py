"""One attention block of a model served in low bits, prompt and single tokens, on synthetic weights.

The linear layers run on MXFP4 operands (rotated by H_128 and quantized, activations as they come,
weights once), keys and values live in the paged 8-bit cache, and attention reads them there:

    x -> quantize -> gemm (q, k, v) -> kv.append -> kv.attention -> quantize -> gemm -> x + ...

    python examples/attention_block.py [--hidden 4096] [--heads 32] [--kv-heads 8] [--tokens 1000] [--steps 8]

prints how far the block's outputs are from the same block in fp32 without quantization.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_gemm_fwht_amd import fp4, kv  # noqa: E402


class AttentionBlock:
    """Weights [out, in] bf16 -> quantized once; one cache for all sequences."""

    def __init__(self, w_qkv, w_out, heads, kv_heads, pages, page_tokens=32):
        self.params = fp4.Params(hadamard_n=128)
        self.heads, self.kv_heads = heads, kv_heads
        self.dim = w_out.shape[1] // heads
        self.w_qkv, self.w_out = fp4.quantize(w_qkv, self.params), fp4.quantize(w_out, self.params)
        self.cache = kv.empty_cache(pages, kv_heads, page_tokens, self.dim, w_qkv.device)

    def __call__(self, x, batch):
        n, hidden = x.shape
        fused = fp4.gemm(fp4.quantize(x, self.params), self.w_qkv).view(n, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = fused.split([self.heads, self.kv_heads, self.kv_heads], 1)  # slices: no copies
        kv.append(self.cache, k, v, batch)
        o = kv.attention(q, self.cache, batch)
        return x + fp4.gemm(fp4.quantize(o.view(n, hidden), self.params), self.w_out)


def plain_block(x, w_qkv, w_out, heads, kv_heads, past):
    """The same in fp32 for one sequence; past: its keys and values so far, extended in place."""
    n, hidden = x.shape
    dim = hidden // heads
    q, k, v = (x.float() @ w_qkv.float().T).view(n, -1, dim).split([heads, kv_heads, kv_heads], 1)
    past["k"] = torch.cat([past["k"], k]) if "k" in past else k
    past["v"] = torch.cat([past["v"], v]) if "v" in past else v
    group, ctx = heads // kv_heads, past["k"].shape[0]
    k, v = (past[i].repeat_interleave(group, 1).transpose(0, 1).contiguous() for i in "kv")
    s = q.transpose(0, 1) @ k.transpose(1, 2) / math.sqrt(dim)
    pos = torch.arange(ctx - n, ctx, device=x.device)
    s = s.masked_fill(torch.arange(ctx, device=x.device) > pos[:, None], -math.inf)
    o = (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, hidden)
    return x.float() + o @ w_out.float().T


def run(hidden=4096, heads=32, kv_heads=8, tokens=1000, steps=8, seed=0, device="cuda"):
    """A prompt of `tokens` tokens and one of a third of that, then `steps` single tokens of each.
    Returns the relative errors (2-norms) of the prompt's outputs and of the single tokens'."""
    g = torch.Generator(device=device).manual_seed(seed)
    dim, page = hidden // heads, 32

    def normal(*shape, size=1.0):
        return (torch.randn(*shape, generator=g, device=device) * size).bfloat16()

    w_qkv = normal((heads + 2 * kv_heads) * dim, hidden, size=1 / math.sqrt(hidden))
    w_out = normal(hidden, hidden, size=1 / math.sqrt(hidden))
    lens = [tokens, max(1, tokens // 3)]
    width = -(-(max(lens) + steps) // page)
    block = AttentionBlock(w_qkv, w_out, heads, kv_heads, pages=2 * width, page_tokens=page)
    table = torch.randperm(2 * width, generator=g, device=device).to(torch.int32).view(2, width)
    past, errors = [{}, {}], []
    for step in range(steps + 1):
        rows = lens if step == 0 else [1, 1]
        ctx = [n + step for n in lens]
        cu = torch.tensor([0, rows[0], sum(rows)], dtype=torch.int32, device=device)
        batch = kv.Batch(cu, torch.tensor(ctx, dtype=torch.int32, device=device), table, max_tokens=max(rows),
                         max_context=max(ctx))
        x = normal(sum(rows), hidden)
        y = block(x, batch).float() - x.float()
        want = torch.cat([plain_block(x[cu[i]:cu[i + 1]], w_qkv, w_out, heads, kv_heads, past[i]) for i in range(2)])
        want = want - x.float()
        errors.append(((y - want).norm() / want.norm()).item())
    return errors[0], max(errors[1:]) if steps else None


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("tokens", 1000), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    prompt, single = run(a.hidden, a.heads, a.kv_heads, a.tokens, a.steps)
    print(f"attention block, {a.tokens} tokens then {a.steps} single ones: relative error of its addition to x "
          f"{prompt:.4f} (prompt), {single:.4f} (single tokens, largest)")
