"""The served decoder layer of examples/decoder_layer.py stage by stage: what each of its calls took and gave is recorded
as the layer runs, and held to the 64-bit forms of layer_stages.py."""
import os
import sys

import numpy as np
import pytest
import torch

import kv_reference
import layer_stages as st

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def values(fp4, q):
    """A coded operand's values (as rotated) and its groups' scales."""
    s = np.exp2(q.scales.view(torch.uint8)[:q.rows * q.cols // 32].double().cpu().numpy() - 127.0).reshape(q.rows, -1)
    return f64(fp4.dequantize(fp4.with_params(q, hadamard_n=0))), s


def copy_of(cache):
    return kv_reference.Cache(*(t.cpu().numpy() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)))


@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (4, 4)])
def test_every_stage_of_a_served_layer(monkeypatch, heads, kv_heads):
    """A prompt of two sequences, then single tokens; the first layer of a model (no x) and a later one."""
    import decoder_layer
    from bit_gemm_fwht_amd import fp4, kv, layer
    g = torch.Generator(device="cuda").manual_seed(5)
    hidden, ff, lens, page = 1024, 2816, [70, 23], 32
    w = decoder_layer.weights(hidden, ff, heads, kv_heads, g)
    inv_freq, scale = layer.rotary_frequencies(hidden // heads, device="cuda")
    assert scale == 1.0
    width = -(-(max(lens) + 2) // page)
    served = decoder_layer.DecoderLayer(w, heads, kv_heads, 2 * width, layer.Rotary(inv_freq), page)
    table = torch.randperm(2 * width, generator=g, device="cuda").to(torch.int32).view(2, width)
    known = {"n1": f64(w["n1"]), "n2": f64(w["n2"])}
    for name, q in (("qkv", served.qkv), ("out", served.out), ("down", served.down)):
        known[name] = values(fp4, q)[0]
    known["gate_up"] = np.concatenate([values(fp4, q)[0] for q in (served.gate_up.gate, served.gate_up.up)])

    r = {}
    calls = []

    def record(module, name, before=None, after=None):
        call = getattr(module, name)

        def recorded(*args, **kw):
            calls.append(name)
            if before:
                before(*args, **kw)
            out = call(*args, **kw)
            if after:
                after(out, *args, **kw)
            return out
        monkeypatch.setattr(module, name, recorded)

    def norm(out, x, weight, residual=None, sum_out=None, **kw):
        first = "a" not in r
        r["a" if first else "b"] = values(fp4, out.q)
        r["stream1" if first else "stream2"] = f64(x if residual is None else out.sum)
        assert residual is None or out.sum is sum_out is residual

    def product(out, a, b):
        name = ("fused", "x2", "y")[calls.count("gemm") - 1]
        r[name] = f64(out)
        coded = values(fp4, a)[0]  # what the operator before it made
        assert np.array_equal(coded, r[{"fused": "a", "x2": "o_q", "y": "h"}[name]][0])
        assert b is {"fused": served.qkv, "x2": served.out, "y": served.down}[name]

    def turned(got, x, rotary, batch, **kw):
        r["q"], r["k"] = f64(got[0]), f64(got[1])

    def before_append(cache, k, v, batch):
        r["cache_before"], r["v"] = copy_of(cache), f64(v)
        assert np.array_equal(f64(k), r["k"])

    def attended(out, q, cache, batch):
        assert np.array_equal(f64(q), r["q"])
        r["cache"], r["o"] = copy_of(cache), f64(out)

    def quantized(out, x, p):
        assert np.array_equal(f64(x), r["o"].reshape(x.shape))
        r["o_q"] = values(fp4, out)

    def gated(out, a, weights, **kw):
        assert np.array_equal(values(fp4, a)[0], r["b"][0]) and weights is served.gate_up
        r["h"] = values(fp4, out.q)

    record(layer, "rmsnorm", after=norm)
    record(fp4, "gemm", after=product)
    record(layer, "rope", after=turned)
    record(kv, "append", before=before_append)
    record(kv, "attention", after=attended)
    record(fp4, "quantize", after=quantized)
    record(layer, "gated", after=gated)
    for step in range(3):
        rows = lens if step == 0 else [1, 1]
        ctx = [n + step for n in lens]
        cu = np.cumsum([0] + rows)
        batch = kv.Batch(torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                         table, max_tokens=max(rows), max_context=max(ctx))
        stream = torch.randn(sum(rows), hidden, generator=g, device="cuda").bfloat16()
        x = None if step == 1 else torch.randn(sum(rows), hidden, generator=g, device="cuda").bfloat16()
        r.clear()
        calls.clear()
        r.update(heads=(heads, kv_heads), cu=cu, context=np.array(ctx), table=table.cpu().numpy(), inv_freq=f64(inv_freq),
                 pos=np.concatenate([np.arange(c - n, c) for n, c in zip(rows, ctx)]), stream0=f64(stream),
                 x=None if x is None else f64(x))
        y, after = served(x, stream, batch)
        assert calls == ["rmsnorm", "gemm", "rope", "append", "attention", "quantize", "gemm", "rmsnorm", "gated", "gemm"]
        assert np.array_equal(f64(y), r["y"]) and np.array_equal(f64(after), r["stream2"])
        r["fused"] = r["fused"].reshape(sum(rows), heads + 2 * kv_heads, -1)
        st.check(dict(r), known)
