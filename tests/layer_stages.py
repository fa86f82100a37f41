"""The stages of a served decoder layer (examples/decoder_layer.py), each held to its 64-bit form on what the stage before
it handed over, in numpy. `Oracle` has the forms; a test may put a wrong one in its place to see that it is noticed.

Bounds: a stored bf16 is off by half a step, 2^-8 of the value; a product's fp32 sum by 1e-5 of the sum of magnitudes;
what is coded in E2M1 by half a step of its group's scale (a quarter below 2 scales, a half below 4, one above, and what
lies past the largest element, 6), with what came before it: 2^-18 of the sum of magnitudes that a rotation adds up."""
import numpy as np

import kv_reference
import layer_reference as ref

HALF = 2.0 ** -8


def fwht(x, n=128):
    """Blockwise H_n / sqrt(n) along the last axis."""
    y = np.array(x, np.float64).reshape(-1, n)
    h = 1
    while h < n:
        y = y.reshape(-1, n // (2 * h), 2, h)
        y = np.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2).reshape(-1, n)
        h *= 2
    return (y / np.sqrt(n)).reshape(np.shape(x))


class Oracle:
    """norm(s, w), rope(x [tokens, heads, dim], pos, inv_freq), attention(q, cache, cu, context, table, scale) as
    kv_reference's, gated(g, u), stream(x, r)."""

    def norm(self, s, w):
        return ref.rmsnorm(s, w, 1e-5)

    def rope(self, x, pos, inv_freq):
        return ref.rope(x, pos, inv_freq, False)

    def attention(self, q, cache, cu, context, table, scale):
        return kv_reference.attention(q, cache, cu, context, table, scale, True, 0)

    def gated(self, g, u):
        return ref.act(g, 0) * u

    def stream(self, x, r):
        return x + r


def coded(what, q, want, err=0.0):
    """q = (values, scales of the groups) of E2M1 codes with the floor rule against the rotated `want`, itself off by
    `err` before the rotation."""
    values, scales = q
    n = 128
    rotated = fwht(want)
    slack = (np.abs(want) * 2.0 ** -18 + err).reshape(-1, n).sum(1).repeat(n).reshape(want.shape) / np.sqrt(n)
    s = np.repeat(scales, 32, axis=1)
    a = np.abs(rotated) / s
    step = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0)) + np.maximum(a - 6.0, 0.0)
    # where `slack` may carry a value across 2 or 4, the wider step
    step = np.maximum(step, np.where(a + slack / s >= 4, 1.0, np.where(a + slack / s >= 2, 0.5, 0.25)))
    assert (np.abs(values - rotated) <= s * step + slack).all(), f"{what}: codes"
    amax = np.abs(rotated).reshape(len(want), -1, 32).max(2)
    room = slack.reshape(len(want), -1, 32).max(2)
    assert (((amax + room >= 4 * scales) | (amax == 0)) & (amax - room < 8 * scales)).all(), f"{what}: scales"


def product(a, b):
    """The product of two coded operands' values, and its sum's bound."""
    return a @ b.T, 1e-5 * (np.abs(a) @ np.abs(b).T)


def stored(what, got, want, tol=0.0):
    assert (np.abs(got - want) <= tol + HALF * (np.abs(want) + tol)).all(), what


def bf16(x):
    """The nearest bf16 of fp32 values, ties to even."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def attention_bound(absv, mag, cnt, out, dim):
    """Scores: dim additions and the scale err by 2^-23 of sum |q k| each, their difference to the maximum by 2^-21 more,
    the exponential by 2 ulp; sums of cnt weights by 2^-23 each, in numerator and denominator. Weights and the output are
    rounded to bf16."""
    w = (2.0 * (dim + 2) * 2.0 ** -23 + 2.0 ** -21) * mag + 2.0 ** -21 + cnt * 2.0 ** -23
    return 1.01 * ((2.0 * w[..., None] + HALF) * absv + HALF * np.abs(out))


def check(r, w, oracle=None):
    """r: what the stages of one call took and gave (float64; coded: (values, scales)); w: the weights' values."""
    o = oracle or Oracle()
    if r["x"] is not None:
        assert np.array_equal(r["stream1"], bf16(o.stream(r["x"], r["stream0"]))), "first stream"
    else:
        assert np.array_equal(r["stream1"], r["stream0"]), "first stream"
    coded("first norm", r["a"], o.norm(r["stream1"], w["n1"]))
    want, tol = product(r["a"][0], w["qkv"])
    stored("q, k, v", r["fused"].reshape(want.shape), want, tol)
    heads, kv_heads = r["heads"]
    f = r["fused"]
    for name, x in (("q", f[:, :heads]), ("k", f[:, heads:heads + kv_heads])):
        n = x.shape[2] // 2
        size = np.abs(x[..., :n]) + np.abs(x[..., n:])
        stored(f"rope of {name}", r[name], o.rope(x, r["pos"], r["inv_freq"]), np.concatenate([size, size], 2) * 2.0 ** -21)
    assert np.array_equal(r["v"], f[:, heads + kv_heads:]), "v"
    before = r["cache_before"]
    kv_reference.append(before, r["k"], r["v"], r["cu"], r["context"], r["table"], True)
    after = r["cache"]
    assert all(np.array_equal(a, b) for a, b in ((before.k, after.k), (before.v, after.v), (before.ks, after.ks), (before.vs, after.vs))), "cache"
    att, _, absv, mag, cnt = o.attention(r["q"], after, r["cu"], r["context"], r["table"], r["q"].shape[2] ** -0.5)
    assert (np.abs(r["o"] - att) <= attention_bound(absv, mag, cnt, att, att.shape[2])).all(), "attention"
    tokens = len(r["o"])
    coded("attention's codes", r["o_q"], r["o"].reshape(tokens, -1))
    stored("output product", r["x2"], *product(r["o_q"][0], w["out"]))
    assert np.array_equal(r["stream2"], bf16(o.stream(r["x2"], r["stream1"]))), "second stream"
    coded("second norm", r["b"], o.norm(r["stream2"], w["n2"]))
    gu, tol = product(r["b"][0], w["gate_up"])
    half = gu.shape[1] // 2
    g, u, tg, tu = gu[:, :half], gu[:, half:], tol[:, :half], tol[:, half:]
    # the activation's slope is at most 1.13
    coded("gated", r["h"], o.gated(g, u), 1.13 * tg * (np.abs(u) + tu) + np.abs(ref.act(g, 0)) * tu)
    stored("down product", r["y"], *product(r["h"][0], w["down"]))
