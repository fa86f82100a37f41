"""CPU test of the stage checks of a served layer (layer_stages.py): a chain worked out in numpy passes, and each mistake
planted in the forms that it is held to is noticed at its own stage."""
import numpy as np
import pytest

import kv_reference
import layer_reference as ref
import layer_stages as st


def code(x):
    """E2M1 values and scales of rows rotated by blocks of H_128, floor rule, nearest even."""
    y = st.fwht(x)
    g = y.reshape(len(y), -1, 32)
    amax = np.abs(g).max(2)
    # (a row that attends to its own token alone has the same values in heads that share a key head: groups of zeros)
    s = 2.0 ** np.maximum(np.floor(np.log2(np.where(amax > 0, amax, 2.0 ** -200))) - 2, -127)
    v = g / s[..., None]
    a = np.abs(v)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return (np.clip(np.round(v / step) * step, -6, 6) * s[..., None]).reshape(y.shape), s


HEADS, KV, DIM, PAGE = 4, 2, 64, 32
HIDDEN, FF = HEADS * DIM, 512


def weights(rng):
    def draw(rows, cols):
        return code(rng.normal(size=(rows, cols)) / np.sqrt(cols))[0]
    return {"n1": 1 + 0.1 * rng.normal(size=HIDDEN), "n2": 1 + 0.1 * rng.normal(size=HIDDEN), "qkv": draw((HEADS + 2 * KV) * DIM, HIDDEN),
            "out": draw(HIDDEN, HIDDEN), "gate_up": draw(2 * FF, HIDDEN), "down": draw(HIDDEN, FF)}


def chain(rng, w, with_x):
    """What the stages of a prompt of two sequences hand over, each rounded as it is stored."""
    o = st.Oracle()
    lens, tokens = (20, 9), 29
    r = {"heads": (HEADS, KV), "cu": np.array([0, 20, 29]), "context": np.array([20, 9]), "table": np.array([[2], [0]]),
         "pos": np.concatenate([np.arange(n) for n in lens]), "inv_freq": 10000.0 ** (-2.0 * np.arange(DIM // 2) / DIM)}
    r["stream0"] = st.bf16(rng.normal(size=(tokens, HIDDEN)))
    r["x"] = st.bf16(rng.normal(size=(tokens, HIDDEN))) if with_x else None
    r["stream1"] = st.bf16(r["x"] + r["stream0"]) if with_x else r["stream0"]
    r["a"] = code(o.norm(r["stream1"], w["n1"]))
    r["fused"] = st.bf16(r["a"][0] @ w["qkv"].T).reshape(tokens, -1, DIM)
    q, k, r["v"] = r["fused"][:, :HEADS], r["fused"][:, HEADS:HEADS + KV], r["fused"][:, HEADS + KV:]
    r["q"], r["k"] = (st.bf16(o.rope(x, r["pos"], r["inv_freq"])) for x in (q, k))
    empty = (np.zeros((3, KV, PAGE, DIM), np.uint8), np.zeros((3, KV, DIM, PAGE), np.uint8), np.zeros((3, KV), np.uint8),
             np.zeros((3, KV), np.uint8))
    r["cache_before"], r["cache"] = kv_reference.Cache(*empty), kv_reference.Cache(*empty)
    kv_reference.append(r["cache"], r["k"], r["v"], r["cu"], r["context"], r["table"], True)
    r["o"] = st.bf16(o.attention(r["q"], r["cache"], r["cu"], r["context"], r["table"], DIM ** -0.5)[0])
    r["o_q"] = code(r["o"].reshape(tokens, -1))
    r["x2"] = st.bf16(r["o_q"][0] @ w["out"].T)
    r["stream2"] = st.bf16(r["x2"] + r["stream1"])
    r["b"] = code(o.norm(r["stream2"], w["n2"]))
    gu = r["b"][0] @ w["gate_up"].T
    r["h"] = code(o.gated(gu[:, :FF], gu[:, FF:]))
    r["y"] = st.bf16(r["h"][0] @ w["down"].T)
    return r


class NoWeight(st.Oracle):
    def norm(self, s, w):
        return ref.rmsnorm(s, 1.0, 1e-5)


class NoRope(st.Oracle):
    def rope(self, x, pos, inv_freq):
        return x


class OtherFrequencies(st.Oracle):
    def rope(self, x, pos, inv_freq):
        return ref.rope(x, pos, inv_freq * 0.9, False)


class OtherPairs(st.Oracle):
    def rope(self, x, pos, inv_freq):
        return ref.rope(x, pos, inv_freq, True)


class NoMask(st.Oracle):
    def attention(self, q, cache, cu, context, table, scale):
        return kv_reference.attention(q, cache, cu, context, table, scale, False, 0)


class Average(st.Oracle):
    def attention(self, q, cache, cu, context, table, scale):
        return kv_reference.attention(0 * q, cache, cu, context, table, scale, True, 0)


class Swapped(st.Oracle):
    def gated(self, g, u):
        return ref.act(u, 0) * g


class NoActivation(st.Oracle):
    def gated(self, g, u):
        return g * u


class NoResidual(st.Oracle):
    def stream(self, x, r):
        return x


MISTAKES = [(NoWeight, "first norm"), (NoRope, "rope of q"), (OtherFrequencies, "rope of q"), (OtherPairs, "rope of q"),
            (NoMask, "attention"), (Average, "attention"), (Swapped, "gated"), (NoActivation, "gated"), (NoResidual, "stream")]


@pytest.mark.parametrize("with_x", [False, True])
def test_the_chain_passes(with_x):
    rng = np.random.default_rng(1)
    w = weights(rng)
    st.check(chain(rng, w, with_x), w)


@pytest.mark.parametrize("mistake,where", MISTAKES, ids=[m.__name__ for m, _ in MISTAKES])
def test_a_mistake_is_noticed(mistake, where):
    rng = np.random.default_rng(2)
    w = weights(rng)
    with pytest.raises(AssertionError, match=where):
        st.check(chain(rng, w, True), w, mistake())


@pytest.mark.parametrize("name,where", [("qkv", "q, k, v"), ("out", "output product"), ("n2", "second norm"), ("gate_up", "gated"),
                                        ("down", "down product")])
def test_another_weight_is_noticed(name, where):
    rng = np.random.default_rng(3)
    w = weights(rng)
    r = chain(rng, w, True)
    with pytest.raises(AssertionError, match=where):
        st.check(r, {**w, name: w[name][::-1]})
