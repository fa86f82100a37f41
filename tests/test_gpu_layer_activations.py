"""GPU tests of the gated feed-forward's activations and their slopes by the result's own size, not by their argument's.

Bounds are counted in E24 = 2^-24, half a step of fp32 relative to the value; the hardware's exponential and reciprocal
are off by an ulp, 2 E24 at most.
- e^-y: exponential 2, its correction 1, and 1.4427 y times the 2^-29 by which ln 2 in fp32 is off: 0.05 y. With
  e <= 1 the sum 1 + e is off by 1 + 3 / 2, its reciprocal by 2 more, and s, e times that, by 3 + 1: 8.5 at most, g s
  by 9.5: VALUE = 10, + 0.05 |z|. 1 - s is off by less: the exponential's 3 enter s = e / (1 + e) by their share 1 / (1 +
  e) alone, which leaves 4 + 1.5 where s is 1 / 2 and less of 1 - s where it is smaller, and a rounding.
- the tanh form's argument z = g (A + B g^2) is off by 4 roundings (square, constants, sum, product), which p passes on
  times |z| (its derivative is p (1 - p) z relative to p): + 4 |z|.
- slopes are p + g p (1 - p) z'(g): each term's factors and products, of the sum of the terms' magnitudes: 2 * 8.5, four
  products and sums, and for tanh the argument's error in both p and 1 - p and 3 roundings in z': SLOPE = 24, + twice
  the value's share of |z|.
- Phi(-a) = e^(-a^2/2) s P(s), a >= 1: exponential 2, its two corrections 1 each; s off by 3 (sum, reciprocal), which
  s P(s) passes on up to 2.1 times, and the polynomial's roundings of constants and sums up to 3.4, together 9.7 at most
  (running error of the eight steps); the fit 0.2, two products 2; with g's product 17, + 0.05 a^2 / 2. Below 1 the sum
  1 / 2 + g R is off by 2.8 of g R, which is at most 0.34, and a rounding of itself, at least 0.16: 7, with g's product
  8. TAIL = 17; for positive g less. Slope: Phi and g e^(-a^2/2) / sqrt(2 pi), which SLOPE covers both.
Values below 2^-126 / (1 - p) may vanish: |g| 2^-125."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
VALUE, TAIL, SLOPE = 10.0, 17.0, 24.0
PER_Z = {0: 0.05, 1: 0.05, 2: 4.05}  # of the exponent
A, B = 2.0 * math.sqrt(2.0 / math.pi), 2.0 * math.sqrt(2.0 / math.pi) * 0.044715
SILU, GELU, TANH = 0, 1, 2
erfc = np.vectorize(math.erfc, otypes=[float])


@pytest.fixture(scope="module")
def fp4():
    from bit_gemm_fwht_amd import fp4 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def layer():
    from bit_gemm_fwht_amd import layer as m
    m.lib()
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def exact(g, act):
    """Value, slope, the sum of the slope's terms' magnitudes and the exponent, in 64 bits without
    cancellation."""
    if act == GELU:
        p = 0.5 * erfc(-g / math.sqrt(2.0))
        rest = g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        return g * p, p + rest, p + np.abs(rest), 0.5 * g * g
    with np.errstate(over="ignore"):
        z = g if act == SILU else g * (A + B * g * g)
        dz = 1.0 if act == SILU else A + 3.0 * B * g * g
        p, q = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
    rest = g * p * q * dz
    return g * p, p + rest, p + np.abs(rest), np.abs(z)


def value_bound(g, act):
    v, _, _, z = exact(g, act)
    return ((TAIL if act == GELU else VALUE) + PER_Z[act] * np.minimum(z, 104.0)) * E24 * np.abs(v) + np.abs(g) * 2.0 ** -125


def slope_bound(g, act):
    _, _, size, z = exact(g, act)
    return (SLOPE + 2.0 * PER_Z[act] * np.minimum(z, 104.0)) * E24 * size + (1.0 + np.abs(g)) ** 3 * 2.0 ** -125


def arguments():
    g = np.concatenate([np.linspace(-104.0, -3.0, 60000), np.linspace(-3.0, 3.0, 60000), np.linspace(3.0, 104.0, 30000),
                        -np.logspace(-30, 0, 2500), np.logspace(-30, 0, 2500)]).astype(np.float32)
    return g[:g.size // 8 * 8]


def within(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(err / np.maximum(tol, 1e-300)).max():.3g} of the bound"


@pytest.mark.parametrize("act", [SILU, GELU, TANH])
def test_value_and_slope(layer, act):
    """dh = u = 1: the gradients are the slope and the value themselves."""
    g = arguments()
    t = torch.from_numpy(g).cuda()
    d = f64(layer.gated_backward(torch.ones(1, g.size, device="cuda"), torch.cat([t, torch.ones_like(t)])[None], act=act).dgu)[0]
    g = g.astype(np.float64)
    v, s, _, _ = exact(g, act)
    within(d[g.size:], v, value_bound(g, act), "value")
    within(d[:g.size], s, slope_bound(g, act), "slope")


def wide_operands(fp4, seed, m, f, k, elem):
    """Products that reach far into both tails, the up projection's about 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, wg, wu = (torch.randn(*s, generator=g, device="cuda") for s in ((m, k), (f, k), (f, k)))
    p = fp4.Params(elem=elem)
    return fp4.quantize(a, p), fp4.quantize(wg * (8.0 / math.sqrt(k)), p), fp4.quantize(wu / math.sqrt(k), p)


# every kernel by its plan, of both element types
KERNELS = [("PLAN_ROWS", 5, 96, 96), ("PLAN_STREAM", 3, 96, 512), ("PLAN_STREAM", 40, 9600, 256), ("PLAN_STREAM", 130, 1376, 512),
           ("PLAN_TILE128", 200, 11008, 256), ("PLAN_TILE128_DEEP", 90, 6016, 256), ("PLAN_TILE128_RAGGED", 150, 512, 288),
           ("PLAN_TILE256", 1100, 3328, 256)]


@pytest.mark.parametrize("act", [SILU, GELU, TANH])
@pytest.mark.parametrize("plan,m,f,k", KERNELS)
def test_forward_in_every_kernel(fp4, layer, plan, m, f, k, act):
    """h against act(g) u of the g and u that the call itself kept in fp32."""
    for elem in (fp4.E2M1, fp4.E4M3):
        aq, gq, uq = wide_operands(fp4, m + f, m, f, k, elem)
        w = layer.GatedWeights(gq, uq, act=act)
        assert layer.gated_plan(m, w, torch.float32).kernel == getattr(layer, plan)
        got = layer.gated(aq, w, out_dtype=torch.float32, keep_gu=True)
        g, u = f64(got.gu)[:, :f], f64(got.gu)[:, f:]
        assert g.min() < -15.0 and g.max() > 15.0
        v = exact(g, act)[0]
        within(f64(got.h), v * u, value_bound(g, act) * np.abs(u) * (1 + E24) + E24 * np.abs(v * u), "h")
