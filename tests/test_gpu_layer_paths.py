"""GPU tests of the variants that the calls between a layer's products choose by size, type and rounding: large calls past
the caches, many rows, wide rows, wide blocks of columns, coded outputs of every kernel. Against 64-bit forms on the
device, codes against fp4_quantize bit for bit. E24 = 2^-24 is half a step of fp32 relative to a value."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: E24}
DTYPES = [torch.bfloat16, torch.float32]


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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, size=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(size).to(dtype)


def near(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def params(fp4, elem, hn, ceil, sr, seed=5):
    return fp4.Params(elem=elem, hadamard_n=hn, scale_mode=fp4.SCALE_E8M0_CEIL if ceil else fp4.SCALE_E8M0_FLOOR,
                      round_mode=fp4.ROUND_SR if sr else fp4.ROUND_RNE, seed=seed)


def same_codes(q, want):
    assert (q.rows, q.cols, q.params) == (want.rows, want.cols, want.params)
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)


# ---- norm ----

# A row's sum runs through at most 8 * 8 additions in a lane, 6 across a wave and 8 across waves.
DEPTH = 80
# More rows than 4 a CU (workgroups that go through several, the last ones not all there), one to eight pieces a lane,
# rows that share a wave and rows that span eight; 6200 x 4096 reads past the caches.
MANY = [(2500, 64), (5003, 256), (9001, 1000), (1300, 4096), (1100, 5120), (1025, 9000), (1200, 14336), (1100, 20480),
        (1030, 32768), (6200, 4096)]


def norm64(s, w, eps):
    s = s.double()
    return s * torch.rsqrt(s.square().mean(1, keepdim=True) + eps) * w.double()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", MANY)
def test_norm_of_many_rows(layer, rows, cols, dtype):
    g = gen(rows + cols)
    x, r = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, size=3.0, dtype=dtype)
    w = rand(g, cols, dtype=torch.bfloat16 if rows & 1 else torch.float32)
    for res in (None, r):
        got = layer.rmsnorm(x, w, eps=0.125, residual=res)
        s = x if res is None else (x.float() + res.float()).to(dtype)
        assert res is None or torch.equal(got.sum, s)
        want = norm64(s, w, 0.125)
        # 1 / sqrt: half the sum's error; the mean, eps, root, quotient and two products round once each
        near(got.y, want, want.abs() * ((DEPTH / 2 + 6) * E24 + HALF_STEP[dtype]), "y")
    a, b = x.clone(), r.clone()
    inside = layer.rmsnorm(a, w, eps=0.125, residual=b, sum_out=a, out=torch.empty_like(x))
    assert inside.sum is a and torch.equal(a, got.sum) and torch.equal(inside.y, got.y) and torch.equal(b, r)
    layer.rmsnorm(a.copy_(x), w, eps=0.125, residual=b, sum_out=b)
    assert torch.equal(b, got.sum)
    y = layer.rmsnorm(x, w, eps=0.125).y
    layer.rmsnorm(a.copy_(x), w, eps=0.125, out=a)
    assert torch.equal(a, y)


@pytest.mark.parametrize("elem,hn,ceil,sr", [(1, 128, 1, 0), (0, 32, 0, 0), (0, 128, 1, 1), (1, 0, 0, 1)])
@pytest.mark.parametrize("rows,cols", [(2500, 128), (5003, 256), (1300, 4096), (1100, 5120), (1200, 14336), (1100, 20480),
                                       (1030, 32768), (6200, 4096)])
def test_norm_codes_of_many_rows(fp4, layer, rows, cols, elem, hn, ceil, sr):
    g = gen(rows + cols)
    x, r, w = rand(g, rows, cols, dtype=torch.bfloat16), rand(g, rows, cols, dtype=torch.bfloat16), rand(g, cols)
    p = params(fp4, elem, hn, ceil, sr)
    full = layer.rmsnorm(x.float(), w, out_q=p)  # the output before it is rounded: fp32 in, fp32 out
    same_codes(full.q, fp4.quantize(full.y, p))
    got = layer.rmsnorm(x, w, out_q=p)
    same_codes(got.q, full.q)
    assert torch.equal(got.y, full.y.bfloat16())
    res = layer.rmsnorm(x, w, residual=r, out_q=p, keep_y=False)
    assert res.y is None and torch.equal(res.sum, (x.float() + r.float()).bfloat16())
    full = layer.rmsnorm(res.sum.float(), w, out_q=p)
    same_codes(res.q, full.q)
    layer.rmsnorm(x, w, residual=r, sum_out=x, out_q=p, keep_y=False, q_out=got.q)
    assert torch.equal(x, res.sum)
    same_codes(got.q, full.q)
    # in fp32 with a residual: its own instances
    x32, r32 = x.float(), r.float()
    res = layer.rmsnorm(x32, w, residual=r32, out_q=p)
    same_codes(res.q, fp4.quantize(res.y, p))
    assert torch.equal(res.sum, x32 + r32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(5, 20480), (300, 24576), (1200, 14336), (1100, 20480), (700, 32768), (2, 26000), (6200, 4096)])
def test_norm_backward_of_wide_rows(layer, rows, cols, dtype):
    """Rows that nearly fill the registers, and a call past the caches; in place of both gradients too."""
    g = gen(rows * 3 + cols)
    s, dy, ds = (rand(g, rows, cols, size=z, dtype=dtype) for z in (2.0, 0.3, 0.5))
    w = rand(g, cols, dtype=torch.bfloat16 if rows & 1 else torch.float32)
    dx, dw = layer.rmsnorm_backward(dy, s, w, eps=0.25, dsum=ds)
    s64, dy64, ds64 = s.double(), dy.double(), ds.double()
    r = torch.rsqrt(s64.square().mean(1, keepdim=True) + 0.25)
    n, a = s64 * r, dy64 * w.double()
    want = ds64 + r * (a - n * (a * n).mean(1, keepdim=True))
    # both sums DEPTH roundings of their magnitudes, the root another half; a few for the rest
    tol = (2 * DEPTH + 16) * E24 * (ds64.abs() + r * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)))
    near(dx, want, tol + HALF_STEP[dtype] * want.abs(), "dx")
    # a column's terms: n (half the sum's depth and 5), a product; the rows of a workgroup one after another, 3 steps
    # across a wave's rows, 7 across its waves, then at most 256 parts in 128 runs of 2, two steps and 32 runs
    depth = DEPTH / 2 + 6 + math.ceil(rows / 256) + 3 + 7 + 2 + 2 + 32
    near(dw, (dy64 * n).sum(0), depth * E24 * (dy64 * n).abs().sum(0), "dw")
    for out in (0, 1):
        t = dy.clone(), ds.clone()
        x2, w2 = layer.rmsnorm_backward(t[0], s, w, eps=0.25, dsum=t[1], out=t[out])
        assert torch.equal(x2, dx) and torch.equal(w2, dw)
    x2, _ = layer.rmsnorm_backward(dy, s, w, eps=0.25, dweight=False)
    near(x2, want - ds64, tol + HALF_STEP[dtype] * (want - ds64).abs(), "dx without a stream")


# ---- rotary positions ----

def rope64(x, pos, f, interleaved, backward=False):
    """The rotation by the fp64 products of position and frequency, and the magnitude |x1| + |x2| of each place."""
    n = f.numel()
    t = pos.double()[:, None, None] * f
    c, s = t.cos(), -t.sin() if backward else t.sin()
    x = x.double()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    y = (a * c - b * s, b * c + a * s)
    size = a.abs() + b.abs()
    join = (lambda u, v: torch.stack([u, v], -1).flatten(-2)) if interleaved else (lambda u, v: torch.cat([u, v], -1))
    return torch.cat([join(*y), x[..., 2 * n:]], -1), torch.cat([join(size, size), torch.zeros_like(x[..., 2 * n:])], -1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_frequencies_above_one(layer, interleaved):
    """Angles of many turns: positions to 2^31 - 1, frequencies from 2^-20 to 2^13. Sine and cosine 2^-22, two products
    and a sum."""
    f = torch.logspace(-20, 13, 32, base=2.0, dtype=torch.float64) * math.sqrt(0.9)
    pos = torch.tensor([0, 1, 3, 1000, 131071, 10 ** 8, 2 ** 30 + 7, 2 ** 31 - 1, -5, -2 ** 31], dtype=torch.int32)
    x = rand(gen(1), 10, 3, 64)
    rotary = layer.Rotary(f.cuda(), layout=layer.INTERLEAVED if interleaved else layer.HALF)
    for backward in (False, True):
        want, size = rope64(x.cpu(), pos, f, interleaved, backward)
        near(layer.rope(x, rotary, pos.cuda(), backward=backward).cpu(), want, size * (2.0 ** -22 + 3 * E24), "rope")


# ---- gated products ----

def operands(fp4, g, m, f, k, elem, tile=False, size=1.5):
    a, wg, wu = rand(g, m, k), rand(g, f, k, size=size / math.sqrt(k)), rand(g, f, k, size=1.0 / math.sqrt(k))
    pa, pw = fp4.Params(elem=elem), fp4.Params(elem=elem, block=(32, 32) if tile else (1, 32))
    return fp4.quantize(a, pa), fp4.quantize(wg, pw), fp4.quantize(wu, pw)


def act64(g, act):
    """Without cancellation in either tail."""
    if act == 0:
        return g * torch.sigmoid(g)
    if act == 1:
        return g * 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
    return g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))


def act_bound(g, act):
    """Half steps of the activation and of its product with u: 17 at most for the first two (5 of them |g|^2's share of
    the exponent's at 13), 11 and 4 of tanh's argument for the third; values below |g| 2^-125 may vanish."""
    v = act64(g, act).abs()
    return ((4.1 * 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3).abs().clamp(max=104.0) if act == 2 else 0.0) + 23.0) * E24 * v \
        + g.abs() * 2.0 ** -125


def check_products(fp4, aq, gq, uq, act, got, dtype):
    """g and u against the products of what the codes stand for; h against the activation of the g and u that were kept
    (in fp32: exactly those of the accumulators; bf16: half a step of each more, the activation's slope at most 1.13)."""
    f = gq.rows
    a, wg, wu = (fp4.dequantize(q).double() for q in (aq, gq, uq))
    # sums of fp32 products; blocks of 8 products lose up to 8 * 2^-13 of their largest on the FP8 matrix core
    part = 1e-5 + (2.0 ** -10 if aq.params.elem == fp4.E4M3 else 0.0)
    half = HALF_STEP[dtype]
    for y, b, name in ((got.gu[:, :f], wg, "g"), (got.gu[:, f:], wu, "u")):
        want, tol = a @ b.T, part * (a.abs() @ b.abs().T)
        near(y, want, tol + half * (want.abs() + tol), name)
    g, u = got.gu[:, :f].double(), got.gu[:, f:].double()
    h = act64(g, act) * u
    tol = act_bound(g, act) * u.abs() + half * h.abs()
    if dtype is torch.bfloat16:
        tol = 1.01 * (tol + half * (1.13 * g.abs() * u.abs() + h.abs()))
    near(got.h, h, tol, "h")


@pytest.mark.parametrize("m,f", [(33, 9216), (48, 11000), (60, 9300), (64, 12288), (40, 12320), (64, 21504)])
def test_gated_wide_blocks_of_columns(fp4, layer, m, f):
    """33 to 64 rows in 8 bits and long K: blocks of 48 columns where they fill the rounds that they take, others beside
    them."""
    aq, gq, uq = operands(fp4, gen(m), m, f, 4096, fp4.E4M3)
    for act, dtype in ((0, torch.float32), (1, torch.bfloat16)):
        w = layer.GatedWeights(gq, uq, act=act)
        assert layer.gated_plan(m, w, dtype).kernel == layer.PLAN_STREAM
        check_products(fp4, aq, gq, uq, act, layer.gated(aq, w, out_dtype=dtype, keep_gu=True), dtype)


def plan_name(layer, plan):
    return next(n for n in dir(layer) if n.startswith("PLAN_") and getattr(layer, n) == plan)


# every kernel, by its plan: few rows of any K, streams, the three kinds of 128-row tiles, 256-row tiles
CODED = [("PLAN_ROWS", 1, 128, 96), ("PLAN_ROWS", 20, 160, 160), ("PLAN_ROWS", 32, 128, 1120), ("PLAN_STREAM", 3, 128, 384),
         ("PLAN_STREAM", 60, 256, 1024), ("PLAN_STREAM", 130, 1408, 512), ("PLAN_TILE128", 200, 11008, 256), ("PLAN_TILE128_DEEP", 90, 6016, 384),
         ("PLAN_TILE128_RAGGED", 33, 128, 96), ("PLAN_TILE128_RAGGED", 150, 640, 288), ("PLAN_TILE256", 1030, 3328, 384)]


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("kind", ["e2m1", "tile", "e4m3"])
@pytest.mark.parametrize("plan,m,f,k", CODED)
def test_gated_codes_of_every_kernel(fp4, layer, plan, m, f, k, kind, act):
    """Weights in groups and in 32 x 32 tiles, the three activations: codes of the fp32 output as fp4_quantize makes them,
    whatever else is stored."""
    aq, gq, uq = operands(fp4, gen(m + f), m, f, k, fp4.E4M3 if kind == "e4m3" else fp4.E2M1, kind == "tile")
    w = layer.GatedWeights(gq, uq, act=act)
    assert plan_name(layer, layer.gated_plan(m, w).kernel) == plan
    for elem, hn, ceil, sr in ((0, 0, 0, 0), (1, 32, 1, 0), (1, 128, 1, 0), (0, 64, 0, 0), (0, 16, 1, 1)):
        if f % max(hn, 1):
            continue
        p = params(fp4, elem, hn, ceil, sr, seed=m * 7 + f)
        full = layer.gated(aq, w, out_dtype=torch.float32, out_q=p, keep_gu=True)
        check_products(fp4, aq, gq, uq, act, full, torch.float32)
        same_codes(full.q, fp4.quantize(full.h, p))
        got = layer.gated(aq, w, out_q=p, keep_gu=True)
        same_codes(got.q, full.q)
        assert torch.equal(got.h, full.h.bfloat16()) and torch.equal(got.gu, full.gu.bfloat16())
        only = layer.gated(aq, w, out_q=p, keep_h=False, q_out=fp4.empty_qtensor(m, f, p, "cuda"))
        assert only.h is None and only.gu is None
        same_codes(only.q, full.q)


# ---- calls larger than the caches ----

@pytest.mark.parametrize("elem,tile", [(0, False), (0, True), (1, False)])
@pytest.mark.parametrize("dtype,m", [(torch.bfloat16, 4096), (torch.float32, 2111)])
def test_gated_past_the_caches(fp4, layer, dtype, m, elem, tile):
    """h of 64 MiB and more: stored past the caches, the same bits as those of fewer rows."""
    f, k, few = 8448, 256, 1024
    assert m * f * (2 if dtype is torch.bfloat16 else 4) >= 64 << 20 > few * f * 4
    aq, gq, uq = operands(fp4, gen(m), m, f, k, elem, tile)
    w = layer.GatedWeights(gq, uq)
    assert layer.gated_plan(m, w).kernel == layer.gated_plan(few, w).kernel == layer.PLAN_TILE256
    got = layer.gated(aq, w, out_dtype=dtype, keep_gu=True)
    check_products(fp4, aq, gq, uq, 0, got, dtype)
    cb, sb = aq.codes.numel() // m, aq.scales.numel() // m
    head = fp4.QTensor(aq.codes[:few * cb], aq.scales[:few * sb], None, few, k, aq.params)
    part = layer.gated(head, w, out_dtype=dtype, keep_gu=True)
    assert torch.equal(got.h[:few], part.h) and torch.equal(got.gu[:few], part.gu)
    assert torch.equal(layer.gated(aq, w, out_dtype=dtype).h, got.h)
    p = params(fp4, 1, 128, 1, 0)
    coded = layer.gated(aq, w, out_dtype=dtype, out_q=p)
    assert torch.equal(coded.h, got.h)
    same_codes(coded.q, fp4.quantize(layer.gated(aq, w, out_dtype=torch.float32).h, p))


def slope64(g, act):
    """The slope and the sum of its terms' magnitudes, without cancellation, and the exponent."""
    if act == 1:
        p, rest, z = 0.5 * torch.special.erfc(-g * math.sqrt(0.5)), g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi), 0.05 * g * g
    else:
        a, b = (1.0, 0.0) if act == 0 else (2.0 * math.sqrt(2.0 / math.pi), 2.0 * math.sqrt(2.0 / math.pi) * 0.044715)
        z = g * (a + b * g * g)
        p, rest = torch.sigmoid(z), g * torch.sigmoid(z) * torch.sigmoid(-z) * (a + 3.0 * b * g * g)
        z = (0.1 if act == 0 else 8.1) * z.abs()
    return p + rest, p + rest.abs(), z


@pytest.mark.parametrize("act", [0, 1, 2])
def test_gated_backward_past_the_caches(fp4, layer, act):
    """96 MiB and more of bf16: read and stored past the caches, kept, in place and coded; the same bits as fewer rows."""
    rows, f, few = 1601, 11008, 130
    assert rows * f * 6 >= 96 << 20 > few * f * 6
    g = gen(rows)
    dh, gu = rand(g, rows, f, dtype=torch.bfloat16), rand(g, rows, 2 * f, size=3.0, dtype=torch.bfloat16)
    got = layer.gated_backward(dh, gu, act=act)
    d, gv, uv = dh.double(), gu[:, :f].double(), gu[:, f:].double()
    half = HALF_STEP[torch.bfloat16]
    slope, size, z = slope64(gv, act)
    # where p is below 2^-126 it may vanish, and with it p (1 + |g| z'): z' is at most 1 + |g| + g^2, so that the factor
    # is below (1 + |g|)^3 (at -10 the third activation's slope is 2e-36 and p 1e-38)
    tol = ((26.0 + z.clamp(max=900.0)) * E24 * size + (1.0 + gv.abs()) ** 3 * 2.0 ** -125) * (d * uv).abs()
    near(got.dgu[:, :f], d * uv * slope, tol + half * (d * uv * slope).abs() + 1e-36, "dg")
    v = d * act64(gv, act)
    near(got.dgu[:, f:], v, act_bound(gv, act) * d.abs() + half * v.abs() + 1e-36, "du")
    part = layer.gated_backward(dh[:few], gu[:few], act=act)
    assert torch.equal(got.dgu[:few], part.dgu)
    for elem, hn, ceil, sr in ((1, 128, 1, 0), (0, 256, 0, 1)):
        p = params(fp4, elem, hn, ceil, sr)
        full = layer.gated_backward(dh.float(), gu.float(), act=act, out_q=p)
        same_codes(full.q, fp4.quantize(full.dgu, p))
        coded = layer.gated_backward(dh, gu, act=act, out_q=p)
        same_codes(coded.q, full.q)
        assert torch.equal(coded.dgu, got.dgu)
        same_codes(layer.gated_backward(dh, gu, act=act, out_q=p, keep=False).q, full.q)
    same = gu.clone()
    assert torch.equal(layer.gated_backward(dh, same, act=act, out=same).dgu, got.dgu)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,tokens,dim,rot", [(torch.bfloat16, 7001, 128, 128), (torch.float32, 3501, 128, 64),
                                                  (torch.bfloat16, 4801, 192, 128), (torch.bfloat16, 11201, 80, 80)])
def test_rope_past_the_caches(layer, dtype, tokens, dim, rot, interleaved):
    """64 MiB and more, in whole cache lines and not: pairs, in place, the same bits as few tokens."""
    hq, hk = 32, 8
    assert tokens * (hq + hk) * dim * (2 if dtype is torch.bfloat16 else 4) >= 64 << 20
    g = gen(tokens)
    fused = rand(g, tokens, hq + 2 * hk, dim, dtype=dtype)
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    f = layer.rotary_frequencies(rot)[0]
    rotary = layer.Rotary(f.cuda(), layout=layer.INTERLEAVED if interleaved else layer.HALF)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") * 100
    for backward in (False, True):
        got = layer.rope((q, k), rotary, pos, backward=backward)
        for x, y in zip((q, k), got):
            want, size = rope64(x, pos, f.cuda(), interleaved, backward)
            near(y, want, size * (2.0 ** -22 + 3 * E24 + HALF_STEP[dtype]), "rope")
            assert torch.equal(y[..., rot:], x[..., rot:])
        few = layer.rope((q[-31:], k[-31:]), rotary, pos[-31:], backward=backward)
        assert torch.equal(got[0][-31:], few[0]) and torch.equal(got[1][-31:], few[1])
    a = fused.clone()
    layer.rope((a[:, :hq], a[:, hq:hq + hk]), rotary, pos, out=(a[:, :hq], a[:, hq:hq + hk]), backward=True)
    assert torch.equal(a[:, :hq], got[0]) and torch.equal(a[:, hq:hq + hk], got[1]) and torch.equal(a[:, hq + hk:], fused[:, hq + hk:])
