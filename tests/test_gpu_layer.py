"""GPU tests of the operators between a layer's products (norm, rotary positions, gated feed-forward and their
backward passes) against plain 64-bit forms; low-bit outputs against fp4_quantize bit for bit.

Tolerances are counted in fp32 roundings (2^-24 of a value each, E24) and one rounding to the output's type
(half a step: 2^-8 for bf16, 2^-24 for fp32). A row's sum of n terms runs through at most 8 * 8 additions in a
lane and 6 + 8 across lanes and waves, so with the products' own roundings it is off by at most DEPTH E24 of
the sum of magnitudes."""
import math

import numpy as np
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
DEPTH = 80
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def fp4():
    from bit_gemm_fwht_amd import fp4 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def kv():
    from bit_gemm_fwht_amd import kv as m
    return m


@pytest.fixture(scope="module")
def layer():
    from bit_gemm_fwht_amd import layer as m
    m.lib()
    return m


def rand(g, *shape, size=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, tol, what=""):
    err = np.abs(f64(got) - want)
    assert err.shape == np.broadcast_shapes(err.shape, np.shape(tol))
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the bound"


def pitched(t, extra):
    """The same values in rows `extra` elements further apart."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), 7.0, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


# ---- norm ----

NORM_SHAPES = [(1, 8), (3, 24), (5, 64), (2, 96), (130, 128), (7, 160), (33, 256), (4, 520), (9, 1000), (3, 2048), (5, 4096),
               (2, 4104), (3, 5120), (2, 11008), (1, 16384), (2, 32768)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm(layer, rows, cols, dtype):
    g = gen(rows * 7 + cols)
    x, r = rand(g, rows, cols, dtype=dtype), rand(g, rows, cols, size=3.0, dtype=dtype)
    w = rand(g, cols, dtype=torch.float32 if rows & 1 else torch.bfloat16)
    for res, weight in ((None, None), (None, w), (r, w), (r, None)):
        eps = 1e-5 if weight is None else 0.125
        got = layer.rmsnorm(x, weight, eps=eps, residual=res)
        s = x if res is None else (x.float() + res.float()).to(dtype)
        if res is None:
            assert got.sum is None
        else:
            assert torch.equal(got.sum, s)
        want = ref.rmsnorm(f64(s), 1.0 if weight is None else f64(weight), eps)
        # 1 / sqrt: half the sum's error; the mean, eps, root, quotient and two products round once each
        within(got.y, want, np.abs(want) * ((DEPTH / 2 + 6) * E24 + HALF_STEP[dtype]), "y")


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_pitches_and_in_place(layer, dtype):
    g = gen(5)
    x, r = rand(g, 13, 1032, dtype=dtype), rand(g, 13, 1032, dtype=dtype)
    w = rand(g, 1032, dtype=dtype)
    want = layer.rmsnorm(x, w, residual=r)
    xp, rp, so, yo = pitched(x, 8), pitched(r, 16), pitched(x, 24), pitched(x, 40)
    got = layer.rmsnorm(xp, w, residual=rp, sum_out=so, out=yo)
    assert torch.equal(got.y, want.y) and torch.equal(got.sum, want.sum)
    assert (so._base[:, 1032:] == 7).all() and (yo._base[:, 1032:] == 7).all()  # nothing outside the rows
    assert torch.equal(xp, x) and torch.equal(rp, r)
    for alias in ("x", "residual"):
        a, b = x.clone(), r.clone()
        got = layer.rmsnorm(a, w, residual=b, sum_out=a if alias == "x" else b)
        assert torch.equal(got.sum, want.sum) and torch.equal(got.y, want.y)
        assert got.sum.data_ptr() == (a if alias == "x" else b).data_ptr()
    a = x.clone()
    plain = layer.rmsnorm(x, w).y
    assert torch.equal(layer.rmsnorm(a, w, out=a).y, plain)


def test_norm_rows_do_not_depend_on_one_another(layer):
    g = gen(6)
    for cols in (64, 1000, 4096):
        x = rand(g, 300, cols)
        whole = layer.rmsnorm(x).y
        for n in (1, 2, 5, 299):
            assert torch.equal(layer.rmsnorm(x[:n]).y, whole[:n])
            assert torch.equal(layer.rmsnorm(x[300 - n:]).y, whole[300 - n:])


def test_norm_of_zeros_and_extremes(layer):
    x = torch.zeros(4, 512, device="cuda")
    x[1] = 1e-30   # squares vanish next to eps
    x[2] = 1e15
    x[3, 3] = -2e18
    y = layer.rmsnorm(x, eps=1e-5).y
    want = ref.rmsnorm(f64(x), 1.0, float(np.float32(1e-5)))
    within(y, want, np.abs(want) * (DEPTH / 2 + 6) * E24 + 1e-44)


Q_MODES = [(e, hn, ceil, sr) for e in (0, 1) for hn in (0, 16, 32, 64, 128, 256) for ceil, sr in ((0, 0), (1, 1))] + \
          [(0, 0, 1, 0), (1, 128, 1, 0), (0, 256, 0, 1)]


def params(fp4, mode, seed=0):
    e, hn, ceil, sr = mode
    return fp4.Params(elem=e, hadamard_n=hn, scale_mode=fp4.SCALE_E8M0_CEIL if ceil else fp4.SCALE_E8M0_FLOOR,
                      round_mode=fp4.ROUND_SR if sr else fp4.ROUND_RNE, seed=seed)


def same_codes(q, want):
    assert (q.rows, q.cols, q.params) == (want.rows, want.cols, want.params)
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)


@pytest.mark.parametrize("mode", Q_MODES)
def test_norm_codes_are_those_of_quantize(fp4, layer, mode):
    for rows, cols in ((1, 256), (37, 512), (5, 1280), (3, 4096), (2, 5120), (3, 11008), (1, 32768)):
        if mode[1] and cols % mode[1]:
            continue
        g = gen(cols + mode[1])
        x, r, w = rand(g, rows, cols, dtype=torch.bfloat16), rand(g, rows, cols, dtype=torch.bfloat16), rand(g, cols)
        x[:, 32:96] = 0  # whole groups of zeros without the residual
        p = params(fp4, mode, seed=rows * 77777 + 3)
        # the output before it is rounded: fp32 in, fp32 out, of the same rows
        full = layer.rmsnorm(x.float(), w, out_q=p)
        same_codes(full.q, fp4.quantize(full.y, p))
        got = layer.rmsnorm(x, w, out_q=p)
        same_codes(got.q, full.q)
        assert torch.equal(got.y, full.y.bfloat16())
        only = layer.rmsnorm(x, w, out_q=p, keep_y=False, q_out=fp4.empty_qtensor(rows, cols, p, "cuda"))
        assert only.y is None
        same_codes(only.q, full.q)
        res = layer.rmsnorm(x, w, residual=r, out_q=p)
        same_codes(res.q, layer.rmsnorm(res.sum.float(), w, out_q=p).q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(700, 64), (2500, 256), (1300, 4096)])
def test_norm_backward(layer, rows, cols, dtype):
    g = gen(rows * 3 + cols)
    s, dy, ds = (rand(g, rows, cols, size=z, dtype=dtype) for z in (2.0, 0.3, 0.5))
    w = rand(g, cols, dtype=torch.bfloat16 if rows & 1 else torch.float32)
    for weight, stream in ((None, None), (w, ds)):
        eps = 1e-5 if weight is None else 0.25
        dx, dw = layer.rmsnorm_backward(dy, s, weight, eps=eps, dsum=stream)
        w64, d64 = 1.0 if weight is None else f64(weight), 0.0 if stream is None else f64(stream)
        want, want_w = ref.rmsnorm_grad(f64(dy), f64(s), w64, eps, d64)
        r = 1.0 / np.sqrt((f64(s) ** 2).mean(1, keepdims=True) + eps)
        n, a = f64(s) * r, f64(dy) * w64
        # both sums DEPTH roundings of their magnitudes, the root another half; a few for the rest
        tol = (2 * DEPTH + 16) * E24 * (np.abs(d64) + r * (np.abs(a) + np.abs(n) * np.abs(a * n).mean(1, keepdims=True)))
        within(dx, want, tol + HALF_STEP[dtype] * np.abs(want), "dx")
        # a column's rows: at most rows / 512 + 4 in a workgroup's register, 3 across a wave's rows, then its slots
        depth = rows / 512 + 4 + 3 + 4096 / 64 + 64 + DEPTH
        within(dw, want_w, depth * E24 * np.abs(f64(dy) * n).sum(0), "dw")


def test_norm_backward_against_differences(layer):
    """dL = <dx, d> + <dw, e> for L = sum c y, by central differences of the 64-bit form."""
    rng = np.random.default_rng(1)
    s, w, c = rng.normal(size=(6, 200)) * 2, rng.normal(size=200), rng.normal(size=(6, 200))
    dx, dw = layer.rmsnorm_backward(*(torch.tensor(v, dtype=torch.float32, device="cuda") for v in (c, s, w)), eps=0.1)
    h = 1e-5
    for _ in range(8):
        d, e = rng.normal(size=s.shape), rng.normal(size=w.shape)
        num = ((c * ref.rmsnorm(s + h * d, w + h * e, 0.1)).sum() - (c * ref.rmsnorm(s - h * d, w - h * e, 0.1)).sum()) / (2 * h)
        ana = (f64(dx) * d).sum() + (f64(dw) * e).sum()
        # inputs rounded to fp32 (2^-24 of each) and the kernel's own few hundred roundings, over 1400 terms of order 1
        assert abs(num - ana) <= 400 * E24 * (np.abs(f64(dx) * d).sum() + np.abs(f64(dw) * e).sum())


def test_norm_backward_without_eps(layer):
    """Rows that do not fill the last workgroup add nothing to the weight's gradient, whatever 1 / 0 makes of them."""
    for rows, cols in ((5, 64), (1, 8), (130, 128), (3, 520)):
        s, dy = rand(gen(rows), rows, cols), rand(gen(cols), rows, cols)
        dx, dw = layer.rmsnorm_backward(dy, s, eps=0.0)
        want, want_w = ref.rmsnorm_grad(f64(dy), f64(s), 1.0, 0.0)
        n = f64(s) / np.sqrt((f64(s) ** 2).mean(1, keepdims=True))
        within(dx, want, (2 * DEPTH + 16) * E24 * (np.abs(f64(dy)) + np.abs(n) * np.abs(f64(dy) * n).mean(1, keepdims=True)) / np.abs(f64(s) / n))
        within(dw, want_w, (4 + 3 + 128 + DEPTH) * E24 * np.abs(f64(dy) * n).sum(0))


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_backward_in_place_and_pitches(layer, dtype):
    g = gen(9)
    s, dy, ds = (rand(g, 21, 776, dtype=dtype) for _ in range(3))
    w = rand(g, 776)
    dx, dw = layer.rmsnorm_backward(dy, s, w, dsum=ds)
    for out in ("dy", "dsum"):
        a, b = dy.clone(), ds.clone()
        x2, w2 = layer.rmsnorm_backward(a, s, w, dsum=b, out=a if out == "dy" else b)
        assert torch.equal(x2, dx) and torch.equal(w2, dw)
    o = pitched(s, 8)
    x2, w2 = layer.rmsnorm_backward(pitched(dy, 8), pitched(s, 16), w, dsum=pitched(ds, 32), out=o, dweight=torch.empty(776, device="cuda"))
    assert torch.equal(x2, dx) and torch.equal(w2, dw) and (o._base[:, 776:] == 7).all()
    x2, none = layer.rmsnorm_backward(dy, s, w, dsum=ds, dweight=False)
    assert none is None and torch.equal(x2, dx)


# ---- rotary positions ----

ROPE_DIMS = [(64, 64), (128, 128), (80, 80), (80, 40), (80, 20), (96, 24), (112, 56), (112, 28), (128, 32), (256, 256), (256, 64),
             (16, 2), (8, 8), (1024, 1024), (72, 6)]


def rope_bound(x, scale, dtype, rot, interleaved):
    n = rot // 2
    out = np.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :n], x[..., n:rot])
    both = np.abs(a) + np.abs(b)
    if interleaved:
        out[..., 0:rot:2] = out[..., 1:rot:2] = both
    else:
        out[..., :n] = out[..., n:rot] = both
    return out * scale * (2.0 ** -22 + 3 * E24 + HALF_STEP[dtype])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", ROPE_DIMS)
def test_rope(layer, dim, rot, interleaved):
    g = gen(dim + rot)
    for dtype in DTYPES:
        tokens, hq, hk = 7, 5, 2
        q, k = rand(g, tokens, hq, dim, dtype=dtype), rand(g, tokens, hk, dim, dtype=dtype)
        pos = torch.tensor([0, 1, 2, 131071, 999983, -5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        f, _ = layer.rotary_frequencies(rot, base=10000.0, device="cuda")
        rotary = layer.Rotary(f, layout=layer.INTERLEAVED if interleaved else layer.HALF, scale=1.25)
        for backward in (False, True):
            got = layer.rope((q, k), rotary, pos, backward=backward)
            for x, y in zip((q, k), got):
                want = ref.rope(f64(x), pos.tolist(), f.tolist(), interleaved, 1.25, backward)
                # the fp64 product of a position near 2^31 is off by 2^-22 of a radian
                tol = rope_bound(f64(x), 1.25, dtype, rot, interleaved) * np.where(np.abs(pos.tolist()) > 2 ** 30, 2.0, 1.0)[:, None, None]
                within(y, want, tol)
                assert torch.equal(y[..., rot:], x[..., rot:])
            a = q.clone()
            layer.rope(a, rotary, pos, out=a, backward=backward)  # one tensor, in place
            assert torch.equal(a, got[0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_copies_the_other_channels_bit_for_bit(layer, interleaved):
    """Channels past the turned ones, whatever they hold; large enough for every variant of the accesses."""
    for dtype, dim, rot, tokens in ((torch.bfloat16, 80, 20, 30), (torch.float32, 96, 24, 30), (torch.bfloat16, 128, 64, 20000)):
        x = rand(gen(2), tokens, 20, dim, dtype=dtype)
        x[..., rot] = -0.0
        x[..., rot + 1] = -math.inf
        x[..., rot + 2] = math.nan
        f, _ = layer.rotary_frequencies(rot, device="cuda")
        rotary = layer.Rotary(f, layout=layer.INTERLEAVED if interleaved else layer.HALF)
        pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
        y = layer.rope(x, rotary, pos)
        bits = torch.int16 if dtype is torch.bfloat16 else torch.int32
        assert torch.equal(y[..., rot:].contiguous().view(bits), x[..., rot:].contiguous().view(bits))
        part = layer.rope(x[:29].contiguous(), rotary, pos[:29])
        assert torch.equal(y[:29, :, :rot], part[..., :rot])
        a = x.clone()
        layer.rope(a, rotary, pos, out=a)
        assert torch.equal(a.view(bits), y.view(bits))


@pytest.mark.parametrize("hq,hk", [(40, 8), (37, 5), (9, 1), (255, 0)])
def test_rope_few_tokens_are_those_of_many(layer, hq, hk):
    """Heads are dealt to workgroups by the number of tokens: the values are the same, in place too."""
    f, _ = layer.rotary_frequencies(96, device="cuda")
    x = rand(gen(hq), 2100, hq + hk, 128)
    pos = torch.arange(2100, dtype=torch.int32, device="cuda") * 61
    for layout in (layer.HALF, layer.INTERLEAVED):
        rotary = layer.Rotary(f, layout=layout)
        want = layer.rope(x, rotary, pos)
        for t0, t1 in ((0, 1), (5, 8), (100, 164), (400, 1000)):
            y = x[t0:t1].clone()
            part = (y[:, :hq], y[:, hq:]) if hk else y
            got = layer.rope(part, rotary, pos[t0:t1])
            assert torch.equal(torch.cat(got, 1) if hk else got, want[t0:t1])
            layer.rope(part, rotary, pos[t0:t1], out=part)
            assert torch.equal(y, want[t0:t1])


def test_rope_batch_positions(layer, kv):
    """Positions of a cache's batch: ragged, empty sequences, rows before a sequence's first token and rows
    behind the last sequence, which keep what was there; slices of one projection, in place and not."""
    g = gen(3)
    lens, ctx = [1, 0, 5, 300, 2, 0, 4], [1000, 3, 5, 700, 1, 0, 131072]  # the fifth has a token less than rows
    tokens = sum(lens) + 3
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    batch = kv.Batch(cu, torch.tensor(ctx, dtype=torch.int32, device="cuda"), torch.zeros(7, 4, dtype=torch.int32, device="cuda"))
    pos = np.concatenate([np.arange(c - n, c) for n, c in zip(lens, ctx)] + [[-1] * 3])
    for dtype in DTYPES:
        fused = rand(g, tokens, 8 + 2 * 2, 64, dtype=dtype)
        q, k = fused[:, :8], fused[:, 8:10]
        f, _ = layer.rotary_frequencies(64, device="cuda")
        rotary = layer.Rotary(f)
        at = torch.tensor(np.maximum(pos, 0), dtype=torch.int32, device="cuda")
        want = layer.rope((q, k), rotary, at)
        gone = torch.tensor(pos < 0, device="cuda")
        outs = tuple(torch.full_like(t, 5.0) for t in want)
        layer.rope((q, k), rotary, batch, out=outs)
        for o, w in zip(outs, want):
            assert torch.equal(o[~gone], w[~gone]) and (o[gone] == 5).all()
        before = fused.clone()
        layer.rope((q, k), rotary, batch, out=(q, k))
        assert torch.equal(q[~gone], want[0][~gone]) and torch.equal(k[~gone], want[1][~gone])
        assert torch.equal(fused[gone], before[gone]) and torch.equal(fused[:, 10:], before[:, 10:])


def test_rope_back_and_forth(layer):
    g = gen(4)
    x = rand(g, 200, 3, 128)
    pos = torch.arange(200, dtype=torch.int32, device="cuda") * 5000
    f, _ = layer.rotary_frequencies(128, device="cuda")
    for lay in (layer.HALF, layer.INTERLEAVED):
        r = layer.Rotary(f, layout=lay)
        y = layer.rope(layer.rope(x, r, pos), r, pos, backward=True)
        within(y, f64(x), 2 * rope_bound(f64(x), 2.0, torch.float32, 128, lay))


# ---- gated feed-forward ----

def operands(fp4, g, m, f, k, elem, tile, hn=0):
    a = rand(g, m, k)
    a[:, :3] *= 8
    wg, wu = rand(g, f, k, size=1.5 / math.sqrt(k)), rand(g, f, k, size=1.0 / math.sqrt(k))
    pa = fp4.Params(elem=elem, hadamard_n=hn)
    pw = fp4.Params(elem=elem, block=(32, 32) if tile else (1, 32), hadamard_n=hn)
    return fp4.quantize(a, pa), fp4.quantize(wg, pw), fp4.quantize(wu, pw)


def plain(fp4, q):
    """The operand's values as the product sees them (a rotation of both operands cancels in it)."""
    return f64(fp4.dequantize(fp4.with_params(q, hadamard_n=0)))


def product_bound(a, b, fp8):
    """1e-5 of the sum of magnitudes; on the FP8 matrix core each block of 8 products also loses what lies 13 bits
    below its largest."""
    tol = 1e-5 * (np.abs(a) @ np.abs(b).T)
    if fp8:
        step = max(1, (1 << 22) // (b.shape[0] * b.shape[1]))
        for i in range(0, a.shape[0], step):
            p = np.abs(a[i:i + step, None] * b[None]).reshape(len(a[i:i + step]), b.shape[0], -1, 8)
            top = p.max(-1, keepdims=True)
            unit = np.where(top > 0, 2.0 ** (np.floor(np.log2(np.where(top > 0, top, 1.0))) - 13), 0.0)
            tol[i:i + step] += np.minimum(p, unit).sum((-1, -2))
    return tol


CODED_SHAPES = [(1, 128, 512), (48, 384, 256), (100, 256, 512), (65, 128, 96), (300, 640, 512), (1030, 3328, 256), (35, 128, 4096),
                (48, 9600, 256), (700, 1280, 512), (513, 128, 384), (90, 1408, 256), (129, 3200, 128)]


def check_gated(layer, fp4, aq, gq, uq, act, dtype, **kw):
    w = layer.GatedWeights(gq, uq, act=act)
    got = layer.gated(aq, w, out_dtype=dtype, keep_gu=True, **kw)
    a, wg, wu = plain(fp4, aq), plain(fp4, gq), plain(fp4, uq)
    g, u = a @ wg.T, a @ wu.T
    fp8 = aq.params.elem == fp4.E4M3
    tg, tu = product_bound(a, wg, fp8), product_bound(a, wu, fp8)
    half = HALF_STEP[dtype]
    f = gq.rows
    within(got.gu[:, :f], g, tg + half * (np.abs(g) + tg), "g")
    within(got.gu[:, f:], u, tu + half * (np.abs(u) + tu), "u")
    h = ref.act(g, act) * u
    # the activation's slope is at most 1.13; its own roundings (an exponential, a quotient, a few products) 2^-20 of |g|
    th = 1.13 * tg * (np.abs(u) + tu) + np.abs(ref.act(g, act)) * tu + 2.0 ** -20 * np.abs(g) * (np.abs(u) + tu)
    within(got.h, h, th + half * (np.abs(h) + th), "h")
    return got


# rows / columns / depth around the kernels' tiles: single rows, 32 and 64 rows, ragged, K of 32, off the tiles' 256
GATED_SHAPES = [(100, 70, 32), (200, 96, 288), (150, 500, 1120), (300, 200, 128), (130, 260, 384), (1, 40, 640), (50, 96, 896), (1, 32, 32), (1, 128, 4096), (3, 100, 96), (17, 64, 256), (32, 96, 512), (33, 160, 1024), (64, 256, 768), (65, 128, 512),
                (70, 40, 256), (129, 200, 768), (200, 512, 288), (256, 384, 256), (300, 1000, 512), (513, 130, 1280),
                (40, 9300, 128), (60, 9300, 256), (35, 64, 4096), (55, 64, 8192), (66, 6000, 512), (130, 4100, 384), (513, 1400, 256),
                (200, 4000, 128), (97, 1376, 512), (260, 1400, 384), (115, 2064, 2048),
                (66, 2064, 1024)]


@pytest.mark.parametrize("kind", ["e2m1", "tile", "e4m3"])
@pytest.mark.parametrize("m,f,k", GATED_SHAPES)
def test_gated(fp4, layer, m, f, k, kind):
    if kind == "tile" and f % 32:
        f = (f + 31) // 32 * 32
    g = gen(m + f + k)
    aq, gq, uq = operands(fp4, g, m, f, k, fp4.E4M3 if kind == "e4m3" else fp4.E2M1, kind == "tile")
    for act, dtype in ((0, torch.float32), (1, torch.bfloat16), (2, torch.float32)):
        check_gated(layer, fp4, aq, gq, uq, act, dtype)


def test_gated_shapes_reach_every_kernel(fp4, layer):
    """The shapes of these tests go by the choice of kernel: each kernel is among them, with and without a launch of its
    own for the codes."""
    def plan(m, f, k, elem=0, out_q=None):
        q = [fp4.empty_qtensor(f, k, fp4.Params(elem=elem), "cuda") for _ in range(2)]
        p = layer.gated_plan(m, layer.GatedWeights(*q), out_q=out_q)
        return p.kernel, p.quantize_pass
    got = {plan(*s)[0] for s in GATED_SHAPES}
    assert got >= {layer.PLAN_ROWS, layer.PLAN_STREAM, layer.PLAN_TILE128_DEEP, layer.PLAN_TILE128_RAGGED}
    assert plan(1100, 3300, 256) == (layer.PLAN_TILE256, 0) and plan(600, 6000, 256) == (layer.PLAN_TILE256, 0)
    assert plan(200, 11008, 256) == (layer.PLAN_TILE128, 0) and plan(255, 13000, 384)[0] == layer.PLAN_TILE128
    assert plan(1100, 1500, 352)[0] == layer.PLAN_TILE128_RAGGED
    modes = {plan(m, f, k, out_q=fp4.Params(hadamard_n=hn)) for m, f, k in CODED_SHAPES for hn in (0, 128)}
    assert {p for _, p in modes} == {0, 1} and (layer.PLAN_TILE256, 0) in modes and (layer.PLAN_TILE128_DEEP, 1) in modes


def test_gated_many_small_tiles(fp4, layer):
    """More tiles of 128 rows than CUs, two workgroups on each."""
    for elem, m, f, k in ((0, 200, 11008, 256), (0, 250, 9001, 384), (1, 131, 10000, 128)):
        aq, gq, uq = operands(fp4, gen(m), m, f, k, elem, False)
        w = layer.GatedWeights(gq, uq, act=layer.GELU_TANH)
        assert layer.gated_plan(m, w).kernel == layer.PLAN_TILE128
        got = layer.gated(aq, w, out_dtype=torch.float32, keep_gu=True)
        a, wg, wu = (torch.from_numpy(plain(fp4, q)).cuda() for q in (aq, gq, uq))
        part = 1e-5 + (2.0 ** -10 if elem else 0.0)
        for y, b in ((got.gu[:, :f], wg), (got.gu[:, f:], wu)):
            assert ((y.double() - a @ b.T).abs() <= part * (a.abs() @ b.abs().T)).all()
        h = torch.nn.functional.gelu(got.gu[:, :f].double(), approximate="tanh") * got.gu[:, f:].double()
        assert ((got.h.double() - h).abs() <= 2.0 ** -20 * got.gu[:, :f].double().abs() * got.gu[:, f:].double().abs()).all()


def test_gated_large_tiles(fp4, layer):
    """A grid that takes the tiles of 256 rows, ragged on both sides, all three operand kinds."""
    for elem, tile, m, f, k in ((0, False, 1100, 3300, 256), (0, True, 1030, 4096, 256), (1, False, 1025, 3302, 256),
                                (0, False, 1500, 3200, 384), (0, True, 1030, 4096, 640), (0, False, 1100, 1500, 352),
                                (1, False, 1100, 1500, 352), (0, True, 1030, 1504, 992)):
        g = gen(m + k)
        aq, gq, uq = operands(fp4, g, m, f, k, elem, tile)
        w = layer.GatedWeights(gq, uq, act=layer.SILU)
        a, wg, wu = (torch.from_numpy(plain(fp4, q)).cuda() for q in (aq, gq, uq))
        gv, uv = a @ wg.T, a @ wu.T
        size = a.abs() @ wg.abs().T, a.abs() @ wu.abs().T
        # blocks of 8 products lose up to 8 * 2^-13 of their largest on the FP8 matrix core
        part = 1e-5 + (2.0 ** -10 if elem else 0.0)
        for dtype in DTYPES:
            got = layer.gated(aq, w, out_dtype=dtype, keep_gu=True)
            half = HALF_STEP[dtype]
            tg, tu = part * size[0], part * size[1]
            h = torch.nn.functional.silu(gv) * uv
            th = 1.13 * tg * (uv.abs() + tu) + torch.nn.functional.silu(gv).abs() * tu + 2.0 ** -20 * gv.abs() * (uv.abs() + tu)
            for y, want, tol in ((got.gu[:, :f], gv, tg), (got.gu[:, f:], uv, tu), (got.h, h, th)):
                assert ((y.double() - want).abs() <= tol + half * (want.abs() + tol)).all()


@pytest.mark.parametrize("mode", [(0, 0, 0, 0), (0, 32, 1, 0), (0, 64, 0, 0), (0, 128, 0, 0), (0, 128, 0, 1), (1, 0, 1, 0), (1, 16, 0, 1),
                                  (1, 64, 1, 0), (1, 128, 1, 0)])
@pytest.mark.parametrize("m,f,k", CODED_SHAPES)
def test_gated_codes_are_those_of_quantize(fp4, layer, m, f, k, mode):
    g = gen(m + f)
    for elem in (0, 1):
        aq, gq, uq = operands(fp4, g, m, f, k, elem, False)
        w = layer.GatedWeights(gq, uq)
        p = params(fp4, mode, seed=m * 991 + 1)
        full = layer.gated(aq, w, out_dtype=torch.float32, out_q=p)
        same_codes(full.q, fp4.quantize(full.h, p))
        got = layer.gated(aq, w, out_q=p, keep_gu=True)
        same_codes(got.q, full.q)
        assert torch.equal(got.h, full.h.bfloat16())
        only = layer.gated(aq, w, out_q=p, keep_h=False, q_out=fp4.empty_qtensor(m, f, p, "cuda"))
        assert only.h is None and only.gu is None
        same_codes(only.q, full.q)


def test_gated_fused_weights_pitches_and_rotation(fp4, layer):
    g = gen(8)
    for m, f, k in ((5, 96, 256), (130, 200, 512), (1030, 3300, 256)):
        aq, gq, uq = operands(fp4, g, m, f, k, fp4.E2M1, False, hn=128)
        want = layer.gated(aq, layer.GatedWeights(gq, uq), keep_gu=True)
        both = fp4.QTensor(torch.cat([gq.codes, uq.codes]), torch.cat([gq.scales, uq.scales]), None, 2 * f, k, gq.params)
        if (f * k // 2) % 16 == 0 and (f * k // 32) % 4 == 0:
            got = layer.gated(aq, layer.GatedWeights(both), keep_gu=True)
            assert torch.equal(got.h, want.h) and torch.equal(got.gu, want.gu)
        for extra in (8, 1):  # whole 16-byte pieces, and rows that are not
            o = torch.full((m, f + extra), 3.0, dtype=torch.bfloat16, device="cuda")
            gu = torch.full((m, 2 * f + extra), 3.0, dtype=torch.bfloat16, device="cuda")
            layer.gated(aq, layer.GatedWeights(gq, uq), out=o[:, :f], keep_gu=gu[:, :2 * f])
            assert torch.equal(o[:, :f], want.h) and torch.equal(gu[:, :2 * f], want.gu)
            assert (o[:, f:] == 3).all() and (gu[:, 2 * f:] == 3).all()


@pytest.mark.parametrize("m,f,k", [(1, 33, 32), (20, 35, 96), (40, 33, 96), (140, 67, 160), (300, 129, 2080)])
def test_gated_scales_that_begin_at_any_byte(fp4, layer, m, f, k):
    """The lower half of a fused weight, and a batch's rows, whose scales begin off a multiple of 4 bytes."""
    g = gen(m + k)
    for elem in (fp4.E2M1, fp4.E4M3):
        aq, gq, uq = operands(fp4, g, m + 1, f, k, elem, False)
        both = fp4.QTensor(torch.cat([gq.codes, uq.codes]), torch.cat([gq.scales, uq.scales]), None, 2 * f, k, gq.params)
        cut = k if elem == fp4.E4M3 else k // 2
        rest = fp4.QTensor(aq.codes.view(-1)[cut:], aq.scales.view(-1)[k // 32:], None, m, k, aq.params)
        assert (f * k // 32) % 4 and (k // 32) % 4
        same = fp4.QTensor(rest.codes.clone(), rest.scales.clone(), None, m, k, aq.params)
        want = layer.gated(same, layer.GatedWeights(gq, uq), keep_gu=True)
        got = layer.gated(rest, layer.GatedWeights(both), keep_gu=True)
        assert torch.equal(got.h, want.h) and torch.equal(got.gu, want.gu)
        assert want.gu.isfinite().all() and want.gu.abs().amax() > 0


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("rows,f", [(1, 8), (1, 128), (3, 104), (7, 1000), (65, 256), (33, 1376), (2, 11008)])
def test_gated_backward(layer, rows, f, act):
    g = gen(rows + f)
    for dtype in DTYPES:
        dh, gu = rand(g, rows, f, dtype=dtype), rand(g, rows, 2 * f, size=3.0, dtype=dtype)
        gu[0, :4] = torch.tensor([0.0, 60.0, -60.0, -200.0])
        got = layer.gated_backward(dh, gu, act=act)
        d, gv, uv = f64(dh), f64(gu)[:, :f], f64(gu)[:, f:]
        want = ref.gated_grad(d, gv, uv, act)
        # value and slope: 2^-20 of their scale (|g| and 1 + |g|), two products' roundings
        tol = 2.0 ** -20 * np.concatenate([np.abs(d * uv) * (1 + np.abs(gv)), np.abs(d * gv)], 1)
        within(got.dgu, want, tol + HALF_STEP[dtype] * np.abs(want) + 1e-38)
        same = gu.clone()
        assert torch.equal(layer.gated_backward(dh, same, act=act, out=same).dgu, got.dgu)
        o = pitched(gu, 16)
        assert torch.equal(layer.gated_backward(pitched(dh, 8), pitched(gu, 24), act=act, out=o).dgu, got.dgu)
        assert (o._base[:, 2 * f:] == 7).all()


def test_gated_backward_far_from_zero(layer):
    """Where the activation is x or 0 its slope is 1 or 0, up to the largest values."""
    g = torch.tensor([[1e4, -1e4, 1e10, -1e10, 3e19, -3e19, 3e38, -3e38]], device="cuda")
    for act in (0, 1, 2):
        got = layer.gated_backward(torch.ones(1, 8, device="cuda"), torch.cat([g, torch.ones_like(g)], 1), act=act).dgu
        assert torch.equal(got[:, :8], (g > 0).float()) and torch.equal(got[:, 8:], g.clamp(min=0))


def test_gated_backward_against_differences(layer):
    rng = np.random.default_rng(2)
    dh, g, u = rng.normal(size=(5, 64)), rng.normal(size=(5, 64)) * 2, rng.normal(size=(5, 64))
    for act in (0, 1, 2):
        gu = torch.tensor(np.concatenate([g, u], 1), dtype=torch.float32, device="cuda")
        d = f64(layer.gated_backward(torch.tensor(dh, dtype=torch.float32, device="cuda"), gu, act=act).dgu)
        h = 1e-5
        for _ in range(5):
            a, b = rng.normal(size=g.shape), rng.normal(size=g.shape)
            num = ((dh * ref.act(g + h * a, act) * (u + h * b)).sum() - (dh * ref.act(g - h * a, act) * (u - h * b)).sum()) / (2 * h)
            ana = (d * np.concatenate([a, b], 1)).sum()
            assert abs(num - ana) <= 2.0 ** -18 * np.abs(d * np.concatenate([a, b], 1)).sum() + 1e-7


@pytest.mark.parametrize("mode", Q_MODES)
def test_gated_backward_codes_are_those_of_quantize(fp4, layer, mode):
    for rows, f in ((1, 256), (5, 512), (130, 256), (3, 11008)):
        if mode[1] and f % mode[1]:
            continue
        g = gen(rows + f)
        dh, gu = rand(g, rows, f, dtype=torch.bfloat16), rand(g, rows, 2 * f, dtype=torch.bfloat16)
        p = params(fp4, mode, seed=12345)
        full = layer.gated_backward(dh.float(), gu.float(), out_q=p)
        same_codes(full.q, fp4.quantize(full.dgu, p))
        got = layer.gated_backward(dh, gu, out_q=p, keep=False)
        assert got.dgu is None
        same_codes(got.q, full.q)


# ---- the calls as programs make them ----

def test_no_rows(fp4, layer, kv):
    p = fp4.Params(hadamard_n=32)
    x = torch.empty(0, 64, device="cuda")
    r = layer.rmsnorm(x, residual=x.clone(), out_q=p)
    assert r.y.shape == (0, 64) and r.sum.shape == (0, 64) and (r.q.rows, r.q.cols) == (0, 64)
    dx, dw = layer.rmsnorm_backward(x, x)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device="cuda"))
    f, _ = layer.rotary_frequencies(64, device="cuda")
    assert layer.rope(torch.empty(0, 4, 64, device="cuda"), layer.Rotary(f), torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 4, 64)
    _, gq, uq = operands(fp4, gen(1), 1, 32, 64, fp4.E2M1, False)
    q = layer.rmsnorm(x, out_q=fp4.Params()).q
    h = layer.gated(q, layer.GatedWeights(gq, uq), keep_gu=True, out_q=fp4.Params())
    assert h.h.shape == (0, 32) and h.gu.shape == (0, 64) and (h.q.rows, h.q.cols) == (0, 32)
    assert layer.gated_backward(h.h, h.gu).dgu.shape == (0, 64)


def test_captured_and_replayed(fp4, layer):
    """Each call recorded into a graph and replayed with new inputs, eager work between the replays; two graphs
    that share one workspace."""
    g = gen(11)
    m, f, k = 40, 256, 512
    p = fp4.Params(elem=fp4.E4M3, hadamard_n=128)  # spans more columns than a tile of few rows: a workspace
    _, gq, uq = operands(fp4, g, m, f, k, fp4.E4M3, False, hn=128)
    w = layer.GatedWeights(gq, uq)
    x, r, wt = rand(g, m, k, dtype=torch.bfloat16), rand(g, m, k, dtype=torch.bfloat16), rand(g, k)
    dh, pos = rand(g, m, f, dtype=torch.bfloat16), torch.arange(m, dtype=torch.int32, device="cuda")
    fr, _ = layer.rotary_frequencies(64, device="cuda")
    rotary = layer.Rotary(fr)
    wsb = torch.empty(layer.rmsnorm_backward_workspace_bytes(m, k), dtype=torch.uint8, device="cuda")
    wsg = torch.empty(m * f * 4, dtype=torch.uint8, device="cuda")

    def step():
        n = layer.rmsnorm(x, wt, residual=r, out_q=p)
        ro = layer.rope(x.view(m, 8, 64), rotary, pos)
        h = layer.gated(n.q, w, out_q=p, keep_gu=True, workspace=wsg)
        d = layer.gated_backward(dh, h.gu, out_q=p)
        dx, dw = layer.rmsnorm_backward(n.sum, x, wt, dsum=r, workspace=wsb)
        return n.y, n.sum, n.q.codes, n.q.scales, ro, h.h, h.gu, h.q.codes, h.q.scales, d.dgu, d.q.codes, dx, dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = step()
        graphs.append((gr, outs))
    for i in range(4):
        x.copy_(rand(g, m, k, dtype=torch.bfloat16))
        dh.copy_(rand(g, m, f, dtype=torch.bfloat16))
        want = [t.clone() for t in step()]
        for gr, outs in graphs:
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_two_streams_at_once(fp4, layer):
    g = gen(12)
    aq, gq, uq = operands(fp4, g, 500, 768, 512, fp4.E2M1, False)
    w = layer.GatedWeights(gq, uq)
    x, dy = rand(g, 3000, 1024), rand(g, 3000, 1024)
    want = layer.gated(aq, w).h, *layer.rmsnorm_backward(dy, x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append((layer.gated(aq, w).h, *layer.rmsnorm_backward(dy, x)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
