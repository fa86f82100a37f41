"""CPU checks of the calls between a layer's products: every rejection happens on the host before any device
call, size queries agree with the calls, tables of frequencies, and the plain reference of the GPU tests against
values worked out by hand and against differences."""
import ctypes
import math

import numpy as np
import pytest

import layer_reference as ref


@pytest.fixture(scope="module")
def layer():
    import os
    from bit_gemm_fwht_amd import fp4, layer as m
    if not os.path.exists(fp4.LIB_PATH):
        from bit_gemm_fwht_amd import build
        build.build()
    m.lib()
    return m


@pytest.fixture(scope="module")
def fp4(layer):
    from bit_gemm_fwht_amd import fp4 as m
    return m


def status(fp4, name):
    return getattr(fp4, "ERR_" + name) if name != "OK" else fp4.OK


def quant(fp4, rows=0, cols=0, **kw):
    p = dict(elem=0, block_rows=1, block_cols=32, scale_mode=0, round_mode=0, hadamard_n=0, seed=0)
    p.update({k: v for k, v in kw.items() if k in p})
    t = dict(codes=0x900000, scales=0xA00000, tensor_scale=None, rows=rows, cols=cols)
    t.update({k: v for k, v in kw.items() if k in t})
    return fp4.QParams(**p), fp4.QTensorC(p=fp4.QParams(**p), **t)


def ptr(c):
    return ctypes.addressof(c)


def norm(layer, **kw):
    a = dict(x=0x10000, residual=0x20000, weight=0x30000, sum=0x40000, y=0x50000, rows=4, cols=64, ldx=64, ldr=64, lds=64, ldy=64,
             dtype=1, w_dtype=0, eps=1e-5)
    a.update(kw)
    return layer.NormC(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"), (dict(cols=0), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"),
    (dict(w_dtype=7), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=math.nan), "INVALID_ARG"),
    (dict(eps=math.inf), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"), (dict(residual=None), "INVALID_ARG"),
    (dict(sum=None), "INVALID_ARG"), (dict(ldx=56), "INVALID_ARG"), (dict(lds=32), "INVALID_ARG"), (dict(ldy=8), "INVALID_ARG"),
    (dict(cols=60, ldx=64), "UNSUPPORTED"), (dict(cols=32776, ldx=40000), "UNSUPPORTED"), (dict(rows=1 << 31), "UNSUPPORTED"),
    (dict(x=0x10008), "ALIGNMENT"), (dict(weight=0x30004), "ALIGNMENT"), (dict(ldx=68), "ALIGNMENT"), (dict(ldr=65), "ALIGNMENT"),
    (dict(sum=0x10000, lds=72), "INVALID_ARG"), (dict(sum=0x20000, lds=72), "INVALID_ARG"), (dict(y=0x40000), "INVALID_ARG"),
    (dict(y=0x20000), "INVALID_ARG"), (dict(y=0x10000, ldy=72), "INVALID_ARG"), (dict(weight=0x40000), "INVALID_ARG"),
])
def test_norm_refusals(layer, fp4, kw, want):
    c = norm(layer, **kw)
    assert layer.lib().fp4_rmsnorm(ptr(c), None, None, None) == status(fp4, want)


QUANT_REFUSALS = [
    (dict(elem=2), "INVALID_ARG"), (dict(round_mode=5), "INVALID_ARG"), (dict(hadamard_n=24), "INVALID_ARG"),
    (dict(block_cols=16), "UNSUPPORTED"), (dict(block_rows=32), "UNSUPPORTED"), (dict(scale_mode=2), "UNSUPPORTED"),
    (dict(scale_mode=4), "UNSUPPORTED"), (dict(hadamard_n=128), "INVALID_ARG"), (dict(codes=None), "INVALID_ARG"),
    (dict(scales=None), "INVALID_ARG"), (dict(codes=0x900008), "ALIGNMENT"), (dict(scales=0x900000), "INVALID_ARG"),
    (dict(codes=0x10000), "INVALID_ARG"), (dict(scales=0x50000), "INVALID_ARG"),
]


@pytest.mark.parametrize("kw,want", QUANT_REFUSALS)
def test_norm_quant_refusals(layer, fp4, kw, want):
    p, q = quant(fp4, **kw)
    assert layer.lib().fp4_rmsnorm(ptr(norm(layer)), ptr(p), ptr(q), None) == status(fp4, want)
    assert q.rows == 0  # nothing described either


def test_norm_other_refusals(layer, fp4):
    L = layer.lib()
    p, q = quant(fp4)
    assert L.fp4_rmsnorm(None, None, None, None) == fp4.ERR_INVALID_ARG
    assert L.fp4_rmsnorm(ptr(norm(layer)), ptr(p), None, None) == fp4.ERR_INVALID_ARG
    assert L.fp4_rmsnorm(ptr(norm(layer)), None, ptr(q), None) == fp4.ERR_INVALID_ARG
    c = norm(layer, cols=40, ldx=40, ldr=40, lds=40, ldy=40)
    assert L.fp4_rmsnorm(ptr(c), ptr(p), ptr(q), None) == fp4.ERR_INVALID_ARG  # groups of 32
    c = norm(layer, rows=0, x=None, residual=None, sum=None, y=None, weight=None)
    assert L.fp4_rmsnorm(ptr(c), None, None, None) == fp4.OK


def grad(layer, **kw):
    a = dict(dy=0x10000, s=0x20000, dsum=0x30000, weight=0x40000, dx=0x50000, dweight=0x60000, rows=4, cols=64, lddy=64, lds=64,
             lddsum=64, lddx=64, dtype=1, w_dtype=0, eps=1e-5)
    a.update(kw)
    return layer.NormGradC(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), "INVALID_ARG"), (dict(s=None), "INVALID_ARG"), (dict(dx=None), "INVALID_ARG"), (dict(rows=-1), "INVALID_ARG"),
    (dict(dtype=3), "INVALID_ARG"), (dict(w_dtype=3), "INVALID_ARG"), (dict(eps=-0.5), "INVALID_ARG"), (dict(lds=40), "INVALID_ARG"),
    (dict(dx=0x20000), "INVALID_ARG"), (dict(dx=0x10000, lddx=72), "INVALID_ARG"), (dict(dx=0x30000, lddx=72), "INVALID_ARG"),
    (dict(dweight=0x50000), "INVALID_ARG"), (dict(dweight=0x40000), "INVALID_ARG"), (dict(dx=0x40000), "INVALID_ARG"),
    (dict(cols=44), "UNSUPPORTED"), (dict(rows=1 << 31), "UNSUPPORTED"), (dict(dy=0x10004), "ALIGNMENT"), (dict(lddsum=66), "ALIGNMENT"),
    (dict(dweight=0x60004), "ALIGNMENT"), (dict(weight=0x40008), "ALIGNMENT"),
])
def test_norm_backward_refusals(layer, fp4, kw, want):
    c = grad(layer, **kw)
    assert layer.lib().fp4_rmsnorm_backward(ptr(c), 0x1000000, 1 << 40, None) == status(fp4, want)


def test_norm_backward_workspace(layer, fp4):
    L = layer.lib()
    for rows, cols in ((1, 8), (4, 64), (1000, 4096), (100000, 32768), (1 << 30, 256)):
        c = grad(layer, rows=rows, cols=cols, lddy=cols, lds=cols, lddsum=cols, lddx=cols)
        need = L.fp4_rmsnorm_backward_workspace_bytes(ptr(c))
        assert 0 < need <= 1 << 27
        assert L.fp4_rmsnorm_backward(ptr(c), None, 0, None) == fp4.ERR_WORKSPACE
        assert L.fp4_rmsnorm_backward(ptr(c), 0x1000000, need - 1, None) == fp4.ERR_WORKSPACE
        assert L.fp4_rmsnorm_backward(ptr(c), 0x1000004, need, None) == fp4.ERR_ALIGNMENT
        assert layer.rmsnorm_backward_workspace_bytes(rows, cols) == need
        c = grad(layer, rows=rows, cols=cols, dweight=None)
        assert L.fp4_rmsnorm_backward_workspace_bytes(ptr(c)) == 0
    assert L.fp4_rmsnorm_backward_workspace_bytes(ptr(grad(layer, cols=12))) == -1
    assert L.fp4_rmsnorm_backward_workspace_bytes(None) == -1


def rope(layer, batch=None, **kw):
    a = dict(x=(0x10000, 0x20000), out=(0x30000, 0x40000), ldx=(512, 256), ldx_head=(128, 128), ldo=(512, 256), ldo_head=(128, 128),
             heads=(4, 2), tokens=3, inv_freq=0x50000, positions=None if batch else 0x60000, batch=batch, scale=1.0, dtype=1,
             head_dim=128, rotary_dim=64, layout=0, backward=0)
    a.update(kw)
    pairs = ("x", "out", "ldx", "ldx_head", "ldo", "ldo_head", "heads")
    return layer.RopeC(**{k + str(i): a[k][i] for k in pairs for i in (0, 1)}, **{k: v for k, v in a.items() if k not in pairs})


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), "INVALID_ARG"), (dict(dtype=4), "INVALID_ARG"), (dict(layout=2), "INVALID_ARG"), (dict(heads=(0, 2)), "INVALID_ARG"),
    (dict(heads=(4, -1)), "INVALID_ARG"), (dict(head_dim=0), "INVALID_ARG"), (dict(rotary_dim=63), "INVALID_ARG"),
    (dict(rotary_dim=0), "INVALID_ARG"), (dict(rotary_dim=130), "INVALID_ARG"), (dict(scale=math.nan), "INVALID_ARG"),
    (dict(inv_freq=None), "INVALID_ARG"), (dict(positions=None), "INVALID_ARG"), (dict(x=(None, 0x20000)), "INVALID_ARG"),
    (dict(out=(0x30000, None)), "INVALID_ARG"), (dict(ldx=(-512, 256)), "INVALID_ARG"), (dict(out=(0x30000, 0x30000)), "INVALID_ARG"),
    (dict(out=(0x20000, 0x40000)), "INVALID_ARG"), (dict(out=(0x10000, 0x40000), ldo=(1024, 256)), "INVALID_ARG"),
    (dict(ldo=(120, 256)), "INVALID_ARG"), (dict(ldo_head=(64, 128)), "INVALID_ARG"), (dict(ldo=(256, 256)), "INVALID_ARG"),
    (dict(head_dim=2048), "UNSUPPORTED"), (dict(head_dim=127), "UNSUPPORTED"), (dict(tokens=1 << 31), "UNSUPPORTED"), (dict(tokens=1 << 62), "UNSUPPORTED"),
    (dict(heads=(70000, 0)), "UNSUPPORTED"), (dict(x=(0x10002, 0x20000)), "ALIGNMENT"), (dict(ldx=(516, 256)), "ALIGNMENT"),
    (dict(inv_freq=0x50004), "ALIGNMENT"), (dict(positions=0x60002), "ALIGNMENT"),
])
def test_rope_refusals(layer, fp4, kw, want):
    c = rope(layer, **kw)
    assert layer.lib().fp4_rope(ptr(c), None) == status(fp4, want)


def test_rope_batch_refusals(layer, fp4):
    from bit_gemm_fwht_amd import kv
    L = layer.lib()
    good = dict(cu_tokens=0x70000, context=0x80000, table=None, tokens=3, seqs=2)
    for kw, want in ((dict(cu_tokens=None), "INVALID_ARG"), (dict(context=None), "INVALID_ARG"), (dict(seqs=0), "INVALID_ARG"),
                     (dict(tokens=4), "INVALID_ARG"), (dict(seqs=1 << 30), "UNSUPPORTED")):
        b = kv.BatchC(**{**good, **kw})
        assert L.fp4_rope(ptr(rope(layer, batch=ptr(b))), None) == status(fp4, want)
    b = kv.BatchC(**good)
    assert L.fp4_rope(ptr(rope(layer, batch=ptr(b), positions=0x60000)), None) == fp4.ERR_INVALID_ARG  # one of the two
    assert L.fp4_rope(ptr(rope(layer, tokens=0)), None) == fp4.OK
    assert L.fp4_rope(None, None) == fp4.ERR_INVALID_ARG


def gated_args(layer, fp4, m=4, f=64, k=256, a=None, w=None, u=None, o=None):
    def q(base, rows, kw):
        p = dict(elem=0, block_rows=1, block_cols=32, scale_mode=0, round_mode=0, hadamard_n=0, seed=0)
        p.update({x: y for x, y in (kw or {}).items() if x in p})
        t = dict(codes=base, scales=base + 0x10000, tensor_scale=None, rows=rows, cols=k)
        t.update({x: y for x, y in (kw or {}).items() if x in t})
        return fp4.QTensorC(p=fp4.QParams(**p), **t)
    out = dict(h=0x700000, gu=0x800000, ldh=f, ldgu=2 * f, dtype=1, act=0)
    out.update(o or {})
    return q(0x100000, m, a), q(0x200000, f, w), q(0x300000, f, w if u is None else u), layer.GatedC(**out)


@pytest.mark.parametrize("kw,want", [
    (dict(a=dict(codes=None)), "INVALID_ARG"), (dict(a=dict(cols=128)), "INVALID_ARG"), (dict(a=dict(rows=-1)), "INVALID_ARG"),
    (dict(w=dict(rows=0)), "INVALID_ARG"), (dict(u=dict(rows=32)), "INVALID_ARG"), (dict(u=dict(scales=None)), "INVALID_ARG"),
    (dict(k=48), "INVALID_ARG"), (dict(a=dict(hadamard_n=64)), "INVALID_ARG"), (dict(u=dict(elem=1)), "INVALID_ARG"),
    (dict(u=dict(block_rows=32)), "INVALID_ARG"), (dict(o=dict(dtype=9)), "INVALID_ARG"), (dict(o=dict(act=3)), "INVALID_ARG"),
    (dict(o=dict(ldh=32)), "INVALID_ARG"), (dict(o=dict(ldgu=100)), "INVALID_ARG"), (dict(o=dict(h=None, gu=None)), "INVALID_ARG"),
    (dict(o=dict(gu=0x700000)), "INVALID_ARG"), (dict(o=dict(h=0x100000)), "INVALID_ARG"),
    (dict(f=40, w=dict(block_rows=32)), "INVALID_ARG"),
    (dict(w=dict(elem=1)), "UNSUPPORTED"), (dict(a=dict(block_rows=32)), "UNSUPPORTED"), (dict(a=dict(scale_mode=2)), "UNSUPPORTED"),
    (dict(a=dict(elem=1), w=dict(elem=1, block_rows=32)), "UNSUPPORTED"), (dict(w=dict(block_cols=16, scale_mode=2)), "UNSUPPORTED"),
    (dict(a=dict(codes=0x100008)), "ALIGNMENT"), (dict(w=dict(scales=0x210002)), "ALIGNMENT"), (dict(o=dict(h=0x700008)), "ALIGNMENT"),
])
def test_gated_refusals(layer, fp4, kw, want):
    a, g, u, o = gated_args(layer, fp4, **kw)
    assert layer.lib().fp4_gemm_gated(ptr(a), ptr(g), ptr(u), ptr(o), None, None, 0x1000000, 1 << 40, None) == status(fp4, want)


def test_gated_quant_refusals_and_workspace(layer, fp4):
    L = layer.lib()
    a, g, u, o = gated_args(layer, fp4, f=512)
    for kw, want in QUANT_REFUSALS + [(dict(hadamard_n=256), "UNSUPPORTED"), (dict(codes=0x100000), "INVALID_ARG"),
                                      (dict(scales=0x800000), "INVALID_ARG")]:
        if kw in (dict(hadamard_n=128), dict(codes=0x10000), dict(scales=0x50000)):
            continue  # fine here
        p, q = quant(fp4, **kw)
        assert L.fp4_gemm_gated(ptr(a), ptr(g), ptr(u), ptr(o), ptr(p), ptr(q), 0x1000000, 1 << 40, None) == status(fp4, want), kw
    for kw in (dict(hadamard_n=128), dict(round_mode=1)):  # a rotation past the columns of a tile of few rows; a rounding of its own
        p, q = quant(fp4, **kw)
        need = L.fp4_gemm_gated_workspace_bytes(ptr(a), ptr(g), ptr(u), ptr(o), ptr(p))
        assert need == 4 * 512 * 4
        assert L.fp4_gemm_gated(ptr(a), ptr(g), ptr(u), ptr(o), ptr(p), ptr(q), None, 0, None) == fp4.ERR_WORKSPACE
        assert L.fp4_gemm_gated(ptr(a), ptr(g), ptr(u), ptr(o), ptr(p), ptr(q), 0x1000008, need, None) == fp4.ERR_ALIGNMENT
    p, q = quant(fp4)
    assert L.fp4_gemm_gated_workspace_bytes(ptr(a), ptr(g), ptr(u), ptr(o), ptr(p)) == 0
    assert L.fp4_gemm_gated_workspace_bytes(ptr(a), ptr(g), None, ptr(o), None) == -1
    a.rows = 0
    assert L.fp4_gemm_gated(ptr(a), ptr(g), ptr(u), ptr(o), ptr(p), ptr(q), None, 0, None) == fp4.OK
    assert (q.rows, q.cols) == (0, 512)


def test_gated_plan(layer, fp4):
    """Few rows, which need no device: the kernel by K, the launch of its own by the rotation and the rounding."""
    L, plan = layer.lib(), layer.GatedPlanC()
    for k, kernel in ((256, layer.PLAN_STREAM), (384, layer.PLAN_STREAM), (96, layer.PLAN_ROWS)):
        a, g, u, o = gated_args(layer, fp4, f=512, k=k)
        for kw, alone in ((None, 0), (dict(hadamard_n=32), 0), (dict(hadamard_n=64), 1), (dict(round_mode=1), 1)):
            p = None if kw is None else quant(fp4, **kw)[0]
            assert L.fp4_gemm_gated_plan(ptr(a), ptr(g), ptr(u), ptr(o), None if p is None else ptr(p), ptr(plan)) == fp4.OK
            assert (plan.kernel, plan.quantize_pass) == (kernel, alone)
            if p is not None:
                assert L.fp4_gemm_gated_workspace_bytes(ptr(a), ptr(g), ptr(u), ptr(o), ptr(p)) == alone * 4 * 512 * 4
    a.rows = 0
    assert L.fp4_gemm_gated_plan(ptr(a), ptr(g), ptr(u), ptr(o), None, ptr(plan)) == fp4.OK and plan.kernel == 0
    assert L.fp4_gemm_gated_plan(ptr(a), ptr(g), ptr(u), ptr(o), None, None) == fp4.ERR_INVALID_ARG


def gated_grad(layer, **kw):
    a = dict(dh=0x10000, gu=0x20000, dgu=0x30000, rows=4, cols=64, lddh=64, ldgu=128, lddgu=128, dtype=1, act=0)
    a.update(kw)
    return layer.GatedGradC(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(dh=None), "INVALID_ARG"), (dict(gu=None), "INVALID_ARG"), (dict(dgu=None), "INVALID_ARG"), (dict(rows=-2), "INVALID_ARG"),
    (dict(act=-1), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"), (dict(ldgu=64), "INVALID_ARG"), (dict(lddgu=64), "INVALID_ARG"),
    (dict(dgu=0x10000), "INVALID_ARG"), (dict(dgu=0x20000, lddgu=136), "INVALID_ARG"), (dict(cols=60, lddh=64), "UNSUPPORTED"),
    (dict(rows=1 << 31), "UNSUPPORTED"), (dict(dh=0x10002), "ALIGNMENT"), (dict(ldgu=132), "ALIGNMENT"),
])
def test_gated_backward_refusals(layer, fp4, kw, want):
    assert layer.lib().fp4_gated_backward(ptr(gated_grad(layer, **kw)), None, None, None) == status(fp4, want)


def test_gated_backward_quant_refusals(layer, fp4):
    L = layer.lib()
    for kw, want in QUANT_REFUSALS:
        if kw == dict(scales=0x50000):
            continue
        p, q = quant(fp4, **kw)
        assert L.fp4_gated_backward(ptr(gated_grad(layer)), ptr(p), ptr(q), None) == status(fp4, want), kw
    p, q = quant(fp4, hadamard_n=64)  # a chunk that would lie across the two halves
    assert L.fp4_gated_backward(ptr(gated_grad(layer, cols=32)), ptr(p), ptr(q), None) == fp4.ERR_INVALID_ARG


def test_python_refusals(layer, fp4):
    import torch
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        layer.rmsnorm(x)
    with pytest.raises(TypeError, match="dtype"):
        layer.rmsnorm(x.half())
    with pytest.raises(ValueError, match="CUDA"):
        layer.rmsnorm_backward(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        layer.gated_backward(x, torch.zeros(2, 128))
    with pytest.raises(ValueError, match="CUDA"):
        layer.Rotary(torch.ones(4, dtype=torch.float64))
    q = fp4.QTensor(torch.zeros(1024, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8), None, 32, 64, fp4.MXFP4)
    with pytest.raises(ValueError):
        layer.GatedWeights(q, q)
    with pytest.raises(ValueError):
        layer.GatedWeights(q, q, act=5)


def test_frequencies(layer):
    f, s = layer.rotary_frequencies(8, base=100.0)
    assert s == 1.0 and np.allclose(f.numpy(), [1.0, 100.0 ** -0.25, 0.1, 100.0 ** -0.75], rtol=1e-15)
    g, _ = layer.rotary_frequencies(8, base=100.0, scaling="linear", factor=4.0)
    assert np.array_equal(g.numpy(), f.numpy() / 4)
    g, _ = layer.rotary_frequencies(8, base=100.0, scaling="ntk", factor=16.0)
    assert g[0] == 1.0 and abs(g[3] / (f[3] / 16.0) - 1) < 1e-14  # the fastest kept, the slowest squeezed by factor
    # bands: turns in 1000 tokens are 159, 50.3, 15.9, 5.03
    g, _ = layer.rotary_frequencies(8, base=100.0, scaling="bands", factor=2.0, original_context=1000, low=10.0, high=50.0)
    part = (100 / (2 * math.pi) - 10) / 40
    assert np.allclose(g.numpy(), f.numpy() * [1, 1, part + (1 - part) / 2, 0.5], rtol=1e-14)
    # yarn: pairs of index 4 ln(1000 / (2 pi turns)) / ln 100: floor(2.01) = 2 for 15.75 turns, ceil(2.9..) for 5.4
    g, s = layer.rotary_frequencies(8, base=100.0, scaling="yarn", factor=8.0, original_context=1000, fast=15.75, slow=5.4)
    assert abs(s - (0.1 * math.log(8) + 1)) < 1e-15
    assert np.allclose(g.numpy(), f.numpy() * [1, 1, 1, 1 / 8], rtol=1e-14)
    for kw in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="bands"),
               dict(rotary_dim=2, scaling="ntk"), dict(rotary_dim=8, base=-1.0), dict(rotary_dim=8, factor=0.0)):
        with pytest.raises(ValueError):
            layer.rotary_frequencies(**kw)


def test_reference_by_hand():
    assert np.allclose(ref.rmsnorm(np.array([[3.0, 4.0]]), np.array([2.0, 1.0]), 0.0), [[6 / math.sqrt(12.5), 4 / math.sqrt(12.5)]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    assert np.allclose(ref.rope(x, [1], [math.pi / 2, math.pi], False), [[[-3, -2, 1, -4]]])
    assert np.allclose(ref.rope(x, [1], [math.pi / 2, math.pi], True), [[[-2, 1, -3, -4]]])
    assert np.allclose(ref.act(np.array([0.0, 1.0]), 0), [0, 1 / (1 + math.exp(-1))])
    assert np.allclose(ref.act(np.array([1.0]), 1), [0.8413447460685429])


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_reference_gradients_against_differences(kind):
    rng = np.random.default_rng(kind)
    g, u, dh = (rng.normal(size=(3, 10)) for _ in range(3))
    d, h = ref.gated_grad(dh, g, u, kind), 1e-6
    for i in range(10):
        e = np.zeros((3, 10))
        e[:, i] = h
        num = dh * (ref.act(g + e, kind) * u - ref.act(g - e, kind) * u) / (2 * h)
        assert np.allclose(num[:, i], d[:, i], atol=1e-8)
    assert np.allclose(d[:, 10:], dh * ref.act(g, kind))
    s, w, dy = rng.normal(size=(2, 9)), rng.normal(size=9), rng.normal(size=(2, 9))
    dx, dw = ref.rmsnorm_grad(dy, s, w, 0.1)
    for i in range(9):
        e = np.zeros((2, 9))
        e[:, i] = h
        num = (dy * (ref.rmsnorm(s + e, w, 0.1) - ref.rmsnorm(s - e, w, 0.1))).sum(1) / (2 * h)
        assert np.allclose(num, dx[:, i], atol=1e-8)
    assert np.allclose((dy * ref.rmsnorm(s, 1.0, 0.1)).sum(0), dw)
