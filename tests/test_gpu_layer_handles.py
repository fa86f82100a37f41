"""GPU tests of what a program keeps from call to call: weights and tables that change are taken as they are."""

import pytest
import torch

pytestmark = pytest.mark.gpu


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


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


ROWS, FF, HIDDEN = 5, 64, 256


def run(layer, a, w):
    return layer.gated(a, w, out_dtype=torch.float32).h


def test_weights_quantized_anew(fp4, layer):
    """Other values, other parameters (whose scales fit the buffers that were there), another shape."""
    group, tile = fp4.Params(), fp4.Params(block=(32, 32))
    rotated = fp4.Params(hadamard_n=64)
    x = rand(1, ROWS, HIDDEN)
    a, ar = fp4.quantize(x, group), fp4.quantize(x, rotated)
    q = [fp4.quantize(rand(2 + i, FF, HIDDEN), group) for i in (0, 1)]
    w = layer.GatedWeights(*q)
    run(layer, a, w)
    for act, p in ((a, group), (a, tile), (ar, rotated)):
        new = [rand(10 + i, FF, HIDDEN) for i in (0, 1)]
        for t, old in zip(new, (w.gate, w.up)):
            fp4.quantize(t, p, out=old)
        want = run(layer, act, layer.GatedWeights(*(fp4.quantize(t, p) for t in new)))
        assert torch.equal(run(layer, act, w), want)
        plan = layer.gated_plan(ROWS, w)
        assert plan.kernel == layer.gated_plan(ROWS, layer.GatedWeights(*(fp4.quantize(t, p) for t in new))).kernel
    half = [rand(20 + i, FF // 2, HIDDEN) for i in (0, 1)]
    for t, old in zip(half, q):
        fp4.quantize(t, group, out=old)
    got = run(layer, a, w)
    assert w.ff == FF // 2 and w.hidden == HIDDEN
    assert torch.equal(got, run(layer, a, layer.GatedWeights(*(fp4.quantize(t, group) for t in half))))


def test_one_of_two_weights_quantized_anew(fp4, layer):
    a = fp4.quantize(rand(1, ROWS, HIDDEN), fp4.Params())
    q = [fp4.quantize(rand(2 + i, FF, HIDDEN), fp4.Params()) for i in (0, 1)]
    w = layer.GatedWeights(*q)
    fp4.quantize(rand(4, FF, HIDDEN), fp4.Params(block=(32, 32)), out=q[1])
    with pytest.raises(fp4.Fp4Error):
        run(layer, a, w)
    fp4.quantize(rand(5, FF // 2, HIDDEN), fp4.Params(), out=q[1])
    with pytest.raises(ValueError, match="gate is"):
        run(layer, a, w)


def test_fused_weight_quantized_anew(fp4, layer):
    a = fp4.quantize(rand(1, ROWS, HIDDEN), fp4.Params())
    both = fp4.quantize(rand(2, 2 * FF, HIDDEN), fp4.Params())
    w = layer.GatedWeights(both)
    for p, n in ((fp4.Params(), FF), (fp4.Params(block=(32, 32)), FF), (fp4.Params(), FF // 2)):
        t = rand(3 + n, 2 * n, HIDDEN)
        fp4.quantize(t, p, out=both)
        assert torch.equal(run(layer, a, w), run(layer, a, layer.GatedWeights(fp4.quantize(t, p)))) and w.ff == n


def test_weights_assigned(fp4, layer):
    a = fp4.quantize(rand(1, ROWS, HIDDEN), fp4.Params())
    q = [fp4.quantize(rand(2 + i, FF, HIDDEN), fp4.Params()) for i in range(4)]
    w = layer.GatedWeights(q[0], q[1])
    run(layer, a, w)
    w.gate = q[2]
    assert torch.equal(run(layer, a, w), run(layer, a, layer.GatedWeights(q[2], q[1])))
    q[1].codes, q[1].scales = q[3].codes, q[3].scales
    assert torch.equal(run(layer, a, w), run(layer, a, layer.GatedWeights(q[2], q[3])))
    w.act = layer.GELU
    assert torch.equal(run(layer, a, w), run(layer, a, layer.GatedWeights(q[2], q[3], act=layer.GELU)))
    q[1].codes = q[3].codes[:16]
    with pytest.raises(ValueError, match="up.codes"):
        run(layer, a, w)
    for name in ("ff", "hidden", "device"):
        with pytest.raises(AttributeError):
            setattr(w, name, 1)


def test_rotary_table_assigned(layer):
    x, pos = rand(1, 7, 3, 64), torch.arange(7, dtype=torch.int32, device="cuda") * 1000
    f = [layer.rotary_frequencies(n, base=b, device="cuda")[0] for n, b in ((64, 10000.0), (64, 500000.0), (32, 10000.0))]
    want = [layer.rope(x, layer.Rotary(t), pos) for t in f]
    r = layer.Rotary(f[0])
    assert torch.equal(layer.rope(x, r, pos), want[0])
    for t, y in zip(f[1:], want[1:]):
        r.inv_freq = t
        assert torch.equal(layer.rope(x, r, pos), y) and r.rotary_dim == 2 * t.shape[0]
    r.inv_freq = f[0].clone()
    assert torch.equal(layer.rope(x, r, pos), want[0])
    r.inv_freq.copy_(f[1])  # in place
    assert torch.equal(layer.rope(x, r, pos), want[1])
    r.layout, r.scale = layer.INTERLEAVED, 2.0
    assert torch.equal(layer.rope(x, r, pos), layer.rope(x, layer.Rotary(f[1], layout=layer.INTERLEAVED, scale=2.0), pos))
    for bad in (f[0].cpu(), f[0].float(), f[0][::2], f[0][:0], f[0][None]):
        with pytest.raises(ValueError, match="inv_freq"):
            r.inv_freq = bad
        with pytest.raises(ValueError, match="inv_freq"):
            layer.Rotary(bad)
    r = layer.Rotary(f[0].clone())
    r.inv_freq.data = f[2]  # the same tensor with other memory and another size
    assert torch.equal(layer.rope(x, r, pos), want[2]) and r.rotary_dim == 32
    r.inv_freq.data = f[0][::2]
    with pytest.raises(ValueError, match="inv_freq"):
        layer.rope(x, r, pos)
    with pytest.raises(AttributeError):
        r.rotary_dim = 128
