"""CPU checks of the limits of the calls between a layer's products: sizes whose bytes leave 64 bits are refused on the
host, in the size query, the plan and the call alike."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def layer():
    import os
    from bit_gemm_fwht_amd import fp4, layer as m
    if not os.path.exists(fp4.LIB_PATH):
        from bit_gemm_fwht_amd import build
        build.build()
    m.lib()
    return m


@pytest.mark.parametrize("m,f,ok", [((1 << 31) - 1, (1 << 31) - 128, False), (1 << 30, 1 << 30, False), (1 << 29, 1 << 30, False),
                                    (1 << 28, 1 << 30, True), ((1 << 31) - 1, 1 << 27, True)])
def test_gated_sizes(layer, m, f, ok):
    """A workspace of 4 M F bytes (a rotation past the columns of a block)."""
    from bit_gemm_fwht_amd import fp4
    L, k = layer.lib(), 64
    p, pq = fp4.QParams(0, 1, 32, 0, 0, 0, 0), fp4.QParams(0, 1, 32, 0, 0, 128, 0)
    a, g, u = (fp4.QTensorC(base, base + 0x10000, None, rows, k, p) for base, rows in ((0x100000, m), (0x200000, f), (0x300000, f)))
    o = layer.GatedC(0x700000, None, f, 0, 1, 0)
    q = fp4.QTensorC(0x900000, 0xA00000, None, 0, 0, pq)
    plan = layer.GatedPlanC()
    args = [ctypes.addressof(x) for x in (a, g, u, o, pq)]
    need = L.fp4_gemm_gated_workspace_bytes(*args)
    status = L.fp4_gemm_gated_plan(*args, ctypes.addressof(plan))
    call = L.fp4_gemm_gated(*args, ctypes.addressof(q), None, 0, None)
    if ok:  # (nothing is launched without its workspace)
        assert need == 4 * m * f and status == fp4.OK and plan.quantize_pass == 1 and call == fp4.ERR_WORKSPACE
    else:
        assert need == -1 and status == call == fp4.ERR_UNSUPPORTED
