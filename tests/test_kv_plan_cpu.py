"""CPU checks of what an attention call over the 8-bit cache accepts and how it is cut up, through the C
ABI alone: sizes near the limits of its counting."""
import ctypes

import pytest

from test_kv_abi_cpu import attn, batch, cache, kv  # noqa: F401  (kv: the fixture)


def query(kv, c, b, a):  # noqa: F811
    p = [ctypes.addressof(x) for x in (c, b, a)]
    return kv.lib().fp4_kv_attention_workspace_bytes(*p), kv.lib().fp4_kv_attention(*p, None, 0, None)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_tables_beyond_32_bit_keys_are_refused(kv, page):  # noqa: F811
    """Keys are counted in 32 bits, lookups a few steps past the last one included."""
    from bit_gemm_fwht_amd import fp4
    most = (2 ** 31 - 4096) // page
    for pages, want in ((most + 1, fp4.ERR_UNSUPPORTED), (2 ** 31 // page, fp4.ERR_UNSUPPORTED),
                        (2 ** 31 - 1, fp4.ERR_UNSUPPORTED), (most, fp4.ERR_WORKSPACE)):
        b = batch(kv, tokens=3, table_pages=pages, table_ld=pages)
        size, status = query(kv, cache(kv, page_tokens=page), b, attn(kv))
        assert status == want and (size == -1) == (want == fp4.ERR_UNSUPPORTED)


def plan(kv, lens, heads, group, dim, page, dtype, window=0, **kw):  # noqa: F811
    width = max(max(-(-c // page) for _, c in lens), 1)
    a = dict(tokens=sum(n for n, _ in lens), table_pages=width, table_ld=width, seqs=len(lens),
             max_tokens=max(n for n, _ in lens), max_context=max(c for _, c in lens))
    a.update(kw)
    p = kv.PlanC()
    args = (cache(kv, pages=1000, kv_heads=heads, page_tokens=page, head_dim=dim), batch(kv, **a),
            attn(kv, q_heads=heads * group, dtype=1 if dtype == "bf16" else 0, window=window), p)
    assert kv.lib().fp4_kv_attention_plan(*(ctypes.addressof(x) for x in args)) == 0
    return p


def test_shapes_of_the_kernel_tests(kv):  # noqa: F811
    """On 256 CUs (which is what is assumed where there is no GPU), the shapes that the GPU tests name after
    kernels take them."""
    from test_gpu_kv_kernels import KERNELS
    for name, (lens, heads, group, dim, page, dtype, kernel, rows) in KERNELS.items():
        p = plan(kv, lens, heads, group, dim, page, dtype)
        assert (p.kernel, p.tile_rows) == (kernel, rows), name


def test_plan_refuses_and_no_rows(kv):  # noqa: F811
    from bit_gemm_fwht_amd import fp4
    L = kv.lib()
    p = kv.PlanC(9, 9, 9, 9)
    c, b, a = cache(kv), batch(kv, tokens=0), attn(kv)
    q = [ctypes.addressof(x) for x in (c, b, a)]
    assert L.fp4_kv_attention_plan(*q, None) == fp4.ERR_INVALID_ARG
    assert L.fp4_kv_attention_plan(*q, ctypes.addressof(p)) == fp4.OK
    assert (p.kernel, p.tile_rows, p.waves, p.workgroups) == (0, 0, 0, 0)
    bad = attn(kv, q_heads=3)
    assert L.fp4_kv_attention_plan(q[0], q[1], ctypes.addressof(bad), ctypes.addressof(p)) == fp4.ERR_INVALID_ARG


def test_more_tiles_than_are_counted_are_refused(kv):  # noqa: F811
    """Tiles of 16 rows, one at least for each sequence and head, up to 2^30."""
    from bit_gemm_fwht_amd import fp4
    for seqs, heads, want in ((2 ** 20, 1024, fp4.OK), (2 ** 20 + 1, 1024, fp4.ERR_UNSUPPORTED),
                              (2 ** 28, 4, fp4.OK), (2 ** 28, 5, fp4.ERR_UNSUPPORTED), (2 ** 28, 60000, fp4.ERR_UNSUPPORTED)):
        args = cache(kv, kv_heads=heads), batch(kv, tokens=1, seqs=seqs), attn(kv, q_heads=heads), kv.PlanC()
        assert kv.lib().fp4_kv_attention_plan(*(ctypes.addressof(x) for x in args)) == want


@pytest.mark.parametrize("lens,heads,group", [([(1, 5000)], 8, 4), ([(1, 5000)], 65535, 1), ([(1, 9000)] * 3000, 64, 1),
                                              ([(9, 5000)] * 20, 16, 2)])
def test_wide_tables_are_still_split(kv, lens, heads, group):  # noqa: F811
    """However many keys a table has room for, contexts are dealt in shares."""
    for width in (40, 4000, 2 ** 20, 2 ** 23, 2 ** 24 - 32):
        p = plan(kv, lens, heads, group, 16, 128, "bf16", max_context=0, table_pages=width, table_ld=width)
        assert p.kernel in (kv.PLAN_ROWS_SPLIT, kv.PLAN_ROWS_NEAR), width


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [16, 128, 256])
@pytest.mark.parametrize("tokens,seqs,heads,group", [
    (2 ** 22, 2 ** 22, 32, 1), (2 ** 22, 2 ** 18, 32, 1), (2 ** 26, 1, 32, 1), (2 ** 27, 1, 32, 2), (2 ** 29, 1, 16, 1),
    (2 ** 24, 1, 1, 64), (2 ** 27, 2 ** 20, 4, 8),
])
def test_launches_stay_within_2_32_threads(kv, tokens, seqs, heads, group, dim, dtype):  # noqa: F811
    for context, window in ((64, 0), (2000, 0), (2 ** 20, 0), (2 ** 20, 16)):
        p = plan(kv, [(1, context)], heads, group, dim, 128, dtype, window, tokens=tokens, seqs=seqs,
                 max_tokens=-(-tokens // seqs), max_context=context)
        assert 0 < p.workgroups * p.waves * 64 < 2 ** 32
