"""CPU checks of the key / value cache calls: every rejection happens on the host before any device
call, the size query agrees with the call, and the plain reference of the GPU tests against values
worked out by hand."""
import ctypes

import numpy as np
import pytest

import kv_reference as ref


@pytest.fixture(scope="module")
def kv():
    import os
    from bit_gemm_fwht_amd import fp4, kv as m
    if not os.path.exists(fp4.LIB_PATH):
        from bit_gemm_fwht_amd import build
        build.build()
    m.lib()
    return m


def cache(kv, **kw):
    a = dict(k_codes=0x10000, v_codes=0x20000, k_scales=0x30000, v_scales=0x40000, pages=10, kv_heads=2,
             page_tokens=32, head_dim=128)
    a.update(kw)
    return kv.CacheC(**a)


def batch(kv, **kw):
    a = dict(cu_tokens=0x50000, context=0x60000, table=0x70000, tokens=0, table_ld=5, seqs=1, table_pages=5,
             max_tokens=0, max_context=0)
    a.update(kw)
    return kv.BatchC(**a)


def attn(kv, **kw):
    a = dict(q=0x100000, out=0x200000, lse=None, ldq=512, ldq_head=128, ldo=512, ldo_head=128, dtype=1, q_heads=4,
             causal=1, window=0, scale=0.1)
    a.update(kw)
    return kv.AttnC(**a)


BAD_PLACES = [
    (dict(k_codes=None), {}, "INVALID_ARG"), (dict(v_codes=None), {}, "INVALID_ARG"),
    (dict(k_scales=None), {}, "INVALID_ARG"), (dict(v_scales=None), {}, "INVALID_ARG"),
    (dict(pages=0), {}, "INVALID_ARG"), (dict(kv_heads=0), {}, "INVALID_ARG"), (dict(head_dim=-16), {}, "INVALID_ARG"),
    (dict(page_tokens=0), {}, "INVALID_ARG"), (dict(v_codes=0x10000), {}, "INVALID_ARG"),
    (dict(page_tokens=24), {}, "UNSUPPORTED"), (dict(page_tokens=8), {}, "UNSUPPORTED"),
    (dict(page_tokens=256), {}, "UNSUPPORTED"), (dict(head_dim=72), {}, "UNSUPPORTED"),
    (dict(head_dim=272), {}, "UNSUPPORTED"), (dict(kv_heads=70000), {}, "UNSUPPORTED"),
    (dict(k_codes=0x10008), {}, "ALIGNMENT"), (dict(v_codes=0x20001), {}, "ALIGNMENT"),
    ({}, dict(cu_tokens=None), "INVALID_ARG"), ({}, dict(context=None), "INVALID_ARG"),
    ({}, dict(table=None), "INVALID_ARG"), ({}, dict(seqs=0), "INVALID_ARG"), ({}, dict(table_pages=0), "INVALID_ARG"),
    ({}, dict(table_ld=4), "INVALID_ARG"), ({}, dict(tokens=-1), "INVALID_ARG"),
    ({}, dict(max_tokens=-1), "INVALID_ARG"), ({}, dict(max_context=-5), "INVALID_ARG"),
    ({}, dict(tokens=1 << 31), "UNSUPPORTED"), ({}, dict(seqs=1 << 30), "UNSUPPORTED"),
]


@pytest.mark.parametrize("c,b,want", BAD_PLACES)
def test_cache_and_batch_are_refused_by_every_call(kv, c, b, want):
    from bit_gemm_fwht_amd import fp4
    L, want = kv.lib(), getattr(fp4, "ERR_" + want)
    cc, bb, a = cache(kv, **c), batch(kv, **{"tokens": 3, **b}), attn(kv)
    pc, pb, pa = (ctypes.addressof(x) for x in (cc, bb, a))
    assert L.fp4_kv_append(pc, pb, 0x100000, 256, 128, 0x200000, 256, 128, 1, 1, None) == want
    assert L.fp4_kv_read(pc, pb, 0x100000, 256, 128, 0x200000, 256, 128, 1, None) == want
    assert L.fp4_kv_attention(pc, pb, pa, None, 0, None) == want
    assert L.fp4_kv_attention_workspace_bytes(pc, pb, pa) == -1


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"),
    (dict(ldk=-256), "INVALID_ARG"), (dict(k=0x10000), "INVALID_ARG"), (dict(v=0x40000), "INVALID_ARG"),
    (dict(k=0x100008), "ALIGNMENT"), (dict(ldk=257), "ALIGNMENT"), (dict(ldv_head=4), "ALIGNMENT"),
    (dict(mode=2), "UNSUPPORTED"), (dict(mode=4), "UNSUPPORTED"), (dict(mode=-1), "UNSUPPORTED"),
])
def test_append_refuses(kv, kw, want):
    from bit_gemm_fwht_amd import fp4
    a = dict(k=0x100000, ldk=256, ldk_head=128, v=0x200000, ldv=256, ldv_head=128, dtype=1, mode=1)
    a.update(kw)
    c, b = cache(kv), batch(kv, tokens=3)
    assert kv.lib().fp4_kv_append(ctypes.addressof(c), ctypes.addressof(b), a["k"], a["ldk"], a["ldk_head"], a["v"],
                                  a["ldv"], a["ldv_head"], a["dtype"], a["mode"], None) == getattr(fp4, "ERR_" + want)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), "INVALID_ARG"), (dict(k=0x200000), "INVALID_ARG"), (dict(ldk=128), "INVALID_ARG"),
    (dict(ldv_head=0), "INVALID_ARG"), (dict(ldv=0), "INVALID_ARG"), (dict(v=0x30000), "INVALID_ARG"),
    (dict(v=0x200004), "ALIGNMENT"), (dict(dtype=-1), "INVALID_ARG"),
])
def test_read_refuses(kv, kw, want):
    """Among others, outputs whose rows would lie over one another."""
    from bit_gemm_fwht_amd import fp4
    a = dict(k=0x100000, ldk=256, ldk_head=128, v=0x200000, ldv=256, ldv_head=128, dtype=1)
    a.update(kw)
    c, b = cache(kv), batch(kv, tokens=3)
    assert kv.lib().fp4_kv_read(ctypes.addressof(c), ctypes.addressof(b), a["k"], a["ldk"], a["ldk_head"], a["v"],
                                a["ldv"], a["ldv_head"], a["dtype"], None) == getattr(fp4, "ERR_" + want)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(dtype=5), "INVALID_ARG"),
    (dict(q_heads=3), "INVALID_ARG"), (dict(q_heads=0), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(out=0x100000), "INVALID_ARG"), (dict(lse=0x200000), "INVALID_ARG"), (dict(out=0x20000), "INVALID_ARG"),
    (dict(ldo=128), "INVALID_ARG"), (dict(ldo_head=64), "INVALID_ARG"), (dict(ldq=-512), "INVALID_ARG"),
    (dict(q=0x100002), "ALIGNMENT"), (dict(ldq=516), "ALIGNMENT"), (dict(ldo_head=132), "ALIGNMENT"),
])
def test_attention_refuses(kv, kw, want):
    from bit_gemm_fwht_amd import fp4
    c, b, a = cache(kv), batch(kv, tokens=3), attn(kv, **kw)
    got = kv.lib().fp4_kv_attention(ctypes.addressof(c), ctypes.addressof(b), ctypes.addressof(a), 0x900000, 1 << 40, None)
    assert got == getattr(fp4, "ERR_" + want)


def test_attention_workspace(kv):
    """A split call without its workspace is refused; no rows need none and queue nothing."""
    from bit_gemm_fwht_amd import fp4
    L = kv.lib()
    c, b, a = cache(kv), batch(kv, tokens=1, table_pages=4000, table_ld=4000), attn(kv)
    p = [ctypes.addressof(x) for x in (c, b, a)]
    need = L.fp4_kv_attention_workspace_bytes(*p)
    assert need > 0
    assert L.fp4_kv_attention(*p, None, need, None) == fp4.ERR_WORKSPACE
    assert L.fp4_kv_attention(*p, 0x900000, need - 1, None) == fp4.ERR_WORKSPACE
    assert L.fp4_kv_attention(*p, 0x900008, need, None) == fp4.ERR_ALIGNMENT
    b.tokens = 0
    assert L.fp4_kv_attention_workspace_bytes(*p) == 0
    assert L.fp4_kv_attention(*p, None, 0, None) == fp4.OK
    assert L.fp4_kv_append(p[0], p[1], None, 0, 0, None, 0, 0, 1, 1, None) == fp4.OK
    assert L.fp4_kv_read(p[0], p[1], None, 0, 0, None, 0, 0, 1, None) == fp4.OK


def test_reference_numbers():
    assert ref.E4M3[0x7E] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[0x38] == 1 and ref.E4M3[0xB8] == -1
    x = np.array([0.0, 1.0, 1.0625, 1.1875, 447.0, 1e9, -0.4375, 2.0 ** -10, 2.0 ** -10 * 1.01, 3 * 2.0 ** -10])
    assert np.array_equal(ref.E4M3[ref.e4m3_encode(x)], [0, 1, 1, 1.25, 448, 448, -0.4375, 0, 2.0 ** -9, 2.0 ** -8])
    assert np.array_equal(ref.e4m3_encode(ref.E4M3[:0x7F]), np.arange(0x7F))
    assert [ref.exponent(a, c) for a, c in ((448, False), (448, True), (449, True), (511, False), (512, False), (0, True))] \
        == [0, 0, 1, 0, 1, -127]


def test_reference_attention_by_hand():
    """Two keys with scores 0 and ln 3, values 1 and 5: (1 + 3 * 5) / 4; and the empty row."""
    c = ref.Cache(np.zeros((1, 1, 16, 16), np.uint8), np.zeros((1, 1, 16, 16), np.uint8),
                  np.full((1, 1), 127, np.uint8), np.full((1, 1), 127, np.uint8))
    c.k[0, 0, 1, 0] = 0x38
    c.v[0, 0, :, 0] = 0x38
    c.v[0, 0, :, 1] = 0x4A
    q = np.zeros((2, 1, 16))
    q[:, 0, 0] = np.log(3.0)
    o, lse, *_ = ref.attention(q, c, [0, 1, 2], [2, 0], np.zeros((2, 1), int), 1.0, True, 0)
    assert np.allclose(o[0], 4.0) and np.allclose(lse[0], np.log(4.0))
    assert not o[1].any() and np.isneginf(lse[1]).all()


def test_reference_append_by_hand():
    """A block at exponent 0 that receives 896 = 2 * 448: exponent 1, the older codes halved."""
    c = ref.Cache(np.full((1, 1, 16, 16), 0x38, np.uint8), np.full((1, 1, 16, 16), 0x38, np.uint8),
                  np.full((1, 1), 127, np.uint8), np.full((1, 1), 127, np.uint8))
    x = np.full((1, 1, 16), 896.0)
    ref.append(c, x, x / 1024, np.array([0, 1]), np.array([4]), np.zeros((1, 1), int), True)
    assert c.ks[0, 0] == 128 and c.vs[0, 0] == 127
    assert (c.k[0, 0, :3] == 0x30).all() and (c.k[0, 0, 3] == 0x7E).all() and (c.k[0, 0, 4:] == 0x38).all()
    assert (ref.E4M3[c.v[0, 0, :, 3]] == 0.875).all() and (c.v[0, 0, :, :3] == 0x38).all()
