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
