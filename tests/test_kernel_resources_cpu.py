"""CPU check of the built library's kernels between a layer's products: what they are said to hold in registers is not
kept in scratch memory. Read from the kernels' own descriptions in the code objects that were built here."""
import os
import struct

import pytest

msgpack = pytest.importorskip("msgpack")


def kernels(path):
    """The metadata of every gfx950 kernel in the library's offload bundles (ELF notes of type 32, msgpack)."""
    with open(path, "rb") as f:
        b = f.read()
    magic, at, out = b"__CLANG_OFFLOAD_BUNDLE__", 0, []
    while (at := b.find(magic, at)) >= 0:
        count, p = struct.unpack_from("<Q", b, at + 24)[0], at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", b, p)
            name = b[p + 24:p + 24 + length]
            p += 24 + length
            if b"gfx950" not in name or not size:
                continue
            e = b[at + offset:at + offset + size]
            sections, = struct.unpack_from("<Q", e, 40)
            each, n = struct.unpack_from("<HH", e, 58)
            for i in range(n):
                if struct.unpack_from("<I", e, sections + i * each + 4)[0] != 7:  # notes
                    continue
                o, = struct.unpack_from("<Q", e, sections + i * each + 24)
                name_size, desc_size, kind = struct.unpack_from("<III", e, o)
                start = o + 12 + (name_size + 3) // 4 * 4
                if kind == 32:
                    out += msgpack.unpackb(e[start:start + desc_size])["amdhsa.kernels"]
        at += len(magic)
    return out


def test_layer_kernels_use_registers_not_scratch():
    from bit_gemm_fwht_amd import fp4
    if not os.path.exists(fp4.LIB_PATH):
        from bit_gemm_fwht_amd import build
        build.build()
    found = [k for k in kernels(fp4.LIB_PATH) if any(n in k[".name"] for n in ("k_rmsnorm", "k_rope", "k_gated", "k_sum_slots"))]
    assert len(found) > 100
    used = {k[".name"]: k[".private_segment_fixed_size"] for k in found if k[".private_segment_fixed_size"]}
    # a few registers of the widest backward norm in bf16, a lane's few words in one of the gated tiles
    assert all(n <= 40 for n in used.values()) and len(used) <= 4, used
