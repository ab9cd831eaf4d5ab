"""Registers of the attention kernels, from the metadata of the built library (CPU only)."""
import re
import struct

import pytest

from sparse_matrix_vector_amd import _lib as L

msgpack = pytest.importorskip("msgpack")


def device_images(data):
    """The gfx950 code objects that the library's offload bundles hold."""
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := data.find(magic, at)) >= 0:
        n, = struct.unpack_from("<Q", data, at + len(magic))
        pos = at + len(magic) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, pos)
            if b"gfx950" in data[pos + 24:pos + 24 + length]:
                yield data[at + offset:at + offset + size]
            pos += 24 + length
        at = pos


def kernels(image):
    """The kernel records of a code object's metadata note."""
    shoff, = struct.unpack_from("<Q", image, 0x28)
    shentsize, shnum = struct.unpack_from("<HH", image, 0x3A)
    for i in range(shnum):
        base = shoff + i * shentsize
        if struct.unpack_from("<I", image, base + 4)[0] != 7:                 # SHT_NOTE
            continue
        pos, size = struct.unpack_from("<QQ", image, base + 0x18)
        end = pos + size
        while pos < end:
            namesz, descsz, kind = struct.unpack_from("<III", image, pos)
            desc = pos + 12 + (namesz + 3) // 4 * 4
            if kind == 32:                                                    # AMDGPU metadata
                yield from msgpack.unpackb(image[desc:desc + descsz])["amdhsa.kernels"]
            pos = desc + (descsz + 3) // 4 * 4


def test_attention_keeps_to_ordinary_registers():
    """Sums and operands in 256 ordinary registers (two waves a SIMD), none in accumulation registers."""
    with open(L.LIB_PATH, "rb") as f:
        data = f.read()
    units = [k for image in device_images(data) for k in kernels(image) if re.search(r"units_kernel", k[".name"])]
    assert len(units) == 60                # two types, three formats, four forms at 64 and 128 columns and two at 256
    for k in units:
        assert k[".agpr_count"] == 0 and k[".vgpr_count"] <= 256, (k[".name"], k[".agpr_count"], k[".vgpr_count"])
