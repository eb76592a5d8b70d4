"""What the built library says of its own kernels: the metadata that the compiler writes beside each of them."""
import os
import struct

import pytest

from mxfp4_latent_mixture_sigmoid_amd import abi

MAGIC, SHT_NOTE, NT_METADATA = b"__CLANG_OFFLOAD_BUNDLE__", 7, 32


def code_objects(data):
    """The gfx950 ELF images in a library."""
    at = data.find(MAGIC)
    while at >= 0:
        count, p = struct.unpack_from("<Q", data, at + 24)[0], at + 32
        for _ in range(count if count < 16 else 0):
            offset, size, length = struct.unpack_from("<3Q", data, p)
            if size and b"gfx950" in data[p + 24:p + 24 + length]:
                yield data[at + offset:at + offset + size]
            p += 24 + length
        at = data.find(MAGIC, at + 24)


def kernels(path):
    """name -> its metadata."""
    msgpack = pytest.importorskip("msgpack")
    found = {}
    for elf in code_objects(open(path, "rb").read()):
        sections, (entry, count) = struct.unpack_from("<Q", elf, 40)[0], struct.unpack_from("<2H", elf, 58)
        for i in range(count):
            kind, = struct.unpack_from("<I", elf, sections + i * entry + 4)
            if kind != SHT_NOTE:
                continue
            at, size = struct.unpack_from("<2Q", elf, sections + i * entry + 24)
            end = at + size
            while at + 12 <= end:
                name, length, kind = struct.unpack_from("<3I", elf, at)
                at += 12 + (name + 3) // 4 * 4
                if kind == NT_METADATA:
                    for k in msgpack.unpackb(elf[at:at + length], strict_map_key=False).get("amdhsa.kernels", []):
                        found[k[".name"]] = k
                at += (length + 3) // 4 * 4
    return found


@pytest.fixture(scope="module")
def built():
    if not os.path.exists(abi.LIB_PATH):
        from mxfp4_latent_mixture_sigmoid_amd import build
        build.build()
    return kernels(abi.LIB_PATH)


@pytest.mark.parametrize("kind", ["wide_kernel", "tile_kernel"])
@pytest.mark.parametrize("product", ["Int8", "Bf16"])
def test_dense_products_keep_their_sums_in_registers(built, kind, product):
    """An epilogue that is not inlined takes the sums by address, so that they live in memory and every instruction of the
    main loop stores its own: 8192 x 7168 x 14336 codes took 11 ms in the place of 0.61."""
    names = [n for n in built if kind in n and f"_{len(product)}{product}" in n]
    assert names, "no such kernel in the library"
    assert {n: built[n][".private_segment_fixed_size"] for n in names} == dict.fromkeys(names, 0)


def test_no_other_kernel_keeps_anything_in_memory(built):
    """But the few-token layer's, whose items that help each other are cold."""
    names = [n for n in built if "decode_kernel" not in n]
    assert len(names) > 100
    assert {n: built[n][".private_segment_fixed_size"] for n in names} == dict.fromkeys(names, 0)
