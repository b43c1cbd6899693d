"""Scratch memory of the kernels of the grouped products, as the compiler notes it in the built library: values that
its loops would read again from memory."""
import os
import struct

import pytest

import bit_gathered_quantized_amd as bgq

msgpack = pytest.importorskip("msgpack")


def code_objects(data):
    """The gfx950 objects in the library's offload bundles."""
    at = data.find(b"__CLANG_OFFLOAD_BUNDLE__")
    while at >= 0:
        entry = at + 32
        for _ in range(struct.unpack_from("<Q", data, at + 24)[0]):
            start, size, name = struct.unpack_from("<QQQ", data, entry)
            if b"gfx950" in data[entry + 24:entry + 24 + name]:
                yield data[at + start:at + start + size]
            entry += 24 + name
        at = data.find(b"__CLANG_OFFLOAD_BUNDLE__", at + 1)


def kernels(elf):
    """Kernel descriptions in an object's notes."""
    (table,), (step, count) = struct.unpack_from("<Q", elf, 40), struct.unpack_from("<HH", elf, 58)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, table + i * step + 4)
        at, size = struct.unpack_from("<QQ", elf, table + i * step + 24)
        if kind != 7:  # notes
            continue
        names, desc, _ = struct.unpack_from("<III", elf, at)
        body = at + 12 + (names + 3) // 4 * 4
        yield from msgpack.unpackb(elf[body:body + desc])["amdhsa.kernels"]


@pytest.fixture(scope="module")
def scratch():
    if not os.path.exists(bgq.LIB_PATH):
        pytest.skip("the library is not built")
    with open(bgq.LIB_PATH, "rb") as f:
        data = f.read()
    return {k[".name"]: k[".private_segment_fixed_size"] for o in code_objects(data) for k in kernels(o)}


def test_tiles_of_256_by_256(scratch):
    """Their results take half of the registers.  What does not fit stays the same in both types of the output: the store's
    addresses are made after the products, not kept through them."""
    big = {n: s for n, s in scratch.items() if "moe_grouped_product" in n and "ELi256E" in n}
    assert len(big) == 8
    assert max(big.values()) <= 64, big


def test_the_other_grouped_kernels(scratch):
    rest = {n: s for n, s in scratch.items() if ("moe_grouped" in n or "moe_mx" in n) and "ELi256E" not in n}
    assert len(rest) > 40
    assert not any(rest.values()), {n: s for n, s in rest.items() if s}
