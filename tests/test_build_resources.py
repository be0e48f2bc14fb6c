"""No kernel of the linear operators spills vector registers: their waits count loads in flight (a
reload from scratch is one more), and scratch traffic shares the path of their weights."""

import os
import struct

import pytest

from mxfp4_quantized_expert_amd import binding

msgpack = pytest.importorskip("msgpack")


def code_objects(data):
    """The gfx950 ELF images of a library's offload bundles."""
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := data.find(magic, at)) >= 0:
        (count,) = struct.unpack_from("<Q", data, at + len(magic))
        entry = at + len(magic) + 8
        for _ in range(count if count < 16 else 0):  # (the loader's own copy of the magic is no bundle)
            offset, size, length = struct.unpack_from("<3Q", data, entry)
            name = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            if b"gfx950" in name and size > 0:
                yield data[at + offset:at + offset + size]
        at += len(magic)


def kernels(elf):
    """The kernels' metadata: the AMDGPU note (type 32) of a code object."""
    table, = struct.unpack_from("<Q", elf, 40)
    width, count = struct.unpack_from("<2H", elf, 58)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, table + i * width + 4)
        offset, size = struct.unpack_from("<2Q", elf, table + i * width + 24)
        if kind != 7:  # notes
            continue
        name, desc, note = struct.unpack_from("<3I", elf, offset)
        if note == 32:
            at = offset + 12 + (name + 3) // 4 * 4
            yield from msgpack.unpackb(elf[at:at + desc], strict_map_key=False)["amdhsa.kernels"]


def test_no_vector_register_spills():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("the library is not built")
    with open(binding.LIB_PATH, "rb") as f:
        data = f.read()
    found = {k[".name"]: k[".vgpr_spill_count"] for elf in code_objects(data) for k in kernels(elf)}
    linear = {n: c for n, c in found.items() if "linear_" in n}
    assert len(linear) >= 30  # the kernels were found at all
    assert not {n: c for n, c in linear.items() if c}
