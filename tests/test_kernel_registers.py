"""The built library's own kernel descriptions (CPU): no few-token kernel keeps more than a handful of values in scratch
memory, where each would be stored and loaded again within the loop over K."""
import os
import struct

import pytest

import combine_expert_histogram_amd.binding as b

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
MOST = 8


def code_objects(blob):
    """The gfx950 ELF images of the library's offload bundles."""
    at = blob.find(MAGIC)
    while at >= 0:
        pos = at + len(MAGIC)
        count, = struct.unpack_from("<Q", blob, pos)
        pos += 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", blob, pos)
            name = blob[pos + 24:pos + 24 + length]
            pos += 24 + length
            if b"gfx950" in name and size:
                yield blob[at + offset:at + offset + size]
        at = blob.find(MAGIC, pos)


def kernels(elf):
    """The entries of the AMDGPU metadata note (type 32)."""
    msgpack = pytest.importorskip("msgpack")
    assert elf[:4] == b"\x7fELF"
    table, = struct.unpack_from("<Q", elf, 0x28)
    entry, count = struct.unpack_from("<HH", elf, 0x3A)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, table + i * entry + 4)
        pos, size = struct.unpack_from("<QQ", elf, table + i * entry + 0x18)
        end = pos + size
        while kind == 7 and pos < end:                           # notes
            names, descs, what = struct.unpack_from("<III", elf, pos)
            desc = pos + 12 + (names + 3) // 4 * 4
            if what == 32 and elf[pos + 12:pos + 18] == b"AMDGPU":
                yield from msgpack.unpackb(elf[desc:desc + descs])["amdhsa.kernels"]
            pos = desc + (descs + 3) // 4 * 4


@pytest.fixture(scope="module")
def found():
    if not os.path.exists(b.LIB_PATH):
        from combine_expert_histogram_amd import build
        build.build()
    with open(b.LIB_PATH, "rb") as f:
        blob = f.read()
    return [k for elf in code_objects(blob) for k in kernels(elf)]


@pytest.mark.parametrize("kernel", ["matvec_kernel", "matvec_wide_kernel", "gate_up_kernel", "down_kernel",
                                    "route_topk_kernel"])
def test_no_kernel_spills_more_than_a_handful(found, kernel):
    these = [k for k in found if kernel in k[".name"]]
    assert these
    spilled = {k[".name"]: k[".vgpr_spill_count"] for k in these if k[".vgpr_spill_count"] > MOST}
    assert not spilled
