"""What the compiler gave the kernels of the built library, from its code objects' metadata (CPU).

The chains of the gated delta rule wait by counts of the memory operations that their loops issue:
a spill inside such a loop would add to them, and a wait would cover too little."""
import os
import struct

import msgpack
import pytest

import state_space_model_amd as ssd

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(blob):
    """The gfx950 ELF images in a library's bundles."""
    at = blob.find(MAGIC)
    while at >= 0:
        (n,) = struct.unpack_from("<Q", blob, at + len(MAGIC))
        pos = at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", blob, pos)
            name = blob[pos + 24:pos + 24 + length].decode()
            pos += 24 + length
            if "gfx950" in name and size:
                yield blob[at + offset:at + offset + size]
        at = blob.find(MAGIC, pos)


def kernels(image):
    """The kernels' entries in an image's metadata note."""
    shoff, = struct.unpack_from("<Q", image, 0x28)
    shentsize, shnum = struct.unpack_from("<HH", image, 0x3A)
    for i in range(shnum):
        kind, = struct.unpack_from("<I", image, shoff + i * shentsize + 4)
        if kind != 7:                                   # SHT_NOTE
            continue
        offset, size = struct.unpack_from("<QQ", image, shoff + i * shentsize + 24)
        end = offset + size
        while offset < end:
            name, desc, note = struct.unpack_from("<III", image, offset)
            body = offset + 12 + (name + 3) // 4 * 4
            if note == 32:                              # NT_AMDGPU_METADATA
                yield from msgpack.unpackb(image[body:body + desc])["amdhsa.kernels"]
            offset = body + (desc + 3) // 4 * 4


@pytest.fixture(scope="module")
def built():
    with open(os.path.join(os.path.dirname(ssd.__file__), "libssd.so"), "rb") as f:
        return {k[".name"]: k for image in code_objects(f.read()) for k in kernels(image)}


def test_kernels_of_the_delta_rule_do_not_spill(built):
    seen = {}
    for name, k in built.items():
        if "k_delta_" in name:
            kind = name[name.index("k_delta_"):].split("I")[0].split("E")[0]
            seen[kind] = seen.get(kind, 0) + 1
            assert k[".private_segment_fixed_size"] == 0, (name, k[".private_segment_fixed_size"])
            assert k[".vgpr_spill_count"] == 0 and k[".sgpr_spill_count"] == 0, name
    # keys of 64 and 128, whole or not; columns shared alone and in pairs
    assert seen["k_delta_tokens"] == seen["k_delta_both_tokens"] == 8, seen
    assert seen["k_delta_columns"] == seen["k_delta_both_columns"] == 4 and seen["k_delta_grads"] == 8, seen
