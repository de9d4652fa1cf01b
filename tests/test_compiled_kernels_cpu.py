"""What the compiler made of the kernels, read from the built library's own
metadata on the CPU.

The 4-bit products keep addresses over a loop with blocks for some of the lanes.
Above 256 vector registers the compiler parks values in the other half of a
lane's registers, and it may do so inside such a block: the other lanes then
read back what was there before, and a memory fault follows where it is an
address.  So no instance may use the other half, and none may spill."""
import os
import re
import struct
import subprocess

import pytest

from expert_ffn_dispatch_amd import _lib
from expert_ffn_dispatch_amd.build import ARCH, HIPCC

READELF = os.path.join(os.path.dirname(os.path.realpath(HIPCC)), "..", "lib", "llvm", "bin", "llvm-readelf")


def code_objects(path):
    """The device programs of a library: every bundle's entry for the GPU."""
    data = open(path, "rb").read()
    for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data):
        at = m.end() + 8
        for _ in range(struct.unpack_from("<Q", data, m.end())[0]):
            offset, size, length = struct.unpack_from("<3Q", data, at)
            name = data[at + 24:at + 24 + length].decode()
            at += 24 + length
            if name.endswith(ARCH):
                yield data[m.start() + offset:m.start() + offset + size]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Name -> its numbers in the metadata."""
    if not os.path.exists(READELF):
        pytest.skip("llvm-readelf is not installed")
    if not os.path.exists(_lib.LIB_PATH):
        from expert_ffn_dispatch_amd import build
        build.build()
    out = {}
    for i, obj in enumerate(code_objects(_lib.LIB_PATH)):
        f = tmp_path_factory.mktemp("co") / f"{i}.o"
        f.write_bytes(obj)
        text = subprocess.run([READELF, "--notes", str(f)], capture_output=True, text=True, check=True).stdout
        for block in re.split(r"\n  - \.agpr_count:", text)[1:]:
            block = " .agpr_count:" + block
            number = dict(re.findall(r"\.(\w+):\s+(\d+)", block))
            out[re.search(r"\.symbol:\s+'?([\w.]+)", block)[1]] = {k: int(v) for k, v in number.items()}
    return out


def test_every_kernel_is_found(kernels):
    for part in ("fp4_stream_kernel", "widen_kernel", "adamw_kernel", "gated_grad_kernel", "matmul_tile_kernel"):
        assert any(part in name for name in kernels), part


def test_4_bit_products_use_one_half_of_the_registers(kernels):
    seen = 0
    for name, k in kernels.items():
        if "fp4_stream_kernel" in name:
            seen += 1
            assert k["agpr_count"] == 0 and k["vgpr_count"] <= 256, (name, k["agpr_count"], k["vgpr_count"])
            assert k["vgpr_spill_count"] == 0 and k["private_segment_fixed_size"] == 0, name
    assert seen >= 2
