"""Registers of the built kernels, from the metadata in the library: what keeps a kernel's registers in scratch memory shows here first."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from conftest import ROOT

READELF = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-readelf")
LIB = os.path.join(ROOT, "block_scaled_quantized_amd", "libmxgemm.so")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"

if not shutil.which(READELF):
    pytest.skip("needs llvm-readelf", allow_module_level=True)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: {field: number}} of every gfx950 code object in the library."""
    if not os.path.exists(LIB):
        from block_scaled_quantized_amd import build
        build.build()
    data = open(LIB, "rb").read()
    found = {}
    for m in re.finditer(MAGIC, data):
        # a bundle: the number of its entries, then of each its offset, size and the length of its target's name
        at, (n,) = m.start() + len(MAGIC) + 8, struct.unpack_from("<Q", data, m.start() + len(MAGIC))
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            target, at = data[at + 24:at + 24 + length], at + 24 + length
            if b"gfx950" not in target or not size:
                continue
            path = tmp_path_factory.mktemp("object") / "code"
            path.write_bytes(data[m.start() + offset:m.start() + offset + size])
            notes = subprocess.run([READELF, "--notes", str(path)], capture_output=True, text=True, check=True).stdout
            for kernel in notes.split("  - .")[1:]:
                name = re.search(r"\.symbol: +(\S+?)\.kd", kernel)
                if name:
                    found[name[1]] = {k: int(v) for k, v in re.findall(r"\.(private_segment_fixed_size|vgpr_spill_count|vgpr_count): +(\d+)", kernel)}
    assert found
    return found


def decode(kernels):
    """The attention kernels of rows of their own: the last parameter of the others is whether rows go on from shared positions."""
    return {k: v for k, v in kernels.items() if "decode_kernelI" in k and "Lb1EEEv" not in k}


def test_every_kernel_is_there(kernels):
    names = " ".join(kernels)
    for part in ("decode_kernel", "prefix_kernel", "norm_kernel", "tile_kernel", "rows_kernel", "step_kernel"):
        assert part in names


def test_decode_without_shared_positions_keeps_its_registers(kernels):
    """Rows of their own do not pay for code that only shared positions need: shares of up to 64 elements with one tile of heads fit three waves per SIMD (168 registers)
    with at most one register in scratch memory, and no variant of up to 128 elements has more."""
    small = {k: v for k, v in decode(kernels).items() if "decode_kernelILi64" in k or "decode_kernelILi128" in k}
    assert small
    for name, v in small.items():
        assert v["private_segment_fixed_size"] <= 8 and v["vgpr_spill_count"] <= 1, (name, v)
        if "ILi64E" in name and "Lb1ELi1E" in name:
            assert v["vgpr_count"] <= 168, (name, v)
