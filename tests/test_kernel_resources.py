"""What the compiler made of the kernels in the built library, read from its code objects'
metadata on a machine without a GPU: a k-tile that is staged in registers must be in registers."""

import os
import re
import struct
import subprocess

import pytest

import software_pipelined_tiled_gemm_amd as spg

READELF = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-readelf")


def _code_objects(path):
    """The gfx950 code objects of a library's offload bundles."""
    data = open(path, "rb").read()
    for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data):
        p = m.end()
        n, = struct.unpack_from("<Q", data, p)
        p += 8
        if n > 8:                                        # the text elsewhere in the file
            continue
        for _ in range(n):
            at, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length]
            p += 24 + length
            if name.endswith(b"gfx950"):
                yield data[m.start() + at:m.start() + at + size]


@pytest.fixture(scope="module")
def scratch(tmp_path_factory):
    """Bytes of scratch memory a lane of every kernel, by its mangled name."""
    if not os.path.exists(spg.LIB_PATH):
        pytest.fail("libspgemm.so is not built; run __graft_entry__.build()")
    f = tmp_path_factory.mktemp("objects") / "one.co"
    found = {}
    for obj in _code_objects(spg.LIB_PATH):
        f.write_bytes(obj)
        notes = subprocess.run([READELF, "--notes", str(f)], capture_output=True, text=True, check=True).stdout
        for kernel in re.split(r"\n  - ", notes)[1:]:
            name = re.search(r"\.symbol:\s+'?([^\s']+)", kernel)
            size = re.search(r"\.private_segment_fixed_size:\s+(\d+)", kernel)
            if name and size:
                found[name.group(1)] = int(size.group(1))
    return found


def test_misaligned_gemm_stages_in_registers(scratch):
    # pipelined_gemm<BF16, B_NK, BM, BN, BK, WM, WN, S, DMA, copy mode, ...>: copy mode 7
    mode7 = {k: v for k, v in scratch.items() if re.search(r"pipelined_gemmI(?:L[bi]\d+E){9}Li7E", k)}
    assert len(mode7) == 12
    assert not {k: v for k, v in mode7.items() if v}


def test_staged_products_stage_in_registers(scratch):
    # every kernel of the products (plain, gated, their gradients, by group) that copies through
    # registers: product_kernel and gradients_kernel have REG behind ET and four (three) flags,
    # grouped_rows, grouped_weights and grouped_gradients behind ET and four, none and two
    patterns = (r"14product_kernelILi\dE(?:Lb[01]E){4}Lb1E", r"16gradients_kernelILi\dE(?:Lb[01]E){1}Lb1E",
                r"12grouped_rowsILi\dE(?:Lb[01]E){3}Lb1E", r"15grouped_weightsILi\dELb1E", r"17grouped_gradientsILi\dE(?:Lb[01]E){2}Lb1E")
    for pattern in patterns:
        found = {k: v for k, v in scratch.items() if re.search(pattern, k)}
        assert found and not {k: v for k, v in found.items() if v}, pattern
