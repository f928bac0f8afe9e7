"""The spreading of an expert's slots over tiles, compiled for the host (no GPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_weight_decode_amd", "csrc")

SOURCE = """
#include "csf_layer.h"
extern "C" void split(uint32_t m, uint32_t tiles, uint32_t j0, uint32_t n, uint32_t *first, uint32_t *count) {
    for (uint32_t i = 0; i < n; ++i) {
        const csf::TileBlocks b = csf::tile_blocks(m, j0 + i, tiles);
        first[i] = b.first;
        count[i] = b.count;
    }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(SOURCE)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", CSRC, str(d / "split.cpp"), "-o", str(d / "split.so")], check=True)
    fn = ctypes.CDLL(str(d / "split.so")).split
    u32 = ctypes.c_uint32
    fn.argtypes = [u32, u32, u32, u32, ctypes.c_void_p, ctypes.c_void_p]

    def call(m, tiles, j0, n):
        first, count = np.empty(n, np.uint32), np.empty(n, np.uint32)
        fn(m, tiles, j0, n, first.ctypes.data, count.ctypes.data)
        return first.astype(np.int64), count.astype(np.int64)

    return call


# up to the ABI's 2^31 - 1 slots, all of them one expert's; from 2^21.5 on blocks * tiles passes 32 bits
@pytest.mark.parametrize("m", [1, 16, 17, 128, 129, 1000, 2964821, 3000000, 4194304, 2 ** 27 + 5, 2 ** 31 - 1])
def test_tiles_cover_an_experts_slots_once(split, m):
    tiles, blocks = (m + 127) // 128, (m + 15) // 16
    end = 0
    for j0 in range(0, tiles, 1 << 20):
        n = min(1 << 20, tiles - j0)
        first, count = split(m, tiles, j0, n)
        assert first[0] == end and np.array_equal(first[1:], (first + count)[:-1])  # one after another
        assert count.min() >= 1 and count.max() <= 8                               # 128 slots at most
        assert count.max() - count.min() <= 1                                      # evenly
        end = int(first[-1] + count[-1])
    assert end == blocks
