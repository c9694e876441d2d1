"""CPU check of how the adapters' first product shares K (csrc/qz_lora_index.cuh,
compiled here with the host compiler)."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "qz_lora_index.cuh"
extern "C" int s_part_begin(int part, int steps, int parts) {
    return qz::lora::part_begin(part, steps, parts);
}
"""


@pytest.fixture(scope="module")
def ix(tmp_path_factory):
    d = tmp_path_factory.mktemp("lora")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "weight_only_quantization_wise_b200", "csrc"), str(src),
                    "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


# K is a multiple of 128 below 2^31, a step 32 of it, 64 warps share it
@pytest.mark.parametrize("K", [128, 4096, 8192, 2 ** 25 + 128, 2 ** 30 - 128, 2 ** 30, 2 ** 30 + 128,
                               2 ** 31 - 128])
def test_warps_share_k(ix, K):
    """The parts follow one another from 0 to the last step and are even."""
    steps = K // 32
    ends = [ix.s_part_begin(w, steps, 64) for w in range(65)]
    assert ends == [w * steps // 64 for w in range(65)]
    assert ends[0] == 0 and ends[64] == steps
    assert max(b - a for a, b in zip(ends, ends[1:])) - min(b - a for a, b in zip(ends, ends[1:])) <= 1
