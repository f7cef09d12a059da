"""The 32-bit sizes of csrc/w4a16_sizes.h, built here with the host compiler, against
64-bit arithmetic."""
import ctypes
import os
import subprocess

import pytest

import w4a16_weight_only_gemm_amd as w4

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_weight_only_gemm_amd", "csrc")


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    d = tmp_path_factory.mktemp("sizes")
    src, lib = d / "s.cpp", str(d / "s.so")
    src.write_text('#include "w4a16_sizes.h"\nusing namespace w4a16_internal;\nextern "C" {\n'
                   "uint32_t matrix_bytes(int blocks, int K) { return packed_matrix_bytes(blocks, K); }\n"
                   "int group_of(int u, int per, int g, int groups) { return unit_group(u, per, g, groups); }\n}\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", lib], check=True)
    out = ctypes.CDLL(lib)
    out.matrix_bytes.restype = ctypes.c_uint32
    return out


def test_packed_matrix_bytes(sizes):
    """Both sides of N x K = 2^31, 2^32 and 2^33 (the limit), and odd sizes."""
    for K in (32, 96, 128, 5120, 16384, 17408, 20480, 1 << 20):
        for nk in (1 << 20, 1 << 31, 1 << 32, 3 << 31, 1 << 33):
            for extra in (-33, -1, 0, 1, 16, 40):
                N = nk // K + extra
                if N < 1 or N > 0x7FFFFFF0 or w4.w4a16_qweight_bytes(N, K) > 0xFFFFFFF0:
                    continue
                assert sizes.matrix_bytes((N + 15) // 16, K) == (N + 15) // 16 * 16 * K // 2, (N, K)


@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_units_of_a_column_block_stay_in_its_matrix(sizes, group):
    """Every tile that the whole expert layer's loads name, of the last column block too, lies
    inside the matrix, and within K it is the unit's own."""
    per, tile_bytes = max(1, 128 // group), 8 * group
    for groups in range(1, 24):
        blocks = 3
        units = (groups + per - 1) // per
        for u in range(units):
            for g in range(per):
                at = sizes.group_of(u, per, g, groups)
                assert 0 <= at < groups and (u * per + g >= groups or at == u * per + g)
                last = ((blocks - 1) * groups + at + 1) * tile_bytes
                assert last <= sizes.matrix_bytes(blocks, groups * group)
