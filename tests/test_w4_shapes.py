"""Which shape of a workgroup the 4-bit forward takes for a problem: the rule of the
source, compiled for the host, over the sizes that the GPU tests list (CPU only)."""
import ctypes
import os
import re
import subprocess

import pytest

import fp8_gemm_backward_amd as lp
import test_gpu_moe_bounds as B
import test_gpu_w4 as T

SOURCE = os.path.join(os.path.dirname(lp.__file__), "csrc", "lp_gemm_w4.hip")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """(shape of (M, N, K, groups): its number, -1 for the large tiles; number of shapes)."""
    text = open(SOURCE).read()
    kernel = open(os.path.join(os.path.dirname(SOURCE), "lp_gemm_kernel.hpp")).read()
    body = text[text.index("struct Shape {"):text.index("template <int F, int kIndex")]
    assert body.count("int choose(") == 1
    waves = re.search(r"constexpr int kWaves = (\d+)", text)[1]
    step = re.search(r"constexpr int kStep = (\d+)", text)[1]
    cus = re.search(r"constexpr int kCUs = (\d+)", kernel)[1]
    at = tmp_path_factory.mktemp("rule")
    (at / "rule.cpp").write_text(f"""
#include <stdint.h>
constexpr int kWaves = {waves}, kStep = {step}, kCUs = {cus};
struct Params {{ int32_t Ptot, Qtot, Ktot; const int32_t* offsets; int32_t groups; }};
{body}
extern "C" int shape(int M, int N, int K, int groups) {{
  int32_t any = 0;
  return choose(Params{{M, N, K, groups ? &any : nullptr, groups ? groups : 1}});
}}
extern "C" int shapes() {{ return kShapeCount; }}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", at / "rule.so", at / "rule.cpp"], check=True)
    lib = ctypes.CDLL(str(at / "rule.so"))
    return (lambda M, N, K, G=0: lib.shape(M, N, K, G)), lib.shapes()


def test_the_listed_sizes_take_every_shape_and_the_large_tiles(rule):
    shape, count = rule
    every = set(range(-1, count))
    assert {shape(*s) for s in T.SHAPES + T.DENSE + T.MIDDLING} == every
    # (the grouped tests leave five rows out of the groups, not out of the call)
    assert {shape(*s) for s in T.GROUPED + T.MIDDLING_GROUPED} == every


def test_the_large_tiles_of_another_stream_are_the_large_tiles(rule):
    shape, _ = rule
    assert all(shape(*s) == -1 for s in B.LARGE_TILES)


def test_the_large_tiles_take_no_contraction_that_a_grouped_call_splits(rule):
    """An MXFP4 weight's tiles have no second launch: contractions of 64 slabs of 64 and more never go to them."""
    shape, _ = rule
    sizes = [1, 100, 255, 256, 257, 1000, 4096, 9001, 32768, 100000]
    for M in sizes:
        for N in [16, 256, 272, 1040, 4096, 8208, 65536]:
            for K in (4096, 4128, 14336, 1 << 17):
                for G in (0, 1, 2, 5, 64, 1024):
                    assert shape(M, N, K, G) >= 0, (M, N, K, G)
