"""The shapes of the GPU tests of the many-row MX FP4 products reach every tile
(the choice is host code, compiled here with g++)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from tests import mx_tile_shapes as S

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_dequantize_matmul_amd", "csrc")
NAMES = {"w4a4": ("k32x64", "k64x64", "k128x128", "k256x256"),
         "w4a16": ("k32x64", "k64x64", "k64x128", "k128x128", "kLarge")}
CUS = 256

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text('''#include "mx_plan.hpp"
extern "C" int w4a4(int64_t M, int64_t N, int64_t cus, int large) { return int(q4::mx_w4a4_tile(M, N, cus, large)); }
extern "C" int w4a16(int64_t M, int64_t N, int64_t cus, int large) { return int(q4::mx_w4a16_tile(M, N, cus, large)); }
''')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", str(d / "plan.cpp"), "-o", str(d / "plan.so")],
                   check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    i = ctypes.c_int64
    return {"w4a4": lambda M, N, large: NAMES["w4a4"][lib.w4a4(i(M), i(N), i(CUS), int(large))],
            "w4a16": lambda M, N, large: NAMES["w4a16"][lib.w4a16(i(M), i(N), i(CUS), int(large))]}


def test_w4a4_shapes_reach_every_variant(plan):
    reached = set()
    for tile, M, N, K in S.cases_w4a4():
        for yt in ("f32", "bf16"):
            assert plan["w4a4"](M, N, S.large_w4a4(K, yt)) == S.tile_w4a4(tile, K, yt), (M, N, K, yt)
            reached.add(S.variant_w4a4(tile, K, yt))
    assert reached == S.variants_w4a4()


def test_w4a16_shapes_reach_every_variant(plan):
    reached = set()
    for tile, M, N, K in S.cases_w4a16():
        assert plan["w4a16"](M, N, S.large_w4a16(K)) == tile, (M, N, K)
        reached.add(S.variant_w4a16(tile, K))
    assert reached == S.variants_w4a16()


def test_unaligned_operands_never_take_the_large_tiles(plan):
    for M in (65, 300, 1000, 5000):
        for N in (100, 2048, 13312):
            assert plan["w4a16"](M, N, False) != "kLarge" and plan["w4a4"](M, N, False) != "k256x256"


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")
@pytest.mark.parametrize("source", ["mx_gemv", "mx_quant", "mx_tiled_w4a16", "mx_tiled_w4a4", "qk_norm_rope"])
def test_no_kernel_spills(source):
    """The compiler's remarks: no kernel keeps values in scratch memory."""
    from int4_dequantize_matmul_amd import build
    r = subprocess.run([build.HIPCC, *build.HIP_FLAGS, "-Rpass-analysis=kernel-resource-usage", "--cuda-device-only",
                        "-c", os.path.join(CSRC, source + ".hip"), "-o", os.devnull], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    scratch = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", r.stderr, re.S)
    assert scratch and not [(n, s) for n, s in scratch if int(s)]
