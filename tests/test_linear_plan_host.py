"""The dense product's weight-gradient plan (tile, token slices) at the sizes
the GPU tests rely on, asked of the library's own host code built here (CPU
only)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_dispatch_grouped_amd", "csrc")
SHIM = """#include "validate.h"
extern "C" void wgrad_plan(int64_t T, int K, int N, int *out) {
  const moe::FfnWgrad w = moe::linear_wgrad_plan(T, K, N);
  out[0] = w.tile; out[1] = w.slices; out[2] = w.chunk; out[3] = w.most;
}
"""

# T, K, N, slices of 256 x 256 tiles: T is no multiple of 64, the last slice is shorter, and rows and columns leave tiles
# partly empty; the last two have more tiles and slices than 256 workgroups
LARGE = [(9001, 2112, 1088, 5), (20011, 1408, 1408, 7), (40001, 1088, 832, 12), (5001, 4160, 2112, 3), (1001, 4160, 4160, 1)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src),
                    os.path.join(CSRC, "validate.cpp"), "-o", str(lib)], check=True)
    fn = ctypes.CDLL(str(lib)).wgrad_plan
    fn.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def call(T, K, N):
        out = (ctypes.c_int * 4)()
        fn(T, K, N, out)
        return dict(zip(("tile", "slices", "chunk", "most"), out))
    return call


@pytest.mark.parametrize("T,K,N,slices", LARGE + [(32768, 2048, 1408, 5)])
def test_large_tiles_in_slices(plan, T, K, N, slices):
    p = plan(T, K, N)
    assert (p["tile"], p["slices"]) == (256, slices), p
    if T % 64:
        assert T % p["chunk"] != 0 and (K % 256 or N % 256)
    units = -(-K // 256) * -(-N // 256) * p["slices"]
    assert (units > 256) == (K == 4160), units


def test_slices_cover_the_tokens_once(plan):
    for T in (1, 63, 64, 255, 256, 700, 2561, 7001, 20011, (1 << 24) - 1):
        for K, N in ((64, 64), (576, 1088), (2048, 1408), (4160, 2112), (65536, 128)):
            p = plan(T, K, N)
            assert p["chunk"] % 64 == 0 and 1 <= p["slices"] <= p["most"]
            assert (p["slices"] - 1) * p["chunk"] < T <= p["slices"] * p["chunk"]
