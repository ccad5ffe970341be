"""The dense block's weight-gradient plan (tile, token slices) at the sizes the
GPU tests rely on, asked of the library's own host code built here (CPU only)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_dispatch_grouped_amd", "csrc")
SHIM = """#include "validate.h"
extern "C" void wgrad_plan(int64_t T, int d, int F, int *out) {
  const moe::FfnWgrad w = moe::ffn_wgrad_plan(T, d, F);
  out[0] = w.tile; out[1] = w.slices; out[2] = w.chunk; out[3] = w.most;
}
"""

# T, d, F, slices of 256 x 256 tiles: T is no multiple of 64, the last slice is shorter, and rows and columns leave tiles
# partly empty
SLICED = [(3011, 576, 1088, 6), (9001, 1088, 1088, 3), (20011, 1408, 1408, 2)]


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

    def call(T, d, F):
        out = (ctypes.c_int * 4)()
        fn(T, d, F, out)
        return dict(zip(("tile", "slices", "chunk", "most"), out))
    return call


@pytest.mark.parametrize("T,d,F,slices", SLICED + [(32768, 2048, 1408, 3)])
def test_large_tiles_in_slices(plan, T, d, F, slices):
    p = plan(T, d, F)
    assert (p["tile"], p["slices"]) == (256, slices), p
    if T % 64:
        assert T % p["chunk"] != 0 and (d % 256 or F % 256)


def test_slices_cover_the_tokens_once(plan):
    for T in (1, 63, 64, 255, 256, 700, 2561, 7001, 20011, (1 << 24) - 1):
        for d, F in ((64, 64), (576, 1088), (2048, 1408), (4096, 2816), (65536, 128)):
            p = plan(T, d, F)
            assert p["chunk"] % 64 == 0 and 1 <= p["slices"] <= p["most"]
            assert (p["slices"] - 1) * p["chunk"] < T <= p["slices"] * p["chunk"]


@pytest.mark.parametrize("d,F,none", [(4096, 2816, True), (7168, 2048, True), (65536, 128, True), (2048, 1408, False),
                                      (64, 64, False)])
def test_workspace_only_where_tokens_are_sliced(plan, d, F, none):
    """Partial sums are kept for two slices or more: sizes that have one slice at any T need no workspace."""
    import token_dispatch_grouped_amd as moe
    most = max(plan(T, d, F)["most"] for T in (1, 1000, 32768, (1 << 24) - 1))
    assert (most == 1) == none
    for T in (1, 700, 7001, 100000):
        need = moe.moe_ffn_workspace_size(moe.make_ffn_shape(T, d, F))[1]
        assert need == 0 if none else need >= 12 * d * F * plan(T, d, F)["slices"]
