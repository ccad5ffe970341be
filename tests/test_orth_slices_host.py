"""Slices of the sums of X X^T, asked of the library's own host code built here
(CPU only)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_dispatch_grouped_amd", "csrc")
SHIM = """#include "validate.h"
extern "C" int slices(int S, int L, int64_t tiles) { return moe::orth_gram_slices(S, L, tiles); }
extern "C" int64_t room(int64_t batch, int rows, int cols) {
  const moe::OrthWorkspace w = moe::orth_workspace(batch, rows, cols);
  return (int64_t)(w.total - w.sums);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("slices")
    src, out = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src),
                    os.path.join(CSRC, "validate.cpp"), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.slices.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    lib.room.argtypes, lib.room.restype = [ctypes.c_int64, ctypes.c_int, ctypes.c_int], ctypes.c_int64
    return lib


def _tiles(batch, S):
    m = -(-S // 128)
    return batch * m * (m + 1) // 2


@pytest.mark.parametrize("batch,S,L", [(1, 2176, 4096), (1, 2304, 4096), (2, 1408, 4096), (1, 2048, 2048), (1, 2560, 8192),
                                       (1, 2816, 8192)])
def test_no_slices_where_they_lose(lib, batch, S, L):
    assert lib.slices(S, L, _tiles(batch, S)) == 1


@pytest.mark.parametrize("batch,S,L,n", [(1, 2048, 8192, 3), (1, 2176, 8192, 3), (2, 1408, 8192, 3), (9, 512, 8192, 5),
                                         (1, 1472, 16384, 6), (1, 2048, 6144, 3), (1, 1536, 4224, 3), (5, 704, 4160, 3),
                                         (20, 320, 4096, 3)])
def test_slices_where_they_win(lib, batch, S, L, n):
    assert lib.slices(S, L, _tiles(batch, S)) == n


def test_partial_sums_fit(lib):
    """Of every batch on these sides: 64 KB a tile and slice, none where nothing is sliced."""
    for S, L, some in ((64, 6144, True), (512, 8192, True), (1472, 6144, True), (2176, 65536, True), (1920, 4096, True),
                       (1984, 4096, False), (2176, 6080, False), (2240, 8192, False), (2816, 8192, False), (512, 4032, False)):
        for batch in range(1, 130):
            n = lib.slices(S, L, _tiles(batch, S))
            assert n == 1 or _tiles(batch, S) * n * 65536 <= lib.room(batch, S, L)
            assert n >= 3 or n == 1
        assert (lib.room(1, S, L) > 0) == some
