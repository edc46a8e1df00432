"""The address arithmetic of the experts' kernels (csrc/expert_access.h), compiled for the host:
no whole piece of 16 bytes may lie outside the row it is taken from."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_embedding_lookup_amd", "csrc")
SOURCE = """
#include "expert_access.h"
extern "C" int whole(uint64_t p, int64_t stride, int64_t width, int size) {
  return ctr::whole_pieces((uintptr_t)p, stride, width, size);
}
extern "C" int64_t piece(int64_t first, int64_t width, int count, int* down) {
  const ctr::PieceAt p = ctr::piece_at(first, width, count);
  *down = p.down;
  return p.column;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("access")
    (d / "access.cpp").write_text(SOURCE)
    lib = str(d / "access.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared",
                           "-I" + CSRC, "-o", lib, str(d / "access.cpp")])
    lib = ctypes.CDLL(lib)
    lib.whole.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    lib.piece.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                          ctypes.POINTER(ctypes.c_int)]
    lib.piece.restype = ctypes.c_int64
    return lib


def test_whole_pieces_only_of_rows_that_are(host):
    """A row taken in whole pieces has no elements left over, wherever it lies: an empty array's
    address is 0."""
    for size in (2, 4):
        for width in range(1, 301):
            for p in (0, 0x10000, 0x10000 + size):
                for stride in (width, width + 8, width + 16 // size):
                    want = p % 16 == 0 and stride * size % 16 == 0 and width * size % 16 == 0
                    assert bool(host.whole(p, stride, width, size)) == want, (size, width, p, stride)


def test_pieces_of_a_tile_lie_inside_their_row(host):
    """Every piece of every tile over rows of 1 to 300 columns: read inside the row, and what is
    there of it found `down` elements later.  (Rows below a piece are read by elements.)"""
    down = ctypes.c_int(0)
    for count in (4, 8):
        for tile in (64, 128):
            for width in range(count, 301):
                for first in range(0, (width + tile - 1) // tile * tile, count):
                    column = host.piece(first, width, count, ctypes.byref(down))
                    case = (count, tile, width, first, column, down.value)
                    assert 0 <= column and column + count <= width, case
                    assert 0 <= down.value < count, case
                    if first < width:
                        assert column + down.value == first, case
