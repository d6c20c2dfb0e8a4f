"""What the layer norm's copies of rows that start anywhere read, on the CPU: the address arithmetic
that the kernels use, compiled for the host. No byte before a matrix or behind a row is read, and
those that are make up the row."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
#include "windows.h"
extern "C" {
void window(uint64_t row, uint64_t bytes, uint64_t offset, uint64_t* at, uint32_t* n) {
    const tpg::CopyWindow w = tpg::copy_window(row, bytes, offset);
    *at = w.at;
    *n = w.bytes;
}
int apart(uint64_t row, uint64_t base, uint64_t offset) { return tpg::begins_apart(row, base, offset); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("windows")
    (d / "windows.cpp").write_text(CODE)
    so = str(d / "windows.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", so, str(d / "windows.cpp"), "-I",
                    os.path.join(ROOT, "tile_primitive_tensor_gb300", "csrc")], check=True)
    lib = ctypes.CDLL(so)
    u64 = ctypes.c_uint64
    lib.window.argtypes = [u64, u64, u64, ctypes.POINTER(u64), ctypes.POINTER(ctypes.c_uint32)]
    lib.apart.argtypes = [u64, u64, u64]
    return lib


@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("cols", [1, 3, 7, 8, 9, 31, 64, 255, 1001])
def test_copies_stay_in_the_matrix(lib, size, cols):
    at, n = ctypes.c_uint64(), ctypes.c_uint32()
    for start in range(0, 16, size):
        for ld in (cols, cols + 1, cols + 5):
            base = 0x7F0000000000 + start
            for r in range(10):
                row, bytes_ = base + r * ld * size, cols * size
                read = set()
                # each lane's piece, and the one behind the last lane's
                for piece in range(-(-bytes_ // 16) + 2):
                    lib.window(row, bytes_, 16 * piece, ctypes.byref(at), ctypes.byref(n))
                    assert at.value % 16 == 0 and n.value <= 16
                    if lib.apart(row, base, 16 * piece):  # (only the row's own bytes are loaded)
                        first = range(row, min(row - row % 16 + 16, row + bytes_))
                    else:
                        first = range(at.value, at.value + n.value)
                    assert all(base <= b < row + bytes_ for b in first)
                    read.update(first)
                assert read >= set(range(row, row + bytes_))
                assert min(read) >= row - row % 16
