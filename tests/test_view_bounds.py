"""Extents of the range-checked views of strided rows (csrc/ss_view.h), compiled for the host: no load that the state
kernels issue, the heads past a group's last among them, reaches behind the operand (CPU)."""
import ctypes
import os
import subprocess

import pytest

from mamba_selective_scan_fwd_amd import build

P = 128          # bytes of a head's 64 channels
PIECE, Q = 64, 256


@pytest.fixture(scope="module")
def view_bytes(tmp_path_factory):
    d = tmp_path_factory.mktemp("view")
    src, lib = os.path.join(d, "view.cpp"), os.path.join(d, "view.so")
    with open(src, "w") as f:
        f.write('#include "ss_view.h"\nextern "C" uint32_t view_bytes(int64_t row, int rows, int64_t cols) {\n'
                '  return ss::view_bytes(row, rows, cols);\n}\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + build.CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).view_bytes
    fn.restype, fn.argtypes = ctypes.c_uint32, [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    return fn


def test_view_bytes(view_bytes):
    assert view_bytes(512, 0, 128) == 0
    assert view_bytes(512, 1, 128) == 128 and view_bytes(512, 256, 128) == 255 * 512 + 128
    assert view_bytes(2 << 21, 256, 2 << 21) == 1 << 30          # the widest rows: offsets stay in 32 bits


@pytest.mark.parametrize("hb_max", [1, 2, 3])
@pytest.mark.parametrize("nheads,ngroups", [(1, 1), (4, 1), (4, 2), (5, 1), (5, 5), (8, 1), (24, 1), (32, 1), (64, 1),
                                            (80, 8)])
def test_state_loads_end_with_the_operand(view_bytes, nheads, ngroups, hb_max):
    """chunk_states: thread tid loads 16 bytes at (piece + tid / 8) * row + hb * 128 + (tid % 8) * 16 of a view that
    begins at head h0's columns, for all hb_max heads of a workgroup and up to three pieces past a chunk's end.  What
    the view's range check lets through must lie in the operand, whose last byte is the last row's last column."""
    hpg = nheads // ngroups
    for gap in (0, 32, 4096):                       # rows apart: columns of something else in between
        row = nheads * P + gap
        for rows in (1, 63, 64, 65, 255, 256):
            end = (rows - 1) * row + nheads * P     # behind the operand's last byte, from the chunk's first row
            for g in range(ngroups):
                for h in range(0, hpg, hb_max):
                    h0, heads = g * hpg + h, min(hpg - h, hb_max)
                    size = view_bytes(row, rows, heads * P)
                    for hb in range(hb_max):
                        for r in range(Q + 3 * PIECE):
                            last = r * row + hb * P + 7 * 16 + 16
                            if last <= size:
                                assert h0 * P + last <= end, (h0, hb, rows, r)
                            # a head's own rows are all read
                            assert (hb >= heads or r >= rows) or last <= size
                            assert r < rows or r * row + hb * P >= size
