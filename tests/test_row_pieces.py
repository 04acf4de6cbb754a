"""Rows on no 16-byte boundary are copied in the 16-byte pieces that cover them. A piece is copied whole only where it
holds nothing but the tensor: the header's arithmetic, compiled for the host, against the tensor's own ends."""

import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_routed_topk_gb300",
                    "csrc")
SOURCE = """
#include "row_pieces.cuh"
extern "C" int whole_row(int any, int64_t row, int64_t rows, int32_t D, int piece) {
    return row > 0 && row < rows - 1 && (any ? moe::neighbours_cover<true>(D, piece) : moe::neighbours_cover<false>(D, piece));
}
extern "C" int one(int any, int64_t row, int64_t rows, int32_t D, int piece, int first) {
    return any ? moe::piece_inside<true>(row, rows, D, first, first + piece - 1)
               : moe::piece_inside<false>(row, rows, D, first, first + piece - 1);
}
"""


@pytest.fixture(scope="module")
def pieces(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("pieces") / "pieces.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-x", "c++", "-", "-o", lib],
                   input=SOURCE.encode(), check=True)
    lib = ctypes.CDLL(lib)
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    lib.whole_row.argtypes, lib.one.argtypes = [i32, i64, i64, i32, i32], [i32, i64, i64, i32, i32, i32]
    return lib


@pytest.mark.parametrize("piece", [4, 8])  # elements of 16 bytes: fp32, and the 16-bit types
@pytest.mark.parametrize("D", [*range(1, 20), 33])
def test_only_pieces_of_the_tensor_are_copied_whole(pieces, piece, D):
    for any_length in (1, 0) if D >= piece - 1 else (1,):
        for rows in (1, 2, 3, 5, 9, 20):
            for base in range(piece):  # elements from a 16-byte boundary to the tensor's first one
                for row in range(rows):
                    lead = (base + row * D) % piece
                    for first in range(-lead, D, piece):
                        at = row * D + first
                        inside = at >= 0 and at + piece <= rows * D
                        if pieces.whole_row(any_length, row, rows, D, piece):
                            assert inside, (rows, base, row, first)
                        assert bool(pieces.one(any_length, row, rows, D, piece, first)) == inside, (rows, base, row, first)


def test_rows_inside_a_large_tensor_take_the_short_way(pieces):
    for rows, D in ((3, 7), (16384, 7001), (2 ** 31 - 1, 2 ** 24)):
        for row in (1, rows // 2, rows - 2):
            assert pieces.whole_row(1, row, rows, D, 8) and pieces.whole_row(0, row, rows, D, 8)
        assert not any(pieces.whole_row(a, row, rows, D, 8) for a in (0, 1) for row in (0, rows - 1))
