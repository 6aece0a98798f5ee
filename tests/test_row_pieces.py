"""Rows read as aligned 16-byte pieces: no piece that is read whole reaches outside its matrix."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "permute_grouped_expert_gb300", "csrc")


@pytest.fixture(scope="module")
def first_cut_row(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_pieces")
    src, lib = str(d / "r.cpp"), str(d / "r.so")
    with open(src, "w") as f:
        f.write('#include "row_pieces.h"\n'
                'extern "C" int64_t cut(int64_t rows, int64_t stride, int n) '
                '{ return moe::first_cut_row(rows, stride, n); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).cut
    fn.restype, fn.argtypes = ctypes.c_int64, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return fn


@pytest.mark.parametrize("n", [4, 8])
def test_whole_pieces_stay_inside(first_cut_row, n):
    """Every piece of every row of small matrices: pieces that start before a row start inside the matrix, those of
    rows before the cut end inside it, and the cut is no earlier than that asks for."""
    for rows in range(1, 21):
        for H in range(1, 20):
            for stride in range(H, H + 10):
                end, cut = (rows - 1) * stride + H, first_cut_row(rows, stride, n)
                beyond = []  # rows with a shared piece that ends behind the matrix
                for r in range(rows):
                    beg = r * stride // n * n
                    for c in range(beg, r * stride + H, n):
                        assert c >= 0
                        whole = c >= r * stride and c + n <= r * stride + H
                        if not whole and c + n > end:
                            beyond.append(r)
                assert all(r >= cut for r in beyond), (rows, H, stride, cut, beyond)
                assert cut >= rows - 1 - (n - 2) // stride or cut == 0


def test_long_matrices(first_cut_row):
    assert first_cut_row(1 << 40, 1 << 40, 8) == (1 << 40) - 1
    assert first_cut_row(1 << 33, 1, 4) == (1 << 33) - 3
    assert first_cut_row(0, 5, 8) == 0
    assert first_cut_row(1, -7, 8) == 0
