"""Which kernel and tile the row-major MXFP4 products take: the GPU tests' cases take
the shapes that they are named by, and between them every shape that there is,
dense and grouped, and the split of a dense product into two launches (no GPU
needed: the choice is plain C++, compiled here by itself)."""
import ctypes as C
import os
import re
import subprocess

import pytest

import bit_grouped_gemm_amd as moe
from test_gpu_mx4_shapes import CASES

HEADER = os.path.join(os.path.dirname(os.path.abspath(moe.__file__)), "csrc", "moe_mx4_shape.h")
KINDS = ("big", "few", "rows")


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    """(shape of a launch, rows of a dense product's first launch)."""
    here = tmp_path_factory.mktemp("mx4_shape")
    src, lib = here / "shape.cpp", here / "shape.so"
    src.write_text(f'#include "{HEADER}"\n'
                   'extern "C" void shape(int R, int N, int K, int E, int* s) {\n'
                   '  const moe::Mx4Shape m = moe::mx4_shape(R, N, K, E);\n'
                   '  s[0] = m.kind; s[1] = m.rows; s[2] = m.cols;\n}\n'
                   'extern "C" int first(int R, int N, int K) { return moe::mx4_first_rows(R, N, K); }\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    L = C.CDLL(str(lib))

    def shape(R, N, K, E):
        s = (C.c_int * 3)()
        L.shape(R, N, K, max(E, 1), s)
        return f"{KINDS[s[0]]}_{s[1]}x{s[2]}"

    return shape, L.first


def test_cases_take_their_shapes(choice):
    shape, first = choice
    for name, R, N, K, E in CASES:
        rows = R if E else first(R, N, K)
        got = shape(rows, N, K, E) + ("" if rows == R else "+" + shape(R - rows, N, K, 0))
        assert got == name, (got, name, R, N, K, E)


def test_cases_have_every_shape(choice):
    text = open(HEADER).read()
    table = re.findall(r"\{\{kMx4(Big|Few|Rows), (\d+), (\w+)\}, \d\}", text)
    every = {f"{kind.lower()}_{rows}x{256 if cols == 'kMx4Cols' else cols}" for kind, rows, cols in table}
    assert len(every) == len(table) == 17
    assert {c[0] for c in CASES if c[4] == 0 and "+" not in c[0]} == every
    assert {c[0] for c in CASES if c[4]} == every
    assert len([c for c in CASES if "+" in c[0]]) >= 3


def test_split_rules(choice):
    """Whole tiles first, at most 255 rows behind them, and nothing to split below 257 rows."""
    shape, first = choice
    for R in (0, 1, 255, 256, 257, 511, 512, 4096, 4099, 16411, 32768, 1 << 30):
        for N, K in ((8, 32), (792, 1440), (4096, 1056), (4096, 7168), (1 << 20, 1 << 20)):
            rows = first(R, N, K)
            assert rows == R or (rows % 256 == 0 and 256 <= rows < R < rows + 256), (R, N, K)
            assert shape(R, N, K, 1) and shape(R, N, K, 1024)
