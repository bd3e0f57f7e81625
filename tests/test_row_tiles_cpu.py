"""The spread of an expert's rows over tiles of the unquantised products, on the
host: the functions that the kernel uses, at every row count that matters."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_expert_ffn_fp32_b200", "csrc")
MOST = 2 ** 31 - 4096                       # pairs of a call

SOURCE = """
#include "row_tiles.h"
extern "C" int tiles(int rows, int tn) { return moe::row_tiles(rows, tn); }
extern "C" int per(int rows, int tn) { return moe::rows_per_tile(rows, moe::row_tiles(rows, tn), tn); }
extern "C" int columns(int n, int cg) { return moe::padded_columns(n, cg); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_tiles")
    src, so = d / "t.cpp", d / "t.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", "-o", str(so), str(src)], check=True)
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("tn", [32, 256])
def test_rows_are_covered_once(lib, tn):
    """Every tile but the last holds `per` rows, the last one 1..per of them."""
    counts = list(range(1, 40 * tn + 2)) + [MOST - i for i in range(300)] + [2139127680 + i for i in range(-300, 300)]
    counts += [2 ** b + i for b in range(12, 31) for i in (-1, 0, 1)]
    for rows in counts:
        nt, per = lib.tiles(rows, tn), lib.per(rows, tn)
        assert nt == -(-rows // tn)
        assert 0 < per <= tn and per % 16 == 0
        assert (nt - 1) * per < rows <= nt * per, (rows, nt, per)


@pytest.mark.parametrize("cg,unit", [(1, 16), (2, 32)])
def test_columns_are_what_the_products_take(lib, cg, unit):
    for n in range(1, 257):
        assert n <= lib.columns(n, cg) < n + unit and lib.columns(n, cg) % unit == 0
