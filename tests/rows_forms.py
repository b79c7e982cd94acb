"""The choice between the streaming and the tiled form of the products over
grouped rows, as the library makes it, and sizes that reach the tiled form."""

from __future__ import annotations

import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256   # of an MI355X

# (rows of each group, N, K); sizes of the tiles 256 x 256, steps of 64 k, four
# codes a load where K is a multiple of 256
EXPERTS = [([333, 0, 41, 230], 9001, 64), ([300, 290, 7], 9001, 320),
           ([513, 88], 8450, 256), ([257, 300, 60, 1], 9100, 1088), ([256, 512], 8192, 1024)]
EXPERTS_LAYOUT = ([200, 0, 3, 400], 9001, 192)
# input gradient: (rows of each group, N, K)
DX = [([333, 0, 41, 326], 64, 8192), ([300, 390, 7], 192, 8256), ([513, 88, 100], 128, 8640),
      ([256, 512], 640, 8192)]
DX_LAYOUT = ([200, 0, 3, 500], 128, 8256)
# (rows, groups) of N = 9001 and, of 700 rows, the input gradient of K = 8192
PLAIN = [(700, 2), (700, 3), (601, 2)]
# (rows, adapters, rank, N, K)
ADAPTERS = [(1500, 5, 16, 9001, 64), (1281, 3, 48, 9101, 320), (2500, 20, 128, 8450, 1024),
            (2000, 2, 256, 9001, 1088), (3000, 300, 16, 9001, 1088)]
ADAPTERS_BROKEN = (2000, 3, 32, 9001, 192)


def load(folder: str) -> ctypes.CDLL:
    """The host rule compiled by itself, with C entry points for the test."""
    src, lib = os.path.join(folder, "form.cpp"), os.path.join(folder, "form.so")
    with open(src, "w") as f:
        f.write('#include "bnbx_rows_form.hpp"\n'
                'extern "C" int tiles(int rows, int groups, int n, int k, int adapters, int rank, '
                'int cus) {\n'
                '  return bnbx::prefer_tiles(rows, groups, n, k, adapters, rank, cus);\n}\n'
                'extern "C" int dx_tiles(int rows, int groups, int k, int cus) {\n'
                '  return bnbx::prefer_dx_tiles(rows, groups, k, cus);\n}\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dequant_gemm_nf4_amd", "csrc"), src, "-o", lib], check=True)
    return ctypes.CDLL(lib)
