"""The choice of form of the 8-bit products, as the library makes it, and sizes that
reach each form."""

from __future__ import annotations

import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256   # of an MI355X

# (rows and columns of a tile, split): M, N, K of the forward product
FORWARD = {
    (256, 256, False): (2047, 6100, 530), (256, 256, True): (539, 2222, 17776),
    (256, 128, False): (1000, 8190, 277), (256, 128, True): (130, 3270, 12508),
    (128, 128, False): (1001, 4090, 1500), (128, 128, True): (300, 2001, 16001),
    (128, 64, False): (290, 4090, 1300), (128, 64, True): (601, 1000, 12010),
    (64, 64, False): (130, 4095, 4096), (64, 64, True): (70, 301, 20001)}
# the same of the gradients: rows and columns of the result and the summed axis
GRADS = {
    (256, 256, False): (2047, 6100, 321), (256, 256, True): (904, 2700, 6988),
    (128, 256, False): (1001, 4100, 777), (128, 256, True): (1180, 129, 16350),
    (128, 128, False): (2000, 2000, 131), (128, 128, True): (200, 4096, 4099),
    (64, 128, False): (1880, 389, 521), (64, 128, True): (700, 700, 5001),
    (32, 128, False): (33, 389, 131), (32, 128, True): (40, 130, 9001)}
# rows of W: how many of them a wave takes with two to four rows of X
FEW = {4096: 1, 4097: 2, 11009: 3, 33000: 8}


def load(folder: str) -> ctypes.CDLL:
    """The host rule compiled by itself, with C entry points for the test."""
    src, lib = os.path.join(folder, "form.cpp"), os.path.join(folder, "form.so")
    with open(src, "w") as f:
        f.write('#include "bnbx_int8_form.hpp"\n'
                'using namespace bnbx;\n'
                'static void tell(const Int8Shape* s, const Int8Form& f, int* out) {\n'
                '  out[0] = s[f.shape].rows, out[1] = s[f.shape].cols;\n'
                '  out[2] = f.splits, out[3] = f.steps_per;\n}\n'
                'extern "C" void forward(int M, int N, int K, int cus, int* out) {\n'
                '  tell(kInt8GemmShapes, int8_gemm_form(M, N, K, cus), out);\n}\n'
                'extern "C" void grad(int R, int C, int T, int cus, int* out) {\n'
                '  tell(kInt8GradShapes, int8_grad_form(R, C, T, cus), out);\n}\n'
                'extern "C" int few_rows(int M, int N, int cus) {\n'
                '  return int8_few_rows(M, N, cus);\n}\n'
                'extern "C" int wave_rows() { return kInt8WaveRows; }\n'
                'extern "C" int shapes(int grad) {\n'
                '  return grad ? sizeof(kInt8GradShapes) / sizeof(Int8Shape)\n'
                '              : sizeof(kInt8GemmShapes) / sizeof(Int8Shape);\n}\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dequant_gemm_nf4_amd", "csrc"), src, "-o", lib], check=True)
    return ctypes.CDLL(lib)


def form(fn, *sizes, cus=CUS):
    """(tile rows, tile columns, splits, steps of each)"""
    out = (ctypes.c_int * 4)()
    fn(*sizes, cus, out)
    return tuple(out)
