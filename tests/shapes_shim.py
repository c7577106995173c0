"""The host's choice of product tiles (``csrc/product_shapes.h``), compiled
with the host compiler."""
import ctypes as C
import os
import subprocess

from tests.conftest import ROOT

TILES = ("64 x 64", "128 x 64", "128 x 128", "256 x 256")
FOUR_BIT = ("few channels", "16 rows, 4 stages", "16 rows, 3 stages", "64 rows")

SOURCE = """
#include "product_shapes.h"
extern "C" int product(int64_t m, int e, int n, int k) { return moe_ep::product_shape_of(m, e, n, k); }
extern "C" int weight_grad(int64_t m, int e, int n, int k) { return moe_ep::weight_grad_shape_of(m, e, n, k); }
extern "C" int four_bit(int64_t m, int e, int n) { return moe_ep::four_bit_shape_of(m, e, n); }
"""


class Shapes:
    """Names of the tiles of a call; experts 0: dense."""

    def __init__(self, folder):
        src, lib = os.path.join(folder, "shapes.cpp"), os.path.join(folder, "shapes.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I",
                        os.path.join(ROOT, "combine_route_mask_amd", "csrc"), "-o", lib, src], check=True)
        self.lib = C.CDLL(lib)
        for f in (self.lib.product, self.lib.weight_grad, self.lib.four_bit):
            f.argtypes = [C.c_int64, C.c_int, C.c_int, C.c_int][:3 if f is self.lib.four_bit else 4]

    def product(self, rows, experts, n, k):
        return TILES[self.lib.product(rows, max(experts, 1), n, k)]

    def weight_grad(self, rows, experts, n, k):
        return TILES[self.lib.weight_grad(rows, max(experts, 1), n, k)]

    def four_bit(self, rows, experts, n):
        return FOUR_BIT[self.lib.four_bit(rows, max(experts, 1), n)]
