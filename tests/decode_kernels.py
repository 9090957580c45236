"""Which product kernels the layer for a few tokens has, which one a call runs,
and shapes that reach each of them (helper of the tests)."""
import ctypes
import re
import shutil
import subprocess

import pytest

import combine_moe_route_histogram_amd as M

FORMATS = ("bf16", "f32", "bf16-mx", "f32-mx")   # the kernels' format argument, 0 to 3

KERNEL_SHAPES = {   # T, H, E, K, I, n_shared
    "bf16": [
        (1, 80, 6, 6, 8056, 2), (1, 2048, 14, 14, 144, 1), (1, 7296, 10, 10, 88, 0), (2, 64, 1, 1, 312, 0),
        (2, 5288, 15, 15, 80, 0), (3, 2488, 11, 11, 168, 0), (4, 16, 1, 1, 344, 1), (5, 64, 1, 1, 272, 0),
        (5, 264, 1, 1, 64, 0), (5, 4568, 6, 3, 168, 1), (7, 144, 9, 9, 2624, 2), (7, 312, 1, 1, 16, 0),
        (8, 144, 1, 1, 9464, 2), (9, 4672, 14, 14, 72, 0), (12, 4896, 13, 4, 120, 0),
        (15, 72, 148, 140, 4136, 0), (15, 136, 197, 151, 296, 1), (15, 360, 147, 138, 24, 2),
        (16, 72, 132, 129, 4160, 0), (16, 88, 10, 2, 5504, 2), (16, 136, 187, 180, 384, 0),
        (16, 280, 144, 133, 64, 0), (16, 9280, 3, 3, 136, 0), (17, 16, 1, 1, 360, 0), (24, 152, 4, 4, 4992, 2),
        (24, 152, 167, 158, 448, 0), (31, 64, 1, 1, 272, 0), (31, 136, 6, 4, 4680, 0),
        (31, 176, 148, 137, 408, 0), (31, 272, 1, 1, 16, 0), (32, 72, 70, 66, 4136, 1),
        (32, 72, 70, 66, 4160, 0), (32, 264, 1, 1, 64, 0), (32, 424, 70, 70, 64, 0), (32, 5888, 9, 2, 72, 1),
        (33, 5824, 9, 9, 72, 1), (50, 16, 1, 1, 456, 0), (50, 136, 175, 140, 320, 0), (50, 344, 1, 1, 16, 0),
        (64, 80, 6, 1, 9408, 0), (64, 2360, 13, 4, 136, 0), (64, 7248, 2, 2, 136, 2), (65, 2432, 11, 3, 152, 1),
        (100, 104, 13, 13, 4544, 0), (100, 152, 5, 5, 5952, 0), (150, 104, 25, 25, 4416, 2),
        (200, 72, 7, 1, 8016, 0), (200, 264, 18, 18, 16, 0), (200, 264, 71, 11, 32, 2),
        (200, 4296, 17, 1, 80, 1),
    ],
    "f32": [
        (1, 32, 1, 1, 408, 1), (1, 72, 5, 5, 5800, 0), (1, 72, 7, 7, 4032, 0), (2, 2368, 12, 12, 72, 0),
        (3, 16, 1, 1, 456, 0), (3, 152, 128, 128, 208, 0), (3, 5544, 6, 6, 80, 0), (3, 7488, 2, 2, 136, 0),
        (4, 400, 1, 1, 16, 0), (5, 264, 1, 1, 64, 0), (5, 1216, 10, 10, 136, 2), (8, 4032, 7, 7, 80, 0),
        (9, 32, 1, 1, 568, 0), (12, 136, 5, 5, 2816, 0), (15, 24, 1, 1, 264, 0), (15, 72, 148, 140, 2104, 0),
        (15, 144, 187, 149, 192, 2), (15, 168, 179, 175, 184, 0), (15, 400, 142, 141, 24, 0),
        (15, 7544, 4, 4, 72, 0), (16, 72, 132, 129, 2080, 0), (16, 280, 173, 156, 32, 1),
        (17, 16, 1, 1, 408, 0), (17, 32, 1, 1, 360, 0), (24, 328, 1, 1, 16, 0), (24, 6528, 5, 5, 72, 0),
        (31, 4304, 5, 5, 88, 2), (31, 7040, 2, 2, 136, 0), (32, 72, 70, 66, 2080, 0), (32, 72, 70, 66, 2104, 1),
        (32, 136, 7, 1, 2904, 0), (32, 144, 6, 6, 2240, 1), (32, 144, 134, 128, 256, 0),
        (32, 280, 66, 66, 16, 0), (32, 504, 1, 1, 32, 0), (40, 264, 1, 1, 16, 1), (50, 72, 12, 3, 2144, 2),
        (64, 72, 6, 1, 4680, 0), (64, 136, 3, 3, 4896, 0), (64, 7232, 4, 4, 72, 0), (65, 72, 10, 10, 2944, 0),
        (100, 16, 1, 1, 360, 0), (150, 152, 183, 174, 136, 0), (150, 344, 100, 18, 32, 0),
        (200, 552, 11, 11, 16, 0), (256, 80, 9, 9, 3264, 1), (256, 136, 193, 10, 152, 0),
    ],
    "bf16-mx": [
        (1, 1088, 1, 1, 64, 0), (2, 96, 1, 1, 1184, 0), (4, 64, 128, 57, 544, 0), (7, 96, 1, 1, 1088, 0),
        (7, 544, 135, 135, 96, 0), (8, 160, 53, 53, 576, 2), (15, 64, 1, 1, 288, 0), (15, 288, 1, 1, 64, 0),
        (200, 288, 2, 2, 4832, 0), (200, 288, 12, 12, 96, 0), (256, 64, 1, 1, 8384, 0),
        (256, 288, 55, 55, 128, 0),
    ],
    "f32-mx": [
        (1, 64, 128, 128, 576, 0), (1, 576, 130, 129, 96, 0), (2, 1056, 1, 1, 64, 0), (3, 96, 1, 1, 1312, 0),
        (5, 64, 118, 118, 544, 0), (12, 96, 1, 1, 1056, 0), (15, 672, 142, 141, 96, 2),
        (16, 1216, 136, 136, 64, 0), (17, 288, 1, 1, 64, 0), (32, 64, 1, 1, 288, 0), (256, 320, 9, 9, 64, 0),
    ],
}


class _Kernel(ctypes.Structure):
    _fields_ = [("row_tiles", ctypes.c_int), ("width", ctypes.c_int), ("fused", ctypes.c_bool),
                ("many", ctypes.c_bool), ("cached", ctypes.c_bool)]


class Plan(ctypes.Structure):
    """DecodePlan of csrc/decode.hpp."""
    _fields_ = [("up", _Kernel), ("down", _Kernel), ("picked", ctypes.c_bool), ("row_tile", ctypes.c_int),
                ("entries", ctypes.c_int), ("up_tiles", ctypes.c_int), ("down_tiles", ctypes.c_int),
                ("slices", ctypes.c_int), ("slice_steps", ctypes.c_int)]


def plan(fmt, shape):
    """The library's decode_plan for T, H, E, K, I, n_shared."""
    fn = M.load()["_ZN3moe11decode_planEbbiiiiii"]
    fn.restype, fn.argtypes = Plan, [ctypes.c_bool] * 2 + [ctypes.c_int] * 6
    return fn(fmt.startswith("bf16"), fmt.endswith("mx"), *shape)


def kernels_of(fmt, shape):
    """Template arguments of the two product kernels of a call: format, gate/up, row tiles, width,
    fused, many, cached."""
    p = plan(fmt, shape)
    return [(FORMATS.index(fmt), up, k.row_tiles, k.width, k.fused, k.many, k.cached)
            for up, k in ((True, p.up), (False, p.down))]


def built_kernels():
    """The same of every product kernel in libmoe.so, from its symbols."""
    nm = shutil.which("nm") or shutil.which("llvm-nm", path="/opt/rocm/llvm/bin")
    if nm is None:
        pytest.skip("nm not available")
    names = subprocess.run([nm, M.lib_path()], capture_output=True, text=True, check=True).stdout
    found = re.findall(r"__device_stub__decode_ffn_kernelILi(\d)ELb(\d)ELi(\d)ELi(\d)ELb(\d)ELb(\d)ELb(\d)E", names)
    return {(int(f), up == "1", int(nt), int(cw), fused == "1", many == "1", cached == "1")
            for f, up, nt, cw, fused, many, cached in found}
