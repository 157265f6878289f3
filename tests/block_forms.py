"""The rules that choose a product's form in 8-bit blocks (csrc/block_forms.h, host code without
HIP), compiled and called on the CPU: which form a case of the tests takes."""
import atexit
import ctypes
import functools
import os
import shutil
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ["own rows", "few rows", "256x256", "256x128", "128x128 twice", "128x128", "128x64",
         "128x32", "64x32", "32x32", "none"]
# sets of waves that split the contraction's blocks, by form
SETS = {"256x256": 1, "256x128": 1, "128x128 twice": 1, "128x128": 1, "128x64": 2, "128x32": 2,
        "64x32": 4, "32x32": 4}
UNITS = 256                                            # compute units of an MI355X

SOURCE = """
#include "block_forms.h"
extern "C" int form(int64_t n, int m, int k, int groups, int offsets, int transposed, int x16,
                    int units) {
    return exl3::block_form(exl3::BlockCall{n, m, k, groups, offsets != 0, transposed != 0},
                            x16 != 0, units);
}
"""


@functools.lru_cache(None)
def _library():
    folder = tempfile.mkdtemp(prefix="block_forms")
    atexit.register(shutil.rmtree, folder, ignore_errors=True)
    src, lib = os.path.join(folder, "form.cpp"), os.path.join(folder, "form.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "trellis_coded_weight_amd", "csrc"), src, "-o", lib],
                   check=True)
    form = ctypes.CDLL(lib).form
    form.argtypes = [ctypes.c_int64] + [ctypes.c_int] * 7
    return form


def form(n, m, k, groups=1, offsets=None, transposed=False, x16=False, units=UNITS):
    """The form's name; offsets: whether rows are given by group (so with more than one group)."""
    offsets = groups > 1 if offsets is None else offsets
    return NAMES[_library()(n, m, k, groups, offsets, transposed, x16, units)]
