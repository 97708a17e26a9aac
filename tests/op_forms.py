"""Sizes that reach every form of the products grouped by expert, and the
library's own rules (a header without HIP, compiled here) that say which form
a size takes."""
import ctypes
import functools
import itertools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "reduction_codec_amd", "csrc")
FORWARD = ["16x32 thin", "16x128", "32x128 span 16", "32x128 span 8", "64x128", "64x256", "128x128", "128x256",
           "32x128 fp32", "32x256 fp32"]
DX = ["64x64 shared", "64x128", "128x256"]
DW = ["128x128 fp32", "128x128", "256x256"]
# 32-wide blocks of a span of the contraction: whole spans are loaded in another way
SPAN = {"16x32 thin": 16, "16x128": 16, "32x128 span 16": 16, "32x128 span 8": 8, "64x128": 8, "64x256": 4, "128x128": 4,
        "128x256": 4, "32x128 fp32": 4, "32x256 fp32": 4}
SOURCE = """
#include "rc_op_rules.hpp"
extern "C" {
int forward(int f32, size_t rows, size_t e, int64_t n, int64_t k) { return (int)rc::forward_form(f32, {rows, e, n, k}); }
int dx(int bf16, size_t rows, size_t e, int64_t n, int64_t k) { return (int)rc::dx_form(bf16, {rows, e, n, k}); }
int dw(int f32, size_t rows, size_t e, int64_t n, int64_t k) { return (int)rc::dw_form(f32, {rows, e, n, k}); }
}
"""


@functools.lru_cache(None)
def rules():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "rules.cpp"), os.path.join(d, "rules.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib],
                       check=True)
        l = ctypes.CDLL(lib)
    for f in (l.forward, l.dx, l.dw):
        f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int64]
    return l


def forms(dtype: str, rows, experts, n, k):
    """{direction: (form, ...)}; forward and its whole spans, dx, dW."""
    l, f32 = rules(), dtype == "fp32"
    fwd = FORWARD[l.forward(f32, rows, experts, n, k)]
    span = 8 if fwd == "16x128" and f32 else SPAN[fwd]
    return {"forward": (fwd, k % (32 * span) == 0), "dx": (DX[l.dx(dtype == "bf16", rows, experts, n, k)],),
            "dw": (DW[l.dw(f32, rows, experts, n, k)],)}


def ragged(experts, mean):
    """Rows of `experts` groups, `mean` on average: one empty, one of a single row, the others around tile edges."""
    each = round(experts * mean / (experts - 2))
    step = itertools.cycle([0, 1, -1, 15, -15, 32, -31, 7, -8])
    counts = [max(0, each + d) for d in itertools.islice(step, experts - 2)] if each > 31 else \
        [max(0, each + d % 5 - 2) for d in itertools.islice(step, experts - 2)]
    counts.insert(1, 0)
    counts.insert(experts // 2, 1)
    return counts


# (row counts, n, k); the rows before the first expert's and after the last one's are BEFORE and AFTER
BEFORE, AFTER = 5, 70
SHAPES = [
    ([3, 0, 17, 1], 200, 2560), ([3, 0, 17, 1], 200, 2592),
    (ragged(24, 5), 1032, 1536), (ragged(24, 5), 1032, 1568),
    (ragged(16, 20), 1032, 1536), (ragged(16, 20), 1032, 1568),
    (ragged(4, 100), 1032, 1536), (ragged(4, 100), 1032, 1568),
    (ragged(16, 70), 1032, 1536), (ragged(16, 70), 1032, 1568),
    (ragged(16, 70), 2056, 1024), (ragged(16, 70), 2056, 800),
    (ragged(8, 200), 1032, 768), (ragged(8, 200), 1032, 800),
    (ragged(8, 310), 4104, 512), (ragged(8, 310), 4104, 544),
    (ragged(8, 400), 8200, 384), (ragged(8, 400), 8200, 416),
    ([3, 0, 70, 1], 1096, 96), ([40, 0, 65, 1], 1032, 160),
    # gradients: several column tiles with a partial last one, 0 to 4 steps after the four-step loop
    (ragged(8, 200), 520, 3296), (ragged(8, 200), 552, 3296), (ragged(8, 200), 584, 3296), (ragged(8, 200), 616, 3296),
    (ragged(8, 200), 640, 3328), (ragged(8, 200), 1032, 3296), (ragged(8, 130), 1088, 3328),
    # more experts than one scan of the bounds takes
    (ragged(200, 70), 264, 544), (ragged(130, 3), 264, 288),
]


def rows_of(counts):
    return BEFORE + sum(counts) + AFTER


def label(shape):
    counts, n, k = shape
    return f"{len(counts)}x{sum(counts) // len(counts)}-{n}x{k}"
