"""The launch plan of the 8-bit products, compiled for the host from the
library's own header."""
import collections
import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROOM = 1 << 30  # bytes: more than any form's pieces take
CUS = 256       # of an MI355X

_SOURCE = r"""
#include "w8a8_plan.h"
extern "C" void plan(int n, int m, int k, int gated, int cus, size_t room, int *o) {
    const vq::Plan p = vq::plan_of(n, m, k, gated != 0, cus, room);
    const vq::Form &f = vq::kForms[p.form];
    const int v[] = {p.form, p.groups, p.whole, p.cuts, f.rows(), f.feats(), f.wk,
                     vq::past_caches(f, n, m, k, gated != 0)};
    for (int i = 0; i < 8; ++i)
        o[i] = v[i];
}
extern "C" int forms() { return vq::kFormCount; }
extern "C" size_t counter_bytes() { return vq::kCounterBytes; }
"""

Plan = collections.namedtuple("Plan", "form groups whole cuts rows feats wk past")


@functools.lru_cache(maxsize=None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(_SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC",
                        "-I" + os.path.join(ROOT, "block_quantized_gemm_amd", "csrc"),
                        "-I" + os.path.join(ROOT, "include"), src, "-o", so], check=True)
        handle = ctypes.CDLL(so)
    handle.plan.argtypes = [ctypes.c_int] * 5 + [ctypes.c_size_t, ctypes.POINTER(ctypes.c_int)]
    handle.plan.restype = None
    handle.counter_bytes.restype = ctypes.c_size_t
    return handle


def plan(n, m, k, gated=False, room=ROOM, cus=CUS):
    o = (ctypes.c_int * 8)()
    lib().plan(n, m, k, gated, cus, room, o)
    return Plan(*o)


def tiles(p, n, m, gated=False):
    """Rows and columns of tiles of a planned launch."""
    feats = p.feats // 2 if gated else p.feats
    return -(-n // p.rows), -(-m // feats)
