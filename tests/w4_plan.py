"""The library's choice of 4-bit kernel (csrc/w4_plan.h), built for the host."""

import ctypes
import os
import subprocess
from collections import namedtuple

from bitlinear_w1_a8_amd import build

SOURCE = """
#include "w4_plan.h"
extern "C" void plan(int64_t t, int64_t n, int64_t k, int g, int64_t cus, int64_t* out) {
  const bl::W4Plan p = bl::w4_plan(t, n, k, g, cus);
  out[0] = p.wn; out[1] = p.wk; out[2] = p.wmf; out[3] = p.team; out[4] = p.tokens;
}
"""

Plan = namedtuple("Plan", "wn wk wmf team tokens")


def compiled(folder):
    """w4_plan(T, N, K, G, CUs) -> Plan, from a library built in `folder`."""
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).plan
    fn.restype = None
    fn.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]

    def plan(t, n, k, g, cus):
        out = (ctypes.c_int64 * 5)()
        fn(t, n, k, g, cus, out)
        return Plan(*out)
    return plan
