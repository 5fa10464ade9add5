"""How the library runs a whole routed layer (csrc/layer_plan.h), built for the host."""

import collections
import ctypes
import os
import subprocess

from bitlinear_w1_a8_amd import build

SOURCE = """
#include "layer_plan.h"
extern "C" void plan(int64_t t, int64_t e, int64_t k, int64_t f, int64_t kk, int64_t n, int raw, int cus, int* out) {
  const bl::LayerPlan p = bl::layer_plan(t, e, k, f, kk, n, raw, cus);
  const int all[] = {p.two, p.own_quant, p.pairs, p.gate_waves, p.down_tiles, p.team};
  for (int i = 0; i < 6; ++i) out[i] = all[i];
}
extern "C" int depth(int64_t k) { return bl::few_depth(k); }
"""

Plan = collections.namedtuple("Plan", "two own_quant pairs gate_waves down_tiles team")


def compiled(folder):
    """layer_plan(T, E, k, F, K, N, raw bytes, CUs) -> Plan, and few_depth(K), from a library built in `folder`."""
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", lib], check=True)
    built = ctypes.CDLL(lib)
    built.plan.argtypes = [ctypes.c_int64] * 6 + [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    built.depth.argtypes = [ctypes.c_int64]

    def plan(*sizes):
        out = (ctypes.c_int * 6)()
        built.plan(*sizes, out)
        return Plan(*out)
    return plan, built.depth
