"""csrc/sample_weight.h compiled for the host, every operation rounded by itself
(no contraction), and the exponential it stands for in long double."""
import ctypes
import os
import subprocess

import numpy as np

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "early_exit_decoding_gb300", "csrc")
SOURCE = r"""
#include "sample_weight.h"
using namespace river;
extern "C" void weights(const float* x, long n, float m, float t, uint64_t* out) {
  uint64_t table[64];
  for (int j = 0; j < 64; ++j) table[j] = weight::entry(j);
  const weight::Rate c = weight::rate_of(t);
  for (long i = 0; i < n; ++i) out[i] = weight::of(x[i], m, c, [&](uint32_t j) { return table[j]; });
}
// (weight - exact) / exact less half a unit's share; exact in units
extern "C" void errors(const float* x, long n, float m, float t, double* rel, double* exact) {
  uint64_t table[64];
  for (int j = 0; j < 64; ++j) table[j] = weight::entry(j);
  const weight::Rate c = weight::rate_of(t);
  for (long i = 0; i < n; ++i) {
    const long double w = expl(((long double)x[i] - m) / t) * 17592186044416.0L;
    const long double off = fabsl((long double)weight::of(x[i], m, c, [&](uint32_t j) { return table[j]; }) - w) - 0.5L;
    rel[i] = (double)(off > 0 ? off / w : 0);
    exact[i] = (double)w;
  }
}
"""


class WeightHost:
    def __init__(self, folder):
        src, lib = os.path.join(folder, "weight.cpp"), os.path.join(folder, "weight_host.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)

    def weights(self, x, m, t):
        """Weights (uint64) of fp32 logits x beside the largest, m."""
        x = np.ascontiguousarray(x, np.float32)
        out = np.empty(x.shape, np.uint64)
        self.lib.weights(x.ctypes.data_as(ctypes.c_void_p), ctypes.c_long(x.size), ctypes.c_float(m), ctypes.c_float(t), out.ctypes.data_as(ctypes.c_void_p))
        return out

    def errors(self, x, m, t):
        """How far each weight is from its exponential, beyond half a unit and relative to it; the exponentials in units."""
        x = np.ascontiguousarray(x, np.float32)
        rel, exact = np.empty(x.shape), np.empty(x.shape)
        self.lib.errors(x.ctypes.data_as(ctypes.c_void_p), ctypes.c_long(x.size), ctypes.c_float(m), ctypes.c_float(t),
                        rel.ctypes.data_as(ctypes.c_void_p), exact.ctypes.data_as(ctypes.c_void_p))
        return rel, exact
