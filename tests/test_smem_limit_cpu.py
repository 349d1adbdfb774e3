"""Shared-memory limits are set once for each kernel and device and then
remembered, for as many pairs as the library has on sixteen devices."""
from __future__ import annotations

import os
import subprocess

from attention_attn_fwd_02_gb300 import build

MAIN = r"""
#include <stdio.h>
#include "smem_limit.h"
static int device, calls;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { ++calls; return cudaSuccess; }
static char kernels[300 * 64];
static int pass(int bytes) {
  calls = 0;
  for (device = 0; device < 16; ++device)
    for (int k = 0; k < 300; ++k)
      if (attn::ensure_smem(kernels + 64 * k, bytes + k) != cudaSuccess) return -1;
  return calls;
}
int main() {
  const int first = pass(70000), again = pass(70000), less = pass(60000), more = pass(80000), last = pass(80000);
  printf("%d %d %d %d %d\n", first, again, less, more, last);
}
"""


def test_limits_are_remembered(tmp_path):
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(MAIN)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, "-I", cuda, str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [4800, 0, 0, 4800, 0]
