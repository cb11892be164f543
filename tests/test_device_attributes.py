"""The opt-in to large shared memory is made once for each kernel and device: checked on the host, against stand-ins
for the runtime's calls."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = "/usr/local/cuda/include"

PROGRAM = r"""
#include "block_diffusion_text_gb300/csrc/dg_internal.h"
#include <cstdio>

static int device = 0, sets = 0, fail = 0;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  ++sets;
  return fail ? cudaErrorInvalidValue : cudaSuccess;
}
static void one(int) {}
static void two(int) {}

int main() {
  auto a = [](int dev) { device = dev; return dg::set_smem_once<&one>(100000); };
  auto b = [](int dev) { device = dev; return dg::set_smem_once<&two>(100000); };
  fail = 1;
  if (a(0) == cudaSuccess || sets != 1) return 1;   // an error is told, and tried again
  fail = 0;
  if (a(0) || a(0) || sets != 2) return 2;          // once on a device
  if (a(1) || a(1) || a(0) || sets != 3) return 3;  // and once on each other one
  if (b(1) || b(0) || b(1) || sets != 5) return 4;  // each kernel for itself
  if (a(63) || a(63) || sets != 6) return 5;
  if (a(70) || sets != 7) return 6;                 // past the table: set every time
  if (a(0) || a(1) || sets != 7) return 7;
  return 0;
}
"""


@pytest.mark.skipif(not (shutil.which("g++") and os.path.isdir(CUDA)), reason="g++ and the CUDA headers")
def test_shared_memory_is_opted_in_on_every_device(tmp_path):
    src = tmp_path / "attr.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "attr"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", ROOT, "-I", CUDA, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
