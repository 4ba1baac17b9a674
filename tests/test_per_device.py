"""CPU check of the numbers that launchers keep per device (PerDevice in qmv_internal.h), compiled with the host compiler
against a stand-in for cudaGetDevice: a device's answer is asked once and is no other device's; zero is an answer; errors
are not kept."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SRC = r'''
#include <cstdio>
#include "qmv_internal.h"
static int device = 0;
extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
int main() {
  static qmv::PerDevice kept;
  const int number[3] = {76, 0, 72};
  int asked = 0;
  for (int round = 0; round < 3; ++round) {
    for (device = 0; device < 3; ++device) {
      int v = -1;
      const cudaError_t e = kept.get(&v, [&](int* n) {
        ++asked;
        if (asked == 1) return cudaErrorUnknown;
        *n = number[device];
        return cudaSuccess;
      });
      std::printf("%d:%d ", (int)e, v);
    }
  }
  device = 64;
  int v = 0;
  std::printf("%d %d\n", asked, (int)kept.get(&v, [](int*) { return cudaSuccess; }));
  return 0;
}
'''


def test_numbers_are_kept_per_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no host C++ compiler or CUDA headers")
    src, exe = tmp_path / "pd.cpp", tmp_path / "pd"
    src.write_text(SRC)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", os.path.join(ROOT, "bit_quantized_moe_gb300", "csrc"), "-I", cuda,
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    unknown, invalid = 999, 101   # cudaErrorUnknown, cudaErrorInvalidDevice
    assert out == [f"{unknown}:-1", "0:0", "0:72", "0:76", "0:0", "0:72", "0:76", "0:0", "0:72", "4", str(invalid)]
