"""What the launchers keep of a device is kept for each device (CPU): the lookups of csrc/ssm.cuh, compiled against stand-ins for
the runtime's calls, on two devices that differ."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

SOURCE = r"""
#include <cstdio>
#include "ssm.cuh"

static int device, asked;
extern "C" cudaError_t cudaGetDevice(int* dev) {
  *dev = device;
  return cudaSuccess;
}
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int dev) {
  *v = dev ? 100 : 152;
  return cudaSuccess;
}
// (device 1's SMs hold half as many; a device past the table's end is refused before it is asked)
static cudaError_t occupancy(int* held, const void*, int threads, size_t) {
  ++asked;
  *held = (device ? 512 : 1024) / threads;
  return cudaSuccess;
}
extern "C" cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* h, const void* f, int t, size_t b) {
  return occupancy(h, f, t, b);
}
extern "C" cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* h, const void* f, int t, size_t b, unsigned) {
  return occupancy(h, f, t, b);
}

static void kernel(int) {}

int main() {
  static palimpsa::HeldCtas known;
  for (int round = 0; round < 2; ++round)
    for (device = 0; device < 2; ++device)
      for (int threads : {128, 256}) {
        int held = 0;
        const cudaError_t e = palimpsa::held_ctas(kernel, threads, 0, &known, &held);
        std::printf("%d %d %d %d %d\n", device, threads, (int)e, held, palimpsa::sms_of_device());
      }
  device = 64;
  int held = 0;
  std::printf("%d %d\n", (int)palimpsa::held_ctas(kernel, 128, 0, &known, &held) == (int)cudaErrorInvalidDevice, asked);
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="no CUDA toolkit")
def test_occupancies_and_sizes_are_kept_for_each_device(tmp_path):
    src, exe = tmp_path / "devices.cpp", tmp_path / "devices"
    src.write_text(SOURCE)
    subprocess.run([NVCC, "-std=c++17", "-cudart", "none", "-I", os.path.join(ROOT, "metaplastic_linear_attention_gb300", "csrc"), str(src), "-o",
                    str(exe)], check=True, capture_output=True, text=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    want = [f"{dev} {threads} 0 {(512 if dev else 1024) // threads} {100 if dev else 152}"
            for _ in range(2) for dev in range(2) for threads in (128, 256)]
    assert got[:8] == want
    assert got[8] == "1 4"     # refused; every device was asked once for either size
