"""The cluster size of a windowed rows launch against a fake CUDA runtime: clusters of sixteen only where the device
says that one fits, asked once a device and kernel."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = next((p for p in ("/usr/local/cuda", os.environ.get("CUDA_HOME", "")) if os.path.exists(f"{p}/include/cuda.h")), None)

HARNESS = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdio.h>
#include "pa_window.h"

static int device, answer, asked, cleared, wide;
static cudaError_t status;
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { ++cleared; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute a, int) {
  wide += a == cudaFuncAttributeNonPortableClusterSizeAllowed;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* cfg) {
  ++asked;
  if (cfg->numAttrs != 1 || cfg->attrs[0].val.clusterDim.x != 16 || cfg->gridDim.x != 16 || cfg->blockDim.x != 192 ||
      cfg->dynamicSmemBytes != 1000) printf("bad question\n");
  *n = answer;
  return status;
}
}
static void kernel(pa::WindowParams) {}
static void ask(pa::ClusterRoom& room, int dev, int cluster) {
  device = dev;
  int32_t c = cluster;
  const cudaError_t e = pa::prepare_rows(&kernel, room, 192, 1000, &c);
  printf("%d %d\n", (int)e, c);
}
int main() {
  pa::ClusterRoom one, two, three;
  answer = 0;                  // no room on device 0: eight instead
  ask(one, 0, 16);
  answer = 4;                  // room on device 1
  ask(one, 1, 16);
  ask(one, 0, 16);             // remembered
  ask(one, 1, 16);
  printf("%d\n", asked);
  ask(two, 0, 16);             // another kernel is asked for
  status = cudaErrorInvalidValue;
  ask(three, 0, 16);           // an error is a no, and does not stay behind
  ask(three, 0, 16);
  printf("%d %d\n", asked, cleared);
  status = cudaSuccess;
  ask(three, 900, 16);         // devices past the memory are asked every time
  ask(three, 900, 16);
  printf("%d\n", asked);
  const int before = wide;
  for (int c : {1, 2, 8}) ask(three, 0, c);  // portable sizes: no question
  printf("%d %d\n", asked, wide - before);
}
"""


@pytest.mark.skipif(CUDA is None or shutil.which("g++") is None, reason="needs g++ and the CUDA headers")
def test_sixteen_only_where_it_fits(tmp_path):
    src, exe = tmp_path / "room.cpp", tmp_path / "room"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", f"-I{CUDA}/include", f"-I{ROOT}/include", f"-I{ROOT}/paged_kv_cache_32_gb300/csrc",
                    str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert lines[:-1] == ["0 8", "0 16", "0 8", "0 16", "2", "0 16", "0 8", "0 8", "4 1", "0 16", "0 16", "6", "0 1", "0 2",
                          "0 8", "6 0"]
