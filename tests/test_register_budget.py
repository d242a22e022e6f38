"""The check before the first launch of a kernel that raises its warps' register limits, against a fake CUDA runtime."""
import os
import shutil
import subprocess

import pytest

from test_cluster_room import CUDA, ROOT

HARNESS = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdio.h>
#include "pa_launch.h"

static int regs, asked;
static cudaError_t status;
extern "C" cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  ++asked;
  a->numRegs = regs;
  return status;
}
static void ask(std::atomic<bool>& known) { printf("%d\n", (int)pa::require_registers(nullptr, 96, known)); }
int main() {
  std::atomic<bool> one{false}, two{false};
  regs = 88;
  ask(one);                           // fewer than the budget: no launch, however often
  ask(one);
  regs = 96;
  ask(one);
  regs = 0;
  ask(one);                           // looked at once
  printf("%d\n", asked);
  status = cudaErrorNoDevice;
  ask(two);                           // an error is passed on, and not kept
  status = cudaSuccess;
  regs = 104;
  ask(two);
  printf("%d\n", asked);
}
"""


@pytest.mark.skipif(CUDA is None or shutil.which("g++") is None, reason="needs g++ and the CUDA headers")
def test_too_few_registers_are_not_launched(tmp_path):
    src, exe = tmp_path / "regs.cpp", tmp_path / "regs"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", f"-I{CUDA}/include", f"-I{ROOT}/include",
                    f"-I{os.path.join(ROOT, 'paged_kv_cache_32_gb300', 'csrc')}", str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert lines == ["9", "9", "0", "0", "3", "100", "0", "5"]  # (9: cudaErrorInvalidConfiguration, 100: no device)
