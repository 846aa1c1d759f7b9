"""The host queries in front of a cluster launch (csrc/t3_vec.cuh), compiled here
with fakes of the CUDA calls: a query that fails leaves no error behind for the
next call's check to find, and an answer is asked for once, "none fit" too."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

SOURCE = r"""
#include <cuda_runtime.h>
#include <cstdio>
static int calls = 0, answer = 0, fails = 0;
static cudaError_t last = cudaSuccess;  // what the next check of any call finds
static cudaError_t failing() { return last = cudaErrorInvalidValue; }
static cudaError_t fake_last() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
template <class F> cudaError_t fake_clusters(int* n, F, const cudaLaunchConfig_t*) {
  ++calls;
  *n = answer;
  return fails ? failing() : cudaSuccess;
}
template <class F> cudaError_t fake_attribute(F, cudaFuncAttribute, int) {
  ++calls;
  return fails ? failing() : cudaSuccess;
}
#include "t3_internal.h"
#define cudaOccupancyMaxActiveClusters fake_clusters
#define cudaFuncSetAttribute fake_attribute
#define cudaGetLastError fake_last
#include "t3_vec.cuh"
template <int> __global__ void kernel() {}
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
  using namespace t3::vec;
  fails = 1;
  CHECK(max_clusters<kernel<0>>(0, 2, 256, 1024) == 0);
  CHECK(last == cudaSuccess);
  CHECK(allow_smem<kernel<0>>(0, 1024) == T3_ECUDA);
  CHECK(last == cudaSuccess);
  fails = 0;  // a failure is not kept
  answer = 7;
  CHECK(max_clusters<kernel<0>>(0, 2, 256, 1024) == 7);
  CHECK(allow_smem<kernel<0>>(0, 1024) == T3_OK);
  calls = 0;
  CHECK(max_clusters<kernel<0>>(0, 2, 256, 1024) == 7 && allow_smem<kernel<0>>(0, 1024) == T3_OK && calls == 0);
  answer = 0;
  CHECK(max_clusters<kernel<0>>(0, 3, 256, 1024) == 0 && calls == 1);
  CHECK(max_clusters<kernel<0>>(0, 3, 256, 1024) == 0 && calls == 1);
  CHECK(max_clusters<kernel<1>>(0, 2, 256, 1024) == 0 && calls == 2);
  std::printf("fine\n");
  return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(NVCC), reason="needs nvcc")
def test_failed_queries_leave_no_error_and_answers_are_kept(tmp_path):
    src, exe = tmp_path / "queries.cu", tmp_path / "queries"
    src.write_text(SOURCE)
    csrc = os.path.join(ROOT, "ternary_weight_int8_t3_gb300", "csrc")
    cmd = [NVCC, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", csrc, "-I", os.path.join(ROOT, "include"),
           "-o", str(exe), str(src)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr
