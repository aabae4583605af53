"""What the decode calls ask the CUDA runtime, with the runtime faked on the host: one answer per kernel and
shared-memory size, whatever the batch sizes that a process serves, and none about kernels that a call does not
launch.  kivi_decode_host.cu holds host code only, so a C++ compiler takes it as it is."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from bit_asymmetric_kv_gb300 import build as kbuild

MAIN = r"""
#include <stdio.h>
#include <stdlib.h>
#include "kivi_internal.h"

static int g_queries, g_window_queries;   // of the occupancy and the attributes
static bool g_window_fails;
static char g_fn[4096];                   // the kernels' addresses: [0, 2048) whole contexts, behind them windows

static cudaError_t asked(const void *fn) {
  ++g_queries;
  if ((const char *)fn >= g_fn + 2048) {
    ++g_window_queries;
    if (g_window_fails) return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 10; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *fn, cudaFuncAttribute, int) { return asked(fn); }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *fn, int, size_t smem) {
  *n = smem > 30000 ? 1 : (const char *)fn >= g_fn + 2048 ? 2 : 3;
  return asked(fn);
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *fn, const cudaLaunchConfig_t *) { *n = 1; return asked(fn); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **) { abort(); }
}
namespace kivi {
static DecodeKernels kernels(int R, int G, int bits, int B, int at) {
  DecodeKernels k = {};
  k.decode = g_fn + at + 16 * R + G / 32 + 4 * (bits / 4);
  k.smem = 20000 + 8 * B / 16 * 16;
  k.smem_limit = 40000;
  return k;
}
DecodeKernels decode_kernels(int R, int G, int bits, bool, int B, int) { return kernels(R, G, bits, B, 0); }
DecodeKernels decode_window_kernels(int R, int G, int bits, int B) { return kernels(R, G, bits, B, 2048); }
}  // namespace kivi

static int sweep(bool window, int *warps, int *failed) {  // queries of all batch sizes, and a sum of the answers
  const int before = g_queries;
  *warps = *failed = 0;
  for (int G = 32; G <= 64; G += 32)
    for (int B = 1; B <= 512; ++B) {
      kivi::PagedGeom g = {};
      if (kivi::paged_decode_geometry(B, 8, 32, G, 2, &g, window) != cudaSuccess) ++*failed;
      *warps += g.n_warps;
    }
  return g_queries - before;
}

int main() {
  int w[6], f[6];
  const int first = sweep(false, &w[0], &f[0]), again = sweep(false, &w[1], &f[1]);
  const int whole_window_queries = g_window_queries;
  const int win = sweep(true, &w[2], &f[2]), win_again = sweep(true, &w[3], &f[3]), third = sweep(false, &w[4], &f[4]);
  printf("{\"first\": %d, \"again\": %d, \"window_in_whole\": %d, \"win\": %d, \"win_again\": %d, \"third\": %d, ", first, again,
         whole_window_queries, win, win_again, third);
  printf("\"same\": %d, \"win_same\": %d, \"failed\": %d, ", w[0] == w[1] && w[0] == w[4], w[2] == w[3] && w[2] < w[0],
         f[0] + f[1] + f[2] + f[3] + f[4]);
  // a window's kernel that the device refuses is the window calls' trouble
  g_window_fails = true;
  kivi::PagedGeom g = {};
  const bool whole_ok = kivi::paged_decode_geometry(7, 8, 8, 32, 4, &g, false) == cudaSuccess;
  const bool window_ok = kivi::paged_decode_geometry(7, 8, 8, 32, 4, &g, true) == cudaSuccess;
  printf("\"whole_ok\": %d, \"window_ok\": %d}\n", whole_ok, window_ok);
}
"""


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    import json

    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("tables")
    (d / "main.cpp").write_text(MAIN)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(kbuild.nvcc()))), "include")
    flags = ["-std=c++17", "-O1", "-I", cuda, "-I", kbuild.CSRC, "-I", os.path.join(kbuild.ROOT, "include"), "-pthread"]
    host = os.path.join(kbuild.CSRC, "kivi_decode_host.cu")
    subprocess.run([cxx, *flags, "-x", "c++", str(d / "main.cpp"), "-x", "c++", host, "-o", str(d / "main")], check=True)
    return json.loads(subprocess.run([str(d / "main")], check=True, capture_output=True, text=True).stdout)


def test_every_batch_size_is_asked_about_once(counts):
    assert counts["first"] > 0 and counts["win"] > 0 and counts["failed"] == 0
    assert counts["again"] == counts["win_again"] == counts["third"] == 0
    assert counts["same"] and counts["win_same"]


def test_whole_context_calls_ask_nothing_about_the_windows_kernel(counts):
    assert counts["window_in_whole"] == 0
    assert counts["whole_ok"] and not counts["window_ok"]
