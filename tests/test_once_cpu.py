"""Set-up that failed once is tried again: csrc/qsw_once.h over a runtime whose calls fail
first."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from quantized_swiglu_mlp_gb300 import build

PROGRAM = r"""
#include "qsw_once.h"

#include <cstdio>
#include <initializer_list>

static int device = 0, lookups = 0, found_from = 0;
extern "C" cudaError_t CUDARTAPI cudaGetDevice(int *d) {
  *d = device;
  return device < 0 ? cudaErrorNoDevice : cudaSuccess;
}
extern "C" cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long,
                                                                  cudaDriverEntryPointQueryResult *r) {
  if (++lookups < found_from) return cudaErrorInitializationError;
  *r = lookups == found_from ? cudaDriverEntryPointSymbolNotFound : cudaDriverEntryPointSuccess;
  *p = &lookups;
  return cudaSuccess;
}

#define CHECK(x) if (!(x)) return printf("line %d: %s\n", __LINE__, #x), 1

int main() {
  static qsw::DeviceOnce once;
  int calls = 0;
  cudaError_t answer = cudaErrorMemoryAllocation;
  auto set_up = [&] { return ++calls, answer; };
  CHECK(qsw::once_per_device(once, set_up) == cudaErrorMemoryAllocation && calls == 1);
  CHECK(qsw::once_per_device(once, set_up) == cudaErrorMemoryAllocation && calls == 2);
  answer = cudaSuccess;
  CHECK(qsw::once_per_device(once, set_up) == cudaSuccess && calls == 3);
  answer = cudaErrorMemoryAllocation;
  CHECK(qsw::once_per_device(once, set_up) == cudaSuccess && calls == 3);
  device = 63;                       // another device has its own
  CHECK(qsw::once_per_device(once, set_up) == cudaErrorMemoryAllocation && calls == 4);
  for (int bad : {-1, 64}) {
    device = bad;
    CHECK(qsw::once_per_device(once, set_up) != cudaSuccess && calls == 4);
  }
  found_from = 3;
  CHECK(!qsw::encode_tiled_fn() && !qsw::encode_tiled_fn() && !qsw::encode_tiled_fn());
  CHECK(reinterpret_cast<void *>(qsw::encode_tiled_fn()) == &lookups && lookups == 4);
  CHECK(qsw::encode_tiled_fn() && lookups == 4);
  return 0;
}
"""


def test_failed_set_up_is_tried_again(tmp_path):
    cxx = os.environ.get("CXX", "g++")
    if not shutil.which(cxx):
        pytest.skip("no C++ compiler")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    source, program = tmp_path / "once.cpp", tmp_path / "once"
    source.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.CSRC, "-isystem", os.path.join(cuda, "include"), str(source),
                        "-o", str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_nothing_else_keeps_a_failure():
    """No source keeps the answer of a set-up, whatever it was."""
    for name in os.listdir(build.CSRC):
        with open(os.path.join(build.CSRC, name)) as f:
            assert "call_once" not in f.read(), name
