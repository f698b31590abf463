"""tensor_map.cu against fakes of the CUDA calls it makes, compiled for the host: a
failed lookup of the driver's encoder is not kept, a found one is, and only memory
that this GPU reaches is taken."""
import glob
import os
import shutil
import subprocess

import memory_bound_normalization_rmsnorm_gb300 as gb

CSRC = os.path.join(os.path.dirname(gb.__file__), "csrc")

PROGRAM = r"""
#include <cuda_runtime.h>
#include "tensor_map.h"
static int g_lookups = 0, g_fail = 1;
static cudaMemoryType g_type;
static int g_dev;
extern "C" cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
extern "C" cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(
    const char *, void **fn, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *q) {
  ++g_lookups;
  *fn = g_fail ? nullptr : reinterpret_cast<void *>(&g_lookups);
  *q = g_fail == 1 ? cudaDriverEntryPointSymbolNotFound : cudaDriverEntryPointSuccess;
  return g_fail == 2 ? cudaErrorInitializationError : cudaSuccess;
}
extern "C" cudaError_t CUDARTAPI cudaPointerGetAttributes(cudaPointerAttributes *a, const void *p) {
  a->type = g_type;
  a->device = g_dev;
  return p ? cudaSuccess : cudaErrorInvalidValue;
}
int main() {
  gbn::MapEncoder e = nullptr;
  for (g_fail = 1; g_fail <= 3; ++g_fail)  // not there; an error; no address
    if (gbn::map_encoder(&e) != NORM_ERR_CUDA || e) return 1;
  g_fail = 0;
  if (gbn::map_encoder(&e) != NORM_OK || reinterpret_cast<void *>(e) != &g_lookups) return 2;
  e = nullptr;
  if (gbn::map_encoder(&e) != NORM_OK || !e || g_lookups != 4) return 3;
  const struct { cudaMemoryType t; int dev; bool good; } cases[] = {
      {cudaMemoryTypeDevice, 1, true}, {cudaMemoryTypeDevice, 0, false},
      {cudaMemoryTypeManaged, 0, true}, {cudaMemoryTypeHost, 1, false},
      {cudaMemoryTypeUnregistered, 1, false}};
  for (const auto &c : cases) {
    g_type = c.t;
    g_dev = c.dev;
    if ((gbn::check_device_memory(&e, 1) == NORM_OK) != c.good) return 4;
  }
  return gbn::check_device_memory(nullptr, 1) == NORM_ERR_MEMORY ? 0 : 5;
}
"""


def test_lookups_and_memory_kinds(tmp_path):
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")))
    main, exe = tmp_path / "t.cpp", tmp_path / "t"
    main.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", os.path.join(cuda, "include"), "-I", CSRC,
                    str(main), os.path.join(CSRC, "tensor_map.cu"), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_nothing_else_looks_the_encoder_up():
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        with open(path) as f:
            found = '"cuTensorMapEncodeTiled"' in f.read()
        assert found == (os.path.basename(path) == "tensor_map.cu"), path
