"""Whether a device has room for clusters of sixteen CTAs: compiled against a fake of the
runtime's calls (CPU only).  Where there is none, or the question fails, eight are taken and no
error stays behind; every call asks, since the answer may be another in another context."""
import os
import subprocess

import pytest

from block_sparse_attention_online_gb300 import build as B

PROGRAM = r"""
#include "cluster_size.h"
#include <cstdio>
#include <cstdlib>

static int asked, room, allowed_at, error_left, kernel;
static cudaError_t answer, of_attribute;
extern "C" cudaError_t cudaGetLastError() { error_left = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int v) {
  if (f != &kernel || a != cudaFuncAttributeNonPortableClusterSizeAllowed || v != 1) std::abort();
  allowed_at = asked + 1;
  if (of_attribute != cudaSuccess) error_left = 1;
  return of_attribute;
}
extern "C" cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c) {
  ++asked;
  if (f != &kernel || allowed_at != asked || c->numAttrs != 1 || c->gridDim.x != 16 ||
      c->attrs->id != cudaLaunchAttributeClusterDimension || c->attrs->val.clusterDim.x != 16 ||
      c->attrs->val.clusterDim.y != 1 || c->attrs->val.clusterDim.z != 1 ||
      c->dynamicSmemBytes != 777 || c->blockDim.x != 256)
    std::abort();
  *n = room;
  if (answer != cudaSuccess) error_left = 1;
  return answer;
}
static void ask() {
  const bool fits = attn_skip::large_cluster_fits(&kernel, 256, 777);
  std::printf("%d %d %d\n", fits, asked, error_left);
}

int main() {
  room = 9;
  ask();
  room = 0;
  ask();                                             // another context without
  room = 1;
  ask();
  answer = cudaErrorInvalidClusterSize;
  ask();                                             // refused: eight, and no error
  answer = cudaSuccess; of_attribute = cudaErrorInvalidValue;
  ask();                                             // not even allowed: not asked
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("cluster_size")
    (at / "main.cpp").write_text(PROGRAM)
    include = os.path.join(os.path.dirname(os.path.dirname(B._nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-I", include, "-I", B.CSRC, str(at / "main.cpp"),
                        "-o", str(at / "main")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(at / "main")


def test_eight_are_the_way_back(program):
    r = subprocess.run([program], capture_output=True, text=True)
    assert r.returncode == 0
    # Whether it fits, calls so far, an error left behind.
    assert r.stdout.split("\n")[:-1] == ["1 1 0", "0 2 0", "1 3 0", "0 4 0", "0 4 0"]
