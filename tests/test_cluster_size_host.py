"""Whether a device has room for clusters of sixteen CTAs: compiled against a fake of the
runtime's calls (CPU only).  Where there is none, or the question fails, eight are taken and no
error stays behind; each device is asked once."""
import os
import subprocess

import pytest

from block_sparse_attention_online_gb300 import build as B

PROGRAM = r"""
#include "cluster_size.h"
#include <cstdio>
#include <cstdlib>

static int device, asked, room, allowed_at, error_left, threads;
static cudaError_t answer, of_device = cudaSuccess, of_attribute = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return of_device; }
extern "C" cudaError_t cudaGetLastError() { error_left = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute a, int v) {
  if (a != cudaFuncAttributeNonPortableClusterSizeAllowed || v != 1) std::abort();
  allowed_at = asked + 1;
  if (of_attribute != cudaSuccess) error_left = 1;
  return of_attribute;
}
extern "C" cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *c) {
  ++asked;
  if (allowed_at != asked || c->numAttrs != 1 || c->attrs->val.clusterDim.x != 16 ||
      c->attrs->val.clusterDim.y != 1 || c->attrs->val.clusterDim.z != 1 || c->gridDim.x != 16 ||
      c->dynamicSmemBytes != 777 || (int)c->blockDim.x != threads)
    std::abort();
  *n = room;
  if (answer != cudaSuccess) error_left = 1;
  return answer;
}
static void line(bool fits) { std::printf("%d %d %d\n", fits, asked, error_left); }

int main() {
  using namespace attn_skip;
  static ClusterRoom a, b, c;
  auto ask = [](ClusterRoom &r) { return large_cluster_fits(&device, threads, 777, r); };
  threads = 256;
  room = 9;
  line(ask(a)); line(ask(a));              // room, asked once
  device = 1; room = 0;
  line(ask(a)); room = 9; line(ask(a));    // another device without
  device = 0; line(ask(a));                // the first one is still known
  device = 1; line(ask(b));                // another kernel
  device = 2; answer = cudaErrorInvalidClusterSize;
  line(ask(b)); answer = cudaSuccess; line(ask(b));  // refused: eight, and no error
  device = 3; of_attribute = cudaErrorInvalidValue;
  line(ask(b)); of_attribute = cudaSuccess;
  device = ClusterRoom::kDevices;          // beyond what is kept: asked each time
  line(ask(c)); line(ask(c));
  of_device = cudaErrorNoDevice; line(ask(c));
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


def test_each_device_is_asked_once_and_eight_are_the_way_back(program):
    r = subprocess.run([program], capture_output=True, text=True)
    assert r.returncode == 0
    assert r.stdout.split("\n")[:-1] == [
        "1 1 0", "1 1 0",   # fits, calls so far, error left
        "0 2 0", "0 2 0",
        "1 2 0",
        "1 3 0",
        "0 4 0", "0 4 0",
        "0 4 0",
        "1 5 0", "1 6 0",
        "0 6 0",
    ]
