"""A kernel's limit of dynamic shared memory is a setting that threads share: it is never taken
below what another thread's launch relies on.  A small program with the runtime's two calls
replaced; nothing here reaches a GPU."""
import os
import re
import subprocess

from grammar_constrained_logit_gb300 import build

PROGRAM = r"""
#include <cuda_runtime.h>
#include <cstdio>
#include <vector>

static int device = 0;
static bool fails = false;
static std::vector<int> set_to[2];
static void (*in_between)() = nullptr;

static cudaError_t fake_device(int* d) { return *d = device, cudaSuccess; }
template <class K>
static cudaError_t fake_set(K*, cudaFuncAttribute, int bytes) {
  if (fails) return cudaErrorInvalidValue;
  if (in_between != nullptr) {  // another thread's call, from its first line to its last
    void (*f)() = in_between;
    in_between = nullptr;
    f();
  }
  set_to[device].push_back(bytes);
  return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#include "common.cuh"

static void kernel(int) {}
static lp::PerDevice<1> allowed;
static cudaError_t call() { return lp::allow_shared(kernel, 98304, allowed); }

int main() {
  fails = true;
  if (call() == cudaSuccess) return 1;  // and it is not taken as done
  fails = false;
  in_between = [] { call(); };
  for (device = 0; device < 2; ++device)
    for (int i = 0; i < 3; ++i)
      if (call() != cudaSuccess) return 2;
  for (int d = 0; d < 2; ++d) {
    if (set_to[d].size() != (d == 0 ? 2 : 1)) return 3;  // once a device, or once a thread of it
    for (int bytes : set_to[d])
      if (bytes != 98304) return 4;
  }
  return 0;
}
"""


def test_limit_is_one_number(tmp_path):
    source, program = tmp_path / "limit.cu", tmp_path / "limit"
    source.write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-O1", f"-I{build.INCLUDE}",
                    f"-I{build.CSRC}", "-o", str(program), str(source)], check=True, timeout=300)
    assert subprocess.run([str(program)], timeout=60).returncode == 0


def test_no_launch_asks_for_a_limit_of_its_own():
    """What the launches of the cache's operators pass is a constant of the kernel's."""
    for name, limits in (("evict.cu", ("kHeldTokens * 4", "2 * kRoundBytes")),
                         ("attend.cu", ("kAnyBytes",)), ("attend_chunk.cu", ("smem",))):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        calls = re.findall(r"allow_shared\([^;]*, ([^,;]+), allowed", text)
        assert sorted(calls) == sorted(limits), (name, calls)
