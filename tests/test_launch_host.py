"""CPU tests of the launch helpers (csrc/gdn_launch.cuh) against a stand-in for the
CUDA runtime: how much dynamic shared memory a kernel is allowed.  The helper is
compiled into a small host program whose runtime calls are replaced; nothing is
launched."""
from __future__ import annotations

import subprocess

import pytest

from linear_attention_recurrence_gated_gb300 import build as gbuild

PROGRAM = r"""
#include <cuda_runtime.h>
#include <atomic>
#include <condition_variable>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <thread>

// A kernel with `kStatic` bytes of static shared memory on a GPU that allows 232448 in
// all and 49152 without opting in.
static const int kStatic = 2304, kOptin = 232448;
static std::atomic<int> allowed{49152 - kStatic};   // dynamic bytes a launch may have
static std::atomic<int> pending{0};                 // the runtime's last error
static std::mutex m;
static std::condition_variable cv;
static int hold_first = 0, sets = 0;

template <typename K> cudaError_t fake_set(K, cudaFuncAttribute, int bytes) {
  std::unique_lock<std::mutex> lock(m);
  const int mine = sets++;
  // the first caller is overtaken by the second one, which ends its whole call
  if (hold_first && mine == 0) cv.wait_for(lock, std::chrono::seconds(2), [] { return sets > 100; });
  if (bytes + kStatic > kOptin) { pending = cudaErrorInvalidValue; return cudaErrorInvalidValue; }
  allowed = bytes;
  return cudaSuccess;
}
template <typename K> cudaError_t fake_get(cudaFuncAttributes *a, K) {
  memset(a, 0, sizeof *a);
  a->sharedSizeBytes = kStatic;
  a->maxDynamicSharedSizeBytes = allowed;
  return cudaSuccess;
}
static cudaError_t fake_device(int *d) { *d = 0; return cudaSuccess; }
static cudaError_t fake_attribute(int *v, cudaDeviceAttr, int) { *v = kOptin; return cudaSuccess; }
static cudaError_t fake_last() { return (cudaError_t)pending.exchange(0); }
#define cudaFuncSetAttribute fake_set
#define cudaFuncGetAttributes fake_get
#define cudaGetDevice fake_device
#define cudaDeviceGetAttribute fake_attribute
#define cudaGetLastError fake_last
#include "gdn_launch.cuh"

__global__ void one() {}
__global__ void two() {}
__global__ void three() {}

// a launch with these dynamic bytes
static bool fits(size_t n) { return (int)n <= allowed; }

int main(int, char **argv) {
  if (!strcmp(argv[1], "static")) {
    for (size_t n : {1024u, 46848u, 46849u, 48000u, 49152u, 49153u, 100000u, 230144u})
      if (gdn::allow_smem<one>(n) != cudaSuccess || !fits(n)) {
        printf("%zu bytes do not fit\n", n);
        return 1;
      }
  } else if (!strcmp(argv[1], "error")) {
    if (gdn::allow_smem<two>(kOptin) == cudaSuccess && fits(kOptin)) return 1;
    if (pending) { printf("an error is left behind\n"); return 1; }
  } else {
    hold_first = 1;
    cudaError_t a, b;
    std::thread t([&] { a = gdn::allow_smem<three>(100000); });
    for (;;) {
      std::unique_lock<std::mutex> lock(m);
      if (sets > 0) break;
      lock.unlock();
      std::this_thread::yield();
    }
    b = gdn::allow_smem<three>(200000);
    { std::unique_lock<std::mutex> lock(m); sets = 1000; }
    cv.notify_all();
    t.join();
    if (a != cudaSuccess || b != cudaSuccess) return 1;
    if (gdn::allow_smem<three>(200000) != cudaSuccess || !fits(200000)) {
      printf("200000 bytes were allowed and are not any more\n");
      return 1;
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    where = tmp_path_factory.mktemp("launch")
    (where / "t.cu").write_text(PROGRAM)
    subprocess.run([gbuild.nvcc(), "-std=c++17", *gbuild.ARCH, "-I", gbuild.CSRC, "-o",
                    str(where / "t"), str(where / "t.cu")], check=True, capture_output=True)
    return str(where / "t")


def passes(program, which):
    r = subprocess.run([program, which], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_static_shared_memory_counts(program):
    """48 KB without opting in are the static and the dynamic bytes together."""
    passes(program, "static")


def test_a_refused_size_leaves_no_error_behind(program):
    """The next call's check of its own launch would report it."""
    passes(program, "error")


def test_first_calls_from_two_threads(program):
    """Threads that call one kernel with different sizes for the first time: whoever
    sets the limit last, the larger size stays allowed."""
    passes(program, "threads")
