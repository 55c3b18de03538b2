"""The shared-memory attribute when two host threads set it for one kernel, on the CPU: the
runtime's two calls are replaced by functions of the test, compiled with the library's own
ensure_smem_attr (csrc/smem_attr.cuh)."""
import ctypes
import os
import subprocess

import pytest

from weight_only_int4_w4_b200 import build

HARNESS = r"""
#include "smem_attr.cuh"
#include <chrono>
#include <thread>
static std::atomic<int> limit{0}, inside{0}, calls{0}, fail{0};
extern "C" cudaError_t cudaGetDevice(int *d) { *d = 3; return cudaSuccess; }
// The small size takes its time: as long as the large one is not there, half a second at most.
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int v) {
  ++calls;
  if (fail) return cudaErrorInvalidValue;
  if (v == 100) {
    inside = 1;
    for (int i = 0; i < 500 && limit != 200; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  }
  limit = v;
  return cudaSuccess;
}
// What a kernel of 200 may use when both threads are done, and what a later call finds.
extern "C" int race() {
  static std::atomic<int> set[w4::kAttrDevices];
  std::thread a([] { w4::ensure_smem_attr(nullptr, 100, set); });
  while (!inside) std::this_thread::yield();
  std::thread b([] { w4::ensure_smem_attr(nullptr, 200, set); });
  a.join();
  b.join();
  w4::ensure_smem_attr(nullptr, 200, set);
  return limit;
}
extern "C" int calls_of(int n) {
  static std::atomic<int> set[w4::kAttrDevices];
  limit = 200;
  calls = 0;
  const int sizes[] = {150, 150, 120, 160, 160, 120};
  for (int i = 0; i < n; ++i) w4::ensure_smem_attr(nullptr, sizes[i % 6], set);
  return calls;
}
extern "C" int after_an_error() {
  static std::atomic<int> set[w4::kAttrDevices];
  fail = 1;
  const int first = w4::ensure_smem_attr(nullptr, 300, set);
  fail = 0;
  return first != 0 && w4::ensure_smem_attr(nullptr, 300, set) == 0 && limit == 300;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("attr")
    (d / "h.cpp").write_text(HARNESS)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc_path()))), "include")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-pthread", "-Wl,-Bsymbolic", "-I" + build.SRC_DIR,
                           "-I" + cuda, "-o", str(d / "h.so"), str(d / "h.cpp")])
    return ctypes.CDLL(str(d / "h.so"))


def test_a_smaller_size_does_not_undo_a_larger_one(lib):
    assert lib.race() == 200


def test_one_driver_call_per_larger_size(lib):
    assert lib.calls_of(12) == 2


def test_a_failed_call_is_made_again(lib):
    assert lib.after_an_error() == 1


def test_the_slots_of_two_variants_are_not_mixed_up(tmp_path):
    """A table [devices][variants] passed by a row would let one variant's slot for a device stand
    for another variant's: only an array of one slot per device is taken."""
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc_path()))), "include")

    def compiles(dims, arg):
        (tmp_path / "t.cpp").write_text(f"""#include "smem_attr.cuh"
            static std::atomic<int> set{dims};
            int f(int v) {{ return w4::ensure_smem_attr(nullptr, 1, set{arg}); }}""")
        return subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-I" + build.SRC_DIR, "-I" + cuda, str(tmp_path / "t.cpp")],
                              capture_output=True).returncode == 0

    assert compiles("[w4::kAttrDevices]", "") and compiles("[2][w4::kAttrDevices]", "[v]")
    assert not compiles("[w4::kAttrDevices][2]", "[v]")
