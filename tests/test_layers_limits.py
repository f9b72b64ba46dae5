"""What the host keeps about kernels between calls (csrc/layer_limits.h, compiled
here): the record of what CUDA was told they may use, with two host threads in it
at once and a fake for CUDA's call, the limits of their waits, and which waits given
up have been reported."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_communication_sharded_gb300", "csrc")

PROGRAM = r"""
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <thread>
#include "layer_limits.h"

using namespace std::chrono_literals;
static std::mutex m;
static std::condition_variable cv;
static bool inside = false, second_done = false;
static int attribute = 0, calls = 0;  // what "CUDA" holds

static int set(int bytes, bool first, bool holds_after) {
  std::unique_lock<std::mutex> l(m);
  ++calls;
  if (holds_after) attribute = bytes;
  if (first) {
    // lets the other thread do what it can, whole or not at all
    inside = true;
    cv.notify_all();
    cv.wait_for(l, 500ms, [] { return second_done; });
  }
  if (!holds_after) attribute = bytes;
  return 0;
}

using scapek::layer::kWaitLimitNs;
using scapek::layer::product_wait_ns;
static_assert(product_wait_ns(1) < 2 * kWaitLimitNs, "a short contraction fails as soon as any wait");
// the longest contraction a block can have, 2^31 rows of 64 a stage, at 1 us a stage
static_assert(product_wait_ns((int64_t{1} << 31) / 64) > ((uint64_t{1} << 31) / 64) * 1000, "and a long one lasts");

int main(int argc, char** argv) {
  const int first = atoi(argv[1]), second = atoi(argv[2]);
  const bool holds_after = atoi(argv[3]);  // the first call takes effect before or after the second's
  static scapek::layer::RaisedLimits limits;
  const int kernel = 0;
  std::thread a([&] { limits.raise(0, &kernel, first, -1, [&](int b) { return set(b, true, holds_after); }); });
  std::thread b([&] {
    {
      std::unique_lock<std::mutex> l(m);
      cv.wait(l, [] { return inside; });
    }
    limits.raise(0, &kernel, second, -1, [&](int x) { return set(x, false, true); });
    std::unique_lock<std::mutex> l(m);
    second_done = true;
    cv.notify_all();
  });
  a.join();
  b.join();
  // every size that was asked for must launch now, from the record or by another call
  for (int bytes : {first, second}) {
    const int r = limits.raise(0, &kernel, bytes, -1, [&](int x) { return set(x, false, true); });
    if (r != 0 || attribute < bytes) {
      printf("%d bytes allowed, the attribute is %d\n", bytes, attribute);
      return 1;
    }
  }
  // errors are passed on and not recorded; another kernel and device are their own
  const int other = 0;
  if (limits.raise(0, &other, 64, -1, [](int) { return 7; }) != 7) return 2;
  int told = 0;
  if (limits.raise(0, &other, 64, -1, [&](int) { return ++told, 0; }) != 0 || told != 1) return 3;
  if (limits.raise(1, &other, 64, -1, [&](int) { return ++told, 0; }) != 0 || told != 2) return 4;
  if (limits.raise(1, &other, 32, -1, [&](int) { return ++told, 0; }) != 0 || told != 2) return 5;
  // no place left: the call says so
  static int many[80];
  int full = 0;
  for (int& k : many) full += limits.raise(2, &k, 1, -1, [](int) { return 0; }) == -1;
  if (full != 80 - scapek::layer::RaisedLimits::kKernels) return 6;

  // Waits given up: each is told once, whatever is added while it is asked for.
  scapek::layer::LastSeen seen;
  if (seen.news(0) != 0 || seen.news(2) != 2 || seen.news(2) != 0) return 7;
  // two readers, of whom the one with the older value comes last
  if (seen.news(5) != 3 || seen.news(4) != 0 || seen.news(5) != 0) return 8;
  // the count passes 32 bits
  scapek::layer::LastSeen far;
  if (far.news(0x7FFFFFFFu) <= 0 || far.news(0xFFFFFFFEu) <= 0 || far.news(3) != 5) return 9;
  std::atomic<unsigned> count{0};
  std::atomic<bool> stop{false};
  std::atomic<long> told_of{0};
  scapek::layer::LastSeen both;
  std::thread readers[2];
  for (std::thread& r : readers)
    r = std::thread([&] {
      while (!stop) told_of += both.news(count.load());
    });
  for (int i = 0; i < 200000; ++i) ++count;
  stop = true;
  for (std::thread& r : readers) r.join();
  told_of += both.news(count.load());
  return told_of == 200000 ? 0 : 10;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("limits")
    src, exe = d / "limits.cpp", d / "limits"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    return str(exe)


@pytest.mark.parametrize("first,second", [(65536, 36864), (36864, 65536), (65536, 65536)])
@pytest.mark.parametrize("early", [0, 1])
def test_two_threads_raise_one_kernel(program, first, second, early):
    r = subprocess.run([program, str(first), str(second), str(early)], capture_output=True, text=True, timeout=30)
    assert r.returncode == 0, r.stdout


def test_probe_refusals():
    from sparse_communication_sharded_gb300 import _scape as C
    from sparse_communication_sharded_gb300 import build as B
    B.build()
    lib = C.load()
    for ns in (0, -5, 2 * 10 ** 9 + 1):
        assert lib.scape_layer_probe_wait(ns, None) == C.SCAPE_EINVAL
        assert "limit_ns" in lib.scape_layer_last_error().decode()


def test_plan_refusals():
    import ctypes

    from sparse_communication_sharded_gb300 import _scape as C
    from sparse_communication_sharded_gb300 import build as B
    B.build()
    lib = C.load()
    a, b, c = (ctypes.byref(ctypes.c_int()) for _ in range(3))
    assert lib.scape_layer_linear_plan(3, 8, 8, 8, 0, a, b, c) == C.SCAPE_EINVAL
    assert lib.scape_layer_linear_plan(0, 8, 0, 8, 0, a, b, c) == C.SCAPE_EINVAL
    assert lib.scape_layer_linear_plan(0, 8, 8, 8, 0, None, b, c) == C.SCAPE_EINVAL
    assert lib.scape_layer_linear_plan(0, 4, 8, 8, 0, a, b, c) == C.SCAPE_OK  # no tiles
