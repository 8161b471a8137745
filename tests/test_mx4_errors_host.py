"""CPU test of who is told of a product's bounded wait that ran out
(zero_mx4_check): every host thread once, whichever asks first."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_optimizer_sm_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include "mx4_errors.hpp"
using zsm::mx_errors_are_news;
#define EXPECT(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  EXPECT(!mx_errors_are_news(0, 0));
  EXPECT(mx_errors_are_news(0, 3));    // three waits ran out
  EXPECT(!mx_errors_are_news(0, 3));   // told once
  EXPECT(!mx_errors_are_news(1, 0));   // of that device only
  bool first = false, again = true, more = false;
  std::thread([&] {                    // another thread is told too, though this one asked before
    first = mx_errors_are_news(0, 3);
    again = mx_errors_are_news(0, 3);
    more = mx_errors_are_news(0, 4);
  }).join();
  EXPECT(first && !again && more);
  EXPECT(mx_errors_are_news(0, 4));    // and so is this one of the fourth, though that one asked before
  EXPECT(!mx_errors_are_news(63, 0) && mx_errors_are_news(63, 1) && !mx_errors_are_news(63, 1));
  EXPECT(!mx_errors_are_news(64, 0) && mx_errors_are_news(64, 1) && mx_errors_are_news(64, 1));
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_thread_is_told(tmp_path):
    src, exe = tmp_path / "told.cpp", str(tmp_path / "told")
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_kernels_only_count_up():
    """The count is added to on the device and never written by the host."""
    with open(os.path.join(CSRC, "mx4_gemm.cu")) as f:
        uses = [line.strip() for line in f if "g_mx_errors" in line]
    assert sum("atomicAdd(&g_mx_errors, 1u)" in u for u in uses) == 2
    assert not any("ToSymbol" in u for u in uses)
