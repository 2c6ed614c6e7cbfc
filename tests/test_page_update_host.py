"""The page bookkeeping's walk over a step's tokens, cut out of the kernel's source and compiled for the
host: every token is visited once, by one thread, and nothing outside the token array, up to the largest
token count that the call takes."""

import os
import shutil
import subprocess

import pytest

from .test_unit_schedule_host import CSRC, _braced

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#define __device__
#define __forceinline__ inline
%s
int main() {
  const int largest = 2147483647;
  for (int threads : {512, 512 * 147, 512 * 148})
    for (int n : {0, 1, 511, 512, 513, 512 * 148, 512 * 148 + 1, 1 << 30, largest - threads, largest - threads + 1, largest})
      for (int first : {0, 1, 511, threads / 2, threads - 1}) {
        long long want = first, count = 0;
        every(first, threads, n, [&](int t) {
          if (t != want || t < 0 || t >= n) {
            std::printf("%%d threads, %%d tokens: thread %%d visits %%d, not %%lld\n", threads, n, first, t, want);
            std::exit(1);
          }
          want += threads, ++count;
        });
        if (count != (n > first ? (n - 1LL - first) / threads + 1 : 0)) return 2;
      }
  return 0;
}
"""


def test_tokens_are_visited_once_and_in_bounds(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src = open(os.path.join(CSRC, "pages.cuh")).read()
    at = src.index("template <typename F>\n__device__ __forceinline__ void every(")
    cpp, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    cpp.write_text(MAIN % _braced(src, at))
    subprocess.check_call(["g++", "-O1", "-fwrapv", "-std=c++17", "-o", str(exe), str(cpp)])
    subprocess.check_call([str(exe)], timeout=120)
    # the tokens are walked in no other way
    assert src.count("p.max_tokens, [&](int t)") == 2 and "t += threads" not in src
