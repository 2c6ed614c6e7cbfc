"""What the decode behind shared prefixes knows of a sequence without a group, and of a job that is not
there, is zero in every field, not whatever its registers held: the structs cut out of the kernel's
source, compiled for the host and made in memory full of ones."""

import os
import shutil
import subprocess

import pytest

from .test_unit_schedule_host import CSRC, _braced

MAIN = r"""
#include <cstdio>
#include <cstring>
#include <new>
%s
template <typename T>
int set_bytes(const char* name) {
  alignas(T) unsigned char memory[sizeof(T)];
  std::memset(memory, 0xff, sizeof memory);
  T* t = new (memory) T;
  int wild = 0;
  for (std::size_t i = 0; i < sizeof(T) / sizeof(int); ++i) {
    int v;
    std::memcpy(&v, reinterpret_cast<unsigned char*>(t) + i * sizeof(int), sizeof v);
    wild += v == -1;
  }
  if (wild) std::printf("%%s: %%d fields without a value\n", name, wild);
  return wild;
}
int main() { return set_bytes<Group>("Group") + set_bytes<Parts>("Parts"); }
"""


def test_structs_start_with_values(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src = open(os.path.join(CSRC, "decode_prefix.cuh")).read()
    cpp, exe = tmp_path / "structs.cpp", tmp_path / "structs"
    cpp.write_text(MAIN % "\n".join(_braced(src, src.index("struct %s {" % n)) for n in ("Group", "Parts")))
    # (without optimisation, and stores to the memory before an object's life kept)
    subprocess.check_call(["g++", "-O0", "-fno-lifetime-dse", "-std=c++17", "-o", str(exe), str(cpp)])
    subprocess.check_call([str(exe)])
