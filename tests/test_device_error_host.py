"""skv_device_error with a fake of the two device words (host only): the library's
argument layer linked with a program in their place."""
import os
import shutil
import subprocess

import pytest

from split_kv_merge_attn_b200 import _build

FAKE = r"""
#include <cstdio>
#include "skv_internal.h"

namespace {
int words[2], fail_read = -1, fail_clear = -1;
int read(int w, int* code) {
  if (fail_read == w) return 2;
  *code = words[w];
  return 0;
}
int clear(int w) {
  if (fail_clear == w) return 2;
  words[w] = 0;
  return 0;
}
}  // namespace
namespace skv {
int read_device_error(int* code) { return read(0, code); }
int clear_device_error() { return clear(0); }
int read_cache_error(int* code) { return read(1, code); }
int clear_cache_error() { return clear(1); }
}  // namespace skv

int main(int, char** argv) {
  std::sscanf(argv[1], "%d,%d,%d,%d", &words[0], &words[1], &fail_read, &fail_clear);
  int code = -1;
  const int status = skv_device_error(&code);
  std::printf("%d %d %d %d", status, code, words[0], words[1]);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("device_error")
    (d / "fake.cpp").write_text(FAKE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-I", _build.INCLUDE, "-I", _build.CSRC, "-isystem", cuda,
                    os.path.join(_build.CSRC, "skv_abi.cpp"), str(d / "fake.cpp"), "-o", str(d / "run"),
                    "-Wl,--unresolved-symbols=ignore-all"], check=True)  # the launchers are not reached
    return str(d / "run")


@pytest.mark.parametrize("first,second,fail_read,fail_clear,status,code,left", [
    (0, 0, -1, -1, 0, 0, (0, 0)), (0x102, 0, -1, -1, 0, 0x102, (0, 0)), (0, 0x301, -1, -1, 0, 0x301, (0, 0)),
    (0x102, 0x301, -1, -1, 0, 0x102, (0, 0)),
    (0x102, 0x301, 0, -1, 4, -1, (0x102, 0x301)),
    (0x102, 0x301, 1, -1, 4, -1, (0x102, 0x301)),  # the second read fails: the first word is still there
    (0, 0x301, -1, 1, 4, -1, (0, 0x301)),
])
def test_nothing_is_lost(program, first, second, fail_read, fail_clear, status, code, left):
    out = subprocess.run([program, f"{first},{second},{fail_read},{fail_clear}"], check=True, capture_output=True, text=True)
    assert [int(x) for x in out.stdout.split()] == [status, code, *left]
