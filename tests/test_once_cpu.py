"""What a process does once (a kernel's limit of shared memory): a failure is not kept."""
import os
import re
import shutil
import subprocess

import pytest

import token_routing_expert_router_gb300._build as build

PROGRAM = r"""
#include <cstdio>
#include "once.h"
enum Error { kSuccess = 0, kMemory = 2 };
int main() {
  static moe::Once once, other;
  int calls = 0;
  auto set = [&] { return ++calls < 3 ? kMemory : kSuccess; };
  const Error a = once(set), b = once(set), c = once(set), d = once(set);
  const bool kept = a == kMemory && b == kMemory && c == kSuccess && d == kSuccess && calls == 3;
  const Error e = other([&] { ++calls; return kSuccess; });
  return kept && e == kSuccess && calls == 4 ? 0 : 1;
}
"""


def test_a_failure_is_tried_again(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", f"-I{build.CSRC}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_no_launcher_keeps_an_error():
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            assert not re.search(r"static\s+(const\s+)?(cudaError_t|auto)\s+\w+\s*=", f.read()), name
