"""What host threads that launch at once share: a note of the prepared devices
(csrc/device_set.h) under the thread sanitizer, and no shared state without one."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_17_gb300", "csrc")

SOURCE = r'''
#include "device_set.h"
#include <cstdio>
#include <thread>
#include <vector>
static pkv::DeviceSet set;
int main() {
  if (set.has(0) || set.has(-1) || set.has(32) || set.has(1 << 30)) return 1;
  std::vector<std::thread> threads;
  for (int t = 0; t < 16; ++t)
    threads.emplace_back([t] {
      for (int i = 0; i < 200; ++i) {
        const int device = (t + i) % 34 - 1;               // -1 .. 32
        if (!set.has(device)) set.add(device);
      }
    });
  for (auto& t : threads) t.join();
  for (int device = 0; device < 32; ++device)
    if (!set.has(device)) return 2;
  // (out of its range: never noted)
  return set.has(-1) || set.has(32) ? 3 : 0;
}
'''


def test_notes_of_threads_do_not_race(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = str(tmp_path / "x.cpp"), str(tmp_path / "x")
    open(src, "w").write(SOURCE)
    flags = ["-std=c++17", "-Wall", "-Werror", "-O1", "-g", "-pthread", "-I", CSRC, src, "-o", exe]
    checked = subprocess.run([cxx, "-fsanitize=thread", *flags], capture_output=True)
    if checked.returncode != 0:                            # (a compiler without the sanitizer)
        subprocess.run([cxx, *flags], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    if "unexpected memory mapping" in got.stderr:
        pytest.skip("the sanitizer does not run on this system")
    assert got.returncode == 0, (got.returncode, got.stderr[-2000:])


def test_no_launcher_keeps_plain_shared_state():
    """Variables that outlive a host function are constant, atomic or a DeviceSet."""
    found = []
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh", ".cpp", ".h")):
            continue
        for i, line in enumerate(open(os.path.join(CSRC, name)), 1):
            m = re.match(r"\s+static\s+(?!const|inline|__device__|__host__)([\w:<>]+)\s+\w+\s*(\[\w+\])?\s*(=|;|\{)", line)
            if m and not m.group(1).startswith("std::atomic<") and m.group(1) != "DeviceSet":
                found.append((name, i, line.strip()))
    assert not found, found
