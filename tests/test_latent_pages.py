"""What the absorbed kernel does about a block table's entries (csrc/latent_index.h),
compiled for the host: whether a place lies behind a unit's keys goes by the place, and
never by the entry's value."""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_17_gb300", "csrc")

SOURCE = r'''
#include "latent_index.h"
using namespace pkv;
extern "C" int page(int b, int blocks, int entry, int64_t num_blocks) {
  const Page p = page_of(b, blocks, entry, num_blocks);
  return p == Page::kLoad ? 0 : p == Page::kBehind ? 1 : 2;
}
'''
LOAD, BEHIND, BAD = 0, 1, 2


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("latent_pages")
    src, so = str(d / "x.cpp"), str(d / "x.so")
    open(src, "w").write(SOURCE)
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC, src,
                    "-o", so], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("entry", [0, 7, 82, 83, -1, -2, -3, -(1 << 31), (1 << 31) - 1])
def test_entries_of_every_value(lib, entry):
    page = lambda b: lib.page(b, 13, entry, ctypes.c_int64(83))  # noqa: E731
    assert [page(b) for b in (0, 5, 12)] == [LOAD if 0 <= entry < 83 else BAD] * 3
    assert [page(b) for b in (13, 14, 99)] == [BEHIND] * 3
