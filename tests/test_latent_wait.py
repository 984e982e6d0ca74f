"""How long the absorbed kernel's planning warp waits for a piece (csrc/latent_index.h),
compiled for the host: every wait has a limit, and this one's grows with the piece."""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_17_gb300", "csrc")
SOURCE = r'''
#include "latent_index.h"
extern "C" uint64_t limit(int tiles) { return pkv::piece_limit_ns(tiles); }
'''


def test_the_limit_is_ten_times_what_a_piece_takes(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, so = str(tmp_path / "x.cpp"), str(tmp_path / "x.so")
    open(src, "w").write(SOURCE)
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC, src,
                    "-o", so], check=True)
    limit = ctypes.CDLL(so).limit
    limit.restype = ctypes.c_uint64
    for keys in (0, 1, 64, 100_000, 100_000_000, 1 << 30):
        tiles = -(-keys // 64)
        took = tiles * 2000                                # ns, at 2 us a tile
        assert 10 * took <= limit(tiles) <= 20 * took or tiles == 0
    assert limit(0) == 0
    call = open(os.path.join(CSRC, "latent.cu")).read()
    assert "poll(q_empty, (units - 1) & 1, kWaitLimitNs + piece_limit_ns(tiles))" in call
