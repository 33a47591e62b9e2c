"""The absorbed decode's cuts, checked on the host: csrc/kda_mla_split.h compiled here as host code (no GPU) against whole
numbers of any size.  A wrong group would send the join to another CTA's results, or outside the workspace."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_127_b200", "csrc")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SHIM = r"""
#include "kda_mla_split.h"
extern "C" long long scaled(long long x, int a, int b) { return kda::mla::scaled(x, a, b); }
extern "C" int group_of(long long place, int groups, long long total) { return kda::mla::group_of(place, groups, total); }
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    if not os.path.exists(NVCC) and shutil.which("nvcc") is None:
        pytest.skip("needs nvcc")
    d = tmp_path_factory.mktemp("split")
    src, lib = d / "shim.cu", d / "libsplit.so"
    src.write_text(SHIM)
    subprocess.run([NVCC if os.path.exists(NVCC) else "nvcc", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC,
                    "-o", str(lib), str(src)], check=True, capture_output=True)
    s = ctypes.CDLL(str(lib))
    s.scaled.argtypes, s.scaled.restype = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int], ctypes.c_longlong
    s.group_of.argtypes, s.group_of.restype = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong], ctypes.c_int
    return s


# the most places: page tables of 2^37 bytes, pages of 1,024 tokens, tiles of 64
TOTALS = [1, 2, 147, 148, 149, 1000, (1 << 24) - 1, 1 << 24, (1 << 29) + 5, (1 << 32) - 1, 1 << 32, (1 << 32) + 1,
          (1 << 32) + 12345, 1 << 33, (1 << 39) + 7]


@pytest.mark.parametrize("total", TOTALS)
def test_groups_and_ranges_agree(split, total):
    rng = random.Random(total)
    for groups in {1, min(2, total), min(37, total), min(74, total), min(148, total)}:
        starts = [total * g // groups for g in range(groups + 1)]
        for g, start in enumerate(starts):
            assert split.scaled(total, g, groups) == start
        places = {0, total - 1, total // 2} | {rng.randrange(total) for _ in range(200)}
        places |= {p for s in starts for p in (s - 1, s, s + 1) if 0 <= p < total}
        for p in places:
            g = split.group_of(p, groups, total)
            assert 0 <= g < groups and starts[g] <= p < starts[g + 1], (p, groups, total, g)
