"""The index arithmetic that the GPU kernels and the marshalling extension share with the host, compiled with g++ and
checked over every size, also where a wrong index would not change a result."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "swiglu_mlp_amd", "csrc")


def compiled(tmp_path, header, code):
    """A library of `code`, which sees csrc/<header>."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, so = tmp_path / "host.cpp", tmp_path / "host.so"
    src.write_text(f'#include "{header}"\n{code}\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fPIC", "-shared", f"-I{CSRC}",
                    str(src), "-o", str(so)], check=True, capture_output=True, text=True, timeout=120)
    return ctypes.CDLL(str(so))


class Lane(ctypes.Structure):
    _fields_ = [("live", ctypes.c_bool), ("turns", ctypes.c_bool), ("upper", ctypes.c_bool), ("c", ctypes.c_uint32),
                ("other", ctypes.c_uint32), ("other_c", ctypes.c_uint32), ("table", ctypes.c_uint32)]


def test_norm_lanes_stay_inside_weights_and_tables(tmp_path):
    # every lane reads its own and its partner's 8 weights, and a lane that turns reads its table entries, whether or
    # not the lane has channels of the head: none may be past the d weights or the rot / 2 entries of a row
    L = compiled(tmp_path, "qk_lanes.hpp", 'extern "C" ck::qkn::Lane lane(uint32_t l, uint32_t d, uint32_t rot, bool half)'
                                           " { return ck::qkn::lane_of(l, d, rot, half); }")
    L.lane.restype = Lane
    L.lane.argtypes = [ctypes.c_uint32] * 3 + [ctypes.c_bool]
    for d in range(8, 257, 8):
        team = 8 if d <= 64 else 16 if d <= 128 else 32
        for half in (True, False):
            for rot in range(0, d + 1, 16 if half else 8):
                lanes = [L.lane(i, d, rot, half) for i in range(team)]
                for i, x in enumerate(lanes):
                    case = (d, rot, half, i)
                    assert x.c + 8 <= d and x.other_c + 8 <= d and x.other < team, case
                    assert x.live == (8 * i < d) and x.c == (8 * i if x.live else 0), case
                    assert x.turns == (x.live and 8 * i < rot), case
                    if not x.turns:
                        assert x.other == i and x.other_c == x.c, case
                        continue
                    assert x.table + (8 if half else 4) <= rot // 2, case
                    if half:
                        assert x.other_c == (x.c - rot // 2 if x.upper else x.c + rot // 2), case
                        assert x.upper == (x.c >= rot // 2) and x.table == min(x.c, x.other_c), case
                        assert x.other_c == 8 * x.other and lanes[x.other].other == i, case
                    else:
                        assert x.other == i and x.table == x.c // 2, case
