"""The index arithmetic that the GPU kernels and the marshalling extension share with the host, compiled with g++ and
checked over every size, also where a wrong index would not change a result."""
import ctypes
import os
import random
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
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fPIC", "-shared", f"-I{CSRC}",
                        str(src), "-o", str(so)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
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


DISJOINT = """
extern "C" bool apart(const int64_t *a, const int64_t *b, int64_t a0, int64_t b0, int64_t bytes_a, int64_t bytes_b)
{
    return ck::disjoint(ck::View::of((const void *)a0, bytes_a, a, a + 4, 4), ck::View::of((const void *)b0, bytes_b, b, b + 4, 4));
}
extern "C" bool distinct(const int64_t *a, int64_t bytes) { return ck::View::of(nullptr, bytes, a, a + 4, 4).distinct(); }
"""


@pytest.fixture(scope="module")
def apart(tmp_path_factory):
    """apart(a, b) of (first byte, element size, sizes, strides), up to four dimensions each."""
    L = compiled(tmp_path_factory.mktemp("views"), "views.hpp", DISJOINT)
    L.apart.restype = ctypes.c_bool
    L.apart.argtypes = [ctypes.c_void_p, ctypes.c_void_p] + [ctypes.c_int64] * 4

    def call(a, b):
        def flat(v):
            pad = 4 - len(v[2])
            return (ctypes.c_int64 * 8)(*([1] * pad + list(v[2]) + [0] * pad + list(v[3])))
        return L.apart(flat(a), flat(b), a[0], b[0], a[1], b[1])
    return call


def elements(v):
    at = {v[0]}
    for n, s in zip(v[2], v[3]):
        at = {x + i * s * v[1] for x in at for i in range(n)}
    return {x + i for x in at for i in range(v[1])}


def test_views_apart(apart):
    row = 48 * 128
    q = (0, 2, (16, 1, 32, 128), (row, row, 128, 1))
    k = (32 * 128 * 2, 2, (16, 1, 8, 128), (row, row, 128, 1))
    assert apart(q, k) and apart(k, q) and not apart(q, q)
    # the stride of a dimension of one element says nothing
    assert apart((0, 2, (16, 1, 32, 128), (row, 7, 128, 1)), k)
    # one token of each sequence beside packed rows of nine; heads before tokens; a key head's own group
    assert apart((0, 2, (3, 1, 32, 128), (9 * row, row, 128, 1)), (8192, 2, (3, 9, 8, 128), (9 * row, row, 128, 1)))
    assert apart((0, 2, (3, 7, 6, 64), (10 * 7 * 64, 64, 7 * 64, 1)), (6 * 7 * 128, 2, (3, 7, 2, 64), (10 * 7 * 64, 64, 7 * 64, 1)))
    assert apart((0, 2, (2, 5, 3, 64), (50 * 64, 10 * 64, 64, 1)), (3 * 128, 2, (2, 5, 2, 64), (50 * 64, 10 * 64, 5 * 64, 1)))
    # one more head of q would be k's first
    assert not apart((0, 2, (16, 1, 33, 128), (row, row, 128, 1)), k)
    assert not apart(k, (0, 2, (16, 1, 33, 128), (row, row, 128, 1)))
    # an empty view; a line of bytes between two sequences, and one into the second
    assert apart(q, (0, 1, (0,), (1,))) and apart((0, 2, (0, 4), (4, 1)), (0, 2, (9, 4), (4, 1)))
    assert apart((0, 2, (2, 100), (1000, 1)), (200, 1, (1800,), (1,)))
    assert not apart((0, 2, (2, 100), (1000, 1)), (200, 1, (1801,), (1,)))


def test_views_called_apart_share_no_byte(apart):
    rng = random.Random(1)

    def view():
        n = rng.randint(0, 4)
        return (rng.randint(0, 60), rng.choice([1, 2]), tuple(rng.choice([0, 1, 1, 2, 2, 3]) for _ in range(n)),
                tuple(rng.choice([0, 1, 1, 2, 3, 4, 6, 8, 12, 24, 36]) for _ in range(n)))

    said = 0
    for _ in range(30000):
        a, b = view(), view()
        if apart(a, b):
            said += 1
            assert not elements(a) & elements(b), (a, b)
        else:
            assert a != b or elements(a), (a, b)
    assert said > 5000


def test_views_without_an_element_twice(tmp_path):
    L = compiled(tmp_path, "views.hpp", DISJOINT)
    L.distinct.restype = ctypes.c_bool
    L.distinct.argtypes = [ctypes.c_void_p, ctypes.c_int64]

    def distinct(sizes, strides, size=2):
        return L.distinct((ctypes.c_int64 * 8)(*sizes, *strides), size)

    # contiguous, columns of packed rows, heads before tokens, tokens before sequences
    for strides in ((600, 120, 24, 1), (4000, 800, 40, 1), (200, 8, 40, 1), (120, 360, 24, 1)):
        assert len(elements((0, 2, (3, 5, 5, 8), strides))) == 1200
        assert distinct((3, 5, 5, 8), strides), strides
    # windows of rows, heads, sequences; two dimensions of one stride
    for strides in ((600, 16, 24, 1), (600, 120, 4, 1), (4, 120, 24, 1), (120, 120, 24, 1)):
        assert len(elements((0, 2, (3, 5, 5, 8), strides))) < 1200
        assert not distinct((3, 5, 5, 8), strides), strides
    rng = random.Random(2)
    for _ in range(10000):
        # dimensions nested in any order, with room between: what a tensor's own layout and its columns are
        size, n, order, st = rng.choice([1, 2]), [rng.randint(1, 3) for _ in range(4)], [0, 1, 2, 3], [0] * 4
        rng.shuffle(order)
        extent = 1
        for i in order:
            st[i] = extent + rng.choice([0, 0, 1, 5])
            extent += (n[i] - 1) * st[i]
        assert distinct(n, st, size), (n, st, size)
        # and any strides at all: never an element twice in what is accepted
        st = [rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24]) for _ in range(4)]
        if distinct(n, st, size):
            assert len(elements((0, size, n, st))) == size * n[0] * n[1] * n[2] * n[3], (n, st, size)
