"""The host's check for overlapping tensors, compiled as it stands and run on addresses alone: runs of
elements in rows of one stride overlap exactly where they share an element, and runs that do share one
are found whatever their strides."""
import ctypes
import os
import random
import subprocess

import pytest

from mamba_chunked_ssd_gb300 import build_lib

SOURCE = """
#include "abi_checks.cuh"
extern "C" int overlaps(long p, long rows, long width, long stride, long q, long rows2, long width2, long stride2) {
    const m2::Tensor a = {(const void*)p, rows, width, stride, false, 1}, b = {(const void*)q, rows2, width2, stride2, false, 1};
    return m2::overlap(a, b);
}
"""


@pytest.fixture(scope="module")
def overlaps(tmp_path_factory):
    at = tmp_path_factory.mktemp("overlap")
    (at / "o.cpp").write_text(SOURCE)
    lib = os.path.join(at, "o.so")
    subprocess.run([build_lib._nvcc(), "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", build_lib.INCLUDE, "-I",
                    build_lib.CSRC, str(at / "o.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).overlaps
    f.argtypes = [ctypes.c_long] * 8
    return lambda a, b: bool(f(*a, *b))


def share(a, b):
    """Whether two tensors (start, rows, bytes of a run, bytes from run to run) have a byte in common."""
    of = lambda p, rows, width, stride: {p + k * stride + i for k in range(rows) for i in range(width)}  # noqa: E731
    return not of(*a).isdisjoint(of(*b))


def test_slices_side_by_side_do_not_overlap(overlaps):
    """dx, dr, di of 64 bf16 channels in one tensor of rows of 192, from any of them to any other."""
    at = 1 << 20
    side = [(at + 128 * k, 200, 128, 384) for k in range(3)]
    for k in range(3):
        for j in range(3):
            assert overlaps(side[k], side[j]) == (k == j)
    dx, dr, di = side
    assert overlaps(dx, (dr[0] - 2, *dr[1:])) and overlaps((di[0] + 2, *di[1:]), dx)  # an element over the next one
    assert not overlaps((di[0] + 2, 1, 128, 384), (dr[0], 1, 128, 384))
    assert not overlaps(dx, (at + 200 * 384, 200, 128, 384))                          # behind the last row
    assert overlaps(dx, (at + 199 * 384, 200, 128, 384))                              # its last row is the other's first


def test_runs_of_one_stride_overlap_exactly_where_they_share_an_element(overlaps):
    r = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(20000):
        stride = r.randint(1, 12)
        a, b = ((1000 + r.randint(0, 40), r.randint(2, 5), r.randint(1, stride), stride) for _ in range(2))
        want = share(a, b)
        assert overlaps(a, b) == want, (a, b)
        seen[want] += 1
    assert min(seen.values()) > 2000


def test_shared_elements_are_found_for_all_strides(overlaps):
    r = random.Random(2)
    seen = 0
    for _ in range(20000):
        s, t = r.randint(1, 12), r.randint(1, 12)
        a = (1000 + r.randint(0, 40), r.randint(0, 5), r.randint(1, s), s)
        b = (1000 + r.randint(0, 40), r.randint(0, 5), r.randint(1, t), t)
        if share(a, b):
            seen += 1
            assert overlaps(a, b), (a, b)
    assert seen > 2000
