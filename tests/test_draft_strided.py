"""The checks for rows at strides that lie over each other, against all pairs of rows
(CPU only; the header is host C++)."""

import ctypes
import os
import random
import subprocess
import time

import pytest

from tests.test_draft_abi import call_filter, lib  # noqa: F401
from tests.test_ops_abi import EINVAL, EWORKSPACE, FAR, ROOT

SRC = """
#include "strided.h"
using namespace specv;
extern "C" int overlap_of(const long long* a, const long long* b) {
  auto rows = [](const long long* r) {
    return Rows{reinterpret_cast<const void*>(r[0]), (size_t)r[1], (size_t)r[2], (int)r[3], (int)r[4],
                (size_t)r[5]};
  };
  return rows_overlap(rows(a), rows(b));
}
extern "C" int overlaps_itself(const long long* a) {
  return self_overlap(Rows{reinterpret_cast<const void*>(a[0]), (size_t)a[1], (size_t)a[2], (int)a[3],
                           (int)a[4], (size_t)a[5]});
}
"""


@pytest.fixture(scope="module")
def checks(tmp_path_factory):
    at = tmp_path_factory.mktemp("strided")
    (at / "t.cpp").write_text(SRC)
    so = str(at / "t.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(ROOT, "include"), "-isystem", "/opt/rocm/include", "-I",
                    os.path.join(ROOT, "speculative_decoding_sampling_amd", "csrc"), str(at / "t.cpp"),
                    "-o", so], check=True)
    return ctypes.CDLL(so)


def rows(r):
    p, sb, sk, B, n, size = r
    return [(p + b * sb + k * sk, p + b * sb + k * sk + size) for b in range(B) for k in range(n)]


def meet(a, b):
    return any(x < v and u < y for x, y in rows(a) for u, v in rows(b))


def packed(r):
    return (ctypes.c_longlong * 6)(*r)


def some(rng, most):
    """(start, strides, counts, bytes) of rows, often close to each other."""
    B, n, size = rng.randint(1, 7), rng.randint(1, 7), rng.choice([1, 2, 3, 4, 8, 30])
    kind = rng.random()
    if kind < 0.4:                                      # nested, either way round, with room
        inner = size + rng.randint(0, most)
        outer = inner * (n if rng.random() < 0.5 else 1) + rng.randint(0, most)
        sb, sk = (outer, inner) if rng.random() < 0.5 else (inner, outer)
    else:
        sb, sk = rng.randint(0, most), rng.randint(0, most)
    return (1 << 20) + rng.randint(0, 200), sb, sk, B, n, size


def test_rows_of_two_arrays_against_every_pair(checks):
    rng = random.Random(1)
    seen = [0, 0]
    for i in range(60000):
        a = some(rng, rng.choice([5, 60, 400]))
        b = some(rng, rng.choice([5, 60, 400]))
        if rng.random() < 0.4:                          # equal strides, as of one buffer
            b = b[:1] + a[1:5] + b[5:]
        elif rng.random() < 0.3:
            b = b[:1] + a[1:2] + b[2:]
        want = meet(a, b)
        assert bool(checks.overlap_of(packed(a), packed(b))) == want, (a, b)
        assert bool(checks.overlap_of(packed(b), packed(a))) == want, (a, b)
        seen[want] += 1
    assert min(seen) > 10000


def test_long_axes_against_every_pair(checks):
    # one axis of up to 300 rows: the remainders go through several steps
    rng = random.Random(2)
    seen = [0, 0]
    for i in range(400):
        a = (1 << 20, rng.randint(1, 5000), 0, rng.randint(1, 300), 1, rng.randint(1, 4))
        b = ((1 << 20) + rng.randint(0, 20000), rng.randint(1, 5000), 0, rng.randint(1, 300), 1, rng.randint(1, 4))
        want = meet(a, b)
        assert bool(checks.overlap_of(packed(a), packed(b))) == want, (a, b)
        seen[want] += 1
    assert min(seen) > 30


def test_far_strides_do_not_overflow(checks):
    # 2^60 bytes between the first and the last row
    big = (1 << 60) // 3
    for shift, want in ((0, True), (8, False), (big, True), (2 * big, True), (2 * big + 8, False)):
        for B, n in ((3, 2), (2, 3)):
            a = (1 << 40, big, 0, 3, 1, 8)
            b = ((1 << 40) + shift, big if B == 3 else 1 << 20, 1 << 20 if B == 3 else big, B, n, 8)
            got = bool(checks.overlap_of(packed(a), packed(b)))
            assert got == want == meet(a, b), (shift, B, n)


@pytest.mark.parametrize("B,L", [(64, 5), (256, 5), (1024, 5), (4096, 1), (5, 1024)])
def test_interleaved_calls_are_checked_in_time(lib, B, L):  # noqa: F811
    # probabilities in the gaps of the logits' rows: legal, so the missing workspace
    # is what is refused; every pair of rows would take 1 to 50 ms at 256 rows or more
    V = 40000
    kw = dict(B=B, L=L, zsb=2 * L * V, zsl=2 * V, p=FAR[0] + 4 * V, psb=2 * L * V, psl=2 * V, tsb=L, usb=L, ws=None)
    best = 1.0
    for _ in range(20):
        t = time.perf_counter()
        st = call_filter(lib, **kw)
        best = min(best, time.perf_counter() - t)
        assert st == EWORKSPACE
    assert best < 0.3e-3, best
    # one element into the next rows, or the ones before
    assert call_filter(lib, **dict(kw, p=kw["p"] + 4)) == EINVAL
    assert call_filter(lib, **dict(kw, p=kw["p"] - 4)) == EINVAL


def test_overlaps_come_before_a_missing_workspace(lib):  # noqa: F811
    assert call_filter(lib, p=FAR[0], ws=None) == EINVAL
    assert call_filter(lib, tsb=1, tsl=4, psb=40000, psl=160000, ws=None) == EWORKSPACE
    assert call_filter(lib, zsb=240000, zsl=80000, p=FAR[0] + 160000, psb=240000, psl=80000, ws=None) == EWORKSPACE
    # a stride that no row takes does not matter
    assert call_filter(lib, B=1, psb=1 << 62, zsb=1 << 62, ws=None) == EWORKSPACE
    assert call_filter(lib, psb=1 << 58, ws=None) == EINVAL


def meets_itself(a):
    r = sorted(rows(a))
    return any(x[1] > y[0] for x, y in zip(r, r[1:]))


def test_rows_of_one_array_against_every_pair(checks):
    rng = random.Random(3)
    seen = [0, 0]
    for i in range(60000):
        a = some(rng, rng.choice([5, 60, 400]))
        want = meets_itself(a)
        assert bool(checks.overlaps_itself(packed(a))) == want, a
        seen[want] += 1
    assert min(seen) > 10000


def test_strides_that_are_not_nested_are_accepted(lib):  # noqa: F811
    # rows at 0, 2, 4 and 3, 5, 7 times their length
    V = 40000
    kw = dict(B=3, L=2, V=V, zsb=2 * V, zsl=V, ws=None)
    assert call_filter(lib, **kw, psb=2 * V, psl=3 * V, tsb=2, tsl=3) == EWORKSPACE
    assert call_filter(lib, **kw, psb=3 * V, psl=2 * V, tsb=3, tsl=4) == EWORKSPACE
    # at 0, 2, 4 and 4, 6, 8; one element short
    assert call_filter(lib, **kw, psb=2 * V, psl=4 * V) == EINVAL
    assert call_filter(lib, **kw, tsb=2, tsl=4) == EINVAL
    assert call_filter(lib, **kw, psb=2 * V, psl=3 * V - 1) == EINVAL
