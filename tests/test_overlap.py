"""CPU test of the check that keeps outputs off the inputs: against sets of
bytes, over random strided matrices in a small range."""
import ctypes
import random
import subprocess

import pytest

from orthonormalized_update_optimizers_b200 import build as B


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    (d / "o.cpp").write_text('''
#include "overlap.h"
extern "C" int o(int64_t p, int64_t r, int64_t w, int64_t l, int64_t q, int64_t s, int64_t x,
                 int64_t m) {
  return ouo::overlap(ouo::Span{(uintptr_t)p, r, w, l}, ouo::Span{(uintptr_t)q, s, x, m});
}
''')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", B.CSRC, "-o", str(d / "o.so"),
                    str(d / "o.cpp")], check=True)
    fn = ctypes.CDLL(str(d / "o.so")).o
    fn.argtypes = [ctypes.c_int64] * 8
    return fn


def _bytes(p, rows, width, pitch):
    return {p + r * pitch + i for r in range(rows) for i in range(width)}


def test_against_sets_of_bytes(overlap):
    rng = random.Random(0)
    seen = [0, 0]
    for _ in range(40000):
        a = (1000 + rng.randrange(60), rng.randrange(5), rng.randrange(9), rng.randrange(1, 14))
        b = (1000 + rng.randrange(60), rng.randrange(5), rng.randrange(9), rng.randrange(1, 14))
        if rng.random() < 0.5:
            b = b[:3] + (a[3],)
        if any(m[1] > 1 and m[3] < m[2] for m in (a, b)):
            continue  # its own rows overlap: refused before
        want = bool(_bytes(*a) & _bytes(*b))
        solid = [m[1] <= 1 or m[3] == m[2] for m in (a, b)]
        if a[3] != b[3] and not any(solid) and a[1] and b[1]:
            assert not overlap(*a, *b) or want
            continue
        assert bool(overlap(*a, *b)) == want, (a, b)
        seen[want] += 1
    assert min(seen) > 3000


def test_columns_of_one_matrix_are_apart(overlap):
    """q, k and v as columns of one buffer, and past 2^31 bytes."""
    pitch, rows = 3 * 8192, 1 << 20
    base = 1 << 40
    for i in range(3):
        for j in range(3):
            got = overlap(base + 8192 * i, rows, 8192, pitch, base + 8192 * j, rows, 8192, pitch)
            assert bool(got) == (i == j)
    assert overlap(base, rows, 8192, pitch, base + (rows - 1) * pitch, 1, 1, 1)
    assert not overlap(base, rows, 8192, pitch, base + (rows - 1) * pitch + 8192, 1, 1, 1)
