"""Whether two strided tensors share memory (csrc/overlap.h), against the sets of their
bytes, for small tensors of all kinds of strides; and far ones, whose places pass 64 bits."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_graph_recurrent_amd", "csrc")


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("overlap") / "driver")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=undefined", "-I",
                    CSRC, "-o", exe, os.path.join(ROOT, "tests", "overlap_driver.cpp")], check=True)

    def run(pairs):
        text = "".join(" ".join(map(str, a + b)) + "\n" for a, b in pairs)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        assert not out.stderr
        both = [int(ln) for ln in out.stdout.split()]
        assert 3 not in both, "side by side, and over one another"
        return [k & 1 == 1 for k in both], [k & 2 == 2 for k in both]
    return lambda pairs, beside=False: run(pairs)[1 if beside else 0]


def held(p):
    at, n0, s0, n1, s1, size = p
    return {at + i * s0 + j * s1 + k for i in range(n0) for j in range(n1) for k in range(size)}


@pytest.mark.parametrize("like", [False, True])
def test_against_the_bytes_themselves(meet, like):
    """Any strides (rows within one another, over one another, all alike); `like`: slices
    of one tensor, which begin at other places."""
    r = np.random.default_rng(5 + like)
    pairs = []
    for _ in range(6000):
        def one(strides=None):
            s0, s1 = strides or (int(r.integers(0, 40)), int(r.integers(0, 40)))
            return (int(r.integers(1, 120)), int(r.integers(1, 6)), s0, int(r.integers(1, 6)), s1,
                    int(r.integers(1, 9)))
        a = one()
        pairs.append((a, one((a[2], a[4])) if like else one()))
    want = [bool(held(a) & held(b)) for a, b in pairs]
    assert 0.2 < np.mean(want) < 0.98
    assert meet(pairs) == want


def test_slices_of_a_projection(meet):
    """Windows [40, 3, 16] cut from a wide one, and the ways in which they do lie over
    one another."""
    T, B, wide = 40, 3, 64
    cut = lambda c, d=16, t=0, n=T: (4096 + 4 * (t * B * wide + c), n, 4 * B * wide, B, 4 * wide,
                                     4 * d)
    apart = [(cut(0), cut(16)), (cut(16), cut(48)), (cut(0, n=20), cut(0, t=20, n=20)),
             (cut(0), (4096 + 4 * T * B * wide, T, 4 * B * 16, B, 64, 64))]
    over = [(cut(0), cut(15)), (cut(0, 17), cut(16)), (cut(0, n=21), cut(0, t=20, n=20)),
            (cut(0), (4096 + 4 * (T * B * wide - wide + 15), 1, 0, 1, 0, 4)), (cut(0), cut(0))]
    # batch rows outermost
    turn = lambda p: (p[0], p[3], 4 * wide * 1000, p[1], 4 * wide, p[5])
    assert meet(apart + over) == [False] * 4 + [True] * 5
    assert meet([(turn(cut(0)), turn(cut(16))), (turn(cut(0)), turn(cut(15)))]) == [False, True]


def test_side_by_side(meet):
    """Slices of a tensor's rows, of its pieces, and such as wrap around a row's end."""
    a = (4096, 8, 256, 1, 0, 64)
    to = lambda at, size=64, n=8, s=256: (4096 + at, n, s, 1, 0, size)
    pairs = [(a, to(64)), (a, to(192)), (a, to(256 + 64)), (a, to(63)), (a, to(193)),
             (a, to(64, s=128)), (a, to(64, 192)), (a, to(64, 193)), (to(128), a)]
    assert meet(pairs, True) == [True, True, True, False, False, False, True, False, True]
    b = (4096, 3, 1024, 4, 256, 64)
    assert meet([(b, (4096 + 64, 3, 1024, 4, 256, 64)), (b, (4096 + 32, 3, 1024, 4, 256, 64)),
                 ((4096, 3, 1000, 4, 256, 64), (4096 + 64, 3, 1000, 4, 256, 64))], True) == \
        [True, False, False]


def test_nothing_meets_nothing_and_far_strides(meet):
    a, big = (64, 4, 16, 1, 0, 16), 2 ** 62
    assert meet([((0, 4, 16, 1, 0, 16), a), (a, (64, 4, 16, 1, 0, 0)), (a, (64, 0, 16, 1, 0, 16)),
                 ((64, 1000, big, 9, big, 16), (128, 1, 0, 1, 0, 64)),
                 ((64, 1000, big, 9, big, 16), (64 + big, 1, 0, 1, 0, 4))]) == \
        [False, False, False, False, True]
