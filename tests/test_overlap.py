"""Whether strided tensors share memory (csrc/overlap.cuh), against sets of bytes."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def unit():
    out = os.path.join(HERE, "_build", "liboverlapunit.so")
    os.makedirs(os.path.dirname(out), exist_ok=True)
    tmp = f"{out}.tmp{os.getpid()}"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", tmp, os.path.join(HERE, "csrc", "overlap_unit.cc")], check=True)
    os.replace(tmp, out)
    return ctypes.CDLL(out)


def args(at, length, *axes):
    flat = [at, length, *itertools.chain(*axes), *[1, 0] * (3 - len(axes))]
    return (ctypes.c_int64 * 8)(*flat)


def starts(at, axes):
    return [at + sum(i * s for i, (_, s) in zip(index, axes)) for index in itertools.product(*(range(n) for n, _ in axes))]


def cells(at, length, axes):
    return [b for s in starts(at, axes) for b in range(s, s + length)]


def test_random_tensors(unit):
    r = random.Random(1)
    seen = [0, 0, 0, 0]
    for _ in range(20000):
        tensors = []
        common = r.choice([None, r.randint(0, 40)])
        for _ in range(2):
            length = r.randint(1, 5)
            axes = [(r.randint(1, 5), r.choice([0, length, r.randint(0, 30), 2 * length * r.randint(1, 4)])) for _ in range(r.randint(1, 3))]
            if common is not None:  # tokens of one projection
                axes[0] = (axes[0][0], common)
            tensors.append((1000 + r.randint(0, 120), length, axes))
        (a, la, xa), (b, lb, xb) = tensors
        ca, cb = cells(a, la, xa), cells(b, lb, xb)
        want, itself = not set(ca).isdisjoint(cb), len(set(ca)) < len(ca)
        assert bool(unit.overlap_unit(args(a, la, *xa), args(b, lb, *xb))) == want, tensors
        assert bool(unit.overlap_unit(args(b, lb, *xb), args(a, la, *xa))) == want, tensors
        assert bool(unit.overlaps_itself_unit(args(a, la, *xa))) == itself, tensors
        seen[want] += 1
        seen[2 + itself] += 1
    assert min(seen) > 1000


def test_large_tensors(unit):
    # slices of one projection of 2^31 tokens, and head-major storage of as many, past 32 bits
    n, d = 2 ** 31 - 1, 256
    row = 48 * d
    q, k = args(4096, d, (n, row), (32, d)), args(4096 + 32 * d, d, (n, row), (8, d))
    assert not unit.overlap_unit(q, k) and unit.overlap_unit(q, q) and not unit.overlaps_itself_unit(q)
    assert unit.overlap_unit(args(4096 + row * (n - 1) + 16, d, (1, 0)), q)
    assert not unit.overlap_unit(args(4096 + row * (n - 1) + 32 * d, d, (1, 0)), q)
    major, other = args(4096, d, (n, 2 * d), (4, n * 2 * d)), args(4096 + d, d, (n, 2 * d), (4, n * 2 * d))
    assert not unit.overlap_unit(major, other) and not unit.overlaps_itself_unit(major)
    assert unit.overlap_unit(major, args(4096 + d - 16, d, (n, 2 * d), (4, n * 2 * d)))
    assert unit.overlaps_itself_unit(args(4096, d, (n, d - 16), (4, n * d))) and unit.overlaps_itself_unit(args(4096, d, (n, row), (49, d)))


@pytest.mark.parametrize("empty", [0, 1, 2])
def test_tensors_without_elements(unit, empty):
    axes = [(3, 64), (4, 16), (2, 8)]
    axes[empty] = (0, axes[empty][1])
    assert not unit.overlap_unit(args(64, 8, *axes), args(64, 8, (9, 8))) and not unit.overlaps_itself_unit(args(64, 8, *axes))
