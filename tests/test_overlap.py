"""binding/overlap.h on the host: every pair of small strided row sets against the sets of
bytes they hold."""
import ctypes
import os
import random
import subprocess

import pytest

import mamba_ssd_chunked_02_gb300 as m2

BINDING = os.path.join(os.path.dirname(m2.__file__), "binding")


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    at = tmp_path_factory.mktemp("overlap")
    (at / "o.cpp").write_text('#include "overlap.h"\nextern "C" int overlap(const m2::Rows* a, const m2::Rows* b)'
                              " { return m2::overlap(*a, *b); }\n")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error",
                    "-I", BINDING, str(at / "o.cpp"), "-o", str(at / "o.so")], check=True)
    f = ctypes.CDLL(str(at / "o.so")).overlap
    rows = ctypes.c_int64 * 6
    return lambda a, b: bool(f(rows(*a), rows(*b)))


def held(at, row, n0, n1, s0, s1):
    return {at + i * s0 + j * s1 + k for i in range(n0) for j in range(n1) for k in range(row)}


def test_against_the_bytes_held(overlap):
    r = random.Random(1)
    seen = [0, 0]
    for _ in range(60000):
        same = r.random() < 0.5
        st = [r.choice([0, 1, 2, 3, 4, 6, 8, 12, 16, 24]) for _ in range(2)]
        sets = []
        for k in range(2):
            s = st if same else [r.choice([0, 1, 2, 3, 4, 6, 8, 12, 16, 24]) for _ in range(2)]
            if same and r.random() < 0.3:
                s = s[::-1]
            sets.append((r.randrange(0, 40), r.randrange(1, 6), r.randrange(1, 5), r.randrange(1, 5), *s))
        want = bool(held(*sets[0]) & held(*sets[1]))
        assert overlap(*sets) == want, sets
        seen[want] += 1
    assert min(seen) > 5000


def test_nothing_held_overlaps_nothing(overlap):
    full = (0, 4, 2, 2, 8, 4)
    for empty in ((0, 0, 2, 2, 8, 4), (0, 4, 0, 2, 8, 4), (0, 4, 2, 0, 8, 4)):
        assert not overlap(full, empty) and not overlap(empty, full)


def test_column_slices_of_one_large_buffer(overlap):
    pitch, b, T, base = 16384, 8, 1 << 20, 1 << 40
    st = (T * pitch, pitch)
    x, y = (base, 8192, b, T, *st), (base + 8192, 8192, b, T, *st)
    assert not overlap(x, y) and overlap(x, (base + 8190, 8192, b, T, *st))
    whole = (base, b * T * pitch, 1, 1, 0, 0)
    assert overlap(whole, y) and not overlap((base + b * T * pitch, 2, 1, 1, 0, 0), y)
    # tokens outermost against sequences outermost
    assert overlap(x, (base, 8192, T, b, pitch, T * pitch)) and not overlap(y, (base, 8192, T, b, pitch, T * pitch))
    assert overlap(x, x) and overlap(y, y)
