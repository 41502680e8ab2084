"""The arithmetic that cuts a latent attention's steps into stretches, compiled for the host,
against whole numbers of any size (CPU)."""

import ctypes
import os
import random
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "paged_kv_cache_51_gb300", "csrc")
SOURCE = """
#include "latent_split.h"
extern "C" int64_t md(int64_t a, int64_t b, int64_t c) { return pkv::mul_div(a, b, c); }
extern "C" int64_t begin(int64_t t, int64_t n, int teams) { return pkv::stretch_begin(t, n, teams); }
extern "C" int of(int64_t step, int64_t n, int teams) { return pkv::stretch_of(step, n, teams); }
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src, so = d / "split.cpp", d / "libsplit.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(so)],
                   check=True)
    lib = ctypes.CDLL(str(so))
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    lib.md.restype, lib.md.argtypes = i64, [i64, i64, i64]
    lib.begin.restype, lib.begin.argtypes = i64, [i64, i64, i32]
    lib.of.restype, lib.of.argtypes = i32, [i64, i64, i32]
    return lib


@pytest.mark.parametrize("teams", [1, 2, 3, 19, 76, 152])
def test_every_step_belongs_to_the_stretch_that_holds_it(split, teams):
    for total in (*range(teams, teams + 40), 1000, 4801):
        begins = [split.begin(t, total, teams) for t in range(teams + 1)]
        assert begins == [t * total // teams for t in range(teams + 1)]
        owners = [split.of(s, total, teams) for s in range(total)]
        assert owners == [t for t in range(teams) for _ in range(begins[t], begins[t + 1])]


@pytest.mark.parametrize("total", [(1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, (1 << 32) + 5,
                                   (1 << 40) + 3, (1 << 51) - 1])
@pytest.mark.parametrize("teams", [1, 7, 76, 152])
def test_totals_past_32_bits(split, total, teams):
    """Products that fit into 32 bits beside divisors that do not, among others."""
    rng = random.Random(total)
    for t in range(teams):
        a, b = t * total // teams, (t + 1) * total // teams
        assert split.begin(t, total, teams) == a
        for s in {a, a + 1, b - 1, rng.randrange(a, b)}:
            assert split.of(s, total, teams) == t, s


def test_products_and_divisors_of_every_size(split):
    rng = random.Random(1)
    for _ in range(20000):
        a, c = rng.getrandbits(rng.randint(1, 55)), rng.getrandbits(rng.randint(1, 62)) + 1
        b = rng.getrandbits(rng.randint(1, 63 - max(1, a.bit_length())))
        assert split.md(a, b, c) == a * b // c, (a, b, c)
