"""The chains by which the distillation kernels find a stage's listed elements (csrc/p24_chain.h),
compiled for the host: the walk ends, and stays among the entries, also on what an expired wait can
leave behind, namely chains that a second list was added to before they were used up."""
import ctypes as C
import os
import random
import subprocess

import pytest

from tests.conftest import ROOT

MOST = 128
SOURCE = """
#include "p24_chain.h"
extern "C" int walk(int first, const int* next, int most, int* seen, int room) {
  int n = 0;
  p24::chain_walk(first, next, most, [&](int e) { if (n < room) seen[n] = e; ++n; });
  return n;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("chain")
    src, lib = os.path.join(d, "chain.cpp"), os.path.join(d, "chain.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    csrc = os.path.join(ROOT, "semi_structured_sparse_prune24_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", f"-I{csrc}", src, "-o", lib], check=True)
    f = C.CDLL(lib).walk

    def run(first, next_):
        seen = (C.c_int * (2 * MOST))()
        n = f(first, (C.c_int * MOST)(*next_), MOST, seen, 2 * MOST)
        return list(seen[:n])
    return run


def push(heads, next_, h, j):
    next_[j], heads[h] = heads[h], j


def test_whole_chains_in_full(walk):
    rng = random.Random(1)
    for k in (0, 1, 5, MOST):
        heads, next_, want = [-1] * 3, [-1] * MOST, [[], [], []]
        for j in rng.sample(range(MOST), k):
            h = rng.randrange(3)
            push(heads, next_, h, j)
            want[h].insert(0, j)
        assert [walk(h, next_) for h in heads] == want


def test_a_list_chained_onto_one_that_was_not_used_up(walk):
    """Entry 3 of two lists in one chain, with 5 between: 3, 5, 3, 5, ... without end."""
    heads, next_ = [-1], [-1] * MOST
    for j in (3, 5, 3):
        push(heads, next_, 0, j)
    assert next_[3] == 5 and next_[5] == 3
    seen = walk(heads[0], next_)
    assert len(seen) <= MOST and set(seen) == {3, 5}


def test_any_leftovers(walk):
    rng = random.Random(2)
    for _ in range(200):
        next_ = [rng.choice([-1, rng.randrange(MOST), rng.randrange(-2 ** 31, 2 ** 31)]) for _ in range(MOST)]
        seen = walk(rng.randrange(MOST), next_)
        assert len(seen) <= MOST and all(0 <= j < MOST for j in seen)
